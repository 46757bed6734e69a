// Activations in 8 bits: pack and unpack.
#include "sscan_glr.h"

namespace sscan {

// A lane holds VEC neighbouring channels of the 16 tokens of a group, so the group's
// largest magnitude needs no other lane, and loads and stores are whole words.  The work
// is bound by memory: 2 (float32: 4) bytes an element on one side and 1 + 1/16 on the
// other.  8 x 4096 x 2048 bf16: packed in 45 us, unpacked in 32 (4.6 and 6.4 TB/s, part of
// the codes still in the last cache); one channel a lane 88 and 142.
template <typename Tin, int VEC>
struct ActWords {   // VEC elements, VEC codes
  typedef Tin elems __attribute__((ext_vector_type(VEC)));
  typedef uint8_t bytes __attribute__((ext_vector_type(VEC)));
};
template <typename Tin>
struct ActWords<Tin, 1> {
  struct elems {
    Tin v;
    __device__ Tin& operator[](int) { return v; }
  };
  struct bytes {
    uint8_t v;
    __device__ uint8_t& operator[](int) { return v; }
  };
};

// Lane `id` of a launch over groups x channel words: channel word q, token group g of row b.
struct ActPlace {
  int64_t b, g, c;
  __device__ ActPlace(int64_t id, int64_t words, int64_t ngrp, int vec) {
    const int64_t row = id / words;
    c = (id - row * words) * vec;
    b = row / ngrp;
    g = row - b * ngrp;
  }
};

template <typename Tin, int VEC>
__global__ __launch_bounds__(256) void act8_pack_kernel(const Tin* x, int64_t stride, int8_t* codes, uint8_t* exps,
                                                        int64_t lanes, int64_t words, int64_t ngrp, int64_t L, int64_t dim) {
  typedef typename ActWords<Tin, VEC>::elems Elems;
  typedef typename ActWords<Tin, VEC>::bytes Bytes;
  const int64_t id = static_cast<int64_t>(workgroup<256>()) * 256 + threadIdx.x;
  if (id >= lanes) return;
  const ActPlace at(id, words, ngrp, VEC);
  const int64_t t0 = at.g * kActGroup, row0 = at.b * L + t0;
  const int rows = L - t0 < kActGroup ? static_cast<int>(L - t0) : kActGroup;
  Elems v[kActGroup];
  // a short group's missing tokens repeat its last one, which changes no maximum
#pragma unroll
  for (int k = 0; k < kActGroup; ++k)
    v[k] = *reinterpret_cast<const Elems*>(x + (row0 + (k < rows ? k : rows - 1)) * stride + at.c);
  int shift[VEC];
  Bytes field;
#pragma unroll
  for (int j = 0; j < VEC; ++j) {
    uint32_t top = 0;
#pragma unroll
    for (int k = 0; k < kActGroup; ++k) top = act8_top(top, to_f32(v[k][j]));
    field[j] = static_cast<uint8_t>(top >> 23);
    shift[j] = act8_shift(top >> 23);
  }
  *reinterpret_cast<Bytes*>(exps + (at.b * ngrp + at.g) * dim + at.c) = field;
#pragma unroll
  for (int k = 0; k < kActGroup; ++k) {
    Bytes q;
#pragma unroll
    for (int j = 0; j < VEC; ++j) q[j] = static_cast<uint8_t>(act8_code(to_f32(v[k][j]), shift[j]));
    if (k < rows) *reinterpret_cast<Bytes*>(codes + (row0 + k) * dim + at.c) = q;
  }
}

template <typename Tin, int VEC>
__global__ __launch_bounds__(256) void act8_unpack_kernel(const int8_t* codes, const uint8_t* exps, Tin* x, int64_t lanes,
                                                          int64_t words, int64_t ngrp, int64_t L, int64_t dim) {
  typedef typename ActWords<Tin, VEC>::elems Elems;
  typedef typename ActWords<Tin, VEC>::bytes Bytes;
  const int64_t id = static_cast<int64_t>(workgroup<256>()) * 256 + threadIdx.x;
  if (id >= lanes) return;
  const ActPlace at(id, words, ngrp, VEC);
  const int64_t t0 = at.g * kActGroup, row0 = at.b * L + t0;
  const int rows = L - t0 < kActGroup ? static_cast<int>(L - t0) : kActGroup;
  Bytes q[kActGroup];
  Bytes field = *reinterpret_cast<const Bytes*>(exps + (at.b * ngrp + at.g) * dim + at.c);
#pragma unroll
  for (int k = 0; k < kActGroup; ++k)
    q[k] = *reinterpret_cast<const Bytes*>(codes + (row0 + (k < rows ? k : rows - 1)) * dim + at.c);
  float scale[VEC];
#pragma unroll
  for (int j = 0; j < VEC; ++j) scale[j] = act8_value(1, field[j]);
#pragma unroll
  for (int k = 0; k < kActGroup; ++k) {
    Elems v;
#pragma unroll
    for (int j = 0; j < VEC; ++j) {
      Tin e;
      store_val(&e, static_cast<float>(static_cast<int8_t>(q[k][j])) * scale[j]);
      v[j] = e;
    }
    if (k < rows) *reinterpret_cast<Elems*>(x + (row0 + k) * dim + at.c) = v;
  }
}

namespace {

// Channels a lane: the most that divides every row's channels and keeps every word of
// both sides aligned (the packed side starts aligned; its rows are dim bytes).
int act_vec(const void* x, size_t elem, int64_t stride, int64_t dim, int most) {
  int vec = most;
  while (vec > 1 && (dim % vec || stride % vec || reinterpret_cast<uintptr_t>(x) % (vec * elem))) vec /= 2;
  return vec;
}

template <typename Tin, int VEC>
hipError_t pack(const void* x, int64_t stride, void* packed, int64_t batch, int64_t L, int64_t dim, hipStream_t s) {
  const int64_t ngrp = (L + kActGroup - 1) / kActGroup, words = dim / VEC, lanes = batch * ngrp * words;
  hipLaunchKernelGGL((act8_pack_kernel<Tin, VEC>), grid_of<256>((lanes + 255) / 256), dim3(256), 0, s,
                     static_cast<const Tin*>(x), stride, static_cast<int8_t*>(packed),
                     static_cast<uint8_t*>(packed) + act8_exps_at(batch, L, dim), lanes, words, ngrp, L, dim);
  return hipGetLastError();
}

template <typename Tin, int VEC>
hipError_t unpack(const void* packed, void* x, int64_t batch, int64_t L, int64_t dim, hipStream_t s) {
  const int64_t ngrp = (L + kActGroup - 1) / kActGroup, words = dim / VEC, lanes = batch * ngrp * words;
  hipLaunchKernelGGL((act8_unpack_kernel<Tin, VEC>), grid_of<256>((lanes + 255) / 256), dim3(256), 0, s,
                     static_cast<const int8_t*>(packed), static_cast<const uint8_t*>(packed) + act8_exps_at(batch, L, dim),
                     static_cast<Tin*>(x), lanes, words, ngrp, L, dim);
  return hipGetLastError();
}

}  // namespace

hipError_t launch_act8_pack(const void* x, int64_t stride, void* packed, int64_t batch, int64_t L, int64_t dim,
                            bool bf16, hipStream_t s) {
  const int vec = act_vec(x, bf16 ? 2 : 4, stride, dim, 4);
  if (bf16) {
    if (vec == 4) return pack<bf16_t, 4>(x, stride, packed, batch, L, dim, s);
    return vec == 2 ? pack<bf16_t, 2>(x, stride, packed, batch, L, dim, s) : pack<bf16_t, 1>(x, stride, packed, batch, L, dim, s);
  }
  if (vec == 4) return pack<float, 4>(x, stride, packed, batch, L, dim, s);
  return vec == 2 ? pack<float, 2>(x, stride, packed, batch, L, dim, s) : pack<float, 1>(x, stride, packed, batch, L, dim, s);
}

hipError_t launch_act8_unpack(const void* packed, void* x, int64_t batch, int64_t L, int64_t dim, bool bf16,
                              hipStream_t s) {
  const int vec = act_vec(x, bf16 ? 2 : 4, dim, dim, 4);
  if (bf16) {
    if (vec == 4) return unpack<bf16_t, 4>(packed, x, batch, L, dim, s);
    return vec == 2 ? unpack<bf16_t, 2>(packed, x, batch, L, dim, s) : unpack<bf16_t, 1>(packed, x, batch, L, dim, s);
  }
  if (vec == 4) return unpack<float, 4>(packed, x, batch, L, dim, s);
  return vec == 2 ? unpack<float, 2>(packed, x, batch, L, dim, s) : unpack<float, 1>(packed, x, batch, L, dim, s);
}

}  // namespace sscan
