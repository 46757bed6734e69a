// Activations in 8 bits: pack and unpack.
#include "sscan_glr.h"

namespace sscan {

template <typename Tin>
__global__ __launch_bounds__(256) void act8_pack_kernel(const Tin* x, int64_t stride, int8_t* codes, uint8_t* exps,
                                                        int64_t batch, int64_t L, int64_t dim) {
  const int64_t id = static_cast<int64_t>(blockIdx.x) * 256 + threadIdx.x;
  const int64_t ngrp = (L + kActGroup - 1) / kActGroup;
  if (id >= batch * ngrp * dim) return;
  const int64_t d = id % dim, g = id / dim % ngrp, b = id / dim / ngrp;
  float v[kActGroup];
  uint32_t top = 0;
  for (int k = 0; k < kActGroup; ++k) {
    const int64_t t = g * kActGroup + k;
    v[k] = t < L ? to_f32(x[(b * L + t) * stride + d]) : 0.f;
    top = act8_top(top, v[k]);
  }
  const uint32_t field = top >> 23;
  exps[id] = static_cast<uint8_t>(field);
  for (int k = 0; k < kActGroup; ++k)
    if (g * kActGroup + k < L) codes[(b * L + g * kActGroup + k) * dim + d] = static_cast<int8_t>(act8_code(v[k], act8_shift(field)));
}

template <typename Tin>
__global__ __launch_bounds__(256) void act8_unpack_kernel(const int8_t* codes, const uint8_t* exps, Tin* x, int64_t batch,
                                                          int64_t L, int64_t dim) {
  const int64_t id = static_cast<int64_t>(blockIdx.x) * 256 + threadIdx.x;
  if (id >= batch * L * dim) return;
  const int64_t d = id % dim, t = id / dim % L, b = id / dim / L;
  const int64_t ngrp = (L + kActGroup - 1) / kActGroup;
  store_val(&x[id], act8_value(codes[id], exps[(b * ngrp + t / kActGroup) * dim + d]));
}

namespace {
unsigned blocks(int64_t n) { return static_cast<unsigned>((n + 255) / 256); }
}  // namespace

hipError_t launch_act8_pack(const void* x, int64_t stride, void* packed, int64_t batch, int64_t L, int64_t dim,
                            bool bf16, hipStream_t s) {
  int8_t* codes = static_cast<int8_t*>(packed);
  uint8_t* exps = static_cast<uint8_t*>(packed) + act8_exps_at(batch, L, dim);
  const unsigned nb = blocks(batch * ((L + kActGroup - 1) / kActGroup) * dim);
  if (bf16)
    hipLaunchKernelGGL((act8_pack_kernel<bf16_t>), dim3(nb), dim3(256), 0, s, static_cast<const bf16_t*>(x), stride, codes,
                       exps, batch, L, dim);
  else
    hipLaunchKernelGGL((act8_pack_kernel<float>), dim3(nb), dim3(256), 0, s, static_cast<const float*>(x), stride, codes,
                       exps, batch, L, dim);
  return hipGetLastError();
}

hipError_t launch_act8_unpack(const void* packed, void* x, int64_t batch, int64_t L, int64_t dim, bool bf16,
                              hipStream_t s) {
  const int8_t* codes = static_cast<const int8_t*>(packed);
  const uint8_t* exps = static_cast<const uint8_t*>(packed) + act8_exps_at(batch, L, dim);
  const unsigned nb = blocks(batch * L * dim);
  if (bf16)
    hipLaunchKernelGGL((act8_unpack_kernel<bf16_t>), dim3(nb), dim3(256), 0, s, codes, exps, static_cast<bf16_t*>(x), batch,
                       L, dim);
  else
    hipLaunchKernelGGL((act8_unpack_kernel<float>), dim3(nb), dim3(256), 0, s, codes, exps, static_cast<float*>(x), batch, L,
                       dim);
  return hipGetLastError();
}

}  // namespace sscan
