// Root-mean-square norm with the residual's addition, its backward pass, and rows in 8 bits.
//
// All three are bound by memory: a few operations an element, each element read and written
// once.  A row's channels stay in registers between its sums and its outputs, in words of 8
// neighbouring channels a lane (16 bytes of bf16), so every access is as wide as the hardware
// has them; rows need no alignment beyond their elements', since global memory takes wide
// accesses at any address.
#include "sscan_layer.h"

namespace sscan {

constexpr int kWord = 8;               // channels of a word
constexpr int kRmsBlocks = 2048;       // workgroups of a forward, at most: rows go on to the next
constexpr int kRmsGroups = 512;        // workgroups of a backward, at most, a partial dweight each

typedef uint32_t u32x2 __attribute__((ext_vector_type(2)));
typedef uint32_t u32x4 __attribute__((ext_vector_type(4)));
typedef u32x2 u32x2_any __attribute__((aligned(1)));
typedef u32x4 u32x4_bf16 __attribute__((aligned(2)));
typedef u32x4 u32x4_f32 __attribute__((aligned(4)));

// A lane's channel, to be compared with dim anew at each use: known to be the same for all
// rows, the comparisons of every word's tail become masks that the loop over rows keeps, for
// which there are not the scalar registers.
__device__ __forceinline__ int anew(int c) {
  asm volatile("" : "+v"(c));
  return c;
}

// Channels c .. c + 7 of a row; those past its end are zero, and not written.
__device__ __forceinline__ void load_word(const bf16_t* row, int c, int dim, float* v) {
  c = anew(c);
  if (c + kWord <= dim) {
    const u32x4 u = *reinterpret_cast<const u32x4_bf16*>(row + c);
#pragma unroll
    for (int j = 0; j < 4; ++j) {
      v[2 * j] = __uint_as_float(u[j] << 16);
      v[2 * j + 1] = __uint_as_float(u[j] & 0xffff0000u);
    }
  } else {
#pragma unroll
    for (int j = 0; j < kWord; ++j) v[j] = c + j < dim ? to_f32(row[c + j]) : 0.f;
  }
}
__device__ __forceinline__ void load_word(const float* row, int c, int dim, float* v) {
  c = anew(c);
  if (c + kWord <= dim) {
#pragma unroll
    for (int h = 0; h < 2; ++h) {
      const u32x4 u = *reinterpret_cast<const u32x4_f32*>(row + c + 4 * h);
#pragma unroll
      for (int j = 0; j < 4; ++j) v[4 * h + j] = __uint_as_float(u[j]);
    }
  } else {
#pragma unroll
    for (int j = 0; j < kWord; ++j) v[j] = c + j < dim ? row[c + j] : 0.f;
  }
}
__device__ __forceinline__ void store_word(bf16_t* row, int c, int dim, const float* v) {
  c = anew(c);
  typedef __bf16 b2 __attribute__((ext_vector_type(2)));
  typedef float f2 __attribute__((ext_vector_type(2)));
  if (c + kWord <= dim) {
    u32x4 u;
#pragma unroll
    for (int j = 0; j < 4; ++j)
      u[j] = __builtin_bit_cast(uint32_t, __builtin_convertvector((f2{v[2 * j], v[2 * j + 1]}), b2));
    *reinterpret_cast<u32x4_bf16*>(row + c) = u;
  } else {
#pragma unroll
    for (int j = 0; j < kWord; ++j)
      if (c + j < dim) store_val(row + c + j, v[j]);
  }
}
__device__ __forceinline__ void store_word(float* row, int c, int dim, const float* v) {
  c = anew(c);
  if (c + kWord <= dim) {
#pragma unroll
    for (int h = 0; h < 2; ++h) {
      u32x4 u;
#pragma unroll
      for (int j = 0; j < 4; ++j) u[j] = __float_as_uint(v[4 * h + j]);
      *reinterpret_cast<u32x4_f32*>(row + c + 4 * h) = u;
    }
  } else {
#pragma unroll
    for (int j = 0; j < kWord; ++j)
      if (c + j < dim) row[c + j] = v[j];
  }
}
// The codes of a word's values.  v inv is off by a few units of its last place, so it rounds to
// the right whole number unless it lies next to a border; words with such a value take the
// exact way.  Adding 1.5 x 2^23 rounds (ties to even) and leaves the code in the low byte.
__device__ __forceinline__ void store_codes(int8_t* row, int c, int dim, const float* v, float scale, float inv) {
  constexpr float k = 12582912.f;
  c = anew(c);
  uint32_t q[kWord];
  float off = 0.f;
#pragma unroll
  for (int j = 0; j < kWord; ++j) {
    const float t = fmaf(v[j], inv, k);
    q[j] = __float_as_uint(t);
    off = fmaxf(off, fabsf(fmaf(v[j], inv, k - t)));
  }
  if (off > 0.4999f) {
#pragma unroll
    for (int j = 0; j < kWord; ++j) q[j] = static_cast<uint32_t>(static_cast<int>(i8_code(v[j], scale, inv)));
  }
  if (c + kWord <= dim) {
    u32x2 u;
#pragma unroll
    for (int h = 0; h < 2; ++h) {
      const uint32_t lo = __builtin_amdgcn_perm(q[4 * h + 1], q[4 * h], 0x0c0c0400u);
      const uint32_t hi = __builtin_amdgcn_perm(q[4 * h + 3], q[4 * h + 2], 0x0c0c0400u);
      u[h] = lo | hi << 16;
    }
    *reinterpret_cast<u32x2_any*>(row + c) = u;
  } else {
#pragma unroll
    for (int j = 0; j < kWord; ++j)
      if (c + j < dim) row[c + j] = static_cast<int8_t>(q[j]);
  }
}

__device__ __forceinline__ float rounded(float v, const float*) { return v; }
__device__ __forceinline__ float rounded(float v, const bf16_t*) {
  bf16_t t;
  store_val(&t, v);
  return to_f32(t);
}

// A lane's value moved by a DPP control word, zero where no lane gives one.
template <int CTRL, int ROWS>
__device__ __forceinline__ uint32_t dpp(uint32_t v) {
  return static_cast<uint32_t>(__builtin_amdgcn_update_dpp(0, static_cast<int>(v), CTRL, ROWS, 0xf, ROWS == 0xf));
}
// The whole wave's sum, or the largest of magnitude bits (a NaN's are above infinity's):
// within rows of 16 lanes, then across them to lane 63.
struct Sum {
  template <int CTRL, int ROWS>
  static __device__ __forceinline__ float with(float v) {
    return v + __uint_as_float(dpp<CTRL, ROWS>(__float_as_uint(v)));
  }
};
struct Top {
  template <int CTRL, int ROWS>
  static __device__ __forceinline__ float with(float v) {
    const uint32_t a = __float_as_uint(v), b = dpp<CTRL, ROWS>(a);
    return __uint_as_float(b > a ? b : a);
  }
};
template <typename Op>
__device__ __forceinline__ float over_wave(float v) {
  v = Op::template with<0x111, 0xf>(v);   // the lane 1, 2, 4, 8 below
  v = Op::template with<0x112, 0xf>(v);
  v = Op::template with<0x114, 0xf>(v);
  v = Op::template with<0x118, 0xf>(v);
  v = Op::template with<0x142, 0xa>(v);   // lane 15 of the row below
  v = Op::template with<0x143, 0xc>(v);   // lane 31
  return __uint_as_float(__builtin_amdgcn_readlane(__float_as_uint(v), 63));
}

// Values joined over the LANES lanes that hold a row: one wave, or all waves of the workgroup
// through LDS.  The two halves of the LDS array are used in turn, so one barrier a call will do:
// who writes a half again has passed the barrier that follows its last reading.
template <int LANES>
struct RowLanes {
  static constexpr int kWaves = LANES / 64;
  float* lds;     // [2][2 kWaves]
  int half = 0;
  __device__ explicit RowLanes(float* l) : lds(l) {}
  // the sums of a and b
  __device__ __forceinline__ void sums(float& a, float& b) {
    a = over_wave<Sum>(a);
    b = over_wave<Sum>(b);
    if (kWaves == 1) return;
    float* at = lds + half * 2 * kWaves;
    half ^= 1;
    if ((threadIdx.x & 63) == 0) {
      at[threadIdx.x >> 6] = a;
      at[kWaves + (threadIdx.x >> 6)] = b;
    }
    __syncthreads();
    a = b = 0.f;
#pragma unroll
    for (int w = 0; w < kWaves; ++w) {
      a += at[w];
      b += at[kWaves + w];
    }
  }
  __device__ __forceinline__ float sum(float a) {
    float none = 0.f;
    sums(a, none);
    return a;
  }
  __device__ __forceinline__ uint32_t top(uint32_t a) {
    a = __float_as_uint(over_wave<Top>(__uint_as_float(a)));
    if (kWaves == 1) return a;
    float* at = lds + half * 2 * kWaves;
    half ^= 1;
    if ((threadIdx.x & 63) == 0) at[threadIdx.x >> 6] = __uint_as_float(a);
    __syncthreads();
    a = 0;
#pragma unroll
    for (int w = 0; w < kWaves; ++w) {
      const uint32_t o = __float_as_uint(at[w]);
      a = o > a ? o : a;
    }
    return a;
  }
};

// A lane's weights: held over the rows, or read at each use where a row takes 1024 lanes, whose
// waves have 128 registers at most.
template <int LANES, int WORDS>
struct Weights {
  static constexpr bool kHeld = LANES < 1024;
  const float* weight;
  int lane, dim;
  float w[kHeld ? WORDS : 1][kWord];
  __device__ Weights(const float* p, int l, int d) : weight(p), lane(l), dim(d) {
    if (!kHeld) return;
#pragma unroll
    for (int i = 0; i < WORDS; ++i) read(i, w[i]);
  }
  __device__ __forceinline__ void read(int i, float* to) const {
    if (weight) {
      load_word(weight, (i * LANES + lane) * kWord, dim, to);
    } else {
#pragma unroll
      for (int j = 0; j < kWord; ++j) to[j] = 1.f;
    }
  }
  __device__ __forceinline__ void get(int i, float* to) const {
    if (!kHeld) return read(i, to);
#pragma unroll
    for (int j = 0; j < kWord; ++j) to[j] = w[kHeld ? i : 0][j];
  }
};

constexpr int block_of(int lanes) { return lanes == 64 ? 256 : lanes; }

// LANES lanes with WORDS words each hold a row; a workgroup of 256 holds four rows of one wave.
// NORM: the norm; otherwise the row as it is, for its codes.
template <typename Tin, typename Tres, bool NORM, int LANES, int WORDS>
__global__ __launch_bounds__(block_of(LANES)) void rms_fwd_kernel(RmsFwdParams p) {
  constexpr int kRows = block_of(LANES) / LANES;
  __shared__ float lds[4 * RowLanes<LANES>::kWaves];
  RowLanes<LANES> join(lds);
  const int lane = kRows == 1 ? threadIdx.x : threadIdx.x % LANES, sub = kRows == 1 ? 0 : threadIdx.x / LANES;
  const Weights<LANES, WORDS> weights(p.weight, lane, p.dim);
  const float per = 1.f / static_cast<float>(p.dim);
  for (int64_t row = static_cast<int64_t>(blockIdx.x) * kRows + sub; row < p.rows; row += static_cast<int64_t>(gridDim.x) * kRows) {
    float v[WORDS][kWord], sum = 0.f;
#pragma unroll
    for (int i = 0; i < WORDS; ++i)
      load_word(static_cast<const Tin*>(p.x) + row * p.sx, (i * LANES + lane) * kWord, p.dim, v[i]);
    if (NORM) {
      if (p.residual) {
#pragma unroll
        for (int i = 0; i < WORDS; ++i) {
          float a[kWord];
          load_word(static_cast<const Tres*>(p.residual) + row * p.dim, (i * LANES + lane) * kWord, p.dim, a);
#pragma unroll
          for (int j = 0; j < kWord; ++j) v[i][j] += a[j];
        }
      }
#pragma unroll
      for (int i = 0; i < WORDS; ++i) {
#pragma unroll
        for (int j = 0; j < kWord; ++j) {
          v[i][j] = rounded(v[i][j], static_cast<const Tres*>(nullptr));
          sum = fmaf(v[i][j], v[i][j], sum);
        }
        if (p.kept) store_word(static_cast<Tres*>(p.kept) + row * p.dim, (i * LANES + lane) * kWord, p.dim, v[i]);
      }
      const float r = __builtin_amdgcn_rsqf(fmaf(join.sum(sum), per, p.eps));
#pragma unroll
      for (int i = 0; i < WORDS; ++i) {
        float w[kWord];
        weights.get(i, w);
#pragma unroll
        for (int j = 0; j < kWord; ++j) v[i][j] = v[i][j] * r * w[j];
        if (p.y) store_word(static_cast<Tin*>(p.y) + row * p.dim, (i * LANES + lane) * kWord, p.dim, v[i]);
      }
    }
    if (p.scales) {      // also of rows without channels, which have no codes
      uint32_t top = 0;
#pragma unroll
      for (int i = 0; i < WORDS; ++i)
#pragma unroll
        for (int j = 0; j < kWord; ++j) top = act8_top(top, v[i][j]);
      top = join.top(top);
      const bool fine = top < 0x7f800000u;
      const float scale = i8_scale(__uint_as_float(top)), inv = 1.f / scale;
      if (lane == 0) p.scales[row] = fine ? scale : __uint_as_float(0x7fc00000u);
#pragma unroll
      for (int i = 0; i < WORDS; ++i) {
        if (!fine) {
#pragma unroll
          for (int j = 0; j < kWord; ++j) v[i][j] = 0.f;
        }
        store_codes(p.codes + row * p.sc, (i * LANES + lane) * kWord, p.dim, v[i], fine ? scale : 1.f, fine ? inv : 1.f);
      }
    }
  }
}

// Rows as in the forward; each workgroup sums its rows' part of dweight in registers.  1024 lanes of
// 4 words (rows of 24577 to 32768 channels) spill 56 to 60 bytes a lane.
// Measured: 32768 x 2048 bf16 with a float32 stream 205 us of 215 at 5 TB/s (the forward 147 of
// 161: part of what both read and write stays cached), 4094 x 1535 float32 30 of 25.  Rows of few
// channels leave lanes of their wave idle: 131072 x 256 bf16 90 of 40 (the forward 30 of 27), 524288 x 64
// 336 of 40 (108 of 27), 65536 x 512 36 of 40.
template <typename Tin, typename Tres, int LANES, int WORDS>
__global__ __launch_bounds__(block_of(LANES)) void rms_bwd_kernel(RmsBwdParams p) {
  constexpr int kRows = block_of(LANES) / LANES;
  __shared__ float lds[4 * RowLanes<LANES>::kWaves];
  __shared__ float sums[kRows > 1 ? kRows * LANES * kWord : 1];
  RowLanes<LANES> join(lds);
  const int lane = kRows == 1 ? threadIdx.x : threadIdx.x % LANES, sub = kRows == 1 ? 0 : threadIdx.x / LANES;
  const Weights<LANES, WORDS> weights(p.weight, lane, p.dim);
  float dw[WORDS][kWord] = {};
  const float per = 1.f / static_cast<float>(p.dim);
  for (int64_t row = static_cast<int64_t>(blockIdx.x) * kRows + sub; row < p.rows; row += static_cast<int64_t>(gridDim.x) * kRows) {
    float v[WORDS][kWord], g[WORDS][kWord], ss = 0.f, gs = 0.f;
#pragma unroll
    for (int i = 0; i < WORDS; ++i) {
      load_word(static_cast<const Tres*>(p.s) + row * p.ss, (i * LANES + lane) * kWord, p.dim, v[i]);
      load_word(static_cast<const Tin*>(p.dy) + row * p.dim, (i * LANES + lane) * kWord, p.dim, g[i]);
    }
#pragma unroll
    for (int i = 0; i < WORDS; ++i) {
      float w[kWord];
      weights.get(i, w);
#pragma unroll
      for (int j = 0; j < kWord; ++j) {
        ss = fmaf(v[i][j], v[i][j], ss);
        gs = fmaf(g[i][j] * w[j], v[i][j], gs);
      }
    }
    join.sums(ss, gs);
    const float r = __builtin_amdgcn_rsqf(fmaf(ss, per, p.eps)), mean = gs * r * per;
#pragma unroll
    for (int i = 0; i < WORDS; ++i) {
      const int c = (i * LANES + lane) * kWord;
      float out[kWord], w[kWord];
      weights.get(i, w);
#pragma unroll
      for (int j = 0; j < kWord; ++j) {
        const float n = v[i][j] * r;
        dw[i][j] = fmaf(g[i][j], n, dw[i][j]);
        out[j] = r * fmaf(-n, mean, g[i][j] * w[j]);
      }
      if (p.dkept) {
        float a[kWord];
        load_word(static_cast<const Tres*>(p.dkept) + row * p.dim, c, p.dim, a);
#pragma unroll
        for (int j = 0; j < kWord; ++j) out[j] += a[j];
      }
      if (p.dx) store_word(static_cast<Tin*>(p.dx) + row * p.sdx, c, p.dim, out);
      if (p.dresidual) store_word(static_cast<Tres*>(p.dresidual) + row * p.dim, c, p.dim, out);
    }
  }
  if (!p.dweight) return;
  float* part = p.partial + static_cast<int64_t>(blockIdx.x) * p.dim;
#pragma unroll
  for (int i = 0; i < WORDS; ++i) {
    if (kRows > 1) {      // the waves' rows, added in their order
      __syncthreads();
#pragma unroll
      for (int j = 0; j < kWord; ++j) sums[(sub * kWord + j) * LANES + lane] = dw[i][j];
      __syncthreads();
      if (sub != 0) continue;
#pragma unroll
      for (int k = 1; k < kRows; ++k)
#pragma unroll
        for (int j = 0; j < kWord; ++j) dw[i][j] += sums[(k * kWord + j) * LANES + lane];
    }
    store_word(part, (i * LANES + lane) * kWord, p.dim, dw[i]);
  }
}

// dweight from the workgroups' sums: 64 channels a workgroup, its 16 waves a 16th of the
// sums each, eight loads in flight.
constexpr int kWeightWaves = 16;
__global__ __launch_bounds__(64 * kWeightWaves) void rms_weight_kernel(const float* partial, float* dweight, int groups, int dim) {
  __shared__ float lds[kWeightWaves][64];
  const int lane = threadIdx.x & 63, wave = threadIdx.x >> 6, c = blockIdx.x * 64 + lane;
  float sum = 0.f;
  if (c < dim) {
    int g = wave;
    for (; g + 7 * kWeightWaves < groups; g += 8 * kWeightWaves) {
      float v[8];
#pragma unroll
      for (int k = 0; k < 8; ++k) v[k] = partial[static_cast<int64_t>(g + k * kWeightWaves) * dim + c];
#pragma unroll
      for (int k = 0; k < 8; ++k) sum += v[k];
    }
    for (; g < groups; g += kWeightWaves) sum += partial[static_cast<int64_t>(g) * dim + c];
  }
  lds[wave][lane] = sum;
  __syncthreads();
  if (wave != 0 || c >= dim) return;
#pragma unroll
  for (int k = 1; k < kWeightWaves; ++k) sum += lds[k][lane];
  dweight[c] = sum;
}

namespace {

// Lanes and words of a row.  Forward: few words a lane, which keeps many rows in flight
// (16411 x 2560 bf16 to 8 bits: 57 us with 256 lanes of 2 words, 62 with 128 of 3, of which
// fewer idle; 32768 x 2048: the same within 3 %; one word on each of 320 to 448 lanes: 57, and 3500
// channels to 8 bits 111 for 98), and rows of fewer words on fewer lanes (16411 x 1400 on 192 of them
// 34 us, on 256 37; rows alone to 8 bits 21 and 23.5).
// Backward: one wave a row while it holds it, which joins a row's sums without a barrier and
// four rows' part of dweight in LDS (4094 x 1535 float32: 30 us, 33 with 256 lanes; 32768 x
// 2048 bf16 the same within 2 %); fewer than 1024 rows leave compute units idle that way.
struct RowPlan {
  int lanes, words;
};

RowPlan forward_plan(int64_t dim) {
  const int words = static_cast<int>((dim + kWord - 1) / kWord);
  const int lanes = words > 256 * 4 ? 1024 : words > 192 ? 256 : words > 64 ? (words + 63) / 64 * 64 : 64;
  return {lanes, (words + lanes - 1) / lanes};
}

RowPlan backward_plan(int64_t rows, int64_t dim) {
  const int words = static_cast<int>((dim + kWord - 1) / kWord);
  const int lanes = words > 256 * 4 ? 1024 : (words > 64 * 4 || rows < 1024 ? 256 : 64);
  return {lanes, (words + lanes - 1) / lanes};
}

int64_t blocks_of(const RowPlan& q, int64_t rows) {
  const int rows_each = block_of(q.lanes) / q.lanes;
  return (rows + rows_each - 1) / rows_each;
}

int groups_of(int64_t rows, int64_t dim) {
  const int64_t n = blocks_of(backward_plan(rows, dim), rows);
  return static_cast<int>(n < kRmsGroups ? n : kRmsGroups);
}

template <int V>
using Int = std::integral_constant<int, V>;

// f(lanes, words) with the plan's numbers as constants: lanes is given, words is 1 .. 4.
template <typename Lanes, typename F>
void with_words(Lanes lanes, int words, F&& f) {
  switch (words) {
    case 1: return f(lanes, Int<1>{});
    case 2: return f(lanes, Int<2>{});
    case 3: return f(lanes, Int<3>{});
    default: return f(lanes, Int<4>{});
  }
}
// Rows of 1024 lanes have 2 words at least.
template <typename F>
void with_many(int words, F&& f) {
  words == 2 ? f(Int<1024>{}, Int<2>{}) : words == 3 ? f(Int<1024>{}, Int<3>{}) : f(Int<1024>{}, Int<4>{});
}

template <typename Tin, typename Tres, bool NORM>
hipError_t fwd(const RmsFwdParams& p, hipStream_t s) {
  const RowPlan q = forward_plan(p.dim);
  const int64_t n = blocks_of(q, p.rows);
  const unsigned grid = static_cast<unsigned>(n < kRmsBlocks ? n : kRmsBlocks);
  const auto launch = [&](auto lanes, auto words) {
    constexpr int kLanes = decltype(lanes)::value, kWords = decltype(words)::value;
    hipLaunchKernelGGL((rms_fwd_kernel<Tin, Tres, NORM, kLanes, kWords>), dim3(grid), dim3(block_of(kLanes)), 0, s, p);
  };
  if (q.lanes == 64) launch(Int<64>{}, Int<1>{});
  else if (q.lanes == 128) launch(Int<128>{}, Int<1>{});
  else if (q.lanes == 192) launch(Int<192>{}, Int<1>{});
  else if (q.lanes == 256) with_words(Int<256>{}, q.words, launch);
  else with_many(q.words, launch);
  return hipGetLastError();
}

template <typename Tin, typename Tres>
hipError_t bwd(const RmsBwdParams& p, hipStream_t s) {
  const int groups = groups_of(p.rows, p.dim);
  const RowPlan q = backward_plan(p.rows, p.dim);
  const auto launch = [&](auto lanes, auto words) {
    constexpr int kLanes = decltype(lanes)::value, kWords = decltype(words)::value;
    hipLaunchKernelGGL((rms_bwd_kernel<Tin, Tres, kLanes, kWords>), dim3(groups), dim3(block_of(kLanes)), 0, s, p);
  };
  if (groups > 0) {
    if (q.lanes == 64) with_words(Int<64>{}, q.words, launch);
    else if (q.lanes == 256) with_words(Int<256>{}, q.words, launch);
    else with_many(q.words, launch);
  }
  if (p.dweight)
    hipLaunchKernelGGL(rms_weight_kernel, dim3((p.dim + 63) / 64), dim3(64 * kWeightWaves), 0, s, p.partial, p.dweight, groups, p.dim);
  return hipGetLastError();
}

}  // namespace

// As many sums as workgroups of a row each would leave, which is no less for more rows or channels:
// a buffer for the longest batch serves the shorter ones, whose plan may take four times the
// workgroups (2048 channels: 256 at 1024 rows, 512 at 1023).
size_t rms_bwd_workspace_bytes(int64_t rows, int64_t dim) {
  return rows > 0 && dim > 0 ? static_cast<size_t>(rows < kRmsGroups ? rows : kRmsGroups) * dim * 4 : 0;
}

hipError_t launch_rms_fwd(const RmsFwdParams& p, bool bf16, bool kept_bf16, hipStream_t s) {
  if (!bf16) return fwd<float, float, true>(p, s);
  return kept_bf16 ? fwd<bf16_t, bf16_t, true>(p, s) : fwd<bf16_t, float, true>(p, s);
}

hipError_t launch_i8_quant(const RmsFwdParams& p, bool bf16, hipStream_t s) {
  return bf16 ? fwd<bf16_t, bf16_t, false>(p, s) : fwd<float, float, false>(p, s);
}

hipError_t launch_rms_bwd(const RmsBwdParams& p, bool bf16, bool kept_bf16, hipStream_t s) {
  if (!bf16) return bwd<float, float>(p, s);
  return kept_bf16 ? bwd<bf16_t, bf16_t>(p, s) : bwd<bf16_t, float>(p, s);
}

}  // namespace sscan
