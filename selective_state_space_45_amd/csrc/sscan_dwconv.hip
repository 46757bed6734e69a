// Depthwise causal convolution over time, dense or packed: forward, backward, one token.
#include "sscan_layer.h"

namespace sscan {

constexpr int kConvTile = 64;   // tokens of a workgroup

// The sequence that token t is in: tokens [lo, hi) of the row, index s among all sequences;
// hi <= t for padding.  Whatever offsets holds, 0 <= lo <= t, hi <= L and s is in range.
struct Sequence {
  int64_t s, lo, hi;
};
__device__ __forceinline__ Sequence sequence_of(const ConvParams& p, int64_t b, int64_t t) {
  if (!p.offsets) return {b, 0, p.L};
  int64_t lo = 0, hi = p.num_seqs;                   // the last s with offsets[s] <= t, or 0
  while (hi - lo > 1) {
    const int64_t mid = (lo + hi) / 2;
    if (p.offsets[mid] <= t) lo = mid;
    else hi = mid;
  }
  const int64_t from = p.offsets[lo], to = p.offsets[lo + 1];
  return {lo, from < 0 ? 0 : (from > t ? t : from), to > p.L ? p.L : to};
}

// The input at token t, which may lie up to K - 1 before its sequence.
template <typename Tin, int K>
__device__ __forceinline__ float input_at(const ConvParams& p, const Sequence& q, int64_t row0, int64_t t, int64_t c) {
  if (t >= q.lo) return to_f32(static_cast<const Tin*>(p.x)[(row0 + t) * p.sx + c]);
  if (K == 1 || !p.h0) return 0.f;
  return p.h0[(q.s * p.dim + c) * (K - 1) + (K - 1) + (t - q.lo)];
}

template <int K>
__device__ __forceinline__ void load_taps(const ConvParams& p, int64_t c, float* w, float& b) {
#pragma unroll
  for (int k = 0; k < K; ++k) w[k] = p.w[c * K + k];
  b = p.b ? p.b[c] : 0.f;
}

__device__ __forceinline__ float silu_slope(float v) {
  const float g = sigmoid(v);
  return g * (1.f + v * (1.f - g));
}

// dv at token t of sequence q (zero past its end), and its K inputs.
template <typename Tin, int K>
__device__ __forceinline__ float dv_at(const ConvParams& p, const Sequence& q, int64_t row0, int64_t t, int64_t c,
                                       const float* w, float b, float* in) {
#pragma unroll
  for (int k = 0; k < K; ++k) in[k] = 0.f;
  if (t >= q.hi) return 0.f;
  float v = b;
#pragma unroll
  for (int k = 0; k < K; ++k) {
    in[k] = input_at<Tin, K>(p, q, row0, t - (K - 1) + k, c);
    v = fmaf(w[k], in[k], v);
  }
  const float dy = to_f32(static_cast<const Tin*>(p.dy)[(row0 + t) * p.dim + c]);
  return p.silu ? dy * silu_slope(v) : dy;
}

// One channel a lane, kConvTile tokens of one batch row.
template <typename Tin, int K>
__global__ __launch_bounds__(64) void dwconv_fwd_kernel(ConvParams p, int64_t nblk, int64_t nct) {
  const int64_t id = workgroup<64>();
  const int64_t c = id % nct * 64 + threadIdx.x, b = id / nct / nblk, t0 = id / nct % nblk * kConvTile;
  if (b >= p.batch || c >= p.dim) return;
  const int64_t row0 = b * p.L, t1 = t0 + kConvTile < p.L ? t0 + kConvTile : p.L;
  float w[K], bias;
  load_taps<K>(p, c, w, bias);
  for (int64_t t = t0; t < t1; ++t) {
    const Sequence q = sequence_of(p, b, t);
    float y = 0.f;
    if (t < q.hi) {
      float v = bias;
#pragma unroll
      for (int k = 0; k < K; ++k) v = fmaf(w[k], input_at<Tin, K>(p, q, row0, t - (K - 1) + k, c), v);
      y = p.silu ? silu(v) : v;
    }
    store_val(static_cast<Tin*>(p.y) + (row0 + t) * p.dim + c, y);
  }
}

// The sequence of index s: its place among the rows' tokens.
__device__ __forceinline__ Sequence sequence(const ConvParams& p, int64_t s, int64_t& row0) {
  row0 = 0;
  if (!p.offsets) {
    row0 = s * p.L;
    return {s, 0, p.L};
  }
  const int64_t from = p.offsets[s], to = p.offsets[s + 1];
  const int64_t lo = from < 0 ? 0 : (from > p.L ? p.L : from);
  return {s, lo, to < lo ? lo : (to > p.L ? p.L : to)};
}

template <typename Tin, int K>
__global__ __launch_bounds__(256) void dwconv_last_kernel(ConvParams p) {
  const int64_t id = static_cast<int64_t>(workgroup<256>()) * 256 + threadIdx.x;
  if (id >= p.num_seqs * p.dim) return;
  const int64_t c = id % p.dim;
  int64_t row0;
  const Sequence q = sequence(p, id / p.dim, row0);
#pragma unroll
  for (int j = 0; j < K - 1; ++j) p.h_last[id * (K - 1) + j] = input_at<Tin, K>(p, q, row0, q.hi - (K - 1) + j, c);
}

template <typename Tin, int K>
__global__ __launch_bounds__(64) void dwconv_bwd_kernel(ConvParams p, int64_t nblk, int64_t nct) {
  const int64_t id = workgroup<64>();
  const int64_t c = id % nct * 64 + threadIdx.x, blk = id / nct, b = blk / nblk, t0 = blk % nblk * kConvTile;
  if (b >= p.batch || c >= p.dim) return;
  const int64_t row0 = b * p.L, t1 = t0 + kConvTile < p.L ? t0 + kConvTile : p.L;
  float w[K], bias, dw[K] = {}, db = 0.f;
  load_taps<K>(p, c, w, bias);
  for (int64_t t = t0; t < t1; ++t) {
    const Sequence q = sequence_of(p, b, t);
    float dx = 0.f;
    if (t < q.hi) {
      float in[K];
#pragma unroll
      for (int j = K - 1; j >= 0; --j) dx = fmaf(w[K - 1 - j], dv_at<Tin, K>(p, q, row0, t + j, c, w, bias, in), dx);
      const float dv = dv_at<Tin, K>(p, q, row0, t, c, w, bias, in);
#pragma unroll
      for (int k = 0; k < K; ++k) dw[k] = fmaf(dv, in[k], dw[k]);
      db += dv;
      const int64_t j = t - (q.hi - (K - 1));
      if (K > 1 && p.dlast && j >= 0) dx += p.dlast[(q.s * p.dim + c) * (K - 1) + j];
    }
    store_val(static_cast<Tin*>(p.dx) + (row0 + t) * p.sdx + c, dx);
  }
#pragma unroll
  for (int k = 0; k < K; ++k) p.partial[(blk * p.dim + c) * (K + 1) + k] = dw[k];
  p.partial[(blk * p.dim + c) * (K + 1) + K] = db;
}

template <typename Tin, int K>
__global__ __launch_bounds__(256) void dwconv_dinitial_kernel(ConvParams p) {
  const int64_t id = static_cast<int64_t>(workgroup<256>()) * 256 + threadIdx.x;
  if (id >= p.num_seqs * p.dim) return;
  const int64_t c = id % p.dim;
  int64_t row0;
  const Sequence q = sequence(p, id / p.dim, row0);
  float w[K], bias, in[K];
  load_taps<K>(p, c, w, bias);
#pragma unroll
  for (int i = 0; i < K - 1; ++i) {
    float d = 0.f;
#pragma unroll
    for (int m = 0; m <= i; ++m) d = fmaf(w[i - m], dv_at<Tin, K>(p, q, row0, q.lo + m, c, w, bias, in), d);
    const int64_t j = i - (q.hi - q.lo);
    if (p.dlast && j >= 0) d += p.dlast[id * (K - 1) + j];
    p.dh0[id * (K - 1) + i] = d;
  }
}

template <int K>
__global__ __launch_bounds__(256) void dwconv_param_kernel(ConvParams p, int64_t blocks) {
  const int64_t c = blockIdx.x * int64_t(256) + threadIdx.x;
  if (c >= p.dim) return;
  float sum[K + 1] = {};
  for (int64_t b = 0; b < blocks; ++b)
#pragma unroll
    for (int k = 0; k <= K; ++k) sum[k] += p.partial[(b * p.dim + c) * (K + 1) + k];
#pragma unroll
  for (int k = 0; k < K; ++k) p.dw[c * K + k] = sum[k];
  if (p.db) p.db[c] = sum[K];
}

template <typename Tin, int K>
__global__ __launch_bounds__(64) void dwconv_step_kernel(ConvStepParams p, int64_t nct) {
  const int64_t id = workgroup<64>();
  const int64_t b = id / nct, c = id % nct * 64 + threadIdx.x;
  if (b >= p.batch || c >= p.dim) return;
  const int64_t from = p.slots ? p.slots[b] : b, to = p.slots_out ? p.slots_out[b] : from;
  float y = 0.f;
  if (from >= 0 && from < p.num_slots) {
    float in[K], v = p.b ? p.b[c] : 0.f;
    in[K - 1] = to_f32(static_cast<const Tin*>(p.x)[b * p.sx + c]);
#pragma unroll
    for (int k = 0; k < K - 1; ++k) in[k] = p.state[(from * p.dim + c) * (K - 1) + k];
#pragma unroll
    for (int k = 0; k < K; ++k) v = fmaf(p.w[c * K + k], in[k], v);
    y = p.silu ? silu(v) : v;
    if (to >= 0 && to < p.num_slots) {
#pragma unroll
      for (int k = 0; k < K - 1; ++k) p.state[(to * p.dim + c) * (K - 1) + k] = in[k + 1];
    }
  }
  store_val(static_cast<Tin*>(p.y) + b * p.dim + c, y);
}

namespace {

int64_t blocks_of(int64_t L) { return (L + kConvTile - 1) / kConvTile; }

template <typename Tin, int K>
hipError_t fwd(const ConvParams& p, hipStream_t s) {
  const int64_t nblk = blocks_of(p.L), nct = (p.dim + 63) / 64;
  if (p.batch * nblk > 0)
    hipLaunchKernelGGL((dwconv_fwd_kernel<Tin, K>), grid_of<64>(p.batch * nblk * nct), dim3(64), 0, s, p, nblk, nct);
  if (K > 1 && p.h_last)
    hipLaunchKernelGGL((dwconv_last_kernel<Tin, K>), grid_of<256>((p.num_seqs * p.dim + 255) / 256), dim3(256), 0, s, p);
  return hipGetLastError();
}

template <typename Tin, int K>
hipError_t bwd(const ConvParams& p, hipStream_t s) {
  const int64_t nblk = blocks_of(p.L), nct = (p.dim + 63) / 64;
  if (p.batch * nblk > 0)
    hipLaunchKernelGGL((dwconv_bwd_kernel<Tin, K>), grid_of<64>(p.batch * nblk * nct), dim3(64), 0, s, p, nblk, nct);
  if (K > 1 && p.dh0 && p.num_seqs > 0)
    hipLaunchKernelGGL((dwconv_dinitial_kernel<Tin, K>), grid_of<256>((p.num_seqs * p.dim + 255) / 256), dim3(256), 0, s, p);
  hipLaunchKernelGGL((dwconv_param_kernel<K>), dim3((p.dim + 255) / 256), dim3(256), 0, s, p, p.batch * nblk);
  return hipGetLastError();
}

template <typename Tin, int K>
hipError_t step(const ConvStepParams& p, hipStream_t s) {
  const int64_t nct = (p.dim + 63) / 64;
  hipLaunchKernelGGL((dwconv_step_kernel<Tin, K>), grid_of<64>(p.batch * nct), dim3(64), 0, s, p, nct);
  return hipGetLastError();
}

}  // namespace

size_t dwconv_bwd_workspace_bytes(int64_t batch, int64_t L, int64_t dim, int taps) {
  return static_cast<size_t>(batch) * blocks_of(L) * dim * (taps + 1) * 4;
}

#define SSCAN_BY_TAPS(call)                                          \
  switch (taps) {                                                    \
    case 1: return bf16 ? call<bf16_t, 1>(p, s) : call<float, 1>(p, s); \
    case 2: return bf16 ? call<bf16_t, 2>(p, s) : call<float, 2>(p, s); \
    case 3: return bf16 ? call<bf16_t, 3>(p, s) : call<float, 3>(p, s); \
    default: return bf16 ? call<bf16_t, 4>(p, s) : call<float, 4>(p, s); \
  }

hipError_t launch_dwconv_fwd(const ConvParams& p, int taps, bool bf16, hipStream_t s) { SSCAN_BY_TAPS(fwd) }
hipError_t launch_dwconv_bwd(const ConvParams& p, int taps, bool bf16, hipStream_t s) { SSCAN_BY_TAPS(bwd) }
hipError_t launch_dwconv_step(const ConvStepParams& p, int taps, bool bf16, hipStream_t s) { SSCAN_BY_TAPS(step) }

}  // namespace sscan
