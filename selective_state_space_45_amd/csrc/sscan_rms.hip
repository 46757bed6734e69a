// Root-mean-square norm with the residual's addition, its backward pass, and rows in 8 bits.
#include "sscan_layer.h"

namespace sscan {

constexpr int kRowLanes = 1024;                       // lanes of a row
constexpr int kRowWords = 65536 / kRowLanes;          // channels of a lane
constexpr int kRmsGroups = 256;                       // workgroups of a backward pass

// Sum, and maximum of magnitude bits (which keeps NaN), over the workgroup.
__device__ __forceinline__ float sum_all(float v, float* lds) {
#pragma unroll
  for (int d = 32; d; d >>= 1) v += __shfl_xor(v, d);
  __syncthreads();
  if ((threadIdx.x & 63) == 0) lds[threadIdx.x >> 6] = v;
  __syncthreads();
  float s = 0.f;
#pragma unroll
  for (int w = 0; w < kRowLanes / 64; ++w) s += lds[w];
  return s;
}
__device__ __forceinline__ uint32_t top_all(uint32_t v, uint32_t* lds) {
#pragma unroll
  for (int d = 32; d; d >>= 1) {
    const uint32_t o = __shfl_xor(v, d);
    v = o > v ? o : v;
  }
  __syncthreads();
  if ((threadIdx.x & 63) == 0) lds[threadIdx.x >> 6] = v;
  __syncthreads();
  uint32_t s = 0;
#pragma unroll
  for (int w = 0; w < kRowLanes / 64; ++w) s = lds[w] > s ? lds[w] : s;
  return s;
}

template <typename T>
__device__ __forceinline__ float rounded(float v) {
  T t;
  store_val(&t, v);
  return to_f32(t);
}

// One workgroup a row, its channels in registers.  NORM: the norm; otherwise the row as it is.
template <typename Tin, typename Tres, bool NORM>
__global__ __launch_bounds__(kRowLanes) void rms_fwd_kernel(RmsFwdParams p) {
  __shared__ float lds[kRowLanes / 64];
  const int64_t row = workgroup<kRowLanes>();
  if (row >= p.rows) return;
  float v[kRowWords], sum = 0.f;
#pragma unroll
  for (int k = 0; k < kRowWords; ++k) {
    const int c = k * kRowLanes + threadIdx.x;
    v[k] = 0.f;
    if (c >= p.dim) continue;
    v[k] = to_f32(static_cast<const Tin*>(p.x)[row * p.sx + c]);
    if (!NORM) continue;
    if (p.residual) v[k] += to_f32(static_cast<const Tres*>(p.residual)[row * p.dim + c]);
    v[k] = rounded<Tres>(v[k]);
    if (p.kept) store_val(static_cast<Tres*>(p.kept) + row * p.dim + c, v[k]);
    sum = fmaf(v[k], v[k], sum);
  }
  uint32_t top = 0;
  if (NORM) {
    const float r = rsqrtf(sum_all(sum, lds) / p.dim + p.eps);
#pragma unroll
    for (int k = 0; k < kRowWords; ++k) {
      const int c = k * kRowLanes + threadIdx.x;
      if (c >= p.dim) continue;
      v[k] = v[k] * r * (p.weight ? p.weight[c] : 1.f);
      if (p.y) store_val(static_cast<Tin*>(p.y) + row * p.dim + c, v[k]);
    }
  }
  if (!p.codes) return;
#pragma unroll
  for (int k = 0; k < kRowWords; ++k) top = act8_top(top, v[k]);
  top = top_all(top, reinterpret_cast<uint32_t*>(lds));
  const bool fine = top < 0x7f800000u;
  const float scale = i8_scale(__uint_as_float(top)), inv = 1.f / scale;
  if (threadIdx.x == 0) p.scales[row] = fine ? scale : __uint_as_float(0x7fc00000u);
#pragma unroll
  for (int k = 0; k < kRowWords; ++k) {
    const int c = k * kRowLanes + threadIdx.x;
    if (c < p.dim) p.codes[row * p.sc + c] = fine ? static_cast<int8_t>(i8_code(v[k], scale, inv)) : 0;
  }
}

// Workgroup g takes rows g, g + groups, ... and sums its rows' part of dweight.
template <typename Tin, typename Tres>
__global__ __launch_bounds__(kRowLanes) void rms_bwd_kernel(RmsBwdParams p) {
  __shared__ float lds[kRowLanes / 64];
  float dw[kRowWords] = {};
  for (int64_t row = blockIdx.x; row < p.rows; row += gridDim.x) {
    const Tres* s = static_cast<const Tres*>(p.s) + row * p.ss;
    const Tin* dy = static_cast<const Tin*>(p.dy) + row * p.dim;
    float ssum = 0.f, gsum = 0.f;
    for (int c = threadIdx.x; c < p.dim; c += kRowLanes) {
      const float v = to_f32(s[c]), g = to_f32(dy[c]) * (p.weight ? p.weight[c] : 1.f);
      ssum = fmaf(v, v, ssum);
      gsum = fmaf(g, v, gsum);
    }
    const float r = rsqrtf(sum_all(ssum, lds) / p.dim + p.eps);
    const float mean = sum_all(gsum, lds) * r / p.dim;
#pragma unroll
    for (int k = 0; k < kRowWords; ++k) {
      const int c = k * kRowLanes + threadIdx.x;
      if (c >= p.dim) continue;
      const float n = to_f32(s[c]) * r, d = to_f32(dy[c]);
      dw[k] = fmaf(d, n, dw[k]);
      float out = r * (d * (p.weight ? p.weight[c] : 1.f) - n * mean);
      if (p.dkept) out += to_f32(static_cast<const Tres*>(p.dkept)[row * p.dim + c]);
      if (p.dx) store_val(static_cast<Tin*>(p.dx) + row * p.sdx + c, out);
      if (p.dresidual) store_val(static_cast<Tres*>(p.dresidual) + row * p.dim + c, out);
    }
  }
  if (!p.dweight) return;
#pragma unroll
  for (int k = 0; k < kRowWords; ++k) {
    const int c = k * kRowLanes + threadIdx.x;
    if (c < p.dim) p.partial[static_cast<int64_t>(blockIdx.x) * p.dim + c] = dw[k];
  }
}

__global__ __launch_bounds__(256) void rms_weight_kernel(const float* partial, float* dweight, int groups, int dim) {
  const int c = blockIdx.x * 256 + threadIdx.x;
  if (c >= dim) return;
  float sum = 0.f;
  for (int g = 0; g < groups; ++g) sum += partial[static_cast<int64_t>(g) * dim + c];
  dweight[c] = sum;
}

namespace {

int groups_of(int64_t rows) { return rows < kRmsGroups ? static_cast<int>(rows) : kRmsGroups; }

template <typename Tin, typename Tres, bool NORM>
hipError_t fwd(const RmsFwdParams& p, hipStream_t s) {
  hipLaunchKernelGGL((rms_fwd_kernel<Tin, Tres, NORM>), grid_of<kRowLanes>(p.rows), dim3(kRowLanes), 0, s, p);
  return hipGetLastError();
}

template <typename Tin, typename Tres>
hipError_t bwd(const RmsBwdParams& p, hipStream_t s) {
  const int groups = groups_of(p.rows);
  if (groups > 0) hipLaunchKernelGGL((rms_bwd_kernel<Tin, Tres>), dim3(groups), dim3(kRowLanes), 0, s, p);
  if (p.dweight)
    hipLaunchKernelGGL(rms_weight_kernel, dim3((p.dim + 255) / 256), dim3(256), 0, s, p.partial, p.dweight, groups, p.dim);
  return hipGetLastError();
}

}  // namespace

size_t rms_bwd_workspace_bytes(int64_t rows, int64_t dim) { return static_cast<size_t>(groups_of(rows)) * dim * 4; }

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
