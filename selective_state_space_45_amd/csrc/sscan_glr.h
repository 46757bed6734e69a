// The gated linear recurrence and 8-bit activations: parameters and device arithmetic
// shared by their kernels.  The operations are defined in include/selscan.h.
#pragma once

#include "sscan_device.h"

namespace sscan {

constexpr int kGlrBlock = 64;   // tokens between saved states (SSCAN_GLR_BLOCK)
constexpr int kActGroup = 16;   // tokens that share a power of two (SSCAN_ACT8_GROUP)

struct GlrFwdParams {
  const void* x;
  const void* r;
  const void* i;
  const void* z;            // nullable
  int64_t sx, sr, si, sz;   // token strides in elements
  const float* lam;
  const float* r_bias;      // nullable
  const float* i_bias;      // nullable
  float decay_scale;
  const float* h0;          // nullable: [sequences][dim]
  const int32_t* offsets;   // nullable: [num_seqs + 1]
  void* y;
  float* h_last;            // nullable
  float* ckpt;              // nullable: [batch][ceil(L / kGlrBlock)][dim]
  int8_t* codes;            // nullable: saved activations, one packed tensor after another
  size_t saved_stride;      // bytes from one packed tensor to the next
  size_t exps_at;           // bytes from a packed tensor's codes to its exponents
  void* workspace;
  int64_t batch, L, dim, num_seqs;
};

struct GlrBwdParams {
  const void* x;            // x, r, i, z null when the activations come from `codes`
  const void* r;
  const void* i;
  const void* z;
  int64_t sx, sr, si, sz;
  const int8_t* codes;      // nullable
  size_t saved_stride, exps_at;
  const float* lam;
  const float* r_bias;
  const float* i_bias;
  float decay_scale;
  const float* h0;          // nullable, read with offsets only
  const int32_t* offsets;   // nullable
  const float* ckpt;
  const void* dy;
  const float* dlast;       // nullable
  void* dx;
  void* dr;
  void* di;
  void* dz;                 // nullable
  int64_t gx, gr, gi, gz;   // token strides of the gradients
  float* dlam;
  float* dr_bias;           // nullable
  float* di_bias;           // nullable
  float* dh0;               // nullable
  void* workspace;
  int64_t batch, L, dim, num_seqs;
};

struct GlrStepParams {
  float* state;
  int64_t num_slots;
  const int32_t* slots;     // nullable
  const int32_t* slots_out; // nullable
  const void* x;
  const void* r;
  const void* i;
  const void* z;            // nullable
  int64_t sx, sr, si, sz;
  const float* lam;
  const float* r_bias;
  const float* i_bias;
  float decay_scale;
  void* y;
  int64_t batch, dim;
};

hipError_t launch_glr_fwd(const GlrFwdParams& p, bool bf16, hipStream_t s);
hipError_t launch_glr_bwd(const GlrBwdParams& p, bool bf16, hipStream_t s);
hipError_t launch_glr_step(const GlrStepParams& p, bool bf16, hipStream_t s);
hipError_t launch_act8_pack(const void* x, int64_t stride, void* packed, int64_t batch, int64_t L, int64_t dim,
                            bool bf16, hipStream_t s);
hipError_t launch_act8_unpack(const void* packed, void* x, int64_t batch, int64_t L, int64_t dim, bool bf16,
                              hipStream_t s);
size_t glr_fwd_workspace_bytes(int64_t batch, int64_t L, int64_t dim);
size_t glr_bwd_workspace_bytes(int64_t batch, int64_t L, int64_t dim);

// Sizes of one packed tensor: codes, padded to 256 bytes, then exponents.
inline size_t act8_exps_at(int64_t batch, int64_t L, int64_t dim) {
  return (static_cast<size_t>(batch) * L * dim + 255) & ~size_t(255);
}
inline size_t act8_total(int64_t batch, int64_t L, int64_t dim) {
  const size_t exps = static_cast<size_t>(batch) * ((L + kActGroup - 1) / kActGroup) * dim;
  return act8_exps_at(batch, L, dim) + ((exps + 255) & ~size_t(255));
}

// Grids.  HIP counts a launch's threads along an axis in 32 bits, so workgroups of THREADS
// beyond 2^31 threads go on in further rows of the grid; the last row is filled up with
// workgroups past the number asked for, which end at once.
template <int THREADS>
constexpr uint32_t kGridRow = (uint32_t(1) << 31) / THREADS;
template <int THREADS>
inline dim3 grid_of(int64_t n) {
  constexpr int64_t row = kGridRow<THREADS>;
  return n <= row ? dim3(static_cast<unsigned>(n)) : dim3(static_cast<unsigned>(row), static_cast<unsigned>((n + row - 1) / row));
}
template <int THREADS>
__device__ __forceinline__ uint32_t workgroup() { return blockIdx.y * kGridRow<THREADS> + blockIdx.x; }

// sigmoid(v) = 1 / (1 + e^-v).  e^-v overflows to infinity for v below -88, whose
// reciprocal is the right 0.
__device__ __forceinline__ float sigmoid(float v) { return hw_rcp(1.f + hw_exp2(-v * kLog2e)); }
// sigmoid(v + bias) given nb = -bias log2(e).
__device__ __forceinline__ float gate(float v, float nb) { return hw_rcp(1.f + hw_exp2(fmaf(v, -kLog2e, nb))); }

// The derivative s (1 - s) of a sigmoid that is s: off by at most 2^-24 (of its largest
// value, 1/4) where s is close to 1.
__device__ __forceinline__ float slope(float s) { return fmaf(-s, s, s); }

// softplus(v) = max(v, 0) + log(1 + w), w = e^-|v|: log(1 + w) = 2 atanh(s),
// s = w / (2 + w) <= 1/3, by its odd series through s^15 (the next term is below 2e-9 of the
// sum).  The product |v| log2(e) has a rounding error that grows with |v| (62 units of w's
// last place at v = -80); what it lacks, with the low part of log2(e) itself, is put back
// into w to first order, and w keeps a relative error of about three units down to
// v = -87, below which it is zero.  |v| is bounded for the infinities' sake.
__device__ __forceinline__ float softplus_acc(float v) {
  constexpr float log2e_low = 1.92596299e-8f;   // log2(e) - kLog2e
  const float av = fminf(fabsf(v), 128.f), t = av * kLog2e;
  const float lack = fmaf(av, log2e_low, fmaf(av, kLog2e, -t));
  float w = hw_exp2(-t);
  w = fmaf(w, -kLn2 * lack, w);
  const float s = w * hw_rcp(2.f + w);
  const float s2 = s * s;
  float p = fmaf(s2, 1.f / 15.f, 1.f / 13.f);
  p = fmaf(s2, p, 1.f / 11.f);
  p = fmaf(s2, p, 1.f / 9.f);
  p = fmaf(s2, p, 1.f / 7.f);
  p = fmaf(s2, p, 1.f / 5.f);
  p = fmaf(s2, p, 1.f / 3.f);
  p = fmaf(s2, p, 1.f);
  return (v > 0.f ? v : (v <= 0.f ? 0.f : v)) + 2.f * s * p;
}

// a = e^-q and 1 - a^2 for q >= 0, given q log2(e).  1 - a^2 loses its leading digits for
// a near 1, so for q < 1/4 it is 2 a sinh(q) with sinh by its series through q^5 (the next
// term is below 5e-8 of it there); elsewhere a^2 < 0.61 and the difference is exact enough.
__device__ __forceinline__ float decay_of(float q2, float& one_minus_a2) {
  constexpr float c1 = 2.f * kLn2, c3 = c1 * kLn2 * kLn2 / 6.f, c5 = c3 * kLn2 * kLn2 / 20.f;
  const float a = hw_exp2(-q2);
  const float s = q2 * q2;
  const float near1 = a * (q2 * fmaf(s, fmaf(s, c5, c3), c1));
  const float far = fmaf(-a, a, 1.f);
  one_minus_a2 = q2 < 0.25f * kLog2e ? near1 : far;
  return a;
}

__device__ __forceinline__ float hw_sqrt(float v) { return __builtin_amdgcn_sqrtf(v); }

// 8-bit codes.  `field` is the float32 exponent field (0 .. 255) of the group's largest
// magnitude; 255 marks a group with an infinity or NaN.  Scaling by powers of two is
// exact (ldexp reaches every exponent a field asks for), so the only rounding is to the
// whole number.
__device__ __forceinline__ int act8_shift(uint32_t field) { return (field < 1u ? 1 : static_cast<int>(field)) - 133; }
// A code, in the low byte.  Adding 1.5 x 2^23 rounds to the whole number (ties to even)
// and leaves it in the low bits.
__device__ __forceinline__ uint32_t act8_code(float v, int shift) {
  constexpr float k = 12582912.f;
  return __float_as_uint(__builtin_amdgcn_fmed3f(__builtin_amdgcn_ldexpf(v, -shift) + k, k - 127.f, k + 127.f));
}
__device__ __forceinline__ float act8_value(int code, uint32_t field) {
  const float v = __builtin_amdgcn_ldexpf(static_cast<float>(code), act8_shift(field));
  return field == 255u ? __uint_as_float(0x7fc00000u) : v;
}
// max |v| that keeps NaN: a NaN's magnitude bits are above infinity's.
__device__ __forceinline__ uint32_t act8_top(uint32_t top, float v) {
  const uint32_t m = __float_as_uint(v) & 0x7fffffffu;
  return m > top ? m : top;
}

}  // namespace sscan
