// What stands around the recurrence in a layer -- norm, 8-bit rows and their products, short
// convolution: parameters and launchers.  The operations are defined in include/selscan.h.
#pragma once

#include "sscan_glr.h"

namespace sscan {

struct RmsFwdParams {
  const void* x;
  int64_t sx;
  const void* residual;   // nullable
  const float* weight;    // nullable
  float eps;
  void* y;                // nullable
  void* kept;             // nullable
  int8_t* codes;          // nullable, with scales
  int64_t sc;
  float* scales;
  int64_t rows;
  int dim;
};

struct RmsBwdParams {
  const void* s;
  int64_t ss;
  const float* weight;    // nullable
  float eps;
  const void* dy;
  const void* dkept;      // nullable
  void* dx;               // nullable
  int64_t sdx;
  void* dresidual;        // nullable
  float* dweight;         // nullable
  float* partial;         // [rms_bwd_groups(rows)][dim], with dweight
  int64_t rows;
  int dim;
};

struct MatmulParams {
  const int8_t* a;
  const int8_t* b;
  int64_t sa, sb;
  const float* as;
  const float* bs;
  const float* bias;      // nullable
  void* out;
  int64_t so;
  int m, n, k;
};

struct ConvParams {
  const void* x;
  int64_t sx;
  const float* w;
  const float* b;         // nullable
  const float* h0;        // nullable: [sequences][dim][taps - 1]
  const int32_t* offsets; // nullable
  void* y;                // forward
  float* h_last;          // forward, nullable
  const void* dy;         // backward from here on
  const float* dlast;     // nullable
  void* dx;
  int64_t sdx;
  float* dw;
  float* db;              // nullable
  float* dh0;             // nullable
  float* partial;
  int64_t batch, L, dim, num_seqs;   // num_seqs: the batch's rows without offsets
  bool silu;
};

struct ConvStepParams {
  float* state;
  int64_t num_slots;
  const int32_t* slots;
  const int32_t* slots_out;
  const void* x;
  int64_t sx;
  const float* w;
  const float* b;
  void* y;
  int64_t batch, dim;
  bool silu;
};

hipError_t launch_rms_fwd(const RmsFwdParams& p, bool bf16, bool kept_bf16, hipStream_t s);
hipError_t launch_rms_bwd(const RmsBwdParams& p, bool bf16, bool kept_bf16, hipStream_t s);
hipError_t launch_i8_quant(const RmsFwdParams& p, bool bf16, hipStream_t s);
hipError_t launch_i8_matmul(const MatmulParams& p, bool bf16, hipStream_t s);
hipError_t launch_dwconv_fwd(const ConvParams& p, int taps, bool bf16, hipStream_t s);
hipError_t launch_dwconv_bwd(const ConvParams& p, int taps, bool bf16, hipStream_t s);
hipError_t launch_dwconv_step(const ConvStepParams& p, int taps, bool bf16, hipStream_t s);
size_t rms_bwd_workspace_bytes(int64_t rows, int64_t dim);
size_t dwconv_bwd_workspace_bytes(int64_t batch, int64_t L, int64_t dim, int taps);

// 8-bit rows.  The scale is the float32 number nearest to top / 127 (a correctly rounded
// division, once a row), so codes are defined bit for bit.
__device__ __forceinline__ float i8_scale(float top) { return fmaxf(__fdiv_rn(top, 127.f), 0x1p-126f); }

// The whole number nearest to the real quotient v / scale, ties to even, given the
// float32 reciprocal `inv` of scale.  v inv is off by a few units of its last place, which
// decides wrongly at most between two neighbours; the remainder v - c scale is exact in
// one fused step and says which (|remainder| against half the scale, the tie by c's parity).
__device__ __forceinline__ float i8_code(float v, float scale, float inv) {
  float c = rintf(v * inv);
  const float rem = fmaf(-c, scale, v), half = 0.5f * scale;
  const bool odd = (static_cast<int>(c) & 1) != 0;
  if (rem > half || (rem == half && odd)) c += 1.f;
  else if (rem < -half || (rem == -half && odd)) c -= 1.f;
  return c;
}

}  // namespace sscan
