// Gated linear recurrence, backward: one lane per channel, the sequences in turn, the
// blocks of tokens in reverse, each recomputed forward from the state saved at its start.
#include "sscan_glr.h"

namespace sscan {

template <typename Tin>
struct GlrTokens {
  const GlrBwdParams& p;
  int64_t d;
  __device__ float at(const void* q, int64_t stride, int k, int64_t t) const {
    if (!p.codes) return to_f32(static_cast<const Tin*>(q)[t * stride + d]);
    const int8_t* codes = p.codes + k * p.saved_stride;
    const uint8_t* exps = reinterpret_cast<const uint8_t*>(codes) + p.exps_at;
    const int64_t b = t / p.L, l = t - b * p.L;
    const int64_t ngrp = (p.L + kActGroup - 1) / kActGroup;
    return act8_value(codes[t * p.dim + d], exps[(b * ngrp + l / kActGroup) * p.dim + d]);
  }
};

template <typename Tin>
__global__ __launch_bounds__(256) void glr_bwd_kernel(GlrBwdParams p) {
  const int64_t d = static_cast<int64_t>(blockIdx.x) * 256 + threadIdx.x;
  if (d >= p.dim) return;
  const int64_t nseq = p.offsets ? p.num_seqs : p.batch;
  const int64_t nblk = (p.L + kGlrBlock - 1) / kGlrBlock;
  const float lam = p.lam[d];
  const float kappa = p.decay_scale * softplus_acc(lam);
  const float rb = p.r_bias ? p.r_bias[d] : 0.f, ib = p.i_bias ? p.i_bias[d] : 0.f;
  const GlrTokens<Tin> in{p, d};
  float slam = 0.f, srb = 0.f, sib = 0.f;
  float hp[kGlrBlock];
  for (int64_t s = 0; s < nseq; ++s) {
  const int64_t id = s * p.dim + d;
  int64_t lo = s * p.L, hi = lo + p.L, row0 = lo;
  if (p.offsets) {
    lo = p.offsets[s], hi = p.offsets[s + 1], row0 = 0;
    lo = lo < 0 ? 0 : lo;
    hi = hi > p.L ? p.L : hi;
  }
  float g = p.dlast ? p.dlast[id] : 0.f;   // the gradient that reaches the state after a token
  for (int64_t end = hi; end > lo;) {
    int64_t begin = row0 + (end - 1 - row0) / kGlrBlock * kGlrBlock;
    float h;
    if (p.offsets && begin <= lo) {
      begin = lo;
      h = p.h0 ? p.h0[id] : 0.f;
    } else {
      h = p.ckpt[((p.offsets ? 0 : s) * nblk + (begin - row0) / kGlrBlock) * p.dim + d];
    }
    for (int64_t t = begin; t < end; ++t) {
      hp[t - begin] = h;
      const float rho = sigmoid(in.at(p.r, p.sr, 1, t) + rb), iota = sigmoid(in.at(p.i, p.si, 2, t) + ib);
      float v;
      const float a = decay_of(kappa * rho, v);
      h = fmaf(a, h, hw_sqrt(v) * (iota * in.at(p.x, p.sx, 0, t)));
    }
    for (int64_t t = end - 1; t >= begin; --t) {
      const float x = in.at(p.x, p.sx, 0, t);
      float drho, diota, v;
      const float rho = sigmoid_d(in.at(p.r, p.sr, 1, t) + rb, drho), iota = sigmoid_d(in.at(p.i, p.si, 2, t) + ib, diota);
      const float a = decay_of(kappa * rho, v);
      const float rm = rsq_or_0(v), m = v * rm, u = iota * x;
      const float hb = hp[t - begin];
      float gy = to_f32(static_cast<const Tin*>(p.dy)[t * p.dim + d]);
      if (p.dz) {
        const float z = in.at(p.z, p.sz, 3, t);
        float dsz;
        const float sz = sigmoid_d(z, dsz);
        store_val(&static_cast<Tin*>(p.dz)[t * p.gz + d], gy * fmaf(a, hb, m * u) * fmaf(z, dsz, sz));
        gy *= z * sz;
      }
      g += gy;
      const float dla = g * (a * hb - u * (a * a) * rm);
      const float du = g * m;
      const float dr = -kappa * dla * drho, di = du * x * diota;
      store_val(&static_cast<Tin*>(p.dx)[t * p.gx + d], du * iota);
      store_val(&static_cast<Tin*>(p.dr)[t * p.gr + d], dr);
      store_val(&static_cast<Tin*>(p.di)[t * p.gi + d], di);
      slam = fmaf(dla, rho, slam);
      srb += dr;
      sib += di;
      g *= a;
    }
    end = begin;
  }
  if (p.dh0) p.dh0[id] = g;
  }
  p.dlam[d] = -p.decay_scale * sigmoid(lam) * slam;
  if (p.dr_bias) p.dr_bias[d] = srb;
  if (p.di_bias) p.di_bias[d] = sib;
}

template <typename Tin>
__global__ __launch_bounds__(256) void glr_bwd_pad_kernel(GlrBwdParams p) {
  int64_t lo = p.offsets[p.num_seqs];
  lo = lo < 0 ? 0 : lo;
  for (int64_t e = lo * p.dim + static_cast<int64_t>(blockIdx.x) * 256 + threadIdx.x; e < p.L * p.dim;
       e += 256ll * gridDim.x) {
    const int64_t t = e / p.dim, d = e - t * p.dim;
    store_val(&static_cast<Tin*>(p.dx)[t * p.gx + d], 0.f);
    store_val(&static_cast<Tin*>(p.dr)[t * p.gr + d], 0.f);
    store_val(&static_cast<Tin*>(p.di)[t * p.gi + d], 0.f);
    if (p.dz) store_val(&static_cast<Tin*>(p.dz)[t * p.gz + d], 0.f);
  }
}

namespace {
template <typename Tin>
void launch(const GlrBwdParams& p, hipStream_t s) {
  hipLaunchKernelGGL((glr_bwd_kernel<Tin>), dim3(static_cast<unsigned>((p.dim + 255) / 256)), dim3(256), 0, s, p);
  if (p.offsets && p.L > 0) hipLaunchKernelGGL((glr_bwd_pad_kernel<Tin>), dim3(256), dim3(256), 0, s, p);
}
}  // namespace

hipError_t launch_glr_bwd(const GlrBwdParams& p, bool bf16, hipStream_t s) {
  if (bf16) launch<bf16_t>(p, s);
  else launch<float>(p, s);
  return hipGetLastError();
}

size_t glr_bwd_workspace_bytes(int64_t, int64_t, int64_t) { return 0; }

}  // namespace sscan
