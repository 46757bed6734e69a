// Gated linear recurrence, forward: one lane per (sequence, channel), token after token.
#include "sscan_glr.h"

namespace sscan {

template <typename Tin>
__global__ __launch_bounds__(256) void glr_fwd_kernel(GlrFwdParams p) {
  const int64_t id = static_cast<int64_t>(blockIdx.x) * 256 + threadIdx.x;
  const int64_t nseq = p.offsets ? p.num_seqs : p.batch;
  if (id >= nseq * p.dim) return;
  const int64_t s = id / p.dim, d = id - s * p.dim;
  int64_t lo = s * p.L, hi = lo + p.L, row0 = lo;
  if (p.offsets) {
    lo = p.offsets[s], hi = p.offsets[s + 1], row0 = 0;
    lo = lo < 0 ? 0 : lo;
    hi = hi > p.L ? p.L : hi;
  }
  const float kappa = p.decay_scale * softplus_acc(p.lam[d]);
  const float rb = p.r_bias ? p.r_bias[d] : 0.f, ib = p.i_bias ? p.i_bias[d] : 0.f;
  const Tin* x = static_cast<const Tin*>(p.x);
  const Tin* r = static_cast<const Tin*>(p.r);
  const Tin* in = static_cast<const Tin*>(p.i);
  const Tin* z = static_cast<const Tin*>(p.z);
  Tin* y = static_cast<Tin*>(p.y);
  const int64_t nblk = (p.L + kGlrBlock - 1) / kGlrBlock;
  float h = p.h0 ? p.h0[id] : 0.f;
  for (int64_t t = lo; t < hi; ++t) {
    if (p.ckpt && (t - row0) % kGlrBlock == 0) p.ckpt[((p.offsets ? 0 : s) * nblk + (t - row0) / kGlrBlock) * p.dim + d] = h;
    const float rho = sigmoid(to_f32(r[t * p.sr + d]) + rb);
    const float iota = sigmoid(to_f32(in[t * p.si + d]) + ib);
    float v;
    const float a = decay_of(kappa * rho, v);
    h = fmaf(a, h, hw_sqrt(v) * (iota * to_f32(x[t * p.sx + d])));
    store_val(&y[t * p.dim + d], z ? h * silu(to_f32(z[t * p.sz + d])) : h);
  }
  if (p.h_last) p.h_last[id] = h;
}

// Zeros at the padding of a packed batch, and 8-bit codes of the saved activations.
template <typename Tin>
__global__ __launch_bounds__(256) void glr_pad_kernel(Tin* y, const int32_t* offsets, int64_t num_seqs, int64_t L,
                                                      int64_t dim) {
  int64_t lo = offsets[num_seqs];
  lo = lo < 0 ? 0 : lo;
  for (int64_t e = lo * dim + static_cast<int64_t>(blockIdx.x) * 256 + threadIdx.x; e < L * dim; e += 256ll * gridDim.x)
    store_val(&y[e], 0.f);
}

template <typename Tin>
__global__ __launch_bounds__(256) void glr_save_kernel(const Tin* x, int64_t stride, int8_t* codes, uint8_t* exps,
                                                       const int32_t* offsets, int64_t num_seqs, int64_t batch,
                                                       int64_t L, int64_t dim) {
  const int64_t id = static_cast<int64_t>(blockIdx.x) * 256 + threadIdx.x;
  const int64_t ngrp = (L + kActGroup - 1) / kActGroup;
  if (id >= batch * ngrp * dim) return;
  const int64_t d = id % dim, g = id / dim % ngrp, b = id / dim / ngrp;
  int64_t used = L;
  if (offsets) used = offsets[num_seqs] < L ? offsets[num_seqs] : L;
  float v[kActGroup];
  uint32_t top = 0;
  for (int k = 0; k < kActGroup; ++k) {
    const int64_t t = g * kActGroup + k;
    v[k] = t < used ? to_f32(x[(b * L + t) * stride + d]) : 0.f;
    top = act8_top(top, v[k]);
  }
  const uint32_t field = top >> 23;
  exps[id] = static_cast<uint8_t>(field);
  for (int k = 0; k < kActGroup; ++k)
    if (g * kActGroup + k < L) codes[(b * L + g * kActGroup + k) * dim + d] = static_cast<int8_t>(act8_code(v[k], act8_shift(field)));
}

namespace {

unsigned blocks(int64_t n) { return static_cast<unsigned>((n + 255) / 256); }

template <typename Tin>
void launch(const GlrFwdParams& p, hipStream_t s) {
  const int64_t nseq = p.offsets ? p.num_seqs : p.batch;
  if (nseq > 0) hipLaunchKernelGGL((glr_fwd_kernel<Tin>), dim3(blocks(nseq * p.dim)), dim3(256), 0, s, p);
  if (p.offsets && p.L > 0)
    hipLaunchKernelGGL((glr_pad_kernel<Tin>), dim3(256), dim3(256), 0, s, static_cast<Tin*>(p.y), p.offsets, p.num_seqs,
                       p.L, p.dim);
  if (p.codes && p.L > 0) {
    const void* src[4] = {p.x, p.r, p.i, p.z};
    const int64_t stride[4] = {p.sx, p.sr, p.si, p.sz};
    const int64_t n = p.batch * ((p.L + kActGroup - 1) / kActGroup) * p.dim;
    for (int k = 0; k < (p.z ? 4 : 3); ++k) {
      int8_t* codes = p.codes + k * p.saved_stride;
      hipLaunchKernelGGL((glr_save_kernel<Tin>), dim3(blocks(n)), dim3(256), 0, s, static_cast<const Tin*>(src[k]),
                         stride[k], codes, reinterpret_cast<uint8_t*>(codes) + p.exps_at, p.offsets, p.num_seqs,
                         p.batch, p.L, p.dim);
    }
  }
}

}  // namespace

hipError_t launch_glr_fwd(const GlrFwdParams& p, bool bf16, hipStream_t s) {
  if (bf16) launch<bf16_t>(p, s);
  else launch<float>(p, s);
  return hipGetLastError();
}

hipError_t launch_act8_pack(const void* x, int64_t stride, void* packed, int64_t batch, int64_t L, int64_t dim,
                            bool bf16, hipStream_t s) {
  int8_t* codes = static_cast<int8_t*>(packed);
  uint8_t* exps = static_cast<uint8_t*>(packed) + act8_exps_at(batch, L, dim);
  const unsigned nb = blocks(batch * ((L + kActGroup - 1) / kActGroup) * dim);
  if (bf16)
    hipLaunchKernelGGL((glr_save_kernel<bf16_t>), dim3(nb), dim3(256), 0, s, static_cast<const bf16_t*>(x), stride, codes,
                       exps, nullptr, int64_t(0), batch, L, dim);
  else
    hipLaunchKernelGGL((glr_save_kernel<float>), dim3(nb), dim3(256), 0, s, static_cast<const float*>(x), stride, codes,
                       exps, nullptr, int64_t(0), batch, L, dim);
  return hipGetLastError();
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
