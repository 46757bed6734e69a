// Gated linear recurrence, one token per row against a pool of states.
#include "sscan_glr.h"

namespace sscan {

// One lane per (row, channel).  A token moves 8 bytes of state a channel besides its
// inputs and output, so the kernel is bound by memory at large batches and by its launch
// at small ones; nothing is shared between channels.
template <typename Tin>
__global__ __launch_bounds__(256) void glr_step_kernel(GlrStepParams p) {
  const int64_t id = static_cast<int64_t>(blockIdx.x) * 256 + threadIdx.x;
  if (id >= p.batch * p.dim) return;
  const int64_t b = id / p.dim, d = id - b * p.dim;
  Tin* y = static_cast<Tin*>(p.y);
  const int64_t slot = p.slots ? p.slots[b] : b;
  if (slot < 0 || slot >= p.num_slots) {
    store_val(&y[id], 0.f);
    return;
  }
  const int64_t to = p.slots_out ? p.slots_out[b] : slot;
  const float rate = p.decay_scale * softplus_acc(p.lam[d]) * kLog2e;
  const float rho = gate(to_f32(static_cast<const Tin*>(p.r)[b * p.sr + d]), p.r_bias ? -kLog2e * p.r_bias[d] : 0.f);
  const float iota = gate(to_f32(static_cast<const Tin*>(p.i)[b * p.si + d]), p.i_bias ? -kLog2e * p.i_bias[d] : 0.f);
  float v;
  const float a = decay_of(rate * rho, v);
  const float h = fmaf(a, p.state[slot * p.dim + d], hw_sqrt(v) * (iota * to_f32(static_cast<const Tin*>(p.x)[b * p.sx + d])));
  if (to >= 0 && to < p.num_slots) p.state[to * p.dim + d] = h;
  store_val(&y[id], p.z ? h * silu(to_f32(static_cast<const Tin*>(p.z)[b * p.sz + d])) : h);
}

hipError_t launch_glr_step(const GlrStepParams& p, bool bf16, hipStream_t s) {
  const unsigned nb = static_cast<unsigned>((p.batch * p.dim + 255) / 256);
  if (bf16) hipLaunchKernelGGL((glr_step_kernel<bf16_t>), dim3(nb), dim3(256), 0, s, p);
  else hipLaunchKernelGGL((glr_step_kernel<float>), dim3(nb), dim3(256), 0, s, p);
  return hipGetLastError();
}

}  // namespace sscan
