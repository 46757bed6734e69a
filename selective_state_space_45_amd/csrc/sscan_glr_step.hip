// Gated linear recurrence, one token per row against a pool of states.
#include "sscan_glr_tile.h"

namespace sscan {

constexpr int kStepRows = 4;   // rows of a workgroup

// A lane has V channels of up to four rows, so that the channels' parameters are formed
// once for them.  A token moves 8 bytes of state a channel besides its inputs and output:
// bound by memory at large batches and by the launch at small ones.  All loads of a row
// start before the first is used, the state's after its slot is known.  256 x 5120 bf16,
// gated: 7.5 us (one row and channel a lane: 8.4); 1 x 1536: 4.0 us, the launch.
template <typename Tin, int V>
__global__ __launch_bounds__(64) void glr_step_kernel(GlrStepParams p, int nct) {
  typedef TokVec<Tin, V> Tok;
  typedef typename TokVec<float, V>::reg State;
  const uint32_t block = workgroup<64>();
  const int64_t b0 = static_cast<int64_t>(block / nct) * kStepRows;
  const int64_t c = (static_cast<int64_t>(block % nct) * 64 + threadIdx.x) * V;
  if (b0 >= p.batch || c >= p.dim) return;
  const uint32_t at = static_cast<uint32_t>(c * sizeof(Tin)), at4 = static_cast<uint32_t>(c * 4);
  const int rows = p.batch - b0 < kStepRows ? static_cast<int>(p.batch - b0) : kStepRows;

  typename Tok::reg rx[kStepRows], rr[kStepRows], ri[kStepRows], rz[kStepRows];
  State st[kStepRows];
  int64_t from[kStepRows], to[kStepRows];
#pragma unroll
  for (int k = 0; k < kStepRows; ++k) {
    const int64_t b = b0 + (k < rows ? k : rows - 1);
    from[k] = p.slots ? p.slots[b] : b;
    to[k] = p.slots_out ? p.slots_out[b] : from[k];
    if (from[k] < 0 || from[k] >= p.num_slots) from[k] = -1;
    if (to[k] < 0 || to[k] >= p.num_slots) to[k] = -1;
    rx[k] = row_load<typename Tok::word, false>(static_cast<const Tin*>(p.x) + b * p.sx, at);
    rr[k] = row_load<typename Tok::word, false>(static_cast<const Tin*>(p.r) + b * p.sr, at);
    ri[k] = row_load<typename Tok::word, false>(static_cast<const Tin*>(p.i) + b * p.si, at);
    if (p.z) rz[k] = row_load<typename Tok::word, false>(static_cast<const Tin*>(p.z) + b * p.sz, at);
    if (from[k] >= 0) st[k] = row_load<State, false>(p.state + from[k] * p.dim, at4);
  }
  float rate[V], nrb[V], nib[V];
#pragma unroll
  for (int v = 0; v < V; ++v) {
    rate[v] = p.decay_scale * softplus_acc(p.lam[c + v]) * kLog2e;
    nrb[v] = p.r_bias ? -kLog2e * p.r_bias[c + v] : 0.f;
    nib[v] = p.i_bias ? -kLog2e * p.i_bias[c + v] : 0.f;
  }
#pragma unroll
  for (int k = 0; k < kStepRows; ++k) {
    if (k >= rows) continue;
    float y[V] = {}, h[V];
    if (from[k] >= 0) {
#pragma unroll
      for (int v = 0; v < V; ++v) {
        float one;
        const float a = decay_of(rate[v] * gate(Tok::get(rr[k], v), nrb[v]), one);
        const float u = hw_sqrt(one) * (gate(Tok::get(ri[k], v), nib[v]) * Tok::get(rx[k], v));
        h[v] = fmaf(a, TokVec<float, V>::get(st[k], v), u);
        y[v] = p.z ? h[v] * silu(Tok::get(rz[k], v)) : h[v];
      }
      if (to[k] >= 0) row_store<State, false>(p.state + to[k] * p.dim, at4, TokVec<float, V>::put(h));
    }
    row_store<typename Tok::word, false>(static_cast<Tin*>(p.y) + (b0 + k) * p.dim, at, Tok::put(y));
  }
}

namespace {

// Two channels a lane where the rows of every tensor hold whole aligned pairs.
template <typename Tin>
void launch(const GlrStepParams& p, hipStream_t s) {
  uintptr_t bits = static_cast<uintptr_t>(p.sx | p.sr | p.si | (p.z ? p.sz : 0) | p.dim) * sizeof(Tin);
  for (const void* q : {p.x, p.r, p.i, p.z, static_cast<const void*>(p.y)}) bits |= reinterpret_cast<uintptr_t>(q);
  const bool two = bits % (2 * sizeof(Tin)) == 0 && reinterpret_cast<uintptr_t>(p.state) % 8 == 0;
  const int nct = static_cast<int>((p.dim + (two ? 127 : 63)) / (two ? 128 : 64));
  const dim3 grid = grid_of<64>(nct * ((p.batch + kStepRows - 1) / kStepRows));
  if (two) hipLaunchKernelGGL((glr_step_kernel<Tin, 2>), grid, dim3(64), 0, s, p, nct);
  else hipLaunchKernelGGL((glr_step_kernel<Tin, 1>), grid, dim3(64), 0, s, p, nct);
}

}  // namespace

hipError_t launch_glr_step(const GlrStepParams& p, bool bf16, hipStream_t s) {
  if (bf16) launch<bf16_t>(p, s);
  else launch<float>(p, s);
  return hipGetLastError();
}

}  // namespace sscan
