// Gated linear recurrence, backward.
#include "sscan_glr_tile.h"

namespace sscan {

// V activations of one token as the backward reads them: elements, or 8-bit codes with
// the powers of two of the wave's group.
template <typename Tin, int V, bool SAVED>
struct GlrAct {
  typedef typename TokVec<Tin, V>::reg reg;
  const Tin* p;
  int64_t stride;
  __device__ GlrAct(const void* from, int64_t s, const GlrBwdParams&, int, int64_t, uint32_t)
      : p(static_cast<const Tin*>(from)), stride(s) {}
  __device__ __forceinline__ reg load(int64_t t, uint32_t c) const { return TokVec<Tin, V>::load(p + t * stride, c * sizeof(Tin)); }
  __device__ __forceinline__ float get(reg r, int v) const { return TokVec<Tin, V>::get(r, v); }
};
template <typename Tin, int V>
struct GlrAct<Tin, V, true> {
  typedef uint32_t reg;
  typedef typename std::conditional<V == 2, uint16_t, uint8_t>::type word;
  const int8_t* p;
  int64_t stride;
  float scale[V];
  __device__ GlrAct(const void*, int64_t, const GlrBwdParams& q, int k, int64_t group, uint32_t c)
      : p(q.codes + k * q.saved_stride), stride(q.dim) {
    const uint8_t* e = reinterpret_cast<const uint8_t*>(p) + q.exps_at + group * q.dim + c;
    uint32_t f = V == 2 ? *reinterpret_cast<const uint16_t*>(e) : *e;
#pragma unroll
    for (int v = 0; v < V; ++v) scale[v] = act8_value(1, f >> (8 * v) & 255u);
  }
  __device__ __forceinline__ reg load(int64_t t, uint32_t c) const {
    return row_load<word>(p + t * stride, c);
  }
  __device__ __forceinline__ float get(reg r, int v) const {
    return static_cast<float>(static_cast<int8_t>(r >> (8 * v))) * scale[v];
  }
};

// One tile, the chain running from the last tokens to the first.  The states inside the
// tile come from the one saved at its start, by the waves' maps as in the forward; the
// gradient that leaves a token towards the one before is e' = a (gy + e), again an affine
// map with the same factor a, so one exchange through shared memory serves both.
template <typename Tin, int V, bool PACKED, bool GATE, bool SAVED>
__global__ __launch_bounds__(64 * kGlrWaves) void glr_bwd_kernel(GlrBwdParams p, GlrChainWords words, float* part,
                                                                 int ntiles, int nct) {
  typedef TokVec<Tin, V> Tok;
  typedef GlrAct<Tin, V, SAVED> Act;
  constexpr int K = kActGroup, W = kGlrWaves;
  __shared__ float sA[W][V][64], sB[W][V][64], sG[W][V][64], sE[V][64];
  __shared__ int sReset[W], sTile;
  const int w = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6), lane = threadIdx.x & 63;
  const uint32_t nchains = static_cast<uint32_t>(p.batch) * nct;
  const uint32_t chain = blockIdx.x % nchains;
  int pos = 0;
  if (ntiles > 1) {
    if (threadIdx.x == 0) sTile = static_cast<int>(atomicAdd(&words.tickets[static_cast<size_t>(chain) * kGlrTicket], 1u));
    __syncthreads();
    pos = __builtin_amdgcn_readfirstlane(sTile);
  }
  const int tile = ntiles - 1 - pos;
  const int64_t b = chain / nct;
  const int64_t c0 = static_cast<int64_t>(chain % nct) * (64 * V);
  const int64_t D = p.dim, L = p.L;
  const int64_t cl = c0 + lane * V;
  const bool mine = cl < D;
  const uint32_t c = static_cast<uint32_t>(mine ? cl : D - V), cb = c * sizeof(Tin);
  const int64_t t0 = static_cast<int64_t>(tile) * kGlrTile + w * K;
  const int rows = static_cast<int>(L - t0 < 0 ? 0 : (L - t0 < K ? L - t0 : K));

  const int64_t ngrp = (L + K - 1) / K;
  const int64_t group = b * ngrp + (t0 / K < ngrp ? t0 / K : ngrp - 1);
  const Act ax(p.x, p.sx, p, 0, group, c), ar(p.r, p.sr, p, 1, group, c), ai(p.i, p.si, p, 2, group, c);
  const Act az(p.z, p.sz, p, GATE ? 3 : 0, group, c);
  typename Act::reg rx[K], rr[K], ri[K], rz[GATE ? K : 1];
  typename Tok::reg rg[K];
#pragma unroll
  for (int k = 0; k < K; ++k) {
    const int64_t t = b * L + (t0 + k < L ? t0 + k : L - 1);
    rr[k] = ar.load(t, c);
    ri[k] = ai.load(t, c);
    rx[k] = ax.load(t, c);
    rg[k] = Tok::load(static_cast<const Tin*>(p.dy) + t * D, cb);
    if (GATE) rz[k] = az.load(t, c);
  }
  GlrSpan sp;
  sp.valid = rows;
  if (PACKED) sp = glr_span(p.offsets, static_cast<int>(p.num_seqs), t0, L);

  float rate[V], rb[V], ib[V], h[V];
#pragma unroll
  for (int v = 0; v < V; ++v) {
    rate[v] = p.decay_scale * softplus_acc(p.lam[c + v]);
    rb[v] = p.r_bias ? p.r_bias[c + v] : 0.f;
    ib[v] = p.i_bias ? p.i_bias[c + v] : 0.f;
    h[v] = p.ckpt[(b * ntiles + tile) * D + c + v];
  }

  float a[K][V], m[K][V], rho[K][V], iota[K][V], before[K][V];
#pragma unroll
  for (int k = 0; k < K; ++k)
#pragma unroll
    for (int v = 0; v < V; ++v) {
      float one;
      rho[k][v] = sigmoid(ar.get(rr[k], v) + rb[v]);
      iota[k][v] = sigmoid(ai.get(ri[k], v) + ib[v]);
      a[k][v] = decay_of(rate[v] * rho[k][v], one);
      m[k][v] = hw_sqrt(one);
    }
  auto input = [&](int k, int v) __attribute__((always_inline)) { return iota[k][v] * ax.get(rx[k], v); };
  auto grad_y = [&](int k, int v) __attribute__((always_inline)) {
    const float dy = Tok::get(rg[k], v);
    return GATE ? dy * silu(az.get(rz[k], v)) : dy;
  };
  auto state0 = [&](int k, int v) __attribute__((always_inline)) {
    return p.h0 ? p.h0[static_cast<int64_t>(sp.seq_of(k)) * D + c + v] : 0.f;
  };
  auto last_grad = [&](int k, int v) __attribute__((always_inline)) {
    return p.dlast ? p.dlast[static_cast<int64_t>(sp.seq_of(k)) * D + c + v] : 0.f;
  };
  // the wave's two maps
  {
    float A[V], B[V], G[V];
#pragma unroll
    for (int v = 0; v < V; ++v) A[v] = 1.f, B[v] = 0.f, G[v] = 0.f;
    auto ahead = [&](int k) __attribute__((always_inline)) {
      const bool start = PACKED && (sp.starts >> k & 1);
#pragma unroll
      for (int v = 0; v < V; ++v) {
        A[v] *= a[k][v];
        B[v] = fmaf(a[k][v], start ? state0(k, v) : B[v], m[k][v] * input(k, v));
      }
    };
    auto back = [&](int k) __attribute__((always_inline)) {
#pragma unroll
      for (int v = 0; v < V; ++v) {
        if (PACKED && (sp.ends >> k & 1)) G[v] = last_grad(k, v);
        G[v] = a[k][v] * (G[v] + grad_y(k, v));
        if (PACKED && (sp.starts >> k & 1)) G[v] = 0.f;
      }
    };
    if (sp.valid == K) {
#pragma unroll
      for (int k = 0; k < K; ++k) ahead(k);
#pragma unroll
      for (int k = K - 1; k >= 0; --k) back(k);
    } else {
#pragma unroll
      for (int k = 0; k < K; ++k)
        if (k < sp.valid) ahead(k);
#pragma unroll
      for (int k = K - 1; k >= 0; --k)
        if (k < sp.valid) back(k);
    }
#pragma unroll
    for (int v = 0; v < V; ++v) sA[w][v][lane] = A[v], sB[w][v][lane] = B[v], sG[w][v][lane] = G[v];
  }
  if (PACKED && lane == 0) sReset[w] = sp.starts != 0;
  __syncthreads();

  if (w < V) {
    float e = 0.f;
    if (!PACKED && p.dlast && pos == 0) e = p.dlast[b * D + c + w];
    if (ntiles > 1) {
      GlrMap all{sA[W - 1][w][lane], sG[W - 1][w][lane], PACKED && sReset[W - 1]};
#pragma unroll
      for (int q = W - 2; q >= 0; --q) all = GlrMap{sA[q][w][lane], sG[q][w][lane], PACKED && sReset[q]}.after(all);
      e = glr_pass(words, chain, 64 * V, w * 64 + lane, pos, ntiles, all, e);
    }
    sE[w][lane] = e;
  }
  // the states that the wave's tokens continue
#pragma unroll
  for (int q = 0; q < W - 1; ++q) {
    if (q >= w) break;
    const bool qr = PACKED && __builtin_amdgcn_readfirstlane(sReset[q]);
#pragma unroll
    for (int v = 0; v < V; ++v) h[v] = qr ? sB[q][v][lane] : fmaf(sA[q][v][lane], h[v], sB[q][v][lane]);
  }
#pragma unroll
  for (int k = 0; k < K; ++k)
#pragma unroll
    for (int v = 0; v < V; ++v) {
      if (PACKED && (sp.starts >> k & 1)) h[v] = state0(k, v);
      before[k][v] = h[v];
      h[v] = fmaf(a[k][v], h[v], m[k][v] * input(k, v));
    }
  __syncthreads();

  float e[V], slam[V], srb[V], sib[V];
#pragma unroll
  for (int v = 0; v < V; ++v) e[v] = sE[v][lane], slam[v] = 0.f, srb[v] = 0.f, sib[v] = 0.f;
#pragma unroll
  for (int q = W - 1; q > 0; --q) {
    if (q <= w) break;
    const bool qr = PACKED && __builtin_amdgcn_readfirstlane(sReset[q]);
#pragma unroll
    for (int v = 0; v < V; ++v) e[v] = qr ? sG[q][v][lane] : fmaf(sA[q][v][lane], e[v], sG[q][v][lane]);
  }
  const int64_t row0 = b * L + t0;
  Tin* dxp = static_cast<Tin*>(p.dx) + row0 * p.gx;
  Tin* drp = static_cast<Tin*>(p.dr) + row0 * p.gr;
  Tin* dip = static_cast<Tin*>(p.di) + row0 * p.gi;
  Tin* dzp = GATE ? static_cast<Tin*>(p.dz) + row0 * p.gz : nullptr;
  auto put = [&](int k, const float* gx, const float* gr, const float* gi, const float* gz) __attribute__((always_inline)) {
    if (!mine) return;
    Tok::store(dxp + k * p.gx, cb, gx);
    Tok::store(drp + k * p.gr, cb, gr);
    Tok::store(dip + k * p.gi, cb, gi);
    if (GATE) Tok::store(dzp + k * p.gz, cb, gz);
  };
  auto token = [&](int k) __attribute__((always_inline)) {
    float gx[V], gr[V], gi[V], gz[V];
#pragma unroll
    for (int v = 0; v < V; ++v) {
      const float P = rho[k][v], I = iota[k][v], A = a[k][v], M = m[k][v], H = before[k][v];
      const float x = ax.get(rx[k], v), in = I * x;
      float gy = Tok::get(rg[k], v);
      if (GATE) {
        const float z = az.get(rz[k], v), sz = sigmoid(z);
        gz[v] = gy * fmaf(A, H, M * in) * fmaf(z, slope(sz), sz);
        gy *= z * sz;
      }
      if (PACKED && (sp.ends >> k & 1)) e[v] = last_grad(k, v);
      const float g = gy + e[v];
      const float dla = g * (A * H - in * A * (A * rcp_or_0(M)));
      const float du = g * M;
      gx[v] = du * I;
      gi[v] = du * x * slope(I);
      gr[v] = -rate[v] * dla * slope(P);
      slam[v] = fmaf(dla, P, slam[v]);
      srb[v] += gr[v];
      sib[v] += gi[v];
      e[v] = A * g;
      if (PACKED && (sp.starts >> k & 1)) {
        if (p.dh0 && mine) p.dh0[static_cast<int64_t>(sp.seq_of(k)) * D + c + v] = e[v];
        e[v] = 0.f;
      }
    }
    put(k, gx, gr, gi, gz);
  };
  if (sp.valid == K) {
#pragma unroll
    for (int k = K - 1; k >= 0; --k) token(k);
  } else {
    float none[V] = {};
#pragma unroll
    for (int k = K - 1; k >= 0; --k) {
      if (k < sp.valid) token(k);
      else if (k < rows) put(k, none, none, none, none);
    }
  }
  if (!PACKED && p.dh0 && mine && tile == 0 && w == 0) {
#pragma unroll
    for (int v = 0; v < V; ++v) p.dh0[b * D + c + v] = e[v];
  }

  // the tile's sums for the parameters, its waves in order
  __syncthreads();
#pragma unroll
  for (int v = 0; v < V; ++v) sA[w][v][lane] = slam[v], sB[w][v][lane] = srb[v], sG[w][v][lane] = sib[v];
  __syncthreads();
  if (w < V) {
    float* to = part + (static_cast<int64_t>(chain) * ntiles + tile) * (3 * 64 * V) + w * 64 + lane;
    float s0 = 0.f, s1 = 0.f, s2 = 0.f;
#pragma unroll
    for (int q = 0; q < W; ++q) s0 += sA[q][w][lane], s1 += sB[q][w][lane], s2 += sG[q][w][lane];
    to[0] = s0;
    to[64 * V] = s1;
    to[2 * 64 * V] = s2;
  }
}

// Parameter gradients: the tiles' sums, over batch rows and tiles in a fixed order.  One
// workgroup per 64 channels and parameter, 16 waves taking every 16th tile.
__global__ __launch_bounds__(1024) void glr_param_kernel(const float* part, const float* lam, float decay_scale, float* dlam,
                                                         float* drb, float* dib, int64_t batch, int64_t ntiles, int64_t D,
                                                         int nct, int V) {
  __shared__ float sum[16][64];
  const int w = threadIdx.x >> 6, lane = threadIdx.x & 63;
  const int kind = blockIdx.x % 3, set = blockIdx.x / 3;
  const int ct = set / V, v = set % V;
  float s = 0.f;
  const int64_t n = batch * ntiles;
  auto at = [&](int64_t k) {
    const int64_t b = k / ntiles, tile = k - b * ntiles;
    return part[((b * nct + ct) * ntiles + tile) * (3 * 64 * V) + (kind * V + v) * 64 + lane];
  };
  int64_t k = w;
  for (; k + 7 * 16 < n; k += 8 * 16) {   // eight loads in flight
    float x[8];
#pragma unroll
    for (int j = 0; j < 8; ++j) x[j] = at(k + j * 16);
#pragma unroll
    for (int j = 0; j < 8; ++j) s += x[j];
  }
  for (; k < n; k += 16) s += at(k);
  sum[w][lane] = s;
  __syncthreads();
  const int64_t d = (static_cast<int64_t>(ct) * 64 + lane) * V + v;
  if (w > 0 || d >= D) return;
#pragma unroll
  for (int q = 1; q < 16; ++q) s += sum[q][lane];
  if (kind == 0) dlam[d] = -decay_scale * sigmoid(lam[d]) * s;
  else if (kind == 1 && drb) drb[d] = s;
  else if (kind == 2 && dib) dib[d] = s;
}

namespace {

template <typename Tin, int V, bool PACKED, bool GATE>
hipError_t launch_one(const GlrBwdParams& p, const GlrChainLayout& lo, float* part, int nct, hipStream_t s) {
  const dim3 grid(static_cast<unsigned>(lo.chains * lo.tiles)), wg(64 * kGlrWaves);
  const GlrChainWords words = lo.at(p.workspace);
  const int nt = static_cast<int>(lo.tiles);
  if (p.codes) hipLaunchKernelGGL((glr_bwd_kernel<Tin, V, PACKED, GATE, true>), grid, wg, 0, s, p, words, part, nt, nct);
  else hipLaunchKernelGGL((glr_bwd_kernel<Tin, V, PACKED, GATE, false>), grid, wg, 0, s, p, words, part, nt, nct);
  return hipGetLastError();
}

size_t part_bytes(const GlrChainLayout& lo) { return static_cast<size_t>(lo.chains) * lo.tiles * lo.lanes * 3 * 4; }

template <typename Tin, int V>
hipError_t launch_v(const GlrBwdParams& p, hipStream_t s) {
  const GlrChainLayout lo(p.batch, p.L, p.dim, V);
  const int nct = static_cast<int>((p.dim + 64 * V - 1) / (64 * V));
  float* part = reinterpret_cast<float*>(static_cast<char*>(p.workspace) + lo.bytes());
  if (p.batch > 0 && p.L > 0) {
    hipError_t e = lo.tiles > 1 ? launch_glr_clear(p.workspace, lo, s) : hipSuccess;
    if (e != hipSuccess) return e;
    if (p.offsets)
      e = p.dz ? launch_one<Tin, V, true, true>(p, lo, part, nct, s) : launch_one<Tin, V, true, false>(p, lo, part, nct, s);
    else
      e = p.dz ? launch_one<Tin, V, false, true>(p, lo, part, nct, s) : launch_one<Tin, V, false, false>(p, lo, part, nct, s);
    if (e != hipSuccess) return e;
  }
  hipLaunchKernelGGL(glr_param_kernel, dim3(static_cast<unsigned>(3 * nct * V)), dim3(1024), 0, s, part, p.lam,
                     p.decay_scale, p.dlam, p.dr_bias, p.di_bias, p.batch, lo.tiles, p.dim, nct, V);
  return hipGetLastError();
}

// Two channels a lane where every row of every tensor holds whole aligned pairs.
template <typename Tin>
bool pairs(const GlrBwdParams& p) {
  uintptr_t at = 0;
  for (const void* q : {p.x, p.r, p.i, p.z, p.dy, static_cast<const void*>(p.dx), static_cast<const void*>(p.dr),
                        static_cast<const void*>(p.di), static_cast<const void*>(p.dz)})
    at |= reinterpret_cast<uintptr_t>(q);
  int64_t odd = p.dim | p.gx | p.gr | p.gi | (p.dz ? p.gz : 0);
  if (!p.codes) odd |= p.sx | p.sr | p.si | (p.z ? p.sz : 0);
  return at % (2 * sizeof(Tin)) == 0 && odd % 2 == 0;
}

template <typename Tin>
hipError_t launch_t(const GlrBwdParams& p, hipStream_t s) {
  return launch_v<Tin, 1>(p, s);
}

}  // namespace

size_t glr_bwd_workspace_bytes(int64_t batch, int64_t L, int64_t dim) {
  // enough for one and for two channels a lane
  const GlrChainLayout a(batch, L, dim, 1), b(batch, L, dim, 2);
  const size_t na = a.bytes() + part_bytes(a), nb = b.bytes() + part_bytes(b);
  return ((na > nb ? na : nb) + 255) & ~size_t(255);
}

hipError_t launch_glr_bwd(const GlrBwdParams& p, bool bf16, hipStream_t s) {
  if (p.dh0 && (p.offsets || p.L == 0)) {
    const hipError_t e = launch_glr_empty(p.offsets, p.dlast, p.dh0, p.offsets ? p.num_seqs : p.batch, p.dim, s);
    if (e != hipSuccess) return e;
  }
  return bf16 ? launch_t<bf16_t>(p, s) : launch_t<float>(p, s);
}

}  // namespace sscan
