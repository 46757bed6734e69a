// Gated linear recurrence, backward.
#include "sscan_glr_tile.h"

namespace sscan {

// An activation tensor as the backward reads it, one channel a lane: elements, or 8-bit
// codes with the power of two of the wave's group.
template <typename Tin, bool LINES, bool SAVED>
struct GlrAct {
  typedef TokVec<Tin, 1> Tok;
  typedef typename Tok::reg reg;
  const Tin* row;
  int64_t stride;
  __device__ GlrAct(const void* from, int64_t s, const GlrBwdParams&, int, int64_t t, int64_t, uint32_t)
      : row(static_cast<const Tin*>(from) + t * s), stride(s) {}
  __device__ __forceinline__ reg load(uint32_t at) const { return row_load<typename Tok::word, LINES>(row, at); }
  __device__ __forceinline__ float get(reg r) const { return Tok::get(r, 0); }
};
template <typename Tin, bool LINES>
struct GlrAct<Tin, LINES, true> {
  typedef int32_t reg;
  const int8_t* row;
  int64_t stride;
  float scale;
  __device__ GlrAct(const void*, int64_t, const GlrBwdParams& q, int k, int64_t t, int64_t group, uint32_t c) {
    const int8_t* codes = q.codes + k * q.saved_stride;
    row = codes + t * q.dim;
    stride = q.dim;
    scale = act8_value(1, row_load<uint8_t, false>(reinterpret_cast<const uint8_t*>(codes) + q.exps_at + group * q.dim, c));
  }
  __device__ __forceinline__ reg load(uint32_t at) const { return row_load<int8_t, LINES>(row, at); }
  __device__ __forceinline__ float get(reg r) const { return static_cast<float>(r) * scale; }
};

// x and dy of a token, held over the wait for the gradient: in bf16 they share a word.
template <typename Tin, typename Act>
struct GlrPair {
  typename Act::reg x;
  typename TokVec<Tin, 1>::reg dy;
  __device__ __forceinline__ void set(typename Act::reg rx, typename TokVec<Tin, 1>::reg rg) { x = rx, dy = rg; }
  __device__ __forceinline__ void forget() { asm("" : "+v"(x)); }
  __device__ __forceinline__ float get_x(const Act& act) const { return act.get(x); }
  __device__ __forceinline__ float get_dy() const { return dy; }
};
template <typename Act>
struct GlrPair<bf16_t, Act> {
  uint32_t both;
  __device__ __forceinline__ void set(typename Act::reg rx, uint32_t rg) {
    both = __builtin_amdgcn_perm(rg, static_cast<uint32_t>(rx), 0x05040100u);
    forget();   // that it was two registers
  }
  __device__ __forceinline__ void forget() { asm("" : "+v"(both)); }
  __device__ __forceinline__ float get_x(const Act& act) const { return act.get(static_cast<int16_t>(both)); }
  __device__ __forceinline__ float get_dy() const { return __uint_as_float(both & 0xffff0000u); }
};

// One tile, the chain running from the last tokens to the first.  The states inside the
// tile come from the one saved at its start, by the waves' maps as in the forward; the
// gradient that leaves a token towards the one before is e' = a (gy + e), again an affine
// map with the same factor a, so one exchange through shared memory serves both.
//
// 14 bytes an element in bf16 against about 60 vector operations, 7 of them at half rate:
// counters show the vector units busy half of the time and the memory at 4.5 TB/s; bound
// by the latency of its phases (a ticket, loads, maps, the wait, stores: 10 us a
// workgroup) at the waves that the registers allow.  One channel a lane: what the
// gradients need of each of 16 tokens but the gradient that arrives is formed before the
// wait for it and stays in registers.  With two channels a lane that does not fit, and
// formed again after the wait it costs more than the second channel saves (8 x 4096 x 2048
// bf16, forward and backward: 0.442 ms, and 0.397 with one).  Four waves a SIMD for dense
// bf16 without a gate (0.361 ms, with three 0.381), though 5 registers spill; the other
// forms spill many more at four (2 x 2047 x 1535 float32, gated, in an earlier form: 0.163
// ms, with three 0.118).  At three the dense forms spill no vector register, gated packed
// ones 9 or 10 in bf16 and 19 to 21 in float32, and all packed ones about 130 scalar
// registers, into lanes of vector registers.  8 x 4096 x 2048 bf16: 0.219 ms.
template <typename Tin, bool LINES, bool PACKED, bool GATE, bool SAVED>
__global__ __launch_bounds__(64 * kGlrWaves, PACKED || GATE || sizeof(Tin) == 4 ? 3 : 4) void glr_bwd_kernel(GlrBwdParams p, GlrChainWords words, float* part,
                                                                 int ntiles, int nct) {
  typedef TokVec<Tin, 1> Tok;
  typedef GlrAct<Tin, LINES, SAVED> Act;
  constexpr int K = kActGroup, W = kGlrWaves;
  __shared__ float sA[W][64], sB[W][64], sG[W][64], sE[64];
  __shared__ int sReset[W], sTile;
  const int w = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6), lane = threadIdx.x & 63;
  const uint32_t nchains = static_cast<uint32_t>(p.batch) * nct, block = workgroup<64 * kGlrWaves>();
  const uint32_t chain = glr_chain(block, nchains);
  int pos = 0;
  if (ntiles > 1) {
    if (threadIdx.x == 0)
      sTile = static_cast<int>(atomicAdd(&words.tickets[static_cast<size_t>(chain) * kGlrTicket], 1u));
    __syncthreads();
    pos = __builtin_amdgcn_readfirstlane(sTile);
    if (pos >= ntiles) return;   // a grid that is filled up has more workgroups than tiles
  } else if (block >= nchains) {
    return;
  }
  const int tile = ntiles - 1 - pos;
  const int64_t b = chain / nct;
  const int64_t D = p.dim, L = p.L;
  // lanes past the last channel work on the last one and store nothing
  const int64_t cl = static_cast<int64_t>(chain % nct) * 64 + lane;
  const bool mine = cl < D;
  const uint32_t c = static_cast<uint32_t>(mine ? cl : D - 1), cb = c * sizeof(Tin);
  const int L32 = static_cast<int>(L), t0 = tile * kGlrTile + w * K;
  const int rows = L32 - t0 < 0 ? 0 : (L32 - t0 < K ? L32 - t0 : K);

  // 16 tokens of each input; tokens past the row's end read its last one
  const int64_t ngrp = (L + K - 1) / K;
  const int64_t group = b * ngrp + (rows ? t0 / K : ngrp - 1), tl = b * L + (rows ? t0 : L - 1);
  Act ax(p.x, p.sx, p, 0, tl, group, c), ar(p.r, p.sr, p, 1, tl, group, c), ai(p.i, p.si, p, 2, tl, group, c);
  Act az(p.z, p.sz, p, GATE ? 3 : 0, tl, group, c);
  typename Act::reg rx[K], rr[K], ri[K], rz[K];
  typename Tok::reg rg[K];
  {
    const Tin* pg = static_cast<const Tin*>(p.dy) + tl * D;
    auto load = [&](auto full) __attribute__((always_inline)) {
      const uint32_t at = here(cb), act_at = here(SAVED ? c : cb);
#pragma unroll
      for (int k = 0; k < K; ++k) {
        rr[k] = ar.load(act_at);
        ri[k] = ai.load(act_at);
        rx[k] = ax.load(act_at);
        rg[k] = row_load<typename Tok::word, LINES>(pg, at);
        if (GATE) rz[k] = az.load(act_at);
        const int64_t more = decltype(full)::value || k + 1 < rows ? 1 : 0;
        ar.row += more * ar.stride, ai.row += more * ai.stride, ax.row += more * ax.stride, pg += more * D;
        if (GATE) az.row += more * az.stride;
      }
      apart<decltype(full)::value>();
    };
    if (rows == K) load(std::true_type{});
    else load(std::false_type{});
  }
  GlrSpan sp;
  sp.valid = rows;
  if (PACKED) sp = glr_span(p.offsets, static_cast<int>(p.num_seqs), t0, L32);

  const float rate = p.decay_scale * softplus_acc(p.lam[c]), rate2 = rate * kLog2e;
  const float nrb = p.r_bias ? -kLog2e * p.r_bias[c] : 0.f, nib = p.i_bias ? -kLog2e * p.i_bias[c] : 0.f;
  float h = p.ckpt[(b * ntiles + tile) * D + c];

  // m = sqrt(1 - a^2) stays above 1e-18, for its reciprocal: it is smaller only at decay
  // rates below 1e-36, whose terms with 1 / m, each times the rate, are below 1e-18 of
  // the others.
  float a[K], m[K], rho[K], iota[K], part_a[K], state[GATE ? K : 1];
#pragma unroll
  for (int k = 0; k < K; ++k) {
    float one;
    rho[k] = gate(ar.get(rr[k]), nrb);
    iota[k] = gate(ai.get(ri[k]), nib);
    a[k] = decay_of(rate2 * rho[k], one);
    m[k] = hw_sqrt(__builtin_elementwise_maximum(one, 1e-36f));   // (a NaN stays one)
  }
  GlrPair<Tin, Act> xg[K];
#pragma unroll
  for (int k = 0; k < K; ++k) xg[k].set(rx[k], rg[k]);
  // Tokens past the end, whatever they hold, pass the state and the gradient on (a = 1,
  // x = dy = 0) and have zero gradients themselves (iota, rho, and part_a below).
  if (sp.valid < K) {
#pragma unroll
    for (int k = 0; k < K; ++k)
      if (k >= sp.valid) {
        a[k] = m[k] = 1.f, rho[k] = iota[k] = 0.f;
        xg[k].set({}, {});
        if (GATE) rz[k] = {};
      }
  }
  auto input = [&](int k) __attribute__((always_inline)) { return iota[k] * xg[k].get_x(ax); };
  auto state0 = [&](int k) __attribute__((always_inline)) {
    return p.h0 ? p.h0[static_cast<int64_t>(sp.seq_of(k)) * D + c] : 0.f;
  };
  auto last_grad = [&](int k) __attribute__((always_inline)) {
    return p.dlast ? p.dlast[static_cast<int64_t>(sp.seq_of(k)) * D + c] : 0.f;
  };
  // the wave's two maps
  {
    float A = 1.f, B = 0.f, G = 0.f;
    auto ahead = [&](int k) __attribute__((always_inline)) {
      A *= a[k];
      B = fmaf(a[k], PACKED && (sp.starts >> k & 1) ? state0(k) : B, m[k] * input(k));
    };
    auto back = [&](int k) __attribute__((always_inline)) {
      if (PACKED && (sp.ends >> k & 1)) G = last_grad(k);
      const float dy = xg[k].get_dy();
      G = a[k] * (G + (GATE ? dy * silu(az.get(rz[k])) : dy));
      if (PACKED && (sp.starts >> k & 1)) G = 0.f;
    };
#pragma unroll
    for (int k = 0; k < K; ++k) ahead(k);
#pragma unroll
    for (int k = K - 1; k >= 0; --k) back(k);
    sA[w][lane] = A, sB[w][lane] = B, sG[w][lane] = G;
  }
  if (PACKED && lane == 0) sReset[w] = sp.starts != 0;
  // products of these are formed again below: kept, they would take 32 registers more
#pragma unroll
  for (int k = 0; k < K; ++k) {
    asm("" : "+v"(m[k]));
    xg[k].forget();
    if (GATE) asm("" : "+v"(rz[k]));
  }
  __syncthreads();

  if (w == 0) {
    float e = 0.f;
    if (!PACKED && p.dlast && pos == 0) e = p.dlast[b * D + c];
    if (ntiles > 1) {
      GlrMap all{sA[W - 1][lane], sG[W - 1][lane], PACKED && sReset[W - 1]};
#pragma unroll
      for (int q = W - 2; q >= 0; --q) all = GlrMap{sA[q][lane], sG[q][lane], PACKED && sReset[q]}.after(all);
      e = glr_pass<64>(words, chain, lane, pos, ntiles, all, e);
    }
    sE[lane] = e;
  }
  // the states that the wave's tokens continue, and with them dlog_a / e' of each token,
  // h_{t-1} - iota x a / m (part_a); m becomes dx / g
#pragma unroll
  for (int q = 0; q < W - 1; ++q)
    if (q < w) h = GlrMap{sA[q][lane], sB[q][lane], PACKED && sReset[q]}(h);
#pragma unroll
  for (int k = 0; k < K; ++k) {
    if (PACKED && (sp.starts >> k & 1)) h = state0(k);
    const float in = input(k);
    part_a[k] = fmaf(-in, a[k] * hw_rcp(m[k]), h);
    h = fmaf(a[k], h, m[k] * in);
    if (GATE) state[k] = h;
    m[k] *= iota[k];
  }
  if (sp.valid < K) {
#pragma unroll
    for (int k = 0; k < K; ++k)
      if (k >= sp.valid) {
        part_a[k] = 0.f;
        if (GATE) state[k] = 0.f;
      }
  }
  __syncthreads();

  float e = sE[lane], slam = 0.f, srb = 0.f, sib = 0.f;
#pragma unroll
  for (int q = W - 1; q > 0; --q)
    if (q > w) e = GlrMap{sA[q][lane], sG[q][lane], PACKED && sReset[q]}(e);
  // rows from the wave's last token to its first; a token past the row's end writes its
  // zeros to the last row, which its own token then overwrites
  const int64_t end = b * L + t0 + rows - 1;
  const int64_t sx = step(p.gx), sr = step(p.gr), si = step(p.gi), sz = step(p.gz);
  Tin* px = static_cast<Tin*>(p.dx) + end * sx;
  Tin* pr = static_cast<Tin*>(p.dr) + end * sr;
  Tin* pi = static_cast<Tin*>(p.di) + end * si;
  Tin* pz = GATE ? static_cast<Tin*>(p.dz) + end * sz : nullptr;
  const uint32_t at = here(cb);
  auto token = [&](int k) __attribute__((always_inline)) {
    float gy = xg[k].get_dy(), gz = 0.f;
    if (GATE) {
      const float z = az.get(rz[k]), sz = sigmoid(z);
      gz = gy * state[k] * fmaf(z, slope(sz), sz);
      gy *= z * sz;
    }
    if (PACKED && (sp.ends >> k & 1)) e = last_grad(k);
    const float g = gy + e;
    e = a[k] * g;
    const float dla = e * part_a[k], gx = g * m[k];
    const float gxx = gx * xg[k].get_x(ax), gi = fmaf(-iota[k], gxx, gxx);
    const float dlp = dla * rho[k], rdl = -rate * dlp, gr = fmaf(-rho[k], rdl, rdl);
    slam += dlp;
    srb += gr;
    sib += gi;
    if (PACKED && (sp.starts >> k & 1)) {
      if (p.dh0) p.dh0[static_cast<int64_t>(sp.seq_of(k)) * D + c] = e;
      e = 0.f;
    }
    row_store<typename Tok::word, LINES>(px, at, Tok::put(&gx));
    row_store<typename Tok::word, LINES>(pr, at, Tok::put(&gr));
    row_store<typename Tok::word, LINES>(pi, at, Tok::put(&gi));
    if (GATE) row_store<typename Tok::word, LINES>(pz, at, Tok::put(&gz));
    px -= k < rows ? sx : 0, pr -= k < rows ? sr : 0, pi -= k < rows ? si : 0;
    if (GATE) pz -= k < rows ? sz : 0;
  };
  if (mine && rows > 0) {
#pragma unroll
    for (int k = K - 1; k >= 0; --k) token(k);
    // padding has no gradient, though a factor of its zeros may be infinite or NaN (lam, or the
    // power of two that 8-bit codes share with a request's last tokens)
    if (PACKED) {
      for (int64_t t = b * L + t0 + sp.valid; t <= end; ++t) {
        const typename Tok::word none = {};
        row_store<typename Tok::word, LINES>(static_cast<Tin*>(p.dx) + t * sx, at, none);
        row_store<typename Tok::word, LINES>(static_cast<Tin*>(p.dr) + t * sr, at, none);
        row_store<typename Tok::word, LINES>(static_cast<Tin*>(p.di) + t * si, at, none);
        if (GATE) row_store<typename Tok::word, LINES>(static_cast<Tin*>(p.dz) + t * sz, at, none);
      }
    }
  }
  if (!PACKED && p.dh0 && mine && tile == 0 && w == 0) p.dh0[b * D + c] = e;

  // the tile's sums for the parameters, its waves in order
  __syncthreads();
  sA[w][lane] = slam, sB[w][lane] = srb, sG[w][lane] = sib;
  __syncthreads();
  if (w < 3) {
    const float(*s)[64] = w == 0 ? sA : (w == 1 ? sB : sG);
    float sum = s[0][lane];
#pragma unroll
    for (int q = 1; q < W; ++q) sum += s[q][lane];
    part[((static_cast<int64_t>(chain) * ntiles + tile) * 3 + w) * 64 + lane] = sum;
  }
}

// Parameter gradients: the tiles' sums, over batch rows and tiles in a fixed order.  One
// workgroup per 16 channels and parameter, 64 sets of 16 lanes taking every 64th tile (16
// channels rather than 64: four times the workgroups, for loads that wait on memory).
__global__ __launch_bounds__(1024) void glr_param_kernel(const float* part, const float* lam, float decay_scale, float* dlam,
                                                         float* drb, float* dib, int64_t batch, int64_t ntiles, int64_t D,
                                                         int nct) {
  __shared__ float sum[64][16];
  const int set = threadIdx.x >> 4, lane = threadIdx.x & 15;
  const uint32_t block = workgroup<1024>();
  const int kind = block % 3, quarter = block / 3 % 4, ct = block / 12;
  if (ct >= nct) return;
  const int64_t n = batch * ntiles;
  auto at = [&](int64_t k) {
    const int64_t b = k / ntiles, tile = k - b * ntiles;
    return part[(((b * nct + ct) * ntiles + tile) * 3 + kind) * 64 + quarter * 16 + lane];
  };
  float s = 0.f;
  int64_t k = set;
  for (; k + 7 * 64 < n; k += 8 * 64) {   // eight loads in flight
    float x[8];
#pragma unroll
    for (int j = 0; j < 8; ++j) x[j] = at(k + j * 64);
#pragma unroll
    for (int j = 0; j < 8; ++j) s += x[j];
  }
  for (; k < n; k += 64) s += at(k);
  sum[set][lane] = s;
  __syncthreads();
  if (set >= 4) return;                   // one wave is left
#pragma unroll
  for (int q = 1; q < 16; ++q) s += sum[set + 4 * q][lane];
  sum[set][lane] = s;
  // the wave's writes before its reads of them below: without it the compiler may put them
  // the other way round, since a lane of set 0 reads none that it wrote
  __builtin_amdgcn_fence(__ATOMIC_ACQ_REL, "wavefront");
  __builtin_amdgcn_wave_barrier();
  const int64_t d = static_cast<int64_t>(ct) * 64 + quarter * 16 + lane;
  if (set > 0 || d >= D) return;
  s = ((s + sum[1][lane]) + sum[2][lane]) + sum[3][lane];
  if (kind == 0) dlam[d] = -decay_scale * sigmoid(lam[d]) * s;
  else if (kind == 1 && drb) drb[d] = s;
  else if (kind == 2 && dib) dib[d] = s;
}

namespace {

template <typename Tin, bool LINES, bool PACKED, bool GATE>
void launch_saved(const GlrBwdParams& p, const GlrChainLayout& lo, float* part, int nct, hipStream_t s) {
  const dim3 grid = grid_of<64 * kGlrWaves>(lo.chains * lo.tiles), wg(64 * kGlrWaves);
  const GlrChainWords w = lo.at(p.workspace);
  const int nt = static_cast<int>(lo.tiles);
  if (p.codes) hipLaunchKernelGGL((glr_bwd_kernel<Tin, LINES, PACKED, GATE, true>), grid, wg, 0, s, p, w, part, nt, nct);
  else hipLaunchKernelGGL((glr_bwd_kernel<Tin, LINES, PACKED, GATE, false>), grid, wg, 0, s, p, w, part, nt, nct);
}

template <typename Tin, bool LINES>
hipError_t launch_lines(const GlrBwdParams& p, const GlrChainLayout& lo, float* part, int nct, hipStream_t s) {
  if (p.offsets)
    p.dz ? launch_saved<Tin, LINES, true, true>(p, lo, part, nct, s) : launch_saved<Tin, LINES, true, false>(p, lo, part, nct, s);
  else
    p.dz ? launch_saved<Tin, LINES, false, true>(p, lo, part, nct, s) : launch_saved<Tin, LINES, false, false>(p, lo, part, nct, s);
  return hipGetLastError();
}

template <typename Tin>
hipError_t launch_t(const GlrBwdParams& p, hipStream_t s) {
  const GlrChainLayout lo(p.batch, p.L, p.dim, 1);
  const int nct = static_cast<int>((p.dim + 63) / 64);
  float* part = reinterpret_cast<float*>(static_cast<char*>(p.workspace) + lo.bytes());
  // without tokens (or for the requests that have none) the gradient passes through
  const bool some = p.offsets || p.L == 0;
  const hipError_t e = launch_glr_begin(p.workspace, lo, p.offsets, p.offsets ? p.num_seqs : p.batch, p.dlast,
                                        some ? p.dh0 : nullptr, p.dim, s);
  if (e != hipSuccess) return e;
  if (p.batch > 0 && p.L > 0) {
    // past the caches where every row of every tensor starts on a cache line
    uintptr_t bits = static_cast<uintptr_t>(p.dim | p.gx | p.gr | p.gi | (p.dz ? p.gz : 0)) * sizeof(Tin);
    bits |= p.codes ? static_cast<uintptr_t>(p.dim) : static_cast<uintptr_t>(p.sx | p.sr | p.si | (p.z ? p.sz : 0)) * sizeof(Tin);
    for (const void* q : {p.x, p.r, p.i, p.z, p.dy, static_cast<const void*>(p.dx), static_cast<const void*>(p.dr),
                          static_cast<const void*>(p.di), static_cast<const void*>(p.dz)})
      bits |= reinterpret_cast<uintptr_t>(q);
    const hipError_t e = bits % kCacheLine == 0 ? launch_lines<Tin, true>(p, lo, part, nct, s)
                                                : launch_lines<Tin, false>(p, lo, part, nct, s);
    if (e != hipSuccess) return e;
  }
  hipLaunchKernelGGL(glr_param_kernel, grid_of<1024>(int64_t(12) * nct), dim3(1024), 0, s, part, p.lam, p.decay_scale,
                     p.dlam, p.dr_bias, p.di_bias, p.batch, lo.tiles, p.dim, nct);
  return hipGetLastError();
}

}  // namespace

size_t glr_bwd_workspace_bytes(int64_t batch, int64_t L, int64_t dim) {
  const GlrChainLayout lo(batch, L, dim, 1);
  return lo.bytes() + ((static_cast<size_t>(lo.chains) * lo.tiles * 3 * 64 * 4 + 255) & ~size_t(255));
}

hipError_t launch_glr_bwd(const GlrBwdParams& p, bool bf16, hipStream_t s) {
  return bf16 ? launch_t<bf16_t>(p, s) : launch_t<float>(p, s);
}

}  // namespace sscan
