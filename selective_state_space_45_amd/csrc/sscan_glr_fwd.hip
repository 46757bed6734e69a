// Gated linear recurrence, forward.
#include "sscan_glr_tile.h"

namespace sscan {

// Exponent fields and codes of a wave's 16 tokens of one tensor, for V channels of a lane.
// FULL: 16 tokens; otherwise the first `valid` of `rows` count, the others as zeros.
template <typename Tin, int V, bool LINES, bool FULL>
__device__ __forceinline__ void glr_save(const typename TokVec<Tin, V>::reg (&raw)[kActGroup], int valid, int rows,
                                         int8_t* codes, uint8_t* exps, int64_t dim, uint32_t c, bool mine) {
  typedef TokVec<Tin, V> Tok;
  typedef typename std::conditional<V == 2, uint16_t, uint8_t>::type word;
  typename Tok::reg top = {};
#pragma unroll
  for (int k = 0; k < kActGroup; ++k)
    if (FULL || k < valid) top = Tok::top(top, raw[k]);
  int shift[V];
  uint32_t fields = 0;
#pragma unroll
  for (int v = 0; v < V; ++v) {
    const uint32_t f = Tok::field(top, v);
    shift[v] = act8_shift(f);
    fields |= f << (8 * v);
  }
  if (!mine) return;
  c = here(c);
  row_store<word, LINES>(exps, c, static_cast<word>(fields));
#pragma unroll
  for (int k = 0; k < kActGroup; ++k) {
    uint32_t q = act8_code(Tok::get(raw[k], 0), shift[0]);
    if (V == 2) q = __builtin_amdgcn_perm(act8_code(Tok::get(raw[k], V - 1), shift[V - 1]), q, 0x0c0c0400u);
    if (!FULL && k >= valid) q = 0;
    if (FULL || k < rows) row_store<word, LINES>(codes, c, static_cast<word>(q));
    codes += dim;
  }
}

// One tile.  8 bytes an element in bf16 (10 with a gate) against about 20 vector
// operations and 6 of the quarter-rate ones, whose time is three quarters of the memory's.
// The map of a wave's 16 tokens needs each of them once, and so does the output: a and u
// stay in registers between the two while the state is on its way, and four waves a SIMD
// cover that wait.  8 x 4096 x 2048 bf16: 0.128 ms, 4.2 TB/s (a large copy reaches 4.9);
// gated 0.145 ms, 4.6 TB/s; 2 x 2048 x 1536 float32: 19 us, 5.3 TB/s.  The gated packed
// form of two channels a lane spills 2 (float32: 8 to 12) of its registers.
template <typename Tin, int V, bool LINES, bool PACKED, bool GATE, bool SAVE>
__global__ __launch_bounds__(64 * kGlrWaves, V == 2 && (GATE && sizeof(Tin) == 4) ? 3 : 4) void glr_fwd_kernel(
    GlrFwdParams p, GlrChainWords words, int ntiles, int nct) {
  typedef TokVec<Tin, V> Tok;
  constexpr int K = kActGroup, W = kGlrWaves;
  __shared__ float sA[W][V][64], sB[W][V][64], sH[V][64];
  __shared__ int sReset[W], sTile;
  const int w = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6), lane = threadIdx.x & 63;
  const uint32_t nchains = static_cast<uint32_t>(p.batch) * nct, block = workgroup<64 * kGlrWaves>();
  const uint32_t chain = glr_chain(block, nchains);
  int tile = 0;
  if (ntiles > 1) {
    if (threadIdx.x == 0)
      sTile = static_cast<int>(atomicAdd(&words.tickets[static_cast<size_t>(chain) * kGlrTicket], 1u));
    __syncthreads();
    tile = __builtin_amdgcn_readfirstlane(sTile);
    if (tile >= ntiles) return;   // a grid that is filled up has more workgroups than tiles
  } else if (block >= nchains) {
    return;
  }
  const int64_t b = chain / nct;
  const int64_t c0 = static_cast<int64_t>(chain % nct) * (64 * V);
  const int64_t D = p.dim, L = p.L;
  // lanes past the last channel work on the last ones and store nothing
  const int64_t cl = c0 + lane * V;
  const bool mine = cl < D;
  const uint32_t c = static_cast<uint32_t>(mine ? cl : D - V), cb = c * sizeof(Tin);
  const int L32 = static_cast<int>(L), t0 = tile * kGlrTile + w * K;
  const int rows = L32 - t0 < 0 ? 0 : (L32 - t0 < K ? L32 - t0 : K);

  // 16 tokens of each input; tokens past the row's end read its last one
  typename Tok::reg rx[K], rr[K], ri[K], rz[K];
  {
    const int64_t t = b * L + (rows ? t0 : L - 1);
    const Tin* px = static_cast<const Tin*>(p.x) + t * p.sx;
    const Tin* pr = static_cast<const Tin*>(p.r) + t * p.sr;
    const Tin* pi = static_cast<const Tin*>(p.i) + t * p.si;
    const Tin* pz = GATE ? static_cast<const Tin*>(p.z) + t * p.sz : nullptr;
    auto load = [&](auto full) __attribute__((always_inline)) {
      const uint32_t at = here(cb);
#pragma unroll
      for (int k = 0; k < K; ++k) {
        rx[k] = row_load<typename Tok::word, LINES>(px, at);
        rr[k] = row_load<typename Tok::word, LINES>(pr, at);
        ri[k] = row_load<typename Tok::word, LINES>(pi, at);
        if (GATE) rz[k] = row_load<typename Tok::word, LINES>(pz, at);
        const int64_t more = decltype(full)::value || k + 1 < rows ? 1 : 0;
        px += more * p.sx, pr += more * p.sr, pi += more * p.si;
        if (GATE) pz += more * p.sz;
      }
      apart<decltype(full)::value>();
    };
    if (rows == K) load(std::true_type{});
    else load(std::false_type{});
  }
  GlrSpan sp;
  sp.valid = rows;
  if (PACKED) sp = glr_span(p.offsets, static_cast<int>(p.num_seqs), t0, L32);

  float rate[V], nrb[V], nib[V];   // times log2(e); the biases negated
#pragma unroll
  for (int v = 0; v < V; ++v) {
    rate[v] = p.decay_scale * softplus_acc(p.lam[c + v]) * kLog2e;
    nrb[v] = p.r_bias ? -kLog2e * p.r_bias[c + v] : 0.f;
    nib[v] = p.i_bias ? -kLog2e * p.i_bias[c + v] : 0.f;
  }
  if (SAVE && rows > 0) {
    const int64_t row0 = b * L + t0, group = b * ((L + K - 1) / K) + t0 / K;
    auto save = [&](int q, const typename Tok::reg(&raw)[K]) __attribute__((always_inline)) {
      int8_t* codes = p.codes + q * p.saved_stride;
      uint8_t* exps = reinterpret_cast<uint8_t*>(codes) + p.exps_at;
      if (sp.valid == K) glr_save<Tin, V, LINES, true>(raw, K, K, codes + row0 * D, exps + group * D, D, c, mine);
      else glr_save<Tin, V, LINES, false>(raw, sp.valid, rows, codes + row0 * D, exps + group * D, D, c, mine);
    };
    save(0, rx);
    save(1, rr);
    save(2, ri);
    if (GATE) save(3, rz);
  }

  // each token's map h -> a h + u, and the wave's
  float a[K][V], u[K][V], A[V], B[V];
#pragma unroll
  for (int k = 0; k < K; ++k)
#pragma unroll
    for (int v = 0; v < V; ++v) {
      float one;
      a[k][v] = decay_of(rate[v] * gate(Tok::get(rr[k], v), nrb[v]), one);
      u[k][v] = hw_sqrt(one) * (gate(Tok::get(ri[k], v), nib[v]) * Tok::get(rx[k], v));
    }
  if (sp.valid < K) {   // tokens past the end leave the state alone
#pragma unroll
    for (int k = 0; k < K; ++k)
      if (k >= sp.valid)
#pragma unroll
        for (int v = 0; v < V; ++v) a[k][v] = 1.f, u[k][v] = 0.f;
  }
  // a sequence's first token: its state depends on the sequence's initial one only.  The
  // last states may overwrite the initial ones, so each is read once, here.
  float first[V] = {};
  if (PACKED && sp.starts && p.h0) {
#pragma unroll
    for (int k = 0; k < K; ++k)
      if (sp.starts >> k & 1) {
        const float* from = p.h0 + static_cast<int64_t>(sp.seq_of(k)) * D + c;
#pragma unroll
        for (int v = 0; v < V; ++v) {
          const float h = from[v];
          u[k][v] = fmaf(a[k][v], h, u[k][v]);
          if (k == 0) first[v] = h;
        }
      }
  }
#pragma unroll
  for (int v = 0; v < V; ++v) {
    A[v] = a[0][v], B[v] = u[0][v];
#pragma unroll
    for (int k = 1; k < K; ++k) {
      const bool start = PACKED && (sp.starts >> k & 1);
      A[v] *= a[k][v];
      B[v] = start ? u[k][v] : fmaf(a[k][v], B[v], u[k][v]);
    }
    sA[w][v][lane] = A[v];
    sB[w][v][lane] = B[v];
  }
  if (PACKED && lane == 0) sReset[w] = sp.starts != 0;
  __syncthreads();

  // wave v < V joins the waves' maps of channel set v, publishes, and looks back
  if (w < V) {
    float h = 0.f;
    if (!PACKED && p.h0 && tile == 0) h = p.h0[b * D + c + w];
    if (ntiles > 1) {
      GlrMap all{sA[0][w][lane], sB[0][w][lane], PACKED && sReset[0]};
#pragma unroll
      for (int q = 1; q < W; ++q) all = GlrMap{sA[q][w][lane], sB[q][w][lane], PACKED && sReset[q]}.after(all);
      h = glr_pass<64 * V>(words, chain, w * 64 + lane, tile, ntiles, all, h);
    }
    sH[w][lane] = h;
  }
  __syncthreads();
  if (rows == 0) return;

  float h[V];
#pragma unroll
  for (int v = 0; v < V; ++v) h[v] = sH[v][lane];
#pragma unroll
  for (int q = 0; q < W - 1; ++q) {
    if (q >= w) break;
    const bool qr = PACKED && __builtin_amdgcn_readfirstlane(sReset[q]);
#pragma unroll
    for (int v = 0; v < V; ++v) h[v] = qr ? sB[q][v][lane] : fmaf(sA[q][v][lane], h[v], sB[q][v][lane]);
  }
  if (p.ckpt && w == 0 && mine) {
    float* ck = p.ckpt + (b * ((L + kGlrBlock - 1) / kGlrBlock) + tile) * D + c;
    const bool start = PACKED && (sp.starts & 1);
#pragma unroll
    for (int v = 0; v < V; ++v) ck[v] = start ? first[v] : h[v];
  }
  if (!mine) return;
  Tin* yrow = static_cast<Tin*>(p.y) + (b * L + t0) * D;
  uint32_t at = cb;
  auto out = [&](int k) __attribute__((always_inline)) {
    const bool start = PACKED && (sp.starts >> k & 1);
    float y[V];
#pragma unroll
    for (int v = 0; v < V; ++v) {
      h[v] = start ? u[k][v] : fmaf(a[k][v], h[v], u[k][v]);
      y[v] = GATE ? h[v] * silu(Tok::get(rz[k], v)) : h[v];
      if (PACKED && k >= sp.valid) y[v] = 0.f;
    }
    row_store<typename Tok::word, LINES>(yrow, at, Tok::put(y));
    yrow += D;
    if (PACKED && (sp.ends >> k & 1) && p.h_last) {
      float* hl = p.h_last + static_cast<int64_t>(sp.seq_of(k)) * D + c;
#pragma unroll
      for (int v = 0; v < V; ++v) hl[v] = h[v];
    }
  };
  if (rows == K) {
    at = here(cb);
#pragma unroll
    for (int k = 0; k < K; ++k) out(k);
    apart<true>();
  } else {
#pragma unroll
    for (int k = 0; k < K; ++k)
      if (k < rows) out(k);
    apart<false>();
  }
  if (!PACKED && p.h_last && t0 + K >= L32) {
#pragma unroll
    for (int v = 0; v < V; ++v) p.h_last[b * D + c + v] = h[v];
  }
}

// What comes before a launch over tiles: the chain's words (16 bytes a lane; the first
// `zeros` of them zero, the rest all ones), and in workgroups of their own the sequences
// without tokens, to[s] = from[s] (zero if from is null).
__global__ __launch_bounds__(256) void glr_begin_kernel(uint4* words, size_t zeros, size_t count, unsigned clearing,
                                                        const int32_t* offsets, int64_t rows, const float* from, float* to,
                                                        int64_t D) {
  if (blockIdx.x < clearing) {
    const size_t n = static_cast<size_t>(clearing) * 256;
    for (size_t k = static_cast<size_t>(blockIdx.x) * 256 + threadIdx.x; k < count; k += n) {
      const uint32_t v = k < zeros ? 0u : kNoWord;
      words[k] = make_uint4(v, v, v, v);
    }
    return;
  }
  for (int64_t s = blockIdx.x - clearing; s < rows; s += gridDim.x - clearing) {
    if (offsets && offsets[s] != offsets[s + 1]) continue;
    for (int64_t d = threadIdx.x; d < D; d += 256) to[s * D + d] = from ? from[s * D + d] : 0.f;
  }
}

hipError_t launch_glr_begin(void* ws, const GlrChainLayout& lo, const int32_t* offsets, int64_t rows, const float* from,
                            float* to, int64_t D, hipStream_t s) {
  const size_t count = lo.bytes() / 16;
  const unsigned clearing = static_cast<unsigned>((count + 1023) / 1024 < 2048 ? (count + 1023) / 1024 : 2048);
  const unsigned rest = to && to != from ? static_cast<unsigned>(rows < 256 ? rows : 256) : 0;
  if (clearing + rest == 0) return hipSuccess;
  hipLaunchKernelGGL(glr_begin_kernel, dim3(clearing + rest), dim3(256), 0, s, static_cast<uint4*>(ws), lo.maps_at / 16,
                     count, clearing, offsets, rows, from, to, D);
  return hipGetLastError();
}

namespace {

template <typename Tin, int V, bool LINES, bool PACKED, bool GATE>
void launch_save(const GlrFwdParams& p, const GlrChainLayout& lo, hipStream_t s) {
  const int nct = static_cast<int>((p.dim + 64 * V - 1) / (64 * V)), nt = static_cast<int>(lo.tiles);
  const dim3 grid = grid_of<64 * kGlrWaves>(lo.chains * lo.tiles), wg(64 * kGlrWaves);
  const GlrChainWords w = lo.at(p.workspace);
  if (p.codes) hipLaunchKernelGGL((glr_fwd_kernel<Tin, V, LINES, PACKED, GATE, true>), grid, wg, 0, s, p, w, nt, nct);
  else hipLaunchKernelGGL((glr_fwd_kernel<Tin, V, LINES, PACKED, GATE, false>), grid, wg, 0, s, p, w, nt, nct);
}

template <typename Tin, int V, bool LINES>
hipError_t launch_v(const GlrFwdParams& p, hipStream_t s) {
  const GlrChainLayout lo(p.batch, p.L, p.dim, V);
  // without tokens (or for the requests that have none) the last state is the initial one
  const bool some = p.offsets || p.L == 0;
  const hipError_t e = launch_glr_begin(p.workspace, lo, p.offsets, p.offsets ? p.num_seqs : p.batch, p.h0,
                                        some ? p.h_last : nullptr, p.dim, s);
  if (e != hipSuccess || p.L == 0) return e;
  if (p.offsets) p.z ? launch_save<Tin, V, LINES, true, true>(p, lo, s) : launch_save<Tin, V, LINES, true, false>(p, lo, s);
  else p.z ? launch_save<Tin, V, LINES, false, true>(p, lo, s) : launch_save<Tin, V, LINES, false, false>(p, lo, s);
  return hipGetLastError();
}

// Two channels a lane where every row of every tensor holds whole aligned pairs (one a
// lane: 8 x 4096 x 2048 bf16 gated 0.171 ms against 0.156, 1 x 131072 x 2560 0.765 against
// 0.626, 2 x 2048 x 1536 float32 27.8 us against 23.9), and rows streamed where each starts
// on a cache line.
template <typename Tin>
hipError_t launch_t(const GlrFwdParams& p, hipStream_t s) {
  uintptr_t bits = static_cast<uintptr_t>(p.sx | p.sr | p.si | (p.z ? p.sz : 0) | p.dim) * sizeof(Tin);
  for (const void* q : {p.x, p.r, p.i, p.z, static_cast<const void*>(p.y)}) bits |= reinterpret_cast<uintptr_t>(q);
  if (p.codes) bits |= static_cast<uintptr_t>(p.dim);   // the codes' rows
  if (bits % kCacheLine == 0) return launch_v<Tin, 2, true>(p, s);
  return bits % (2 * sizeof(Tin)) == 0 ? launch_v<Tin, 2, false>(p, s) : launch_v<Tin, 1, false>(p, s);
}

}  // namespace

size_t glr_fwd_workspace_bytes(int64_t batch, int64_t L, int64_t dim) {
  // enough for one and for two channels a lane
  const size_t a = GlrChainLayout(batch, L, dim, 1).bytes(), b = GlrChainLayout(batch, L, dim, 2).bytes();
  return a > b ? a : b;
}

hipError_t launch_glr_fwd(const GlrFwdParams& p, bool bf16, hipStream_t s) {
  return bf16 ? launch_t<bf16_t>(p, s) : launch_t<float>(p, s);
}

}  // namespace sscan
