// Tiles of the gated linear recurrence: how its forward and backward kernels cut the
// work, load it, and pass the state from one tile to the next.
//
// A tile is 64 V neighbouring channels of one batch row (V per lane) over kGlrTile
// consecutive tokens; wave w of its workgroup holds tokens 16 w .. 16 w + 15 in
// registers.  The tiles of one batch row and channel range form a chain.  A run of
// tokens is an affine map of the state that enters it, h -> A h + B, so each wave first
// forms its own (A, B), the workgroup joins them, and the state entering the tile comes
// from the tile before by a single pass over memory (glr_pass below): every input is
// read once whatever the length, and a long sequence of few channels still fills the
// chip, since all its tiles are workgroups of their own.  (Workgroups of 8 waves and 128
// tokens: 8 x 4096 x 2048 bf16 gated 0.192 ms against 0.164, with the chain as it then
// was.  Workgroups that stay and take tile after tile, with or without the next one's
// tokens already in registers: 0.18 and 0.29 against 0.154, for the registers they take.)
#pragma once

#include "sscan_glr.h"

namespace sscan {

constexpr int kGlrWaves = kGlrBlock / kActGroup;   // waves of a tile, 16 tokens each
constexpr uintptr_t kCacheLine = 128;
constexpr int kGlrTile = kGlrBlock;                // tokens of a tile: the spacing of saved states

// An element `at` bytes into a row that is the same for the whole wave: the row's address
// in scalar registers and the lane's 32-bit offset are added in the load itself.  The
// empty asm keeps the compiler from adding the offset to a common base first, which
// leaves a 64-bit vector addition to every load.  LINES: the wave's rows are whole cache
// lines; then they are streamed, since nothing here reads them again (forward and
// backward at 8 x 4096 x 2048 bf16: 0.372 ms, 0.396 without).  Lines that two waves share
// gain from staying (2 x 2047 x 1535 float32: 0.135 ms streamed, 0.120 not).
template <typename T>
using GlobalPtr = __attribute__((address_space(1))) T*;
template <typename T, bool LINES>
__device__ __forceinline__ T row_load(const void* row, uint32_t at) {
  uintptr_t r = reinterpret_cast<uintptr_t>(row);
  asm("" : "+s"(r));
  const GlobalPtr<const T> p = reinterpret_cast<GlobalPtr<const T>>(r + at);
  return LINES ? __builtin_nontemporal_load(p) : *p;
}
template <typename T, bool LINES>
__device__ __forceinline__ void row_store(void* row, uint32_t at, T v) {
  uintptr_t r = reinterpret_cast<uintptr_t>(row);
  asm("" : "+s"(r));
  const GlobalPtr<T> p = reinterpret_cast<GlobalPtr<T>>(r + at);
  if (LINES) __builtin_nontemporal_store(v, p);
  else *p = v;
}

// A lane's offset, to be used in one block of code: the compiler then sees there that it
// has 32 bits, which the load's form needs.
__device__ __forceinline__ uint32_t here(uint32_t at) {
  asm("" : "+v"(at));
  return at;
}

// A row's stride, to be added from row to row: known to the compiler it becomes all its
// multiples, for which there are not the scalar registers.
__device__ __forceinline__ int64_t step(int64_t stride) {
  asm volatile("" : "+s"(stride));
  return stride;
}

// Marks the begin and the end of the code for a whole wave of 16 tokens and of that for a
// short one: where they are alike the compiler takes them together before or after the
// branch, with every address and product of either in vector registers.
template <bool FULL>
__device__ __forceinline__ void apart() {
  if (FULL) asm volatile("; 16 tokens");
  else asm volatile("; fewer");
}

// V channels of one token: one word per lane.  top: the word's magnitudes, whose maxima
// over words give the largest exponents.
template <typename Tin, int V>
struct TokVec;

template <>
struct TokVec<bf16_t, 1> {
  typedef uint32_t reg;
  typedef bf16_t word;
  static __device__ __forceinline__ float get(reg r, int) { return __uint_as_float(r << 16); }
  static __device__ __forceinline__ word put(const float* v) { return __builtin_bit_cast(bf16_t, static_cast<__bf16>(v[0])); }
  static __device__ __forceinline__ reg top(reg t, reg r) { return (r & 0x7fffu) > t ? r & 0x7fffu : t; }
  static __device__ __forceinline__ uint32_t field(reg t, int) { return t >> 7; }
};
template <>
struct TokVec<bf16_t, 2> {
  typedef uint32_t reg;
  typedef uint32_t word;
  static __device__ __forceinline__ float get(reg r, int v) { return __uint_as_float(v ? r & 0xffff0000u : r << 16); }
  static __device__ __forceinline__ word put(const float* v) {
    typedef __bf16 b2 __attribute__((ext_vector_type(2)));
    typedef float f2 __attribute__((ext_vector_type(2)));
    return __builtin_bit_cast(uint32_t, __builtin_convertvector((f2{v[0], v[1]}), b2));
  }
  static __device__ __forceinline__ reg top(reg t, reg r) {
    typedef uint16_t u2 __attribute__((ext_vector_type(2)));
    return __builtin_bit_cast(uint32_t, __builtin_elementwise_max(__builtin_bit_cast(u2, t),
                                                                  __builtin_bit_cast(u2, r & 0x7fff7fffu)));
  }
  static __device__ __forceinline__ uint32_t field(reg t, int v) { return v ? t >> 23 : (t >> 7) & 255u; }
};
template <>
struct TokVec<float, 1> {
  typedef float reg;
  typedef float word;
  static __device__ __forceinline__ float get(reg r, int) { return r; }
  static __device__ __forceinline__ word put(const float* v) { return v[0]; }
  static __device__ __forceinline__ reg top(reg t, reg r) { return __uint_as_float(act8_top(__float_as_uint(t), r)); }
  static __device__ __forceinline__ uint32_t field(reg t, int) { return __float_as_uint(t) >> 23; }
};
template <>
struct TokVec<float, 2> {
  typedef float reg __attribute__((ext_vector_type(2)));
  typedef reg word;
  static __device__ __forceinline__ float get(reg r, int v) { return v ? r.y : r.x; }
  static __device__ __forceinline__ word put(const float* v) { return reg{v[0], v[1]}; }
  static __device__ __forceinline__ reg top(reg t, reg r) {
    return reg{TokVec<float, 1>::top(t.x, r.x), TokVec<float, 1>::top(t.y, r.y)};
  }
  static __device__ __forceinline__ uint32_t field(reg t, int v) { return __float_as_uint(v ? t.y : t.x) >> 23; }
};

// The sequences that a wave's 16 tokens t0 .. t0 + 15 belong to (packed requests).
struct GlrSpan {
  uint32_t starts = 0, ends = 0;   // bit k: token t0 + k begins / ends its sequence
  int valid;                       // tokens of the wave that are no padding: 0 .. 16
  int seq = 0;                     // lane k (mod 16): the sequence of token t0 + k
  __device__ int seq_of(int k) const { return __builtin_amdgcn_readlane(seq, k); }
};

// A token's sequence is the number of offsets[1 ..] at or below it, found by bisection.
// The wave looks for its first token's through the scalar cache, beside the tokens' own
// loads; only if a boundary falls among its tokens does each of 16 lanes look for its
// own.  (By vector loads alone, which return after those of the tokens, a prefill of 37
// requests, 16411 tokens of 2560 channels in bf16, takes 0.107 ms, so 0.102.)  Any
// contents of offsets give indices inside [0, num_seqs).
template <typename P>
__device__ __forceinline__ int glr_find(P offsets, int num_seqs, int t) {
  int lo = 0, n = num_seqs;
  while (n > 0) {
    const int half = n >> 1;
    const bool right = offsets[1 + lo + half] <= t;
    lo = right ? lo + half + 1 : lo;
    n = right ? n - half - 1 : half;
  }
  return lo;
}
__device__ __forceinline__ GlrSpan glr_span(const int32_t* offsets, int num_seqs, int t0, int L) {
  typedef const __attribute__((address_space(4))) int32_t* Scalar;
  const Scalar so = reinterpret_cast<Scalar>(reinterpret_cast<uintptr_t>(offsets));
  GlrSpan sp;
  sp.valid = 0;
  const int t = t0 < L ? t0 : L;
  const int s = glr_find(so, num_seqs, t);
  if (s >= num_seqs || t0 >= L) return sp;             // padding only
  const int begin = so[s], end = so[s + 1];            // begin <= t < end
  if (end >= t + 16) {
    sp.seq = s;
    sp.starts = begin == t;
    sp.ends = end == t + 16 ? 0x8000u : 0u;
    sp.valid = L - t0 < 16 ? L - t0 : 16;
    return sp;
  }
  const int mine = t + static_cast<int>(threadIdx.x & 15);
  const int q = glr_find(offsets, num_seqs, mine);
  const bool used = q < num_seqs && mine < L;
  sp.seq = q < num_seqs ? q : num_seqs - 1;
  const int first = offsets[sp.seq], past = offsets[sp.seq + 1];
  sp.starts = static_cast<uint32_t>(__ballot(used && first == mine)) & 0xffffu;
  sp.ends = static_cast<uint32_t>(__ballot(used && past == mine + 1)) & 0xffffu;
  // padding is at the tail: the used tokens come first
  sp.valid = __builtin_popcount(static_cast<uint32_t>(__ballot(used)) & 0xffffu);
  return sp;
}

// ---------------------------------------------------------------------------
// The chain.  Its tiles form groups of 8.  Every tile publishes its map (A, B) as soon
// as it has it; a group's last tile publishes the group's map, its tiles' maps joined in
// order, and, once it knows the state S_g that enters the group, the one that leaves,
// S_{g+1} = A_g S_g + B_g.  A tile waits for the maps before it in its group, which wait
// for nothing, and looks back over two groups for the nearest state there is, carried
// through the groups' maps after it and then the tiles'.  These are the same operations
// wherever the state is found: results do not depend on timing.  (131072 tokens of 2560
// channels in bf16, 20 chains: 0.79 ms with a state for every tile and 64 tiles looked
// back over, 0.71 with groups; after other steps 0.637 with groups of 4, 0.621 with 8 and
// four groups back, 0.607 with two back.  The same tiles without the wait: 0.56.)
//
// A map's A is at least 0; its sign bit marks a run that contains a sequence's start:
// what it leaves is B, whatever enters.
//
// Each published word carries its own readiness: a word of all ones (which a kernel
// writes before) is no value, and a value that would be all ones, a NaN, is
// stored as another NaN.  So one relaxed atomic access, coherent across the XCDs, both
// tests and reads; no other memory passes between tiles, and no order beyond that of
// the word itself is needed.
//
// Every wait ends: a workgroup takes its tile's number from the chain's counter, so the
// tiles it may wait for were taken by workgroups that have already begun, and the
// earliest tile waits for none.
// ---------------------------------------------------------------------------
constexpr int kGlrGroup = 8;   // tiles of a group
constexpr int kGlrBack = 2;    // groups that one look back covers

// Counters lie a cache line apart: side by side, all of a launch's first workgroups queue
// at a few lines, 4 us before the first load (2 x 2048 x 1536 float32: 28.7 us, apart 23.3).
constexpr int kGlrTicket = 32;

struct GlrChainWords {
  uint32_t* tickets;    // [chains], kGlrTicket words apart, zero
  uint64_t* maps;       // [chains][tiles][64 V], all ones
  uint64_t* group_maps; // [chains][groups][64 V], all ones
  uint32_t* states;     // [chains][groups][64 V], all ones
};

// Bytes of a launch's words: tickets (to a multiple of 256), then the others.
struct GlrChainLayout {
  int64_t chains, tiles, groups, lanes;
  size_t maps_at, group_maps_at, states_at, total;
  GlrChainLayout(int64_t batch, int64_t L, int64_t dim, int V) {
    lanes = 64 * V;
    chains = batch * ((dim + lanes - 1) / lanes);
    tiles = (L + kGlrTile - 1) / kGlrTile;
    groups = (tiles + kGlrGroup - 1) / kGlrGroup;
    maps_at = (static_cast<size_t>(chains) * kGlrTicket * 4 + 255) & ~size_t(255);
    group_maps_at = maps_at + static_cast<size_t>(chains) * tiles * lanes * 8;
    states_at = group_maps_at + static_cast<size_t>(chains) * groups * lanes * 8;
    total = states_at + static_cast<size_t>(chains) * groups * lanes * 4;
  }
  // a single tile needs no words
  size_t bytes() const { return tiles > 1 ? (total + 255) & ~size_t(255) : 0; }
  GlrChainWords at(void* ws) const {
    char* p = static_cast<char*>(ws);
    return {reinterpret_cast<uint32_t*>(p), reinterpret_cast<uint64_t*>(p + maps_at),
            reinterpret_cast<uint64_t*>(p + group_maps_at), reinterpret_cast<uint32_t*>(p + states_at)};
  }
};

// The chain of a workgroup.  Workgroups go round-robin over the 8 XCDs; two neighbouring
// chains share cache lines (of the 8-bit codes' rows, 64 bytes of 128 each in the backward,
// and of rows that start inside a line), so they go to one XCD: 16 chains are taken in the
// order 0, 2, .., 14, 1, 3, ..  (Forward and backward from 8 bits, 8 x 4096 x 2048: 0.404 ms,
// in plain order 0.418; 2 x 2047 x 1535 float32: 0.099 and 0.107.)
__device__ __forceinline__ uint32_t glr_chain(uint32_t block, uint32_t nchains) {
  const uint32_t c = block % nchains;
  return c < nchains / 16 * 16 ? (c & ~15u) | (c & 7u) << 1 | (c >> 3 & 1u) : c;
}

constexpr uint32_t kNoWord = 0xffffffffu;

// One lane's word of row `k` from a row of LANES words each, in one access that is coherent
// across the chip: the row's distance is part of the instruction (within its 4096 bytes).
template <int LANES, typename T>
__device__ __forceinline__ T word_load(const T* row, uint32_t lane, int k) {
  const GlobalPtr<T> at = reinterpret_cast<GlobalPtr<T>>(reinterpret_cast<uintptr_t>(row) + static_cast<uint32_t>(lane * sizeof(T)));
  return __hip_atomic_load(at + k * LANES, __ATOMIC_RELAXED, __HIP_MEMORY_SCOPE_AGENT);
}
template <typename T>
__device__ __forceinline__ void word_store(T* row, uint32_t lane, T v) {
  const GlobalPtr<T> at = reinterpret_cast<GlobalPtr<T>>(reinterpret_cast<uintptr_t>(row) + static_cast<uint32_t>(lane * sizeof(T)));
  __hip_atomic_store(at, v, __ATOMIC_RELAXED, __HIP_MEMORY_SCOPE_AGENT);
}

struct GlrMap {
  float A, B;
  bool reset;
  // this map after `before`
  __device__ GlrMap after(const GlrMap& before) const {
    return reset ? *this : GlrMap{A * before.A, fmaf(A, before.B, B), before.reset};
  }
  __device__ float operator()(float h) const { return reset ? B : fmaf(A, h, B); }
  __device__ uint64_t word() const {
    const uint32_t a = reset ? 0x80000000u : (A != A ? 0x7fc00000u : __float_as_uint(A));
    const uint32_t b = __float_as_uint(B);
    return (static_cast<uint64_t>(b == kNoWord ? 0x7fc00000u : b) << 32) | a;
  }
  static __device__ GlrMap of(uint64_t w) {
    const uint32_t a = static_cast<uint32_t>(w);
    return {__uint_as_float(a), __uint_as_float(static_cast<uint32_t>(w >> 32)), (a >> 31) != 0};
  }
};
__device__ __forceinline__ bool there(uint64_t w) { return static_cast<uint32_t>(w >> 32) != kNoWord; }

// One wave's part of the chain: 64 of the tile's channels, one per lane.  pos: the tile's
// place in the chain, of ntiles > 1.  own: the tile's map; initial: the state that
// enters the chain (read at pos 0 only).  Returns the state that enters the tile.  All 64
// lanes call it.
template <int LANES>
__device__ __forceinline__ float glr_pass(const GlrChainWords& w, int64_t chain, uint32_t lane, int pos, int ntiles,
                                          const GlrMap& own, float initial) {
  const int g = pos / kGlrGroup, j = pos % kGlrGroup, ngroups = (ntiles + kGlrGroup - 1) / kGlrGroup;
  // words of the tile's group, of the group before it, and of the state that enters it
  uint64_t* maps = w.maps + (chain * ntiles + g * kGlrGroup) * LANES;
  uint64_t* gmaps = w.group_maps + (chain * ngroups + g) * LANES;
  uint32_t* states = w.states + (chain * ngroups + g) * LANES;
  auto put_state = [&](int group, float h) {
    const uint32_t b = __float_as_uint(h);
    word_store(states + (group - g) * LANES, lane, b == kNoWord ? 0x7fc00000u : b);
  };
  if (pos == 0) put_state(0, initial);
  const bool closes = j == kGlrGroup - 1 && g + 1 < ngroups;   // the last tile of a group with another after it
  if (j < kGlrGroup - 1 && pos + 1 < ntiles)
    word_store(maps + j * LANES, lane, own.word());
  if (pos == 0) return initial;

  uint64_t m[kGlrGroup - 1];
  bool have = false;
  GlrMap all = own;
  for (;;) {
    uint32_t s[kGlrBack];
    uint64_t gm[kGlrBack];
    if (!have)
#pragma unroll
      for (int k = 0; k < kGlrGroup - 1; ++k)
        if (k < j) m[k] = k < 4 ? word_load<LANES>(maps, lane, k) : word_load<LANES>(maps + 4 * LANES, lane, k - 4);
#pragma unroll
    for (int k = 0; k < kGlrBack; ++k) {
      s[k] = kNoWord;
      gm[k] = ~uint64_t(0);
      if (k <= g) {
        s[k] = word_load<LANES>(states, lane, -k);
        if (k + 1 <= g && k + 1 < kGlrBack)
          gm[k] = word_load<LANES>(gmaps, lane, -(k + 1));
      }
    }
    if (!have) {
      bool ok = true;
#pragma unroll
      for (int k = 0; k < kGlrGroup - 1; ++k) ok = ok && (k >= j || there(m[k]));
      have = __all(ok);
      if (have && closes) {
        all = GlrMap::of(m[0]);
#pragma unroll
        for (int k = 1; k < kGlrGroup - 1; ++k) all = GlrMap::of(m[k]).after(all);
        all = own.after(all);
        if (__all(all.reset)) put_state(g + 1, all.B);
        else word_store(gmaps, lane, all.word());
      }
    }
    int found = -1;
    bool through = true;
#pragma unroll
    for (int k = 0; k < kGlrBack; ++k) {
      if (found < 0 && through && __all(s[k] != kNoWord)) found = k;
      through = through && __all(there(gm[k]));
    }
    if (have && found >= 0) {
      float h = 0.f;
#pragma unroll
      for (int k = kGlrBack - 1; k >= 0; --k)
        h = k == found ? __uint_as_float(s[k]) : (k < found ? GlrMap::of(gm[k])(h) : h);
      if (closes && !__all(all.reset)) put_state(g + 1, all(h));
#pragma unroll
      for (int k = 0; k < kGlrGroup - 1; ++k)
        if (k < j) h = GlrMap::of(m[k])(h);
      return h;
    }
    __builtin_amdgcn_s_sleep(1);
  }
}

// Fills the chain's words before a launch (tickets with zeros, the rest with ones), and
// sets to[s] = from[s] (zero if null) for the sequences without tokens: those of equal
// offsets, or all if offsets is null.
hipError_t launch_glr_begin(void* ws, const GlrChainLayout& lo, const int32_t* offsets, int64_t rows, const float* from,
                            float* to, int64_t D, hipStream_t s);

}  // namespace sscan
