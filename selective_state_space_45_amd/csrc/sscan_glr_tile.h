// Tiles of the gated linear recurrence: how its forward and backward kernels cut the
// work, load it, and pass the state from one tile to the next.
//
// A tile is 64 V neighbouring channels of one batch row (V per lane) over kGlrTile
// consecutive tokens; wave w of its workgroup holds tokens 16 w .. 16 w + 15 in
// registers.  The tiles of one batch row and channel range form a chain.  A run of
// tokens is an affine map of the state that enters it, h -> A h + B, so each wave first
// forms its own (A, B), the workgroup joins them, and the state entering the tile comes
// from the tile before by a single pass over memory (GlrChain below): every input is
// read once whatever the length, and a long sequence of few channels still fills the
// chip, since all its tiles are workgroups of their own.
#pragma once

#include "sscan_glr.h"

namespace sscan {

constexpr int kGlrWaves = kGlrBlock / kActGroup;   // waves of a tile, 16 tokens each
constexpr int kGlrTile = kGlrBlock;                // tokens of a tile: the spacing of saved states
constexpr int kGlrWindow = 8;                      // tiles that one look back covers

// V channels of one token: loaded and stored as one word per lane.
template <typename Tin, int V>
struct TokVec;

template <>
struct TokVec<bf16_t, 1> {
  typedef uint32_t reg;
  static __device__ __forceinline__ reg load(const bf16_t* p) { return *p; }
  static __device__ __forceinline__ float get(reg r, int) { return __uint_as_float(r << 16); }
  static __device__ __forceinline__ void store(bf16_t* p, const float* v) { store_val(p, v[0]); }
};
template <>
struct TokVec<bf16_t, 2> {
  typedef uint32_t reg;
  static __device__ __forceinline__ reg load(const bf16_t* p) { return *reinterpret_cast<const uint32_t*>(p); }
  static __device__ __forceinline__ float get(reg r, int v) { return __uint_as_float(v ? r & 0xffff0000u : r << 16); }
  static __device__ __forceinline__ void store(bf16_t* p, const float* v) {
    typedef __bf16 b2 __attribute__((ext_vector_type(2)));
    typedef float f2 __attribute__((ext_vector_type(2)));
    *reinterpret_cast<b2*>(p) = __builtin_convertvector((f2{v[0], v[1]}), b2);
  }
};
template <>
struct TokVec<float, 1> {
  typedef float reg;
  static __device__ __forceinline__ reg load(const float* p) { return *p; }
  static __device__ __forceinline__ float get(reg r, int) { return r; }
  static __device__ __forceinline__ void store(float* p, const float* v) { *p = v[0]; }
};
template <>
struct TokVec<float, 2> {
  typedef float reg __attribute__((ext_vector_type(2)));
  static __device__ __forceinline__ reg load(const float* p) { return *reinterpret_cast<const reg*>(p); }
  static __device__ __forceinline__ float get(reg r, int v) { return v ? r.y : r.x; }
  static __device__ __forceinline__ void store(float* p, const float* v) { *reinterpret_cast<reg*>(p) = reg{v[0], v[1]}; }
};

// The sequences that a wave's 16 tokens t0 .. t0 + 15 belong to (packed requests).
struct GlrSpan {
  uint32_t starts = 0, ends = 0;   // bit k: token t0 + k begins / ends its sequence
  int valid;                       // tokens of the wave that are no padding: 0 .. 16
  int seq = 0;                     // lane k (mod 16): the sequence of token t0 + k
  __device__ int seq_of(int k) const { return __builtin_amdgcn_readlane(seq, k); }
};

// Each of 16 lanes finds its token's sequence by bisection: the number of offsets[1 ..]
// at or below the token.  The loads run beside those of the tokens.  Any contents of
// offsets give indices inside [0, num_seqs).
__device__ __forceinline__ GlrSpan glr_span(const int32_t* offsets, int num_seqs, int64_t t0, int64_t L) {
  GlrSpan sp;
  const int t = static_cast<int>(t0) + static_cast<int>(threadIdx.x & 15);
  int lo = 0, n = num_seqs;
  while (n > 0) {
    const int half = n >> 1;
    const bool right = offsets[1 + lo + half] <= t;
    lo = right ? lo + half + 1 : lo;
    n = right ? n - half - 1 : half;
  }
  const bool used = lo < num_seqs && t < L;
  sp.seq = lo < num_seqs ? lo : num_seqs - 1;
  const int begin = offsets[sp.seq], end = offsets[sp.seq + 1];
  const uint32_t in = static_cast<uint32_t>(__ballot(used)) & 0xffffu;
  sp.starts = static_cast<uint32_t>(__ballot(used && begin == t)) & 0xffffu;
  sp.ends = static_cast<uint32_t>(__ballot(used && end == t + 1)) & 0xffffu;
  sp.valid = __builtin_popcount(in);   // padding is at the tail: the used tokens come first
  return sp;
}

// ---------------------------------------------------------------------------
// The chain.  Tile k publishes its map (A, B) as soon as it has it, and the state it
// leaves once it knows the one that enters.  A later tile looks back over the window of
// tiles before it for the nearest state, and applies the maps between, in order: the
// same operations as going tile by tile, so results do not depend on timing.  Tiles
// that contain a sequence's start know the state they leave at once.
//
// Each published word carries its own readiness: a word of all ones (which a fill
// kernel writes before) is no value, and a value that would be all ones, a NaN, is
// stored as another NaN.  So one relaxed atomic access, coherent across the XCDs, both
// tests and reads; no other memory passes between tiles, and no order beyond that of
// the word itself is needed.
//
// Every wait ends: a workgroup takes its tile's number from the chain's counter, so the
// tiles it may wait for were taken by workgroups that have already begun, and the
// earliest tile waits for none.
// ---------------------------------------------------------------------------
struct GlrChainWords {
  uint32_t* tickets;   // [chains], zero
  uint64_t* maps;      // [chains][tiles][64 V], all ones
  uint32_t* states;    // [chains][tiles][64 V], all ones
};

// Bytes of a launch's words: tickets (to a multiple of 256), maps, states.
struct GlrChainLayout {
  int64_t chains, tiles, lanes;
  size_t maps_at, states_at, total;
  GlrChainLayout(int64_t batch, int64_t L, int64_t dim, int V) {
    lanes = 64 * V;
    chains = batch * ((dim + lanes - 1) / lanes);
    tiles = (L + kGlrTile - 1) / kGlrTile;
    maps_at = (static_cast<size_t>(chains) * 4 + 255) & ~size_t(255);
    states_at = maps_at + static_cast<size_t>(chains) * tiles * lanes * 8;
    total = states_at + static_cast<size_t>(chains) * tiles * lanes * 4;
  }
  // a single tile needs no words
  size_t bytes() const { return tiles > 1 ? (total + 255) & ~size_t(255) : 0; }
  GlrChainWords at(void* ws) const {
    char* p = static_cast<char*>(ws);
    return {reinterpret_cast<uint32_t*>(p), reinterpret_cast<uint64_t*>(p + maps_at),
            reinterpret_cast<uint32_t*>(p + states_at)};
  }
};

constexpr uint32_t kNoWord = 0xffffffffu;
__device__ __forceinline__ uint32_t word_of(float v) {
  const uint32_t b = __float_as_uint(v);
  return b == kNoWord ? 0x7fc00000u : b;
}

// One wave's view of the chain: 64 of the tile's channels, one per lane.
struct GlrChain {
  GlrChainWords w;
  int64_t first;     // index of the words of tile 0 of the chain, for this lane
  int64_t pitch;     // words from one tile to the next
  int tile;          // position in the chain, from the end that is computed first

  __device__ void publish_map(float A, float B) const {
    __hip_atomic_store(&w.maps[first + tile * pitch], (static_cast<uint64_t>(word_of(B)) << 32) | __float_as_uint(A),
                       __ATOMIC_RELAXED, __HIP_MEMORY_SCOPE_AGENT);
  }
  __device__ void publish_state(float h) const {
    __hip_atomic_store(&w.states[first + tile * pitch], word_of(h), __ATOMIC_RELAXED, __HIP_MEMORY_SCOPE_AGENT);
  }

  // The state that enters this tile (tile > 0).  Called by all 64 lanes.
  __device__ float look_back() const {
    const int n = tile < kGlrWindow ? tile : kGlrWindow;
    for (;;) {
      uint32_t st[kGlrWindow];
      uint64_t mp[kGlrWindow];
#pragma unroll
      for (int k = 0; k < kGlrWindow; ++k) {
        const int64_t at = first + (tile - 1 - (k < n ? k : n - 1)) * pitch;   // past the chain's begin: a tile again, unused
        st[k] = __hip_atomic_load(&w.states[at], __ATOMIC_RELAXED, __HIP_MEMORY_SCOPE_AGENT);
        mp[k] = __hip_atomic_load(&w.maps[at], __ATOMIC_RELAXED, __HIP_MEMORY_SCOPE_AGENT);
      }
      // the nearest tile whose state is there for every lane, with all maps between
      int found = -1;
      bool maps = true;
#pragma unroll
      for (int k = 0; k < kGlrWindow; ++k) {
        if (found < 0 && maps && k < n && __all(st[k] != kNoWord)) found = k;
        maps = maps && __all(static_cast<uint32_t>(mp[k] >> 32) != kNoWord);
      }
      if (found >= 0) {
        float h = 0.f;
#pragma unroll
        for (int k = kGlrWindow - 1; k >= 0; --k) {
          const float A = __uint_as_float(static_cast<uint32_t>(mp[k])), B = __uint_as_float(static_cast<uint32_t>(mp[k] >> 32));
          h = k == found ? __uint_as_float(st[k]) : (k < found ? fmaf(A, h, B) : h);
        }
        return h;
      }
      __builtin_amdgcn_s_sleep(1);
    }
  }
};

// Fills the words before a launch: tickets with zeros, the rest with ones.
hipError_t launch_glr_clear(void* ws, const GlrChainLayout& lo, hipStream_t s);
// to[s] = from[s] (zero if null), for the sequences without tokens (all, if offsets is null).
hipError_t launch_glr_empty(const int32_t* offsets, const float* from, float* to, int64_t rows, int64_t D, hipStream_t s);

}  // namespace sscan
