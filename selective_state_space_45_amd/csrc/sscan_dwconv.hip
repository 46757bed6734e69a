// Depthwise causal convolution over time, dense or packed: forward, backward, one token.
//
// Bound by memory, and the backward nearly as much by its arithmetic.  A wave runs along a block of
// tokens of one batch row with neighbouring channels in its lanes, 8 bytes of a row each, the
// inputs of the last taps in registers and the next rows already on their way, so that each row is
// read once but for the few that two blocks share.  Rows need no alignment beyond their elements'.
// Where a sequence begins and ends is the same for the whole wave: it is looked up once per block
// and then followed in scalar registers.  Tokens go in groups of as many as are on their way:
// a group inside one sequence without a test or a move, any other by a loop over its tokens (with
// the tests in every token the forward of 8 x 4096 x 2048 bf16 took 66 us, now 51; the backward
// 132, now 108).  At 5 TB/s their reads and writes take 54 and 81 us; the backward issues about
// 130 vector instructions for each 4 channels of a token and wave, some 60 us of them.  Rows of fewer
// than 256 bf16 channels leave lanes repeating the last word: 524288 x 64 forward 57 us of 27, backward 132
// of 40 (131072 x 256: 26 and 48).
#include "sscan_layer.h"

namespace sscan {

constexpr int kConvWaves = 4;   // waves of a workgroup, one block of tokens after another

// V neighbouring channels of a row, at any address its elements may have.
template <typename Tin, int V>
struct Word {
  typedef Tin vec __attribute__((ext_vector_type(V)));
  typedef vec any __attribute__((aligned(sizeof(Tin))));
  static __device__ __forceinline__ vec load(const Tin* row, uint32_t at) {
    uintptr_t r = reinterpret_cast<uintptr_t>(row);   // the row's address stays in scalar registers
    asm("" : "+s"(r));
    return *reinterpret_cast<__attribute__((address_space(1))) const any*>(r + at);
  }
  static __device__ __forceinline__ void store(Tin* row, uint32_t at, const float* v) {
    uintptr_t r = reinterpret_cast<uintptr_t>(row);
    asm("" : "+s"(r));
    vec out;
#pragma unroll
    for (int j = 0; j < V; ++j) {
      Tin e;
      store_val(&e, v[j]);
      out[j] = e;
    }
    *reinterpret_cast<__attribute__((address_space(1))) any*>(r + at) = out;
  }
};

// The sequence that the wave's token is in: tokens [lo, hi) of the batch row, index s among
// all sequences; padding has hi = kNone.  Whatever offsets holds, indexes stay in range.
constexpr int kNone = INT32_MAX;
struct Sequence {
  int64_t s;
  int lo, hi;
};
__device__ __forceinline__ void bounds(const int32_t* offsets, int nseq, int L, int t, Sequence& q) {
  const int from = offsets[q.s], to = offsets[q.s + 1];
  q.lo = from < 0 ? 0 : (from > t ? t : from);
  q.hi = to > L ? L : to;
  if (q.hi <= t) q.hi = kNone, q.lo = kNone;
}
// The last s from `lo` on with offsets[s] <= t, or lo.
__device__ __forceinline__ int last_begun(const int32_t* offsets, int lo, int nseq, int t) {
  int hi = nseq;
  while (hi - lo > 1) {
    const int mid = lo + (hi - lo) / 2;
    if (offsets[mid] <= t) lo = mid;
    else hi = mid;
  }
  return lo;
}
__device__ __forceinline__ Sequence sequence_of(const int32_t* offsets, int nseq, int L, int64_t b, int t) {
  if (!offsets) return {b, 0, L};
  Sequence q{last_begun(offsets, 0, nseq, t), 0, 0};
  bounds(offsets, nseq, L, t, q);
  return q;
}
// The sequence that begins at t, where one ended: the next, or one after empty ones, of which there
// may be any number.
__device__ __forceinline__ void follow(const int32_t* offsets, int nseq, int L, int t, Sequence& q) {
  if (!offsets) {
    q.lo = q.hi = kNone;
    return;
  }
  int s = static_cast<int>(q.s);
  if (s + 1 < nseq && offsets[s + 1] <= t) ++s;
  if (s + 1 < nseq && offsets[s + 1] <= t) s = last_begun(offsets, s + 1, nseq, t);
  q.s = s;
  bounds(offsets, nseq, L, t, q);
}

// Taps, bias and states of V channels.
template <int K, int V>
struct Taps {
  float w[K][V], b[V];
  __device__ __forceinline__ Taps(const ConvParams& p, int64_t c) {
#pragma unroll
    for (int v = 0; v < V; ++v) {
#pragma unroll
      for (int k = 0; k < K; ++k) w[k][v] = p.w[(c + v) * K + k];
      b[v] = p.b ? p.b[c + v] : 0.f;
    }
  }
};
// Element i of the state [sequences][dim][K - 1] of V channels (zeros without one).
template <int K, int V>
__device__ __forceinline__ void state_at(const float* state, int64_t s, int64_t dim, int64_t c, int i, float* out) {
#pragma unroll
  for (int v = 0; v < V; ++v) out[v] = state ? state[(s * dim + c + v) * (K - 1) + i] : 0.f;
}

__device__ __forceinline__ float silu_slope(float v) {
  const float g = sigmoid(v);
  return g * (1.f + v * (1.f - g));
}

// The work of a wave: its batch row, tokens t0 .. t1 - 1, and channels of a lane, of which
// those past the last whole word repeat it (and write the same values).
struct Part {
  int64_t b, c;
  int t0, t1;
  __device__ __forceinline__ Part(const ConvParams& p, uint32_t block, int tokens, int nblk, int nct, int V) {
    const int wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
    const int64_t set = block / nct;
    b = set / nblk;
    const int64_t t = (set - b * nblk) * (static_cast<int64_t>(kConvWaves) * tokens) + static_cast<int64_t>(wave) * tokens;
    t0 = static_cast<int>(t < p.L ? t : p.L);
    t1 = static_cast<int>(t + tokens < p.L ? t + tokens : p.L);
    c = (static_cast<int64_t>(block % nct) * 64 + (threadIdx.x & 63)) * V;
    if (c > p.dim - V) c = p.dim - V;
  }
};

// Inputs before token t of a sequence: of the row, or of the state before it.
template <typename Tin, int K, int V>
__device__ __forceinline__ void history(const ConvParams& p, const Sequence& q, const Tin* x, uint32_t at, int64_t c, int t,
                                        float (&in)[K][V]) {
#pragma unroll
  for (int j = 1; j < K; ++j) {
    float* to = in[K - 1 - j];
    if (q.hi == kNone) {
#pragma unroll
      for (int v = 0; v < V; ++v) to[v] = 0.f;
    } else if (t - j >= q.lo) {
      const typename Word<Tin, V>::vec r = Word<Tin, V>::load(x + (t - j) * p.sx, at);
#pragma unroll
      for (int v = 0; v < V; ++v) to[v] = to_f32(r[v]);
    } else {
      state_at<K, V>(p.h0, q.s, p.dim, c, K - 1 + (t - j - q.lo), to);
    }
  }
}

// One lane for each sequence and channel: the state after it.
template <typename Tin, int K>
__device__ __forceinline__ void last_state(const ConvParams& p, int64_t id) {
  if (!p.h_last || id >= p.num_seqs * p.dim) return;   // a grid that is filled up has more lanes
  const int64_t s = id / p.dim, c = id - s * p.dim;
  int64_t row0 = 0, lo = 0, hi = p.L;
  if (p.offsets) {
    lo = p.offsets[s] < 0 ? 0 : (p.offsets[s] > p.L ? p.L : p.offsets[s]);
    hi = p.offsets[s + 1] < lo ? lo : (p.offsets[s + 1] > p.L ? p.L : p.offsets[s + 1]);
  } else {
    row0 = s * p.L;
  }
#pragma unroll
  for (int j = 0; j < K - 1; ++j) {
    const int64_t t = hi - (K - 1) + j;
    p.h_last[id * (K - 1) + j] = t >= lo ? to_f32(static_cast<const Tin*>(p.x)[(row0 + t) * p.sx + c])
                                         : (p.h0 ? p.h0[id * (K - 1) + (K - 1) + (t - lo)] : 0.f);
  }
}

// Blocks of `tokens` tokens (a multiple of kRows).  Workgroups from `main` on write last states.
template <typename Tin, int K, int V>
__global__ __launch_bounds__(64 * kConvWaves) void dwconv_fwd_kernel(ConvParams p, const int32_t* __restrict__ offsets, int tokens,
                                                                     int nblk, int nct, uint32_t main) {
  constexpr int kRows = 4;      // rows on their way at a time
  typedef Word<Tin, V> W;
  const uint32_t block = workgroup<64 * kConvWaves>();
  if (block >= main) return last_state<Tin, K>(p, static_cast<int64_t>(block - main) * (64 * kConvWaves) + threadIdx.x);
  const Part at(p, block, tokens, nblk, nct, V);
  if (at.t0 >= at.t1) return;
  const int L = static_cast<int>(p.L), nseq = static_cast<int>(p.num_seqs);
  const Tin* x = static_cast<const Tin*>(p.x) + at.b * p.L * p.sx;
  Tin* y = static_cast<Tin*>(p.y) + at.b * p.L * p.dim;
  const uint32_t lane = static_cast<uint32_t>(at.c * sizeof(Tin));
  typename W::vec next[kRows];
  const auto load = [&](int t) {      // rows past the block's end repeat its last one
#pragma unroll
    for (int k = 0; k < kRows; ++k) next[k] = W::load(x + (t + k < at.t1 ? t + k : at.t1 - 1) * p.sx, lane);
  };
  load(at.t0);
  const Taps<K, V> taps(p, at.c);
  Sequence q = sequence_of(offsets, nseq, L, at.b, at.t0);
  float in[K][V];
  history<Tin, K, V>(p, q, x, lane, at.c, at.t0, in);
  const auto token = [&](int now, typename W::vec vx, auto with_silu) {
    float out[V];
#pragma unroll
    for (int v = 0; v < V; ++v) {
      in[K - 1][v] = to_f32(vx[v]);
      float sum = taps.b[v];
#pragma unroll
      for (int i = 0; i < K; ++i) sum = fmaf(taps.w[i][v], in[i][v], sum);
      out[v] = decltype(with_silu)::value ? silu(sum) : sum;
#pragma unroll
      for (int i = 0; i < K - 1; ++i) in[i][v] = in[i + 1][v];
    }
    W::store(y + now * p.dim, lane, out);
  };
  const auto run = [&](auto with_silu) {
    for (int t = at.t0; t < at.t1; t += kRows) {
      typename W::vec rows[kRows];
#pragma unroll
      for (int k = 0; k < kRows; ++k) rows[k] = next[k];
      if (t + kRows < at.t1) load(t + kRows);
      if (t + kRows <= at.t1 && t + kRows <= q.hi && q.hi != kNone) {      // all of one sequence
#pragma unroll
        for (int k = 0; k < kRows; ++k) token(t + k, rows[k], with_silu);
        continue;
      }
#pragma unroll 1
      for (int k = 0; k < kRows && t + k < at.t1; ++k) {
        if (t + k == q.hi) {
          follow(offsets, nseq, L, t + k, q);
          history<Tin, K, V>(p, q, x, lane, at.c, t + k, in);
        }
        if (q.hi == kNone) {          // padding
          const float zero[V] = {};
          W::store(y + (t + k) * p.dim, lane, zero);
        } else {
          token(t + k, rows[0], with_silu);
        }
#pragma unroll
        for (int j = 0; j < kRows - 1; ++j) rows[j] = rows[j + 1];
      }
    }
  };
  if (p.silu) run(std::true_type{});
  else run(std::false_type{});
}

// One lane for each sequence and channel: the gradient of the state before it, from the
// sequence's first tokens.
template <typename Tin, int K>
__device__ __forceinline__ void dinitial_state(const ConvParams& p, int64_t id) {
  if (!p.dh0 || id >= p.num_seqs * p.dim) return;   // a grid that is filled up has more lanes
  const int64_t s = id / p.dim, c = id - s * p.dim;
  int64_t row0 = 0, lo = 0, hi = p.L;
  if (p.offsets) {
    lo = p.offsets[s] < 0 ? 0 : (p.offsets[s] > p.L ? p.L : p.offsets[s]);
    hi = p.offsets[s + 1] < lo ? lo : (p.offsets[s + 1] > p.L ? p.L : p.offsets[s + 1]);
  } else {
    row0 = s * p.L;
  }
  const Taps<K, 1> taps(p, c);
  float in[2 * K] = {}, dv[K] = {};                   // inputs from K - 1 tokens before on, gradients of the first K - 1
#pragma unroll
  for (int j = 0; j < K - 1; ++j) in[j] = p.h0 ? p.h0[id * (K - 1) + j] : 0.f;
#pragma unroll
  for (int m = 0; m < K - 1; ++m) {
    if (lo + m >= hi) continue;
    in[K - 1 + m] = to_f32(static_cast<const Tin*>(p.x)[(row0 + lo + m) * p.sx + c]);
    float v = taps.b[0];
#pragma unroll
    for (int k = 0; k < K; ++k) v = fmaf(taps.w[k][0], in[m + k], v);
    const float dy = to_f32(static_cast<const Tin*>(p.dy)[(row0 + lo + m) * p.dim + c]);
    dv[m] = p.silu ? dy * silu_slope(v) : dy;
  }
#pragma unroll
  for (int i = 0; i < K - 1; ++i) {
    float d = 0.f;
#pragma unroll
    for (int m = 0; m <= i; ++m) d = fmaf(taps.w[i - m][0], dv[m], d);
    const int64_t j = i - (hi - lo);
    if (p.dlast && j >= 0) d += p.dlast[id * (K - 1) + j];
    p.dh0[id * (K - 1) + i] = d;
  }
}

// Along a block and the K - 1 tokens after it that its last tokens reach: token t's gradient dv
// completes dx of token t - (K - 1); where a sequence ends, the last K - 1 of its dx are
// completed without later ones, and with the last state's gradient.  The workgroup's sums of
// the parameters' gradients go to its row of `partial`, [K + 1][dim], the bias's last.
template <typename Tin, int K, int V>
__global__ __launch_bounds__(64 * kConvWaves) void dwconv_bwd_kernel(ConvParams p, const int32_t* __restrict__ offsets, int tokens,
                                                                     int nblk, int nct, uint32_t main) {
  constexpr int kRows = 4;      // rows of each side on their way at a time
  typedef Word<Tin, V> W;
  __shared__ float sums[kConvWaves - 1][K + 1][V][64];
  const uint32_t block = workgroup<64 * kConvWaves>();
  if (block >= main) return dinitial_state<Tin, K>(p, static_cast<int64_t>(block - main) * (64 * kConvWaves) + threadIdx.x);
  const Part at(p, block, tokens, nblk, nct, V);
  const int L = static_cast<int>(p.L), nseq = static_cast<int>(p.num_seqs);
  const uint32_t lane = static_cast<uint32_t>(at.c * sizeof(Tin));
  float dw[K + 1][V] = {};
  if (at.t0 < at.t1) {
    const Tin* x = static_cast<const Tin*>(p.x) + at.b * p.L * p.sx;
    const Tin* dy = static_cast<const Tin*>(p.dy) + at.b * p.L * p.dim;
    Tin* dx = static_cast<Tin*>(p.dx) + at.b * p.L * p.sdx;
    const int end = at.t1 + K - 1 < L ? at.t1 + K - 1 : L;
    typename W::vec nx[kRows], ng[kRows];
    const auto load = [&](int t) {      // rows past the end repeat the last one
#pragma unroll
      for (int k = 0; k < kRows; ++k) {
        const int64_t r = t + k < end ? t + k : end - 1;
        nx[k] = W::load(x + r * p.sx, lane);
        ng[k] = W::load(dy + r * p.dim, lane);
      }
    };
    load(at.t0);
    const Taps<K, V> taps(p, at.c);
    Sequence q = sequence_of(offsets, nseq, L, at.b, at.t0);
    float in[K][V], dv[K][V] = {};      // of the tokens up to now, the newest last
    history<Tin, K, V>(p, q, x, lane, at.c, at.t0, in);
    // dx of token u, `from` tokens before the newest: later gradients than that are not there
    const auto complete = [&](int u, int from, const float* more) {
      float out[V];
#pragma unroll
      for (int v = 0; v < V; ++v) {
        out[v] = more ? more[v] : 0.f;
#pragma unroll
        for (int j = 0; j < K; ++j)
          if (j <= from) out[v] = fmaf(taps.w[K - 1 - j][v], dv[K - 1 - from + j][v], out[v]);
      }
      W::store(dx + u * p.sdx, lane, out);
    };
    // the last tokens of the sequence, which ends at t; the newest gradient is of token t - 1
    const auto finish = [&](int t) {
#pragma unroll
      for (int j = K - 2; j >= 0; --j) {
        const int u = t - 1 - j;
        if (u < q.lo || u < at.t0 || u >= at.t1) continue;
        float more[V];
        state_at<K, V>(p.dlast, q.s, p.dim, at.c, K - 2 - j, more);
        complete(u, j, more);
      }
    };
    // Token `now`; `inner`: it is one of the block's, and so is the token whose dx it completes, of
    // the same sequence.
    const auto token = [&](int now, typename W::vec vx, typename W::vec vg, auto with_silu, auto inner) {
      constexpr bool kInner = decltype(inner)::value;
#pragma unroll
      for (int v = 0; v < V; ++v) {
        in[K - 1][v] = to_f32(vx[v]);
        float d = to_f32(vg[v]);
        if (decltype(with_silu)::value) {
          float sum = taps.b[v];
#pragma unroll
          for (int i = 0; i < K; ++i) sum = fmaf(taps.w[i][v], in[i][v], sum);
          d *= silu_slope(sum);
        }
#pragma unroll
        for (int i = 0; i < K - 1; ++i) dv[i][v] = dv[i + 1][v];
        dv[K - 1][v] = d;
      }
      if (kInner || now < at.t1) {
#pragma unroll
        for (int v = 0; v < V; ++v) {
#pragma unroll
          for (int i = 0; i < K; ++i) dw[i][v] = fmaf(dv[K - 1][v], in[i][v], dw[i][v]);
          dw[K][v] += dv[K - 1][v];
        }
      }
      if (kInner || (now - (K - 1) >= q.lo && now - (K - 1) >= at.t0)) complete(now - (K - 1), K - 1, nullptr);
#pragma unroll
      for (int i = 0; i < K - 1; ++i)
#pragma unroll
        for (int v = 0; v < V; ++v) in[i][v] = in[i + 1][v];
    };
    const auto run = [&](auto with_silu) {
      for (int t = at.t0; t < end; t += kRows) {
        typename W::vec rx[kRows], rg[kRows];
#pragma unroll
        for (int k = 0; k < kRows; ++k) rx[k] = nx[k], rg[k] = ng[k];
        if (t + kRows < end) load(t + kRows);
        if (t - (K - 1) >= at.t0 && t - (K - 1) >= q.lo && t + kRows <= at.t1 && t + kRows <= q.hi && q.hi != kNone) {
#pragma unroll
          for (int k = 0; k < kRows; ++k) token(t + k, rx[k], rg[k], with_silu, std::true_type{});
          continue;
        }
#pragma unroll 1
        for (int k = 0; k < kRows; ++k) {
          const int now = t + k;
          if (now >= end) break;
          if (now == q.hi) {
            finish(now);
            follow(offsets, nseq, L, now, q);
            history<Tin, K, V>(p, q, x, lane, at.c, now, in);
          }
          if (q.hi == kNone) {          // padding
            const float zero[V] = {};
            if (now < at.t1) W::store(dx + now * p.sdx, lane, zero);
          } else {
            token(now, rx[0], rg[0], with_silu, std::false_type{});
          }
#pragma unroll
          for (int j = 0; j < kRows - 1; ++j) rx[j] = rx[j + 1], rg[j] = rg[j + 1];
        }
      }
    };
    if (p.silu) run(std::true_type{});
    else run(std::false_type{});
    if (end == q.hi) finish(end);
  }
  // the waves' sums, added in their order
  const int wave = threadIdx.x >> 6, l = threadIdx.x & 63;
  if (wave > 0) {
#pragma unroll
    for (int i = 0; i <= K; ++i)
#pragma unroll
      for (int v = 0; v < V; ++v) sums[wave - 1][i][v][l] = dw[i][v];
  }
  __syncthreads();
  if (wave > 0) return;
  const int64_t set = block / nct;
#pragma unroll
  for (int i = 0; i <= K; ++i)
#pragma unroll
    for (int v = 0; v < V; ++v) {
      float sum = dw[i][v];
#pragma unroll
      for (int w = 0; w < kConvWaves - 1; ++w) sum += sums[w][i][v][l];
      p.partial[(set * (K + 1) + i) * p.dim + at.c + v] = sum;
    }
}

// The parameters' gradients from the workgroups' sums: 64 channels of one parameter a workgroup,
// its 16 waves a 16th of the sums each, eight loads in flight.
constexpr int kParamWaves = 16;
template <int K>
__global__ __launch_bounds__(64 * kParamWaves) void dwconv_param_kernel(ConvParams p, int64_t sets) {
  __shared__ float lds[kParamWaves][64];
  const uint32_t block = workgroup<64 * kParamWaves>();
  const int lane = threadIdx.x & 63, wave = threadIdx.x >> 6, i = block % (K + 1);
  const int64_t c = static_cast<int64_t>(block / (K + 1)) * 64 + lane;
  float sum = 0.f;
  if (c < p.dim) {
    const float* from = p.partial + i * p.dim + c;
    const int64_t row = (K + 1) * p.dim;
    int64_t g = wave;
    for (; g + 7 * kParamWaves < sets; g += 8 * kParamWaves) {
      float v[8];
#pragma unroll
      for (int k = 0; k < 8; ++k) v[k] = from[(g + k * kParamWaves) * row];
#pragma unroll
      for (int k = 0; k < 8; ++k) sum += v[k];
    }
    for (; g < sets; g += kParamWaves) sum += from[g * row];
  }
  lds[wave][lane] = sum;
  __syncthreads();
  if (wave != 0 || c >= p.dim) return;
#pragma unroll
  for (int k = 1; k < kParamWaves; ++k) sum += lds[k][lane];
  if (i < K) p.dw[c * K + i] = sum;
  else if (p.db) p.db[c] = sum;
}

// One token: a lane a channel, whose state is read and written once, 12 bytes of it next to the
// neighbour's.  256 x 5120 bf16: 8.9 us, its bytes at 5 TB/s 7.3.
template <typename Tin, int K>
__global__ __launch_bounds__(64) void dwconv_step_kernel(ConvStepParams p, int64_t nct) {
  const int64_t id = workgroup<64>();
  const int64_t b = id / nct, c = id % nct * 64 + threadIdx.x;
  if (b >= p.batch || c >= p.dim) return;
  const int64_t from = p.slots ? p.slots[b] : b, to = p.slots_out ? p.slots_out[b] : from;
  float y = 0.f;
  if (from >= 0 && from < p.num_slots) {
    float in[K], v = p.b ? p.b[c] : 0.f;
    in[K - 1] = to_f32(static_cast<const Tin*>(p.x)[b * p.sx + c]);
#pragma unroll
    for (int k = 0; k < K - 1; ++k) in[k] = p.state[(from * p.dim + c) * (K - 1) + k];
#pragma unroll
    for (int k = 0; k < K; ++k) v = fmaf(p.w[c * K + k], in[k], v);
    y = p.silu ? silu(v) : v;
    if (to >= 0 && to < p.num_slots) {
#pragma unroll
      for (int k = 0; k < K - 1; ++k) p.state[(to * p.dim + c) * (K - 1) + k] = in[k + 1];
    }
  }
  store_val(static_cast<Tin*>(p.y) + b * p.dim + c, y);
}

namespace {

constexpr int kConvFull = 4096;   // waves that keep memory busy

// Tokens of a wave's block, workgroups along the tokens and channels, workgroups in all.
struct ConvPlan {
  int tokens, nblk, nct;
  int64_t main;
};

// Blocks of 64 tokens, of which the first and the last few take the slower way; shorter ones while
// the waves are too few to keep memory busy (in blocks of 16, 32, 64: backward of 8 x 4096 x 2048
// bf16, 4096 waves in blocks of 64, 139, 119, 108 us; of 4094 x 1535 float32, 768 waves, 20.6,
// 22.6, 24.7 us; forward of 16411 x 2560 bf16, 2570 waves, 38, 39, 39).
ConvPlan plan_of(int64_t batch, int64_t L, int64_t dim, int V) {
  ConvPlan q;
  q.nct = static_cast<int>((dim + 64 * V - 1) / (64 * V));
  for (q.tokens = 64; q.tokens > 16; q.tokens /= 2)
    if (batch * ((L + q.tokens - 1) / q.tokens) * q.nct >= kConvFull) break;
  q.nblk = static_cast<int>((L + kConvWaves * q.tokens - 1) / (kConvWaves * q.tokens));
  q.main = batch * q.nblk * q.nct;
  return q;
}

// Channels of a lane: 8 bytes of a row, or one where the row has fewer.
int lane_channels(int64_t dim, size_t elem) { return dim >= static_cast<int64_t>(8 / elem) ? static_cast<int>(8 / elem) : 1; }

int64_t lanes_of(int64_t n) { return (n + 64 * kConvWaves - 1) / (64 * kConvWaves); }

template <typename Tin, int K, int V>
void fwd(const ConvParams& p, hipStream_t s) {
  const ConvPlan q = plan_of(p.batch, p.L, p.dim, V);
  const int64_t more = K > 1 && p.h_last ? lanes_of(p.num_seqs * p.dim) : 0;
  if (q.main + more > 0)
    hipLaunchKernelGGL((dwconv_fwd_kernel<Tin, K, V>), grid_of<64 * kConvWaves>(q.main + more), dim3(64 * kConvWaves), 0, s, p, p.offsets,
                       q.tokens, q.nblk, q.nct, static_cast<uint32_t>(q.main));
}

template <typename Tin, int K, int V>
void bwd(const ConvParams& p, hipStream_t s) {
  const ConvPlan q = plan_of(p.batch, p.L, p.dim, V);
  const int64_t more = K > 1 && p.dh0 ? lanes_of(p.num_seqs * p.dim) : 0;
  if (q.main + more > 0)
    hipLaunchKernelGGL((dwconv_bwd_kernel<Tin, K, V>), grid_of<64 * kConvWaves>(q.main + more), dim3(64 * kConvWaves), 0, s, p, p.offsets,
                       q.tokens, q.nblk, q.nct, static_cast<uint32_t>(q.main));
  hipLaunchKernelGGL((dwconv_param_kernel<K>), grid_of<64 * kParamWaves>((p.dim + 63) / 64 * (K + 1)), dim3(64 * kParamWaves), 0, s, p,
                     p.batch * q.nblk);
}

template <typename Tin, int K>
void step(const ConvStepParams& p, hipStream_t s) {
  const int64_t nct = (p.dim + 63) / 64;
  hipLaunchKernelGGL((dwconv_step_kernel<Tin, K>), grid_of<64>(p.batch * nct), dim3(64), 0, s, p, nct);
}

// f(element, taps) with both as types.
template <typename F>
hipError_t by_type(int taps, bool bf16, F&& f) {
  const auto of = [&](auto elem) {
    switch (taps) {
      case 1: return f(elem, std::integral_constant<int, 1>{});
      case 2: return f(elem, std::integral_constant<int, 2>{});
      case 3: return f(elem, std::integral_constant<int, 3>{});
      default: return f(elem, std::integral_constant<int, 4>{});
    }
  };
  if (bf16) of(bf16_t{});
  else of(float{});
  return hipGetLastError();
}

}  // namespace

// The most that plan_of can ask for any call up to these sizes, in either type, so that a buffer for
// the longest batch serves the shorter ones.  Blocks of 64 tokens: a set of sums for each 256.  Shorter
// blocks: one for at least 64 tokens, and fewer than kConvFull / nct sets, since blocks of twice the
// length were fewer than kConvFull waves; with dim <= nct 64 V that is kConvFull 64 V numbers of each
// parameter, V at most 4.
size_t dwconv_bwd_workspace_bytes(int64_t batch, int64_t L, int64_t dim, int taps) {
  if (batch <= 0 || L <= 0 || dim <= 0) return 0;
  const int64_t least = batch * ((L + 255) / 256) * dim, most = batch * ((L + 63) / 64) * dim, bound = kConvFull * 64 * 4;
  const int64_t shorter = most < bound ? most : bound;
  return static_cast<size_t>(least > shorter ? least : shorter) * (taps + 1) * 4;
}

hipError_t launch_dwconv_fwd(const ConvParams& p, int taps, bool bf16, hipStream_t s) {
  return by_type(taps, bf16, [&](auto elem, auto k) {
    typedef decltype(elem) Tin;
    if (lane_channels(p.dim, sizeof(Tin)) > 1) fwd<Tin, decltype(k)::value, 8 / sizeof(Tin)>(p, s);
    else fwd<Tin, decltype(k)::value, 1>(p, s);
  });
}

hipError_t launch_dwconv_bwd(const ConvParams& p, int taps, bool bf16, hipStream_t s) {
  return by_type(taps, bf16, [&](auto elem, auto k) {
    typedef decltype(elem) Tin;
    if (lane_channels(p.dim, sizeof(Tin)) > 1) bwd<Tin, decltype(k)::value, 8 / sizeof(Tin)>(p, s);
    else bwd<Tin, decltype(k)::value, 1>(p, s);
  });
}

hipError_t launch_dwconv_step(const ConvStepParams& p, int taps, bool bf16, hipStream_t s) {
  return by_type(taps, bf16, [&](auto elem, auto k) { step<decltype(elem), decltype(k)::value>(p, s); });
}

}  // namespace sscan
