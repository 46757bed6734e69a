// Products of rows in 8-bit integers with the scales of both sides.
//
// out[m, n] = (sum_k a[m, k] b[n, k]) (as[m] bs[n]) + bias[n].  Both sides have k along their
// rows, so both go through LDS the same way: 128 bytes of each row at a time, in 16-byte
// chunks, which are what a lane of a matrix instruction takes (v_mfma_i32_32x32x32_i8: lane l
// holds row l % 32, bytes 16 (l / 32) .. + 15 of 32).  The order of k is the same on both
// sides and otherwise free, since the sums are whole numbers.
#include "sscan_layer.h"
#include <cstdlib>

namespace sscan {

typedef int i32x4 __attribute__((ext_vector_type(4)));
typedef int i32x16 __attribute__((ext_vector_type(16)));
typedef float f32x4 __attribute__((ext_vector_type(4)));
typedef i32x4 i32x4_any __attribute__((aligned(1)));

constexpr int kChunk16 = 16;           // bytes of a chunk

// All waves of the workgroup are here, with nothing of theirs under way but the newest VM
// loads into LDS.  What the compiler sees as memory stays on its side.
template <int VM>
__device__ __forceinline__ void all_here() {
  asm volatile("" ::: "memory");
  __builtin_amdgcn_s_waitcnt((VM & 15) | 7 << 4 | 0 << 8 | (VM >> 4) << 14);
  __builtin_amdgcn_s_barrier();
  asm volatile("" ::: "memory");
}

// 16 bytes for each lane straight to LDS, in the lanes' order from the wave's address `to`, from
// an address of its own or from a common one and an offset.  In assembly, since the compiler
// takes any reading of LDS to wait for all such loads; all_here() waits for them.
#pragma clang diagnostic push
#pragma clang diagnostic ignored "-Winline-asm"   // m0 is reserved, and is what such a load goes by
__device__ __forceinline__ void bring(uint32_t to, uintptr_t from) {
  asm volatile("s_mov_b32 m0, %0\n\ts_nop 0\n\tglobal_load_lds_dwordx4 %1, off" ::"s"(to), "v"(from) : "m0");
}
__device__ __forceinline__ void bring(uint32_t to, uintptr_t base, uint32_t at) {
  asm volatile("s_mov_b32 m0, %0\n\ts_nop 0\n\tglobal_load_lds_dwordx4 %1, %2" ::"s"(to), "v"(at), "s"(base) : "m0");
}
#pragma clang diagnostic pop

__device__ __attribute__((aligned(16))) const int8_t g_zeros[kChunk16] = {};

// One side's rows of a tile on their way to LDS, DEPTH bytes of k at a time.  A chunk of row r
// goes to a slot of the row's DEPTH bytes that differs from row to row (slot_of), so that 16
// lanes that read one chunk of 16 rows take all 64 banks once.  The lanes of a wave bring
// slot after slot of row after row: LDS is then filled in the lanes' order, which is what a
// load straight to LDS does.
template <int DEPTH>
__device__ __forceinline__ int slot_of(int row, int chunk) {
  return DEPTH == 128 ? (chunk ^ (row >> 1)) & 7 : (chunk ^ (row >> 2)) & 3;
}
template <int ROWS, int WAVES, int DEPTH, bool DIRECT>
struct Side {
  static constexpr int kChunks = DEPTH / kChunk16, kStep = 64 / kChunks * WAVES;   // rows of one load of all waves
  static constexpr int kLoads = ROWS / kStep;
  static_assert(ROWS % kStep == 0 && kStep % 16 == 0, "the lane's chunk is the same in all its rows");
  const int8_t* base;
  uint32_t at[kLoads];       // DIRECT: bytes from base to the lane's rows
  int64_t stride;
  int row0, last, chunk;     // the lane's first row, the last row there is, its chunk
  i32x4 held[DIRECT ? 1 : kLoads];

  __device__ __forceinline__ Side(const int8_t* p, int64_t st, int64_t r0, int rows) : stride(st) {
    base = p + r0 * st;
    row0 = threadIdx.x / kChunks;
    last = static_cast<int>(rows - r0 < ROWS ? rows - r0 : ROWS) - 1;
    chunk = slot_of<DEPTH>(row0, threadIdx.x % kChunks);
#pragma unroll
    for (int i = 0; i < kLoads; ++i) at[i] = static_cast<uint32_t>(row(i) * st + chunk * kChunk16);
  }
  // rows past the end repeat the last one: their sums are not written
  __device__ __forceinline__ int row(int i) const { return row0 + kStep * i < last ? row0 + kStep * i : last; }

  // Where in LDS the wave's first load of the rows goes.
  static __device__ __forceinline__ uint32_t place(int8_t* lds) {
    return __builtin_amdgcn_readfirstlane(static_cast<uint32_t>(
        reinterpret_cast<uintptr_t>((__attribute__((address_space(3))) int8_t*)lds) + (threadIdx.x >> 6) * 64 * kChunk16));
  }
  // Load i of bytes k .. k + DEPTH, all there.
  __device__ __forceinline__ void one(uint32_t to, int k, int i) const {
    bring(to + i * kStep * DEPTH, reinterpret_cast<uintptr_t>(base + k), at[i]);
  }
  // Bytes k .. k + DEPTH of the rows, of which `left` are there; zeros for the others.
  __device__ __forceinline__ void load(int8_t* lds, int k, int left) {
    if (DIRECT) {
      const uint32_t to = place(lds);
      if (left >= DEPTH) {
#pragma unroll
        for (int i = 0; i < kLoads; ++i) one(to, k, i);
      } else {
        const uintptr_t from = reinterpret_cast<uintptr_t>(base + k), zeros = reinterpret_cast<uintptr_t>(g_zeros);
#pragma unroll
        for (int i = 0; i < kLoads; ++i) bring(to + i * kStep * DEPTH, chunk * kChunk16 < left ? from + at[i] : zeros);
      }
    } else {
#pragma unroll
      for (int i = 0; i < kLoads; ++i) {
        const int8_t* from = base + row(i) * stride + k + chunk * kChunk16;
        const int n = left - chunk * kChunk16;
        if (n >= kChunk16) {
          held[i] = *reinterpret_cast<const i32x4_any*>(from);
        } else {
          uint32_t w[4] = {};
          for (int j = 0; j < n; ++j) w[j / 4] |= static_cast<uint32_t>(static_cast<uint8_t>(from[j])) << 8 * (j % 4);
          held[i] = i32x4{static_cast<int>(w[0]), static_cast<int>(w[1]), static_cast<int>(w[2]), static_cast<int>(w[3])};
        }
      }
    }
  }
  // What load() left in registers, to LDS.
  __device__ __forceinline__ void put(int8_t* lds) {
    if (DIRECT) return;
#pragma unroll
    for (int i = 0; i < kLoads; ++i)
      *reinterpret_cast<i32x4*>(lds + i * kStep * DEPTH + threadIdx.x * kChunk16) = held[i];
  }
};

// Four neighbouring outputs of a row in Tout.
__device__ __forceinline__ void stage(float* p, f32x4 v) { *reinterpret_cast<f32x4*>(p) = v; }
__device__ __forceinline__ void stage(bf16_t* p, f32x4 v) {
  typedef __bf16 b4 __attribute__((ext_vector_type(4)));
  typedef uint16_t u4 __attribute__((ext_vector_type(4)));
  *reinterpret_cast<u4*>(p) = __builtin_bit_cast(u4, __builtin_convertvector(v, b4));
}

// A workgroup's tile of BM x BN sums; its WM x WN waves have a part of MI x NI blocks of 32 x 32
// each.  LDS holds two depths of k: while one is multiplied the next is on its way.  The
// instruction's rows are n and its columns m, so that a lane ends with neighbouring outputs.
template <typename Tout, int BM, int BN, int WM, int WN, int DEPTH, int GROUPS, bool DIRECT>
__global__ __launch_bounds__(64 * WM * WN, GROUPS * WM * WN / 4) void i8_tile_kernel(MatmulParams p, int ntm, int ntn) {
  constexpr int kWaves = WM * WN, kRows = BM / WM, kCols = BN / WN, MI = kRows / 32, NI = kCols / 32;
  typedef Side<BM, kWaves, DEPTH, DIRECT> A;
  typedef Side<BN, kWaves, DEPTH, DIRECT> B;
  constexpr int kLoads = A::kLoads + B::kLoads, kA = BM * DEPTH, kStage = (BM + BN) * DEPTH;
  constexpr int kPitch = kCols + 16 / sizeof(Tout), kRoom = 32 * kPitch * sizeof(Tout);   // outputs of 32 rows
  __shared__ __attribute__((aligned(16))) int8_t lds[2 * kStage > kWaves * kRoom ? 2 * kStage : kWaves * kRoom];
  __shared__ __attribute__((aligned(16))) float cols[2][BN];        // the columns' scales and biases
  const int tile = static_cast<int>(xcd_remap(blockIdx.x, static_cast<int64_t>(ntm) * ntn));
  // tiles go down 4 rows of tiles, then along n: the 32 tiles that an XCD has at a time share
  // 4 tiles' rows of a and 8 of b
  const int group = tile / (4 * ntn), in = tile - group * 4 * ntn;
  const int high = ntm - group * 4 < 4 ? ntm - group * 4 : 4;
  const int tm = group * 4 + in % high, tn = in / high;
  const int64_t m0 = static_cast<int64_t>(tm) * BM, n0 = static_cast<int64_t>(tn) * BN;
  const int lane = threadIdx.x & 63, wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
  const int wm = wave / WN, wn = wave % WN;

  for (int c = threadIdx.x; c < BN; c += 64 * kWaves) {
    const int64_t n = n0 + c < p.n ? n0 + c : p.n - 1;
    cols[0][c] = p.bs[n];
    cols[1][c] = p.bias ? p.bias[n] : 0.f;
  }
  A sa(p.a, p.sa, m0, p.m);
  B sb(p.b, p.sb, n0, p.n);
  i32x16 acc[MI][NI] = {};
  i32x4 fa[2][MI], fb[2][NI];

  // block i's chunk 2 ks + l / 32 of row l % 32
  const int r = lane & 31, h = lane >> 5;
  const auto fetch = [&](const int8_t* from, int ks, int to, int i) {
    const int slot = slot_of<DEPTH>(r, 2 * ks + h);
    if (i < NI)
      fb[to][i] = *reinterpret_cast<const i32x4*>(from + kA + (wn * kCols + i * 32 + r) * DEPTH + slot * kChunk16);
    else
      fa[to][i - NI] = *reinterpret_cast<const i32x4*>(from + (wm * kRows + (i - NI) * 32 + r) * DEPTH + slot * kChunk16);
  };
  // A step: blocks `with` are multiplied while those of step ks of `from` are read and, one at a
  // time, loads for a later depth are begun.  The order is fixed: left to itself the compiler
  // reads blocks when they are needed, and the matrix unit waits for them.
  constexpr int Q = MI * NI, R = MI + NI;
  const auto step = [&](int with, const int8_t* from, int ks, auto&& begin) {
#pragma unroll
    for (int q = 0; q < Q; ++q) {
#pragma unroll
      for (int i = 2 * q * R / Q; i < 2 * (q + 1) * R / Q && i < R; ++i) fetch(from, ks, with ^ 1, i);
#pragma unroll
      for (int i = q * kLoads / Q; i < (q + 1) * kLoads / Q; ++i) begin(i);
      acc[q / NI][q % NI] = __builtin_amdgcn_mfma_i32_32x32x32_i8(fb[with][q % NI], fa[with][q / NI], acc[q / NI][q % NI], 0, 0, 0);
      __builtin_amdgcn_sched_barrier(0);
    }
  };
  const auto nothing = [](int) {};

  // The depths of k: what k has beyond whole depths comes first, filled up with zeros, so that
  // all later ones are whole.
  const int rest = p.k % DEPTH, depths = (p.k + DEPTH - 1) / DEPTH;
  const auto start = [&](int t) { return t == 0 ? 0 : t * DEPTH - (rest ? DEPTH - rest : 0); };
  const auto load = [&](int8_t* to, int t) {
    const int n = t == 0 && rest ? rest : DEPTH;
    sa.load(to, start(t), n);
    sb.load(to + kA, start(t), n);
  };
  const auto put = [&](int8_t* to) {
    sa.put(to);
    sb.put(to + kA);
  };
  if (depths > 0) {
    load(lds, 0);
    put(lds);
    if (DIRECT && depths > 1) {
      load(lds + kStage, 1);
      all_here<kLoads>();
    } else {
      all_here<0>();
    }
#pragma unroll
    for (int i = 0; i < R; ++i) fetch(lds, 0, 0, i);
  }
  // Each step's blocks are read while the step before is multiplied, across depths too: the
  // barrier comes before a depth's last step, when all of its blocks are in registers.  (The
  // last depth reads what is not there yet, and does not use it.)
  for (int t = 0; t < depths; ++t) {
    int8_t* now = lds + (t & 1) * kStage;
    int8_t* next = lds + (~t & 1) * kStage;
    if (!DIRECT && t + 1 < depths) load(next, t + 1);
    step(0, now, 1, nothing);
    if (DEPTH == 128) step(1, now, 2, nothing);
    if (!DIRECT && t + 1 < depths) put(next);
    if (DEPTH == 128) step(0, now, 3, nothing);
    all_here<0>();
    const bool more = DIRECT && t + 2 < depths;
    const uint32_t ta = A::place(now), tb = B::place(now + kA);
    const int k = start(t + 2);
    step(1, next, 0, [&](int i) {
      if (!more) return;
      if (i < A::kLoads) sa.one(ta, k, i);
      else sb.one(tb, k, i - A::kLoads);
    });
  }

  // Outputs: 32 rows of a wave's part at a time through LDS of its own, so that a row's
  // outputs leave in 16-byte words.
  all_here<0>();
  constexpr int kPer = 16 / sizeof(Tout), kChunks = kCols / kPer;
  Tout* room = reinterpret_cast<Tout*>(lds + wave * kRoom);
#pragma unroll
  for (int i = 0; i < MI; ++i) {
    const int64_t mi = m0 + wm * kRows + i * 32;
    const float as = p.as[mi + r < p.m ? mi + r : p.m - 1];
#pragma unroll
    for (int j = 0; j < NI; ++j)
#pragma unroll
      for (int g = 0; g < 4; ++g) {
        const int c = j * 32 + g * 8 + h * 4;
        const f32x4 bs = *reinterpret_cast<const f32x4*>(&cols[0][wn * kCols + c]);
        const f32x4 bias = *reinterpret_cast<const f32x4*>(&cols[1][wn * kCols + c]);
        f32x4 v;
#pragma unroll
        for (int e = 0; e < 4; ++e) v[e] = fmaf(static_cast<float>(acc[i][j][4 * g + e]), as * bs[e], bias[e]);
        stage(room + r * kPitch + c, v);
      }
    asm volatile("s_waitcnt lgkmcnt(0)" ::: "memory");
#pragma unroll
    for (int q = 0; q < 32 * kChunks / 64; ++q) {
      const int at = q * 64 + lane, row = at / kChunks, c = at % kChunks * kPer;
      const int64_t m = mi + row;
      const int n = static_cast<int>(n0) + wn * kCols + c;
      typedef Tout word __attribute__((ext_vector_type(kPer)));
      typedef word word_any __attribute__((aligned(sizeof(Tout))));
      const word v = *reinterpret_cast<const word*>(room + row * kPitch + c);
      if (m >= p.m) continue;
      Tout* to = static_cast<Tout*>(p.out) + m * p.so + n;
      if (n + kPer <= p.n) {
        *reinterpret_cast<word_any*>(to) = v;
      } else {
#pragma unroll
        for (int e = 0; e < kPer; ++e)
          if (n + e < p.n) to[e] = v[e];
      }
    }
    asm volatile("s_waitcnt lgkmcnt(0)" ::: "memory");
  }
}

size_t i8_matmul_workspace_bytes(int64_t, int64_t, int64_t) { return 0; }

namespace {

// Rows that loads straight to LDS can take: whole 16-byte chunks, and a tile's rows within 32 bits.
bool direct(const MatmulParams& p) {
  const auto fine = [&](const int8_t* q, int64_t stride, int rows) {
    return reinterpret_cast<uintptr_t>(q) % 16 == 0 && (rows == 1 || (stride % 16 == 0 && stride < (1 << 23)));
  };
  return p.k % 16 == 0 && fine(p.a, p.sa, p.m) && fine(p.b, p.sb, p.n);
}

template <typename Tout, int BM, int BN, int WM, int WN, int DEPTH, int GROUPS, bool DIRECT>
hipError_t tiles(const MatmulParams& p, hipStream_t s) {
  const int ntm = (p.m - 1) / BM + 1, ntn = (p.n - 1) / BN + 1;
  hipLaunchKernelGGL((i8_tile_kernel<Tout, BM, BN, WM, WN, DEPTH, GROUPS, DIRECT>), dim3(static_cast<unsigned>(ntm) * ntn),
                     dim3(64 * WM * WN), 0, s, p, ntm, ntn);
  return hipGetLastError();
}

template <typename Tout>
hipError_t product(const MatmulParams& p, hipStream_t s) {
  const int64_t big = static_cast<int64_t>((p.m - 1) / 256 + 1) * ((p.n - 1) / 256 + 1);
  const int64_t mid = static_cast<int64_t>((p.m - 1) / 128 + 1) * ((p.n - 1) / 128 + 1);
  if (!direct(p)) return mid >= 256 ? tiles<Tout, 128, 128, 2, 2, 128, 2, false>(p, s) : tiles<Tout, 64, 64, 2, 2, 128, 2, false>(p, s);
  const char* e = getenv("MM_V");
  const int v = e ? atoi(e) : 0;
  if (v == 1) return tiles<Tout, 256, 256, 2, 2, 128, 1, true>(p, s);
  if (v == 2) return tiles<Tout, 256, 256, 2, 4, 128, 1, true>(p, s);
  if (v == 3) return tiles<Tout, 256, 128, 2, 2, 64, 2, true>(p, s);
  if (v == 4) return tiles<Tout, 128, 128, 2, 2, 128, 2, true>(p, s);
  if (v == 5) return tiles<Tout, 128, 128, 2, 2, 64, 3, true>(p, s);
  if (v == 6) return tiles<Tout, 128, 256, 2, 2, 64, 2, true>(p, s);
  if (v == 7) return tiles<Tout, 256, 128, 4, 2, 128, 1, true>(p, s);
  if (v == 8) return tiles<Tout, 64, 64, 2, 2, 128, 2, true>(p, s);
  if (v == 9) return tiles<Tout, 128, 64, 2, 2, 128, 2, true>(p, s);
  if (big >= 256) return tiles<Tout, 256, 256, 2, 2, 128, 1, true>(p, s);
  return mid >= 256 ? tiles<Tout, 128, 128, 2, 2, 128, 2, true>(p, s) : tiles<Tout, 64, 64, 2, 2, 128, 2, true>(p, s);
}

}  // namespace

hipError_t launch_i8_matmul(const MatmulParams& p, size_t, bool bf16, hipStream_t s) {
  return bf16 ? product<bf16_t>(p, s) : product<float>(p, s);
}

}  // namespace sscan
