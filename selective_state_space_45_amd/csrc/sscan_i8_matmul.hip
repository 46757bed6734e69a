// Products of rows in 8-bit integers with the scales of both sides.
//
// out[m, n] = (sum_k a[m, k] b[n, k]) (as[m] bs[n]) + bias[n].  Both sides have k along their
// rows, so both go through LDS the same way: 64 bytes of each row at a time, in 16-byte
// chunks, which are what a lane of a matrix instruction takes (v_mfma_i32_16x16x64_i8: lane l
// holds row l % 16, bytes 16 (l / 16) .. + 15 of 64).  The order of k is the same on both
// sides and otherwise free, since the sums are whole numbers.
//
// The matrix units alone, on random codes, reach 4100 TOP/s with this instruction (at 1.95 GHz) and
// 3450 with v_mfma_i32_32x32x32_i8, on zeros 4850 and 4970: power sets the clock.  Large products stay
// below that for two reasons.  32768 x 4096 x k takes 50 us and 0.77 us for each 64 of k (k = 512,
// 1024, 2048, 4096: 98, 153, 248, 446 us).  The 50 us do not grow with k: all workgroups come to
// their outputs together, 268 MB or 54 us of memory, while the matrix units stand still.  And in
// 64 of k they are busy for 1024 of 1180 to 1290 cycles, at 1.8 GHz.  (On zeros, at 2.35 GHz, 2048 takes
// 224 us.)
#include "sscan_layer.h"

namespace sscan {

typedef int i32x4 __attribute__((ext_vector_type(4)));
typedef float f32x4 __attribute__((ext_vector_type(4)));
typedef i32x4 i32x4_any __attribute__((aligned(1)));

constexpr int kUnits = 256;            // compute units
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

// Loads straight to LDS, in the lanes' order from the wave's address `to`: 16 bytes for each lane
// at an offset from a common address, or 4 at an address of its own.  In assembly, since the
// compiler takes any reading of LDS to wait for all such loads; all_here() waits for them.
#pragma clang diagnostic push
#pragma clang diagnostic ignored "-Winline-asm"   // m0 is reserved, and is what such a load goes by
__device__ __forceinline__ void bring(uint32_t to, uintptr_t base, uint32_t at) {
  asm volatile("s_mov_b32 m0, %0\n\ts_nop 0\n\tglobal_load_lds_dwordx4 %1, %2" ::"s"(to), "v"(at), "s"(base) : "m0");
}
__device__ __forceinline__ void bring_word(uint32_t to, const void* from) {
  asm volatile("s_mov_b32 m0, %0\n\ts_nop 0\n\tglobal_load_lds_dword %1, off" ::"s"(to), "v"(from) : "m0");
}
#pragma clang diagnostic pop

// Where a load to LDS goes that begins at p for the workgroup's first wave, BYTES of a wave after
// another.
template <int BYTES>
__device__ __forceinline__ uint32_t place_of(int8_t* p) {
  return __builtin_amdgcn_readfirstlane(static_cast<uint32_t>(
      reinterpret_cast<uintptr_t>((__attribute__((address_space(3))) int8_t*)p) + (threadIdx.x >> 6) * BYTES));
}

// LDS holds kStages depths of k, kDepth bytes of each row: a pair of depths is multiplied while the
// next is on its way.  Both depths of a pair are begun together, so that they meet in the
// 128-byte lines that memory is read in (begun one by one, three depths ahead, every line passed
// from L2 to a compute unit twice: 8192^3 463 us, now 433; a compute unit then got about 43 bytes a
// nanosecond, whatever the tile).
constexpr int kDepth = 64, kStages = 4;

// Where a row of 64 bytes in LDS has its 16-byte chunk c: at slot (c ^ -(row / 4)) & 3.  A reading of
// 16 bytes a lane goes in four parts, of lanes 0-3, 12-15, 20-27 and 4-11, 16-19, 28-31, and the same
// of the upper half (found by pairs of lanes that read one bank): with a matrix instruction's
// rows in the lanes, each part then takes all 64 banks once (with c ^ row / 4, which does so for 16
// lanes in a row, a reading took 8 cycles, not 4).
__device__ __forceinline__ int slot_of(int row, int chunk) { return (chunk ^ -(row >> 2)) & 3; }

// One side's rows of a tile on their way to LDS.  The lanes of a wave bring slot after slot of row
// after row: LDS is then filled in the lanes' order, which is what a load straight to LDS does.
template <int ROWS, int WAVES, bool DIRECT>
struct Side {
  static constexpr int kStep = 16 * WAVES, kLoads = ROWS / kStep;   // rows of one load of all waves
  static_assert(ROWS % kStep == 0, "the lane's chunk is the same in all its rows");
  const int8_t* base;
  uint32_t at[kLoads];       // DIRECT: bytes from base to the lane's rows
  int64_t stride;
  int row0, last, chunk;     // the lane's first row, the last row there is, its chunk
  i32x4 held[DIRECT ? 1 : kLoads];

  // The rows from r0 on of `rows` rows.
  __device__ __forceinline__ void aim(const int8_t* p, int64_t st, int64_t r0, int rows) {
    stride = st;
    base = p + r0 * st;
    row0 = threadIdx.x / 4;
    last = static_cast<int>(rows - r0 < ROWS ? rows - r0 : ROWS) - 1;
    chunk = slot_of(row0, threadIdx.x % 4);
#pragma unroll
    for (int i = 0; i < kLoads; ++i) at[i] = static_cast<uint32_t>(row(i) * st + chunk * kChunk16);
  }
  // rows past the end repeat the last one: their sums are not written
  __device__ __forceinline__ int row(int i) const { return row0 + kStep * i < last ? row0 + kStep * i : last; }

  // DIRECT: load i of the next two depths of the rows, all there: the second finds its half of the
  // lines on their way.
  __device__ __forceinline__ void two(uint32_t to, uint32_t then, int i) const {
    bring(to + i * kStep * kDepth, reinterpret_cast<uintptr_t>(base), at[i]);
    bring(then + i * kStep * kDepth, reinterpret_cast<uintptr_t>(base) + kDepth, at[i]);
  }
  // The same by way of registers, from any address, zeros past the `left` bytes that are there.
  __device__ __forceinline__ void hold(int left) {
#pragma unroll
    for (int i = 0; i < kLoads; ++i) {
      const int8_t* from = base + row(i) * stride + chunk * kChunk16;
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
  __device__ __forceinline__ void put(int8_t* lds) const {
#pragma unroll
    for (int i = 0; i < kLoads; ++i)
      *reinterpret_cast<i32x4*>(lds + i * kStep * kDepth + threadIdx.x * kChunk16) = held[i];
  }
};

// Four neighbouring outputs of a row in Tout.
__device__ __forceinline__ void stage_out(float* p, f32x4 v) { *reinterpret_cast<f32x4*>(p) = v; }
__device__ __forceinline__ void stage_out(bf16_t* p, f32x4 v) {
  typedef __bf16 b4 __attribute__((ext_vector_type(4)));
  typedef uint16_t u4 __attribute__((ext_vector_type(4)));
  *reinterpret_cast<u4*>(p) = __builtin_bit_cast(u4, __builtin_convertvector(v, b4));
}

// Workgroups take tiles of BM x BN sums one after another; their WM x WN waves have a part of
// MI x NI blocks of 16 x 16 each.  The loads go on from tile to tile, also while a tile's outputs
// leave.  The instruction's rows are n and its columns m, so that a lane ends with neighbouring
// outputs.  GROUPS workgroups share a compute unit.
template <typename Tout, int BM, int BN, int WM, int WN, int GROUPS, bool DIRECT>
__global__ __launch_bounds__(64 * WM * WN, GROUPS * WM * WN / 4) void i8_tile_kernel(MatmulParams p, int ntm, int ntn) {
  constexpr int kWaves = WM * WN, kLanes = 64 * kWaves, kRows = BM / WM, kCols = BN / WN, MI = kRows / 16, NI = kCols / 16;
  typedef Side<BM, kWaves, DIRECT> A;
  typedef Side<BN, kWaves, DIRECT> B;
  constexpr int kLoads = A::kLoads + B::kLoads, kA = BM * kDepth, kStage = (BM + BN) * kDepth;
  static_assert((kStage & (kStage - 1)) == 0, "stages follow one another by a mask");
  constexpr int kPer = 16 / sizeof(Tout), kSpan = 4 * kPer;   // outputs of a word, and of a row that leave at a time
  // of three tiles: b's scales, biases, a's scales, filled up to whole loads of all waves
  constexpr int kScaleLoads = (2 * BN + BM + kLanes - 1) / kLanes, kScales = kScaleLoads * kLanes;
  __shared__ __attribute__((aligned(16))) int8_t lds[kStages * kStage];
  __shared__ __attribute__((aligned(16))) float scale[3][kScales];
  __shared__ __attribute__((aligned(16))) Tout room[kWaves][32 * kSpan];
  const int tiles = ntm * ntn;
  const int lane = threadIdx.x & 63, wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
  const int wm = wave / WN, wn = wave % WN;
  // Where the workgroup's tile of turn v begins.  Tiles go down 4 rows of tiles, then along n:
  // the 32 tiles that an XCD has at a time share 4 tiles' rows of a and 8 of b.
  const auto place = [&](int v, int64_t& m0, int64_t& n0) {
    const int tile = static_cast<int>(xcd_remap(v, tiles));
    const int group = tile / (4 * ntn), in = tile - group * 4 * ntn;
    const int high = ntm - group * 4 < 4 ? ntm - group * 4 : 4;
    m0 = static_cast<int64_t>(group * 4 + in % high) * BM;
    n0 = static_cast<int64_t>(in / high) * BN;
  };

  // A depth is MI slots, each a block of a's rows times all of b's: the order within a slot, and
  // of slots, is fixed (left to itself the compiler reads blocks when they are needed, and the
  // matrix unit waits for them).  A slot reads a's block for kAhead slots later, the last kAhead
  // slots of a depth also b's blocks of the next.  The loads of a pair begin in the last kAhead
  // slots of the pair before.  In large tiles they go on over kBegin slots, as evenly as leaves them
  // the time to arrive (8192^3 in 4, 8, 11, 13 slots: 457, 437, 433, 447 us); in small ones that
  // time is what a pair takes, and they all begin there (256 x 2560 x 5120 15.0 us, now 14.6).  Room
  // for 8 depths in LDS does not help: a pair of 128 x 128 already fills the 32 KB that the lines
  // pass through (256 x 10240 x 2560 16.7 us, with 8 depths 21.3).
  constexpr int kAhead = MI > 3 ? 3 : MI - 1, kRing = kAhead + 1;
  static_assert(MI % kRing == 0 && MI % 2 == 0, "places of blocks are constants");
  constexpr int kBegin = MI > 4 ? MI + kAhead : kAhead;
  i32x4 acc[MI][NI] = {}, fa[kRing], fb[2][NI];
  // a block's chunk l / 16 of row l % 16
  const int r = lane & 15, h = lane >> 4, mine_at = r * kDepth + slot_of(r, h) * kChunk16;
  const auto fetch_a = [&](const int8_t* from, int i) {
    fa[i % kRing] = *reinterpret_cast<const i32x4*>(from + (wm * kRows + i * 16) * kDepth + mine_at);
  };
  const auto fetch_b = [&](const int8_t* from, int half, int i) {
    fb[half][i] = *reinterpret_cast<const i32x4*>(from + kA + (wn * kCols + i * 16) * kDepth + mine_at);
  };
  const auto slot = [&](const int8_t* now, const int8_t* next, int half, int i, auto&& begin) {
    const int late = i - (MI - kAhead);             // 0 .. kAhead - 1 in the last slots
    if (late < 0) fetch_a(now, i + kAhead);
    else fetch_a(next, i + kAhead - MI);
    if (late >= 0) {
#pragma unroll
      for (int j = late * NI / kAhead; j < (late + 1) * NI / kAhead; ++j) fetch_b(next, half ^ 1, j);
    }
    const int step = half == 1 ? late : i + kAhead;       // 0 .. in the slots that begin loads
#pragma unroll
    for (int l = step * kLoads / kBegin; l < (step + 1) * kLoads / kBegin; ++l)
      if (l < kLoads) begin(l);
#pragma unroll
    for (int j = 0; j < NI; ++j)
      acc[i][j] = __builtin_amdgcn_mfma_i32_16x16x64_i8(fb[half][j], fa[i % kRing], acc[i][j], 0, 0, 0);
    __builtin_amdgcn_sched_barrier(0);
  };

  // The depths of k go in pairs, the last one filled up with zeros (DIRECT: all are whole).  The
  // workgroup loads depth after depth, tile after tile; (lv, lt) is the next to load.
  constexpr int kTurn = DIRECT ? 2 : 1;      // depths that are loaded at a time
  const int depths = (p.k + 2 * kDepth - 1) / (2 * kDepth) * 2;
  A sa;
  B sb;
  int lv = blockIdx.x, lt = 0;
  const auto aim = [&]() {
    int64_t m0, n0;
    place(lv, m0, n0);
    sa.aim(p.a, p.sa, m0, p.m);
    sb.aim(p.b, p.sb, n0, p.n);
  };
  const auto begin = [&](uint32_t to, uint32_t then, int l) {
    if (l < A::kLoads) sa.two(to, then, l);
    else sb.two(to + kA, then + kA, l - A::kLoads);
  };
  const auto hold = [&]() {
    const int left = p.k - lt * kDepth;
    sa.hold(left);
    sb.hold(left);
  };
  const auto put = [&](int8_t* to) {
    sa.put(to);
    sb.put(to + kA);
  };
  // (Past the workgroup's last depth its loads repeat that one, and nothing reads them: a test in
  // each slot costs more, 8192^3 443 us for 432.)
  const auto advance = [&]() {
    lt += kTurn;
    if (lt < depths) {
      sa.base += kTurn * kDepth;
      sb.base += kTurn * kDepth;
    } else if (lv + static_cast<int>(gridDim.x) < tiles) {
      lt = 0;
      lv += gridDim.x;
      aim();
    } else {
      lt = depths - kTurn;
    }
  };
  // A tile's scales, straight to one of three places in turn: a wave that is still with the
  // outputs of two tiles before keeps its own.
  const auto get_scales = [&](int v, int turn) {
    int64_t m0, n0;
    place(v, m0, n0);
#pragma unroll
    for (int l = 0; l < kScaleLoads; ++l) {
      const int c = l * kLanes + threadIdx.x;
      const int64_t n = n0 + c % BN < p.n ? n0 + c % BN : p.n - 1, m = m0 + (c - 2 * BN) < p.m ? m0 + (c - 2 * BN) : p.m - 1;
      const float* from = c < BN ? p.bs + n : c < 2 * BN ? (p.bias ? p.bias : p.bs) + n : c < 2 * BN + BM ? p.as + m : p.as;
      bring_word(place_of<256>(reinterpret_cast<int8_t*>(scale[turn] + l * kLanes)), from);
    }
  };
  get_scales(blockIdx.x, 0);
  if (depths > 0) {
    aim();
#pragma unroll
    for (int d = 0; d < 2; d += kTurn) {
      if (DIRECT) {
#pragma unroll
        for (int l = 0; l < kLoads; ++l) begin(place_of<1024>(lds), place_of<1024>(lds + kStage), l);
      } else {
        hold();
        put(lds + d * kStage);
      }
      advance();
    }
    if (!DIRECT) hold();
  }
  all_here<0>();
  if (depths > 0) {
    if (DIRECT) {
#pragma unroll
      for (int l = 0; l < (kAhead < kBegin ? kAhead : kBegin) * kLoads / kBegin; ++l)
        begin(place_of<1024>(lds + 2 * kStage), place_of<1024>(lds + 3 * kStage), l);
    }
#pragma unroll
    for (int i = 0; i < kAhead; ++i) fetch_a(lds, i);
#pragma unroll
    for (int i = 0; i < NI; ++i) fetch_b(lds, 0, i);
  }

  int stage = 0, turn = 0;
  for (int v = blockIdx.x; v < tiles; v += gridDim.x) {
    int64_t m0, n0;
    place(v, m0, n0);
    const int then = turn == 2 ? 0 : turn + 1;
    // Blocks are read ahead across depths and tiles too: the barrier comes before the last kAhead
    // slots of a depth, when all of its blocks are in registers and, at the end of a pair, the next
    // pair has arrived.  (The workgroup's last depth reads what is not there, and does not use it.)  Every instruction here that is none of the matrix units' counts, since
    // a SIMD's two waves stand at the barrier together.
    for (int t = 0; t < depths; t += 2) {
#pragma unroll
      for (int half = 0; half < 2; ++half) {
        int8_t* now = lds + stage;
        stage = (stage + kStage) & (kStages * kStage - 1);
        int8_t* next = lds + stage;
        if (!DIRECT) {      // what was read a depth ago is for the depth after the next
          put(lds + ((stage + kStage) & (kStages * kStage - 1)));
          advance();
          hold();
        }
        const uint32_t to = place_of<1024>(lds + ((stage + (half == 0 ? 1 : 2) * kStage) & (kStages * kStage - 1)));
        const uint32_t then = place_of<1024>(lds + ((stage + (half == 0 ? 2 : 3) * kStage) & (kStages * kStage - 1)));
#pragma unroll
        for (int i = 0; i < MI - kAhead; ++i)
          slot(now, next, half, i, [&](int l) {
            if (DIRECT && half == 0) begin(to, then, l);
          });
        if (!DIRECT || half == 0) all_here<63>();
        else all_here<0>();
#pragma unroll
        for (int i = MI - kAhead; i < MI; ++i)
          slot(now, next, half, i, [&](int l) {
            if (DIRECT) begin(to, then, l);
          });
        if (DIRECT && half == 0) advance();
      }
    }
    // The tile's scales have arrived: DIRECT, with the next pair of depths; by way of registers, a
    // depth waits for what was read a depth ago, but near the end of k, and with no tile to follow,
    // nothing is read: at least its first depth reads the fourth, if that is not among the last two.
    if (depths == 0 || (!DIRECT && depths <= 4)) all_here<0>();
    get_scales(v + static_cast<int>(gridDim.x) < tiles ? v + static_cast<int>(gridDim.x) : v, then);

    // Outputs: 32 rows of 64 bytes at a time through LDS of the wave's own, so that they leave in
    // 16-byte words, four to a row.
    const float* bs = scale[turn] + wn * kCols;
    Tout* mine = room[wave];
    // the tile's first output, and the rows and columns of it that there are
    Tout* first = static_cast<Tout*>(p.out) + m0 * p.so + n0;
    const int tall = static_cast<int>(p.m - m0 < BM ? p.m - m0 : BM), wide = static_cast<int>(p.n - n0 < BN ? p.n - n0 : BN);
    const auto outputs = [&](auto whole) {
      int l = lane;      // anew in each tile: what follows from it is not kept over the depths
      asm volatile("" : "+v"(l));
      const int r = l & 15, h = l >> 4;
#pragma unroll
      for (int i = 0; i < MI / 2; ++i) {
        const int mi = wm * kRows + i * 32;
        float as[2];
#pragma unroll
        for (int u = 0; u < 2; ++u) as[u] = scale[turn][2 * BN + wm * kRows + i * 32 + u * 16 + r];
#pragma unroll
        for (int j = 0; j < kCols / kSpan; ++j) {
#pragma unroll
          for (int g = 0; g < kSpan / 16; ++g) {
            const int c = j * kSpan + g * 16 + h * 4;
            const f32x4 vb = *reinterpret_cast<const f32x4*>(bs + c);
            f32x4 bias = {};
            if (p.bias) bias = *reinterpret_cast<const f32x4*>(bs + BN + c);
#pragma unroll
            for (int u = 0; u < 2; ++u) {
              f32x4 out;
#pragma unroll
              for (int e = 0; e < 4; ++e)
                out[e] = fmaf(static_cast<float>(acc[2 * i + u][j * kSpan / 16 + g][e]), as[u] * vb[e], bias[e]);
              const int col = g * 16 + h * 4;
              stage_out(mine + (u * 16 + r) * kSpan + slot_of(r, col / kPer) * kPer + col % kPer, out);
            }
          }
          asm volatile("s_waitcnt lgkmcnt(0)" ::: "memory");
#pragma unroll
          for (int q = 0; q < 2; ++q) {
            const int row = q * 16 + l / 4, c = l % 4 * kPer;
            const int m = mi + row;
            const int n = wn * kCols + j * kSpan + c;
            typedef Tout word __attribute__((ext_vector_type(kPer)));
            typedef word word_any __attribute__((aligned(sizeof(Tout))));
            const word w = *reinterpret_cast<const word*>(mine + row * kSpan + slot_of(row, l % 4) * kPer);
            Tout* to = first + m * p.so + n;
            if (decltype(whole)::value || (m < tall && n + kPer <= wide)) {
              *reinterpret_cast<word_any*>(to) = w;
            } else if (m < tall) {
#pragma unroll
              for (int e = 0; e < kPer; ++e)
                if (n + e < wide) to[e] = w[e];
            }
          }
          asm volatile("s_waitcnt lgkmcnt(0)" ::: "memory");
        }
      }
    };
    if (tall == BM && wide == BN) outputs(std::true_type{});
    else outputs(std::false_type{});
#pragma unroll
    for (int i = 0; i < MI; ++i)
#pragma unroll
      for (int j = 0; j < NI; ++j) acc[i][j] = i32x4{};
    turn = then;
  }
  all_here<0>();   // no load to LDS outlives the workgroup
}

// Up to 16 rows of a: b is read once, from memory into registers, and the launch and one latency of
// memory are most of the time.  A workgroup has 16 rows of b; its waves split k, in steps of 64
// bytes, and their sums are joined in LDS.  Any alignment: a lane's 16 bytes of a row are loaded
// as they lie, the last ones of k byte by byte.  1 x 5120 x 2560: 8.5 us a call, 9.6 by tiles;
// 16 rows about the same either way, and from 32 on the tiles are ahead.
constexpr int kFewWaves = 8, kFewRows = 16;
template <typename Tout>
__global__ __launch_bounds__(64 * kFewWaves) void i8_few_kernel(MatmulParams p) {
  __shared__ i32x4 sums[kFewWaves][64];
  const int lane = threadIdx.x & 63, wave = threadIdx.x >> 6, r = lane & 15, h = lane >> 4;
  const int64_t n0 = static_cast<int64_t>(workgroup<64 * kFewWaves>()) * 16;
  if (n0 >= p.n) return;
  const int8_t* a = p.a + static_cast<int64_t>(r < p.m ? r : p.m - 1) * p.sa;
  const int8_t* b = p.b + (n0 + r < p.n ? n0 + r : p.n - 1) * p.sb;
  const auto get = [&](const int8_t* row, int k) {
    if (k + kChunk16 <= p.k) return i32x4(*reinterpret_cast<const i32x4_any*>(row + k));
    uint32_t w[4] = {};
    for (int j = 0; k + j < p.k; ++j) w[j / 4] |= static_cast<uint32_t>(static_cast<uint8_t>(row[k + j])) << 8 * (j % 4);
    return i32x4{static_cast<int>(w[0]), static_cast<int>(w[1]), static_cast<int>(w[2]), static_cast<int>(w[3])};
  };
  const int steps = (p.k + 63) / 64, each = (steps + kFewWaves - 1) / kFewWaves;
  const int begin = wave * each, end = begin + each < steps ? begin + each : steps;
  i32x4 acc = {};
#pragma unroll 4
  for (int s = begin; s < end; ++s) {
    const int k = s * 64 + h * kChunk16;
    acc = __builtin_amdgcn_mfma_i32_16x16x64_i8(get(b, k), get(a, k), acc, 0, 0, 0);
  }
  sums[wave][lane] = acc;
  __syncthreads();
  if (wave != 0 || r >= p.m) return;
#pragma unroll
  for (int w = 1; w < kFewWaves; ++w) acc += sums[w][lane];
  const float as = p.as[r];
#pragma unroll
  for (int e = 0; e < 4; ++e) {
    const int64_t n = n0 + h * 4 + e;
    if (n < p.n)
      store_val(static_cast<Tout*>(p.out) + r * p.so + n,
                fmaf(static_cast<float>(acc[e]), as * p.bs[n], p.bias ? p.bias[n] : 0.f));
  }
}

namespace {

// Rows that loads straight to LDS can take: whole pairs of depths, at multiples of 16 bytes, and a
// tile's rows within 32 bits of offsets.
bool direct(const MatmulParams& p) {
  const auto fine = [&](const int8_t* q, int64_t stride, int rows) {
    return reinterpret_cast<uintptr_t>(q) % 16 == 0 && (rows == 1 || (stride % 16 == 0 && stride < (1 << 23)));
  };
  return p.k % (2 * kDepth) == 0 && fine(p.a, p.sa, p.m) && fine(p.b, p.sb, p.n);
}

template <typename Tout, int BM, int BN, int WM, int WN, int GROUPS>
void tiles(const MatmulParams& p, hipStream_t s) {
  const int ntm = (p.m - 1) / BM + 1, ntn = (p.n - 1) / BN + 1;
  const int64_t n = static_cast<int64_t>(ntm) * ntn, most = kUnits * GROUPS;
  const dim3 grid(static_cast<unsigned>(n < most ? n : most)), block(64 * WM * WN);
  if (direct(p)) hipLaunchKernelGGL((i8_tile_kernel<Tout, BM, BN, WM, WN, GROUPS, true>), grid, block, 0, s, p, ntm, ntn);
  else hipLaunchKernelGGL((i8_tile_kernel<Tout, BM, BN, WM, WN, GROUPS, false>), grid, block, 0, s, p, ntm, ntn);
}

int64_t tiles_of(const MatmulParams& p, int side) {
  return static_cast<int64_t>((p.m - 1) / side + 1) * ((p.n - 1) / side + 1);
}

// The tile's side.  Small tiles while the compute units hold them all at once, two each: what a
// depth of k takes then is latency, which grows with the tile (one set of inputs again and
// again, which stays in L2; three in turn take 21 us for the first: 256 x 2560 x 5120, in 160 tiles
// of 64 x 64 15 us, in 40 of 128 x 128 28, in 10 of 256 x 256 55; but 256 x 10240 x 2560, in 640 of
// 64 x 64 21 us, in 160 of 128 x 128 17; 2048 x 4096 x 2048, 512 tiles of 128 x 128 22 us, 128 of
// 256 x 256 28).  Otherwise the largest, which reads least (4096 x 2560 x
// 2560: 160 of 256 x 256 36 us, 640 of 128 x 128 40).  Where they go in rounds of which the last is
// partly filled, the rows beyond the whole rounds go by the smaller tiles, if those fit at once (float32:
// 16411 x 1280 x 2560, 325 tiles, 72 us in one launch, 67 with the last 3355 rows in 270 small
// tiles; 4200 x 4096 x 4096 96 and 78; 9000 x 2048 x 2048 57 and 49; 6000 x 2560 x 5120 71 and 70).
template <typename Tout>
void product(const MatmulParams& p, hipStream_t s) {
  const dim3 few_grid = grid_of<64 * kFewWaves>((static_cast<int64_t>(p.n) + 15) / 16);
  if (p.m <= kFewRows) {
    hipLaunchKernelGGL((i8_few_kernel<Tout>), few_grid, dim3(64 * kFewWaves), 0, s, p);
    return;
  }
  if (tiles_of(p, 64) <= 2 * kUnits) return tiles<Tout, 64, 64, 2, 2, 3>(p, s);
  if (tiles_of(p, 128) <= 2 * kUnits) return tiles<Tout, 128, 128, 2, 2, 2>(p, s);
  const int64_t all = tiles_of(p, 256), across = (p.n - 1) / 256 + 1;
  const int64_t high = all / kUnits * kUnits / across * 256;       // rows in whole rounds
  if (high > 0 && high < p.m) {
    MatmulParams rest = p;
    rest.m = static_cast<int>(p.m - high);
    rest.a += high * p.sa;
    rest.as += high;
    rest.out = static_cast<Tout*>(p.out) + high * p.so;
    if (tiles_of(rest, 128) <= 2 * kUnits) {
      MatmulParams most = p;
      most.m = static_cast<int>(high);
      tiles<Tout, 256, 256, 2, 4, 1>(most, s);
      return product<Tout>(rest, s);
    }
  }
  tiles<Tout, 256, 256, 2, 4, 1>(p, s);
}

}  // namespace

hipError_t launch_i8_matmul(const MatmulParams& p, bool bf16, hipStream_t s) {
  if (bf16) product<bf16_t>(p, s);
  else product<float>(p, s);
  return hipGetLastError();
}

}  // namespace sscan
