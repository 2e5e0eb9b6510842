// K7: products in 8-bit floating point (e4m3) with fp32 scales, one per activation row and 128
// columns and one per 128 x 128 block of a weight matrix, dense or grouped by expert:
//
//   y[r][n] = sum_b sx[r][b] sw[e(r)][n / 128][b] * P_b,   P_b = sum_{c in block b} xq[r][c] wq[e][n][c]
//
// Every P_b is formed by the tensor cores (tcgen05, kind::f8f6f4: products exact, sums fp32 in tensor
// memory) over the block's 128 columns; scales are general fp32 numbers, so P_b is then read back
// and folded into fp32 registers with one fused multiply-add per element and block.  The gated form
// multiplies a gate and an up half, and its epilogue forms h = SiLU(gate) * up and quantises it for
// the next product (one power-of-two scale per row and 128 features: one tile).
//
// Work: units of 128 rows x 256 columns (gated: 128 gate and the 128 matching up columns), in order
// of expert, column tile, row tile; one CTA per SM.  Whole waves of units go one unit to a CTA.  Where
// the rest (U mod SMs units) is at most half the grid, each of its units is cut along K into as many
// pieces as there are CTAs for it (none shorter than kMinPiece blocks) and joined by the CTA that
// finishes last (partials and a counter in the workspace; the sum runs in piece order whoever joins, so
// results repeat bit for bit); a larger rest stays whole and the CTAs behind it idle.  Nobody waits
// for another CTA.
//
// What bounds it: per SM and block the products take 512 cycles, and two blocks (2 x 256 columns) are
// all that tensor memory holds, so a block's turn is half of products + signals + reading back.  4736 x
// 1024 x 16384, one unit of 128 blocks an SM: 84 us alone and 141,000 cycles at 1.68 GHz, so 1,100 a block
// with the launch's start and end, the tensor pipe 50 % active; 80 us a launch back to back (2.0
// PFLOP/s).  4096 x 5120 x 3584, 126 blocks on the fullest SM: 98 us alone, 86 back to back (1.75 PFLOP/s).
// Tried and slower: 128-column products with four half stages (rows read twice from shared memory),
// sixteen epilogue warps of 64 columns, scales loaded two blocks ahead (registers).
//
// Order of launches: a launch before the one in front of this one has completed when this one starts
// (every kernel here lets its dependents start only after its own wait), so the offsets and the
// weights are read at once, and only the rows, their scales, the counters and the outputs wait for
// the launch in front.  The first weight tiles of a CTA then travel while slower CTAs of that launch
// still finish.
//
// Warps: 0 TMA producer (4 stages of 16 KB rows + 32 KB weights; few rows: only their 16-row boxes),
// 1 MMA issuer (4 MMAs of 128 x 256 x 32 a block into one of two tensor-memory stages), 2 tensor
// memory, 4-11 epilogue (two warps per 32-row quarter, 128 columns each; warps whose rows are all
// beyond the group only keep the barriers).
#pragma once
#include <cuda.h>

#include "pw_common.cuh"
#include "pw_ffn.cuh"
#include "pw_rows.cuh"
#include "pw_tc.cuh"

namespace pw {
namespace k7 {

constexpr int kTileM = 128, kTileN = 256, kBlk = 128;
constexpr int kStages = 4;
constexpr int kABytes = kTileM * kBlk, kBBytes = kTileN * kBlk;
constexpr int kStageBytes = kABytes + kBBytes;
constexpr int kSmallRows = 16;  // rows of the small activation box
constexpr int kThreads = 384;
constexpr int kEpiThreads = 256;
// registers a thread: 56 in the producer warpgroup, 224 in the two epilogue warpgroups (128
// accumulators and two buffers of 32); their sum may not exceed what the block is launched with
constexpr int kProducerRegs = 56, kEpilogueRegs = 224;
constexpr int kSplitRegs = 128 * kProducerRegs + kEpiThreads * kEpilogueRegs;
static_assert(kSplitRegs <= 65536, "register file");
constexpr int kTmemCols = 512, kAccCols = 256;
// Shortest piece, in K blocks: shorter ones cost more in joining than they spread.  (This kernel: 3001
// ragged rows over 60 experts, K 2040, 81 us whole and 87 in pieces of 8; 64 rows x 5120 x 3584 24.5
// us in pieces of 14 or more, 25.2 of 9, 34.7 of 4.  The few-rows kernel: 16 rows 16.5 us in pieces of
// 9, 18.6 of 14.)
constexpr int kMinPiece = 12;

constexpr int kOffBar = kStages * kStageBytes;
constexpr int kNumBars = 2 * kStages + 4 + 1;
constexpr int kOffMisc = kOffBar + ((kNumBars * 8 + 15) / 16) * 16;
constexpr int kOffAmax = kOffMisc + 32;
constexpr int kOffStage = kOffAmax + 2 * kTileM * 4;  // output staging, 32 rows x 80 bytes a warp
constexpr int kOffTiles = kOffStage + (kEpiThreads / 32) * 32 * 80;  // [E + 1] row tiles before each expert
constexpr int smem_bytes(int E) { return kOffTiles + 2 * (E + 1) * 4; }
static_assert(smem_bytes(PW_MAX_EXPERTS) <= 227 * 1024, "shared memory budget");

struct alignas(64) Params {
  CUtensorMap xmap;    // rows, box 128 columns x 128 rows
  CUtensorMap xsmall;  // rows, box 128 columns x 16 rows
  CUtensorMap wmap;    // weights [E][N][K], box 128 columns x 256 rows (gated: 64)
  const float* sx;
  const float* sw;
  const int32_t* offsets;  // [E + 1] or NULL: one expert, all M rows
  int M, N, K, E;
  int kb, nb, nt;  // K blocks, N scale blocks, column tiles
  void* y;
  size_t ld_y;
  int vec;  // rows of y may be stored 16 bytes at a time
  uint8_t* hq;  // gated: e4m3 [M][I], fp32 scales [M][I / 128]
  float* hs;
  int I;
  float* part;       // [CTA][256][rcap]
  int rcap;
  int32_t* counter;  // [CTAs], zero at launch
};

// ---- schedule (the same in every role) ----
struct Sched {
  int waves, rem, pieces, run;  // run: K blocks of the remainder, cut into `pieces`
};
// The units behind the last whole wave are cut where each can have two CTAs or more: every such unit
// into the same number of pieces, so that a unit has the fewest pieces to join.  (Cutting them into
// equal runs for all CTAs, wherever a unit ends, costs more in joins than it spreads: 4 tokens x
// 28672 x 4096, 112 units, 34.6 us against 29.0 with 112 CTAs at work; 112 SMs draw what HBM gives.)
__device__ __forceinline__ Sched make_sched(int units, int kb, int grid, int min_piece) {
  Sched s;
  s.waves = units / grid;
  s.rem = units - s.waves * grid;
  s.run = s.rem * kb;
  s.pieces = s.rem ? s.rem * max(1, min(grid / s.rem, kb / min_piece)) : 0;
  return s;
}
__device__ __forceinline__ int piece_begin(const Sched& s, int p) {
  return static_cast<int>(static_cast<long long>(s.run) * p / s.pieces);
}
__device__ __forceinline__ int piece_of(const Sched& s, int x) {  // the piece that holds K block x
  return static_cast<int>((static_cast<long long>(x + 1) * s.pieces - 1) / s.run);
}
struct Piece {
  int unit, k0, k1;
  int first, count, slot;  // the unit's pieces are those of CTAs first ..; one workspace slot a CTA
};
// The i-th piece of a CTA: its units of the whole waves, then its piece of the remainder (within one
// unit: pieces is a multiple of rem).
__device__ __forceinline__ bool get_piece(const Sched& s, int kb, int i, Piece& p) {
  const int cta = blockIdx.x;
  p.first = 0;
  p.count = 1;
  p.slot = 0;
  if (i < s.waves) {
    p.unit = cta + i * static_cast<int>(gridDim.x);
    p.k0 = 0;
    p.k1 = kb;
    return true;
  }
  if (i > s.waves || cta >= s.pieces) return false;  // pieces = 0 without a remainder
  const int a = piece_begin(s, cta), b = piece_begin(s, cta + 1), j = a / kb;
  p.unit = s.waves * static_cast<int>(gridDim.x) + j;
  p.k0 = a - j * kb;
  p.k1 = p.k0 + b - a;
  p.first = piece_of(s, j * kb);
  p.count = piece_of(s, (j + 1) * kb - 1) - p.first + 1;
  p.slot = cta;
  return true;
}

// The 256 epilogue threads (threads 128-383), after their partials are written: true in all of them
// if this is the last of the unit's `count` pieces; the others' partials are then visible.
constexpr int kEpiBarrier = 1;
__device__ __forceinline__ bool last_piece(int32_t* counter, int count, int* s_last) {
  named_sync(kEpiBarrier, kEpiThreads);
  if (threadIdx.x == 128) {  // releases what the barrier gathered, acquires what others released
    int before;
    asm volatile("atom.add.acq_rel.gpu.global.s32 %0, [%1], 1;" : "=r"(before) : "l"(counter) : "memory");
    *s_last = before == count - 1;
  }
  named_sync(kEpiBarrier, kEpiThreads);
  return *s_last != 0;
}

struct Unit {
  int e, row0, rows, n;  // expert, first row, rows (<= the tile's), column tile
};
template <int TM>
__device__ __forceinline__ Unit find_unit(const Params& p, const int* tiles, const int* first, int u) {
  const int v = u / p.nt;
  int lo = 0, hi = p.E - 1;  // the last expert with tiles[e] <= v that has tiles
  while (lo < hi) {
    const int mid = (lo + hi + 1) >> 1;
    if (tiles[mid] <= v) lo = mid;
    else hi = mid - 1;
  }
  Unit r;
  r.e = lo;
  const int mt = tiles[lo + 1] - tiles[lo];
  const int local = u - p.nt * tiles[lo];
  r.n = local / mt;
  const int m = local - r.n * mt;
  r.row0 = first[lo] + m * TM;
  r.rows = min(TM, first[lo + 1] - r.row0);
  return r;
}

// ---- waits ----
// Bounded wait on an mbarrier, as mbar_wait, but the clock and the limit (a global load) are read
// only after several suspended tries: this kernel hands tensor-memory stages back and forth every
// few hundred cycles, and reading the limit first lengthens every wait (4736 x 1024 x 16384, back to back:
// 83.3 us with mbar_wait, 81.7 us so).
__device__ __forceinline__ bool wait_slow(uint64_t* bar, uint32_t parity, volatile int* abort_flag) {
  const unsigned long long t0 = global_ns();
  const unsigned long long limit = wait_limit_ns();
  for (;;) {
    if (mbar_try_wait(bar, parity)) return true;
    if (*abort_flag) return false;
    if (global_ns() - t0 > limit) {
      set_status(PW_ERR_TIMEOUT);
      *abort_flag = 1;
      return false;
    }
  }
}
__device__ __forceinline__ bool wait_bar(uint64_t* bar, uint32_t parity, volatile int* abort_flag) {
#pragma unroll 1
  for (int i = 0; i < 8; ++i) {
    if (mbar_try_wait(bar, parity)) return true;
    if (*abort_flag) return false;
  }
  return wait_slow(bar, parity, abort_flag);
}

// The whole warp waits; the answer is the same in every lane, so no later warp-wide step meets a
// split warp.
__device__ __forceinline__ bool warp_wait(uint64_t* bar, uint32_t parity, volatile int* abort_flag) {
  return __all_sync(0xffffffffu, wait_bar(bar, parity, abort_flag));
}

// Both barriers, for the warp that feeds the tensor cores: the two tries run together and one vote
// serves both (a block's turn of that warp has to stay under the block's 512 cycles of products).
__device__ __forceinline__ bool warp_wait2(uint64_t* a, uint32_t pa, uint64_t* b, uint32_t pb,
                                           volatile int* abort_flag) {
  const bool ra = mbar_try_wait(a, pa), rb = mbar_try_wait(b, pb);
  if (__all_sync(0xffffffffu, ra && rb)) return true;
  return __all_sync(0xffffffffu, wait_bar(a, pa, abort_flag) && wait_bar(b, pb, abort_flag));
}

// Test hook (pw_test_hold_down_items): an issuing warp waits for products that never come, so that
// every bounded wait of the block runs out.  True in normal use.
__device__ __forceinline__ bool not_held(uint64_t* never, volatile int* abort_flag) {
  if (*static_cast<volatile int*>(&g_test_hold) == 0) return true;
  return warp_wait(never, 0, abort_flag);
}

// ---- tcgen05 / TMA ----
// Shared-memory descriptor of a K-major operand with 128-byte swizzle (8 rows x 128 bytes atoms,
// 1024 bytes apart).
__device__ __forceinline__ uint64_t sw128_desc(uint32_t saddr) {
  return static_cast<uint64_t>((saddr >> 4) & 0x3fffu) | (1ull << 16) | (64ull << 32) | (1ull << 46) |
         (2ull << 61);
}
// kind::f8f6f4, e4m3 x e4m3 (both K-major) -> fp32, M = 128, N = 256.
constexpr uint32_t kInstr = (1u << 4) | ((kTileN >> 3) << 17) | ((kTileM >> 4) << 24);

__device__ __forceinline__ void mma_f8(uint32_t d, uint64_t a, uint64_t b, uint32_t instr,
                                       uint32_t accumulate) {
  asm volatile(
      "{\n\t.reg .pred p;\n\t"
      "setp.ne.b32 p, %4, 0;\n\t"
      "tcgen05.mma.cta_group::1.kind::f8f6f4 [%0], %1, %2, %3, p;\n\t}"
      ::"r"(d), "l"(a), "l"(b), "r"(instr), "r"(accumulate)
      : "memory");
}

// True in one lane of the (converged) warp.
__device__ __forceinline__ bool elect_one() {
  uint32_t p;
  asm volatile(
      "{\n\t.reg .pred p;\n\t"
      "elect.sync _|p, 0xffffffff;\n\t"
      "selp.u32 %0, 1, 0, p;\n\t}"
      : "=r"(p));
  return p != 0;
}

__device__ __forceinline__ void tma_2d(uint32_t dst, const CUtensorMap* map, int x, int y, uint64_t* bar) {
  asm volatile(
      "cp.async.bulk.tensor.2d.shared::cluster.global.mbarrier::complete_tx::bytes [%0], "
      "[%1, {%2, %3}], [%4];" ::"r"(dst),
      "l"(map), "r"(x), "r"(y), "r"(smem_u32(bar))
      : "memory");
}
__device__ __forceinline__ void tma_3d(uint32_t dst, const CUtensorMap* map, int x, int y, int z,
                                       uint64_t* bar) {
  asm volatile(
      "cp.async.bulk.tensor.3d.shared::cluster.global.mbarrier::complete_tx::bytes [%0], "
      "[%1, {%2, %3, %4}], [%5];" ::"r"(dst),
      "l"(map), "r"(x), "r"(y), "r"(z), "r"(smem_u32(bar))
      : "memory");
}
__device__ __forceinline__ void prefetch_map(const CUtensorMap* map) {
  asm volatile("prefetch.tensormap [%0];" ::"l"(map) : "memory");
}

// 32 columns of this warp's lane quarter, asynchronously; the registers hold them after tmem_wait.
__device__ __forceinline__ void tmem_ld32(uint32_t addr, uint32_t (&r)[32]) {
  asm volatile(
      "tcgen05.ld.sync.aligned.32x32b.x32.b32 "
      "{%0, %1, %2, %3, %4, %5, %6, %7, %8, %9, %10, %11, %12, %13, %14, %15, "
      "%16, %17, %18, %19, %20, %21, %22, %23, %24, %25, %26, %27, %28, %29, %30, %31}, [%32];"
      : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3]), "=r"(r[4]), "=r"(r[5]), "=r"(r[6]), "=r"(r[7]),
        "=r"(r[8]), "=r"(r[9]), "=r"(r[10]), "=r"(r[11]), "=r"(r[12]), "=r"(r[13]), "=r"(r[14]),
        "=r"(r[15]), "=r"(r[16]), "=r"(r[17]), "=r"(r[18]), "=r"(r[19]), "=r"(r[20]), "=r"(r[21]),
        "=r"(r[22]), "=r"(r[23]), "=r"(r[24]), "=r"(r[25]), "=r"(r[26]), "=r"(r[27]), "=r"(r[28]),
        "=r"(r[29]), "=r"(r[30]), "=r"(r[31])
      : "r"(addr));
}
// The registers pass through the wait so that nothing that uses them moves above it.
__device__ __forceinline__ void tmem_wait(uint32_t (&r)[32]) {
  asm volatile("tcgen05.wait::ld.sync.aligned;"
               : "+r"(r[0]), "+r"(r[1]), "+r"(r[2]), "+r"(r[3]), "+r"(r[4]), "+r"(r[5]), "+r"(r[6]),
                 "+r"(r[7]), "+r"(r[8]), "+r"(r[9]), "+r"(r[10]), "+r"(r[11]), "+r"(r[12]),
                 "+r"(r[13]), "+r"(r[14]), "+r"(r[15]), "+r"(r[16]), "+r"(r[17]), "+r"(r[18]),
                 "+r"(r[19]), "+r"(r[20]), "+r"(r[21]), "+r"(r[22]), "+r"(r[23]), "+r"(r[24]),
                 "+r"(r[25]), "+r"(r[26]), "+r"(r[27]), "+r"(r[28]), "+r"(r[29]), "+r"(r[30]),
                 "+r"(r[31])
               :
               : "memory");
}

// The same for two buffers, one wait.
__device__ __forceinline__ void tmem_wait2(uint32_t (&a)[32], uint32_t (&b)[32]) {
  tmem_wait(a);
#pragma unroll
  for (int i = 0; i < 32; i += 8)
    asm volatile("" : "+r"(b[i]), "+r"(b[i + 1]), "+r"(b[i + 2]), "+r"(b[i + 3]), "+r"(b[i + 4]),
                 "+r"(b[i + 5]), "+r"(b[i + 6]), "+r"(b[i + 7]));
}

// acc[0..31] += r * s, two elements an instruction.
__device__ __forceinline__ void fold32(float* acc, const uint32_t (&r)[32], float s) {
  const uint64_t s2 = (static_cast<uint64_t>(__float_as_uint(s)) << 32) | __float_as_uint(s);
#pragma unroll
  for (int i = 0; i < 32; i += 2) {
    const uint64_t x = (static_cast<uint64_t>(r[i + 1]) << 32) | r[i];
    uint64_t a = (static_cast<uint64_t>(__float_as_uint(acc[i + 1])) << 32) | __float_as_uint(acc[i]);
    asm("fma.rn.f32x2 %0, %1, %2, %0;" : "+l"(a) : "l"(x), "l"(s2));
    acc[i] = __uint_as_float(static_cast<uint32_t>(a));
    acc[i + 1] = __uint_as_float(static_cast<uint32_t>(a >> 32));
  }
}

// SiLU(g) * u.  With t = e^-|g| the sigmoid is 1 / (1 + t), or t / (1 + t) for a negative g: t never
// overflows and the denominator is in [1, 2], where the fast division holds (2 units in the last place;
// e^-g itself would pass 2^126 at g = -87.4, from where that division returns 0).  The fast exponential
// is off by up to 2 + 1.2 |g| units, so for negative g the result is too, by 2^-18 of its value at -20
// and 2^-16 at -87: far below the half step, 2^-4, of the e4m3 value it becomes next.  (With expf
// the prompt layer of 4096 tokens takes 2 % longer.)
__device__ __forceinline__ float gated(float g, float u) {
  const float t = __expf(-fabsf(g));
  return __fdividef(g < 0.0f ? g * t : g, 1.0f + t) * u;
}

// A warp's 32 rows x 128 columns (a thread holds one row's) to y, through a staging buffer of 32 rows
// x 64 bytes (rows 80 bytes apart: conflict free both ways), so that a store instruction writes
// 64-byte runs of 8 rows and not 16 bytes of 32.  rows: rows of the warp that exist; n: first column.
constexpr int kStageRow = 80;
template <int TY>
__device__ __forceinline__ void store_rows(uint8_t* stage, void* y, size_t row0, size_t ld, int rows, int n,
                                           int N, int vec, const float (&acc)[128], int lane) {
  constexpr int S = ElemSize<TY>::value, C = 64 / S;  // columns of a run
#pragma unroll
  for (int c0 = 0; c0 < 128; c0 += C) {
    if (n + c0 >= N) break;
    __syncwarp();
#pragma unroll
    for (int c = 0; c < C; c += 16 / S) {
      float v[16 / S];
#pragma unroll
      for (int i = 0; i < 16 / S; ++i) v[i] = acc[c0 + c + i];
      store_elems<TY, 16 / S>(stage + lane * kStageRow + c * S, v);
    }
    __syncwarp();
    if (vec && n + c0 + C <= N) {
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        const int r = 8 * i + (lane >> 2), c = (lane & 3) * 16;
        const uint4 w = *reinterpret_cast<const uint4*>(stage + r * kStageRow + c);
        if (r < rows)
          *reinterpret_cast<uint4*>(static_cast<uint8_t*>(y) + ((row0 + r) * ld + n + c0) * S + c) = w;
      }
    } else {
      for (int i = 0; i < 32 * C / 32; ++i) {
        const int r = (32 / C) * i + lane / C, c = lane % C;
        if (r < rows && n + c0 + c < N) {
          void* d = elem_at(y, (row0 + r) * ld + n + c0 + c, S);
          if (S == 4)
            *static_cast<uint32_t*>(d) = *reinterpret_cast<const uint32_t*>(stage + r * kStageRow + c * 4);
          else
            *static_cast<uint16_t*>(d) = *reinterpret_cast<const uint16_t*>(stage + r * kStageRow + c * 2);
        }
      }
    }
  }
}

// Row tiles (of TM rows) before each expert, from the offsets: tiles[E + 1], first[E + 1] in shared
// memory.  Offsets that decrease or leave [0, M] are recorded; a group that would start before an
// earlier offset gets no rows, so groups are disjoint (no row has two writers) and there are at most
// M / TM + E tiles whatever the offsets hold.  Whole block.
template <int TM>
__device__ __forceinline__ void row_tiles(const Params& p, int* tiles, int* first) {
  const int E = p.E;
  for (int e = threadIdx.x; e <= E; e += blockDim.x) {
    const int o = p.offsets ? __ldcg(p.offsets + e) : (e ? p.M : 0);
    first[e] = min(max(o, 0), p.M);
    if (o < 0 || o > p.M) set_status(PW_ERR_BOUNDS);
  }
  __syncthreads();
  if (threadIdx.x < 32) {
    const int lane = threadIdx.x;
    int carry = 0;
    int top = -1;  // from the first 32 experts on whose offsets decrease: the largest offset before
    for (int e0 = 0; e0 < E; e0 += 32) {
      const int e = e0 + lane, a = e < E ? first[e] : 0;
      int rows = e < E ? first[e + 1] - a : 0;
      if (rows < 0) set_status(PW_ERR_BOUNDS);
      if (__any_sync(0xffffffffu, rows < 0) || top >= 0) {
        int m = max(a, top);  // largest offset up to this one
#pragma unroll
        for (int d = 1; d < 32; d <<= 1) m = max(m, __shfl_up_sync(0xffffffffu, m, d));
        if (a < m) rows = 0;
        top = __shfl_sync(0xffffffffu, m, 31);
      }
      int v = rows > 0 ? (rows + TM - 1) / TM : 0;
#pragma unroll
      for (int d = 1; d < 32; d <<= 1) {
        const int o = __shfl_up_sync(0xffffffffu, v, d);
        if (lane >= d) v += o;
      }
      if (e < E) tiles[e + 1] = carry + v;
      carry += __shfl_sync(0xffffffffu, v, 31);
    }
    if (lane == 0) tiles[0] = 0;
  }
}

// GATED: the gate_up product (N = 2I; I % 128 == 0).  TO: type of y (GATED: unused).
template <bool GATED, int TO>
__global__ void __launch_bounds__(kThreads, 1) scaled_kernel(const __grid_constant__ Params p) {
  uint8_t* const smem = k4::g_smem;
  uint64_t* full = reinterpret_cast<uint64_t*>(smem + kOffBar);
  uint64_t* empty = full + kStages;
  uint64_t* acc_full = empty + kStages;
  uint64_t* acc_empty = acc_full + 2;
  uint64_t* mma_done = acc_empty + 2;
  uint32_t* tmem_slot = reinterpret_cast<uint32_t*>(smem + kOffMisc);
  volatile int* abort_flag = reinterpret_cast<volatile int*>(tmem_slot + 1);
  int* s_last = reinterpret_cast<int*>(tmem_slot + 2);
  float* s_amax = reinterpret_cast<float*>(smem + kOffAmax);
  int* s_tiles = reinterpret_cast<int*>(smem + kOffTiles);  // [E + 1]
  const int E = p.E;
  int* s_first = s_tiles + E + 1;                           // [E + 1]
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;

  if (smem_u32(smem) & 1023) {  // the swizzled buffers start on 1024-byte boundaries
    if (threadIdx.x == 0) set_status(PW_ERR_UNSUPPORTED);
    return;
  }
  if (threadIdx.x == 0) {
    for (int s = 0; s < kStages; ++s) {
      mbar_init(&full[s], 1);
      mbar_init(&empty[s], 1);
    }
    for (int b = 0; b < 2; ++b) {
      mbar_init(&acc_full[b], 1);
      mbar_init(&acc_empty[b], kEpiThreads / 32);
    }
    mbar_init(mma_done, 1);
    *abort_flag = 0;
    mbar_fence_init();
    prefetch_map(&p.xmap);
    prefetch_map(&p.xsmall);
    prefetch_map(&p.wmap);
  }
  if (warp == 2) {
    asm volatile("tcgen05.alloc.cta_group::1.sync.aligned.shared::cta.b32 [%0], %1;" ::"r"(
                     smem_u32(tmem_slot)),
                 "r"(kTmemCols)
                 : "memory");
    asm volatile("tcgen05.relinquish_alloc_permit.cta_group::1.sync.aligned;" ::: "memory");
  }
  row_tiles<kTileM>(p, s_tiles, s_first);
  k5::tc_fence_before();
  __syncthreads();
  k5::tc_fence_after();
  const uint32_t tmem_base = *tmem_slot;
  const Sched sched = make_sched(s_tiles[E] * p.nt, p.kb, gridDim.x, kMinPiece);
  const uint32_t smem_base = smem_u32(smem);

  if (warp < 4) {
    asm volatile("setmaxnreg.dec.sync.aligned.u32 %0;" ::"n"(kProducerRegs));
    const bool leader = elect_one();  // one lane issues; control flow and operands stay uniform
    if (warp == 0) {
      // ---------------- producer ----------------
      // the first kStages weight tiles are on their way before the launch in front has ended; the
      // rows (its output) follow
      uint32_t g = 0;
      Piece pc;
      bool ok = true;
      auto rows_of = [&](const Unit& u, int b, uint32_t stage) {
        const uint32_t a = smem_base + stage * kStageBytes;
        if (u.rows > kTileM / 2) {
          tma_2d(a, &p.xmap, b * kBlk, u.row0, &full[stage]);
        } else {
          for (int q = 0; q * kSmallRows < u.rows; ++q)
            tma_2d(a + q * kSmallRows * kBlk, &p.xsmall, b * kBlk, u.row0 + q * kSmallRows, &full[stage]);
        }
      };
      auto follow = [&]() {  // the rows of the blocks before g
        griddep_wait();
        if (leader) {
          uint32_t h = 0;
          Piece q;
          for (int i = 0; h < g && get_piece(sched, p.kb, i, q); ++i) {
            const Unit u = find_unit<kTileM>(p, s_tiles, s_first, q.unit);
            for (int b = q.k0; b < q.k1 && h < g; ++b, ++h) rows_of(u, b, h);
          }
          griddep_launch();
        }
        __syncwarp();
      };
      bool waited = false;
      for (int i = 0; ok && get_piece(sched, p.kb, i, pc); ++i) {
        const Unit u = find_unit<kTileM>(p, s_tiles, s_first, pc.unit);
        const int boxes = (u.rows + kSmallRows - 1) / kSmallRows;
        const uint32_t bytes = kBBytes + (u.rows > kTileM / 2 ? kABytes : boxes * kSmallRows * kBlk);
        for (int b = pc.k0; b < pc.k1; ++b, ++g) {
          if (g == kStages && !waited) {
            follow();
            waited = true;
          }
          const int s = g % kStages;
          if (!(ok = warp_wait(&empty[s], ((g / kStages) & 1) ^ 1, abort_flag))) break;
          if (leader) {
            mbar_arrive_expect_tx(&full[s], bytes);
            const uint32_t w = smem_base + s * kStageBytes + kABytes;
            if (GATED) {  // 64 gate, 64 up, 64 gate, 64 up rows: each epilogue half has both
              for (int q = 0; q < 4; ++q)
                tma_3d(w + q * (kBBytes / 4), &p.wmap, b * kBlk,
                       (q & 1 ? p.I : 0) + u.n * 128 + (q >> 1) * 64, u.e, &full[s]);
            } else {
              tma_3d(w, &p.wmap, b * kBlk, u.n * kTileN, u.e, &full[s]);
            }
            if (waited) rows_of(u, b, s);
          }
          __syncwarp();
        }
      }
      if (!waited) follow();
      // every issued copy has landed before the block exits
      if (leader)
        for (uint32_t x = (g > kStages ? g - kStages : 0); x < g; ++x)
          mbar_wait(&full[x % kStages], (x / kStages) & 1);
    } else if (warp == 1) {
      // ---------------- MMA issuer ----------------
      bool ok = not_held(mma_done, abort_flag);
      griddep_wait();  // nothing to multiply before; the bounded waits below start after it
      const uint64_t ad0 = sw128_desc(smem_base);
      uint32_t g = 0;
      Piece pc;
      for (int i = 0; ok && get_piece(sched, p.kb, i, pc); ++i) {
        for (int b = pc.k0; b < pc.k1; ++b, ++g) {
          const int s = g % kStages, t = g & 1;
          if (!(ok = warp_wait2(&full[s], (g / kStages) & 1, &acc_empty[t], ((g >> 1) & 1) ^ 1, abort_flag)))
            break;
          k5::tc_fence_after();
          const uint64_t ad = ad0 + static_cast<uint64_t>(s) * (kStageBytes / 16);
          const uint32_t d = tmem_base + t * kAccCols;
          if (leader) {
#pragma unroll
            for (int j = 0; j < 4; ++j)  // 32 bytes of K each
              mma_f8(d, ad + 2 * j, ad + kABytes / 16 + 2 * j, kInstr, j > 0);
            k5::mma_commit(&acc_full[t]);
            k5::mma_commit(&empty[s]);
          }
        }
      }
      __syncwarp();
      if (leader) {
        k5::mma_commit(mma_done);
        mbar_wait(mma_done, 0);
      }
    }
  } else {
    // ---------------- epilogue ----------------
    asm volatile("setmaxnreg.inc.sync.aligned.u32 %0;" ::"n"(kEpilogueRegs));
    const int ew = warp - 4, quarter = ew & 3, half = ew >> 2;
    const int r = quarter * 32 + lane;
    const uint32_t lane_addr = tmem_base + (static_cast<uint32_t>(quarter * 32) << 16) + half * 128;
    uint32_t g = 0;
    Piece pc;
    bool dead = false;  // a wait gave up: keep every barrier, write zeros
    griddep_wait();
    bool more = get_piece(sched, p.kb, 0, pc);
    Unit u;
    const float *sx, *sw0, *sw1;
    float a_next, w0_next, w1_next;
    auto begin = [&]() {  // the unit of pc, and its first scales on their way
      u = find_unit<kTileM>(p, s_tiles, s_first, pc.unit);
      sx = p.sx + static_cast<size_t>(u.row0 + min(r, u.rows - 1)) * p.kb;
      int n0 = GATED ? u.n : 2 * u.n + half;  // 128-row scale block of columns 0-63 of the half
      int n1 = GATED ? p.I / 128 + u.n : n0;  // and of columns 64-127
      n0 = min(n0, p.nb - 1);
      n1 = min(n1, p.nb - 1);
      sw0 = p.sw + (static_cast<size_t>(u.e) * p.nb + n0) * p.kb;
      sw1 = p.sw + (static_cast<size_t>(u.e) * p.nb + n1) * p.kb;
      a_next = __ldg(sx + pc.k0);
      w0_next = __ldg(sw0 + pc.k0);
      w1_next = GATED ? __ldg(sw1 + pc.k0) : 0.0f;
    };
    if (more) begin();
    for (int i = 0; more; ++i) {
      const bool mine = quarter * 32 < u.rows;  // the warp has rows
      const bool live = r < u.rows;
      float acc[128];
#pragma unroll
      for (int c = 0; c < 128; ++c) acc[c] = 0.0f;
      for (int b = pc.k0; b < pc.k1; ++b, ++g) {
        const int t = g & 1;
        const float s0 = a_next * w0_next, s1 = GATED ? a_next * w1_next : s0;
        if (b + 1 < pc.k1) {
          a_next = __ldg(sx + b + 1);
          w0_next = __ldg(sw0 + b + 1);
          if (GATED) w1_next = __ldg(sw1 + b + 1);
        }
        if (!warp_wait(&acc_full[t], (g >> 1) & 1, abort_flag)) {
          dead = true;
        } else {
          k5::tc_fence_after();
          if (mine) {
            uint32_t v0[32], v1[32];
            const uint32_t ta = lane_addr + t * kAccCols;
            // the stage is given back as soon as its last columns are in registers
            tmem_ld32(ta, v0);
            tmem_ld32(ta + 32, v1);
            tmem_wait2(v0, v1);
            fold32(acc, v0, s0);
            tmem_ld32(ta + 64, v0);
            fold32(acc + 32, v1, s0);
            tmem_ld32(ta + 96, v1);
            tmem_wait2(v0, v1);
            k5::tc_fence_before();
            __syncwarp();
            if (lane == 0) mbar_arrive(&acc_empty[t]);
            fold32(acc + 64, v0, s1);
            fold32(acc + 96, v1, s1);
            continue;
          }
        }
        k5::tc_fence_before();
        __syncwarp();
        if (lane == 0) mbar_arrive(&acc_empty[t]);
      }
      if (dead) {
#pragma unroll
        for (int c = 0; c < 128; ++c) acc[c] = 0.0f;
      }
      const Piece done = pc;
      const Unit du = u;
      const size_t row = static_cast<size_t>(du.row0) + r;
      more = get_piece(sched, p.kb, i + 1, pc);
      if (more) begin();  // the next unit's loads pass while this one is written
      if (done.count > 1) {
        // partial tile to the workspace; the last piece to arrive adds all of them in piece order
        const size_t slot_floats = static_cast<size_t>(kTileN) * p.rcap;
        if (live) {
          float* d = p.part + done.slot * slot_floats + static_cast<size_t>(half * 128) * p.rcap + r;
#pragma unroll
          for (int c = 0; c < 128; ++c) __stcg(d + static_cast<size_t>(c) * p.rcap, acc[c]);
        }
        if (!last_piece(p.counter + (done.unit - sched.waves * static_cast<int>(gridDim.x)), done.count, s_last))
          continue;
        if (live) {
          auto piece_at = [&](int q) {
            return p.part + q * slot_floats + static_cast<size_t>(half * 128) * p.rcap + r;
          };
          if (done.count == 2) {  // the other piece onto this one, in registers: the order is no matter
            const float* d = piece_at(2 * done.first + 1 - static_cast<int>(blockIdx.x));
#pragma unroll
            for (int c = 0; c < 128; ++c) acc[c] += __ldcg(d + static_cast<size_t>(c) * p.rcap);
          } else {
#pragma unroll
            for (int c0 = 0; c0 < 128; c0 += 32) {
              float v[32];
#pragma unroll
              for (int c = 0; c < 32; ++c) v[c] = 0.0f;
              for (int q = done.first; q < done.first + done.count; ++q) {
                const float* d = piece_at(q) + static_cast<size_t>(c0) * p.rcap;
#pragma unroll
                for (int c = 0; c < 32; ++c) v[c] += __ldcg(d + static_cast<size_t>(c) * p.rcap);
              }
#pragma unroll
              for (int c = 0; c < 32; ++c) acc[c0 + c] = v[c];
            }
          }
        }
      }
      if constexpr (GATED) {
        float m = 0.0f;
#pragma unroll
        for (int c = 0; c < 64; ++c) {
          acc[c] = gated(acc[c], acc[64 + c]);
          m = fmaxf(m, finite_abs(acc[c]));
        }
        named_sync(kEpiBarrier, kEpiThreads);  // the previous tile's maxima are read
        s_amax[half * kTileM + r] = m;
        named_sync(kEpiBarrier, kEpiThreads);
        m = fmaxf(s_amax[r], s_amax[kTileM + r]);
        const int ex = scale_exponent(m);
        const float inv = pow2(-ex);
        if (live) {
          if (half == 0) p.hs[row * (p.I / 128) + du.n] = pow2(ex);
          uint4* d = reinterpret_cast<uint4*>(p.hq + row * p.I + du.n * 128 + half * 64);
#pragma unroll
          for (int c = 0; c < 64; c += 16) {
            uint32_t w[4];
#pragma unroll
            for (int q = 0; q < 4; ++q)
              w[q] = e4m3_pair(acc[c + 4 * q] * inv, acc[c + 4 * q + 1] * inv) |
                     (e4m3_pair(acc[c + 4 * q + 2] * inv, acc[c + 4 * q + 3] * inv) << 16);
            d[c / 16] = make_uint4(w[0], w[1], w[2], w[3]);
          }
        }
      } else if (mine) {
        store_rows<TO>(smem + kOffStage + ew * 32 * kStageRow, p.y, static_cast<size_t>(du.row0) + quarter * 32,
                       p.ld_y, min(32, du.rows - quarter * 32), du.n * kTileN + half * 128, p.N, p.vec, acc, lane);
      }
    }
  }

  k5::tc_fence_before();
  __syncthreads();
  if (warp == 2) {
    k5::tc_fence_after();
    asm volatile("tcgen05.dealloc.cta_group::1.sync.aligned.b32 %0, %1;" ::"r"(tmem_base),
                 "r"(kTmemCols)
                 : "memory");
  }
}

}  // namespace k7
}  // namespace pw
