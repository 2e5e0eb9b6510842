// K8: the scaled product of pw_scaled.cuh for few rows per expert (a decode step).  The operands
// change sides: 128 weight rows are the tensor cores' M and up to 64 tokens their N, so a unit (256
// weight rows x 64 tokens; gated: 128 gate rows and the 128 matching up rows) wastes nothing on rows
// that do not exist, a lane of tensor memory is a feature, and partials, joins and outputs are
// contiguous across lanes.  What bounds it is the weights' bytes, each read once: 5 stages of 32 KB
// keep 160 KB an SM in flight.  64 experts of 8 rows, 5120 x 3584: 184 us, 6.4 TB/s; 4 rows x 28672 x
// 4096 (117 MB, 112 units): 24 us, of which about 5 until the first tile is there.
// From 64 rows an expert on the large-rows kernel is as fast or faster (64 x 28672 x 4096: 36 us here,
// 31 there; 64 experts of 32 rows: 194 here, 206 there).
//
// A block's scale of a token is a column's here: the epilogue multiplies it with the weights' scale
// once per (token, block) and reads it back from shared memory as it folds.
//
// Warps: 0 TMA producer, 1 and 3 MMA issuers (an accumulator of up to 64 columns each, four blocks in
// flight in tensor memory; issuing is what a block costs most when half the SMs have a unit: 76 units
// of 4 rows, K 4096, 20.5 us with one warp for both, 19.4 with two), 2 tensor memory, 4-11 epilogue:
// warp 4 + w has lanes (features) of quarter w % 4 of accumulator w / 4.
#pragma once
#include "pw_scaled.cuh"

namespace pw {
namespace k8 {

using k7::Params;
using k7::Piece;
using k7::Sched;
using k7::Unit;
using k7::kBlk;

constexpr int kTokens = 64;  // tokens of a unit
constexpr int kRows = 256;   // weight rows of a unit: two accumulators of 128
constexpr int kStages = 5;
constexpr int kWBytes = kRows * kBlk, kXBytes = kTokens * kBlk;
constexpr int kStageBytes = kWBytes + kXBytes;
constexpr int kThreads = 384, kEpiThreads = 256;
constexpr int kMinPiece = 8;                        // K blocks of the shortest piece (see k7::kMinPiece)
constexpr int kAccStages = 4;                       // K blocks in tensor memory
constexpr int kTmemCols = kAccStages * 2 * kTokens;  // 512
constexpr int kBox = k7::kSmallRows;                // tokens of an activation box, and of an MMA's step of N

constexpr int kOffBar = kStages * kStageBytes;
constexpr int kNumBars = 2 * kStages + 2 * kAccStages + 1;
constexpr int kOffMisc = kOffBar + ((kNumBars * 8 + 15) / 16) * 16;
constexpr int kOffScale = kOffMisc + 32;                     // [8 warps][2][64] scales of a block
constexpr int kOffEx = kOffScale + 8 * 2 * kTokens * 4;      // [16][128] exchange of 16 tokens
constexpr int kOffTiles = kOffEx + kBox * 128 * 4;
constexpr int smem_bytes(int E) { return kOffTiles + 2 * (E + 1) * 4; }
static_assert(smem_bytes(PW_MAX_EXPERTS) <= 227 * 1024, "shared memory budget");
static_assert(kTmemCols == 512 && kStageBytes % 1024 == 0, "layout");

// kind::f8f6f4, e4m3 x e4m3 -> fp32, M = 128, N = n (a multiple of 16).
__device__ __forceinline__ uint32_t instr(int n) {
  return (1u << 4) | (static_cast<uint32_t>(n >> 3) << 17) | (static_cast<uint32_t>(128 >> 4) << 24);
}

__device__ __forceinline__ void tmem_ld16(uint32_t addr, uint32_t (&r)[16]) {
  asm volatile(
      "tcgen05.ld.sync.aligned.32x32b.x16.b32 "
      "{%0, %1, %2, %3, %4, %5, %6, %7, %8, %9, %10, %11, %12, %13, %14, %15}, [%16];"
      : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3]), "=r"(r[4]), "=r"(r[5]), "=r"(r[6]), "=r"(r[7]),
        "=r"(r[8]), "=r"(r[9]), "=r"(r[10]), "=r"(r[11]), "=r"(r[12]), "=r"(r[13]), "=r"(r[14]),
        "=r"(r[15])
      : "r"(addr));
}
__device__ __forceinline__ void tmem_wait16(uint32_t (&r)[16]) {
  asm volatile("tcgen05.wait::ld.sync.aligned;"
               : "+r"(r[0]), "+r"(r[1]), "+r"(r[2]), "+r"(r[3]), "+r"(r[4]), "+r"(r[5]), "+r"(r[6]),
                 "+r"(r[7]), "+r"(r[8]), "+r"(r[9]), "+r"(r[10]), "+r"(r[11]), "+r"(r[12]),
                 "+r"(r[13]), "+r"(r[14]), "+r"(r[15])
               :
               : "memory");
}

// The i-th piece of a CTA: its piece of the remainder first (within one unit: pieces >= rem), then its
// units of the whole waves, so that a join is not what the launch ends with (64 tokens through 64
// experts 294.6 us, last 300.4).  One workspace slot a CTA.
__device__ __forceinline__ bool piece_first(const Sched& s, int kb, int i, Piece& p) {
  const int cta = blockIdx.x;
  const bool extra = cta < s.pieces;  // pieces = 0 without a remainder
  p.first = 0;
  p.count = 1;
  if (extra && i == 0) {
    const int a = k7::piece_begin(s, cta), j = a / kb;
    p.unit = s.waves * static_cast<int>(gridDim.x) + j;
    p.k0 = a - j * kb;
    p.k1 = min(kb, k7::piece_begin(s, cta + 1) - j * kb);
    p.first = k7::piece_of(s, j * kb);
    p.count = k7::piece_of(s, (j + 1) * kb - 1) - p.first + 1;
    return true;
  }
  const int w = extra ? i - 1 : i;
  p.unit = cta + w * static_cast<int>(gridDim.x);
  p.k0 = 0;
  p.k1 = kb;
  return w < s.waves;
}

template <bool GATED, int TO>
__global__ void __launch_bounds__(kThreads, 1) few_kernel(const __grid_constant__ Params p) {
  uint8_t* const smem = k4::g_smem;
  uint64_t* full = reinterpret_cast<uint64_t*>(smem + kOffBar);
  uint64_t* empty = full + kStages;
  uint64_t* acc_full = empty + kStages;
  uint64_t* acc_empty = acc_full + kAccStages;
  uint64_t* mma_done = acc_empty + kAccStages;
  uint32_t* tmem_slot = reinterpret_cast<uint32_t*>(smem + kOffMisc);
  volatile int* abort_flag = reinterpret_cast<volatile int*>(tmem_slot + 1);
  int* s_last = reinterpret_cast<int*>(tmem_slot + 2);
  float* s_ex = reinterpret_cast<float*>(smem + kOffEx);
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
      mbar_init(&empty[s], 2);
    }
    for (int b = 0; b < kAccStages; ++b) {
      mbar_init(&acc_full[b], 2);
      mbar_init(&acc_empty[b], kEpiThreads / 32);
    }
    mbar_init(mma_done, 2);
    *abort_flag = 0;
    mbar_fence_init();
    k7::prefetch_map(&p.xsmall);
    k7::prefetch_map(&p.wmap);
  }
  if (warp == 2) {
    asm volatile("tcgen05.alloc.cta_group::1.sync.aligned.shared::cta.b32 [%0], %1;" ::"r"(
                     smem_u32(tmem_slot)),
                 "r"(kTmemCols)
                 : "memory");
    asm volatile("tcgen05.relinquish_alloc_permit.cta_group::1.sync.aligned;" ::: "memory");
  }
  k7::row_tiles<kTokens>(p, s_tiles, s_first);
  k5::tc_fence_before();
  __syncthreads();
  k5::tc_fence_after();
  const uint32_t tmem_base = *tmem_slot;
  const Sched sched = k7::make_sched(s_tiles[E] * p.nt, p.kb, gridDim.x, kMinPiece);
  const uint32_t smem_base = smem_u32(smem);

  if (warp < 4 && warp != 2) {
    const bool leader = k7::elect_one();  // one lane issues; control flow and operands stay uniform
    uint32_t g = 0;
    Piece pc;
    bool ok = true;
    if (warp == 0) {
      // ---------------- producer ----------------
      // the first kStages weight tiles are on their way before the launch in front has ended; the
      // tokens (its output) follow
      auto tokens_of = [&](const Unit& u, int b, uint32_t stage) {
        const uint32_t x = smem_base + stage * kStageBytes + kWBytes;
        for (int q = 0; q * kBox < u.rows; ++q)
          k7::tma_2d(x + q * kBox * kBlk, &p.xsmall, b * kBlk, u.row0 + q * kBox, &full[stage]);
      };
      auto follow = [&]() {  // the tokens of the blocks before g
        griddep_wait();
        if (leader) {
          uint32_t h = 0;
          Piece q;
          for (int i = 0; h < g && piece_first(sched, p.kb, i, q); ++i) {
            const Unit u = k7::find_unit<kTokens>(p, s_tiles, s_first, q.unit);
            for (int b = q.k0; b < q.k1 && h < g; ++b, ++h) tokens_of(u, b, h);
          }
          griddep_launch();
        }
        __syncwarp();
      };
      bool waited = false;
      for (int i = 0; ok && piece_first(sched, p.kb, i, pc); ++i) {
        const Unit u = k7::find_unit<kTokens>(p, s_tiles, s_first, pc.unit);
        const int boxes = (u.rows + kBox - 1) / kBox;
        const uint32_t bytes = kWBytes + boxes * kBox * kBlk;
        for (int b = pc.k0; b < pc.k1; ++b, ++g) {
          if (g == kStages && !waited) {
            follow();
            waited = true;
          }
          const int s = g % kStages;
          if (!(ok = k7::warp_wait(&empty[s], ((g / kStages) & 1) ^ 1, abort_flag))) break;
          if (leader) {
            mbar_arrive_expect_tx(&full[s], bytes);
            const uint32_t w = smem_base + s * kStageBytes;
            if (GATED) {
              k7::tma_3d(w, &p.wmap, b * kBlk, u.n * 128, u.e, &full[s]);
              k7::tma_3d(w + kWBytes / 2, &p.wmap, b * kBlk, p.I + u.n * 128, u.e, &full[s]);
            } else {
              k7::tma_3d(w, &p.wmap, b * kBlk, u.n * kRows, u.e, &full[s]);
            }
            if (waited) tokens_of(u, b, s);
          }
          __syncwarp();
        }
      }
      if (!waited) follow();
      // every issued copy has landed before the block exits
      if (leader)
        for (uint32_t x = (g > kStages ? g - kStages : 0); x < g; ++x)
          mbar_wait(&full[x % kStages], (x / kStages) & 1);
    } else {
      // ---------------- MMA issuers: warp 1 accumulator 0, warp 3 accumulator 1 ----------------
      const int h = warp >> 1;
      ok = k7::not_held(mma_done, abort_flag);
      griddep_wait();  // nothing to multiply before; the bounded waits below start after it
      const uint64_t xd0 = k7::sw128_desc(smem_base + kWBytes);
      for (int i = 0; ok && piece_first(sched, p.kb, i, pc); ++i) {
        const Unit u = k7::find_unit<kTokens>(p, s_tiles, s_first, pc.unit);
        const uint32_t id = instr((u.rows + kBox - 1) / kBox * kBox);
        for (int b = pc.k0; b < pc.k1; ++b, ++g) {
          const int s = g % kStages, t = g % kAccStages;
          if (!(ok = k7::warp_wait2(&full[s], (g / kStages) & 1, &acc_empty[t], ((g / kAccStages) & 1) ^ 1,
                                    abort_flag)))
            break;
          k5::tc_fence_after();
          const uint64_t xd = xd0 + static_cast<uint64_t>(s) * (kStageBytes / 16);
          const uint64_t wd = xd - (2 - h) * (kWBytes / 2 / 16);
          const uint32_t d = tmem_base + (2 * t + h) * kTokens;
          if (leader) {
#pragma unroll
            for (int j = 0; j < 4; ++j)  // 32 bytes of K each
              k7::mma_f8(d, wd + 2 * j, xd + 2 * j, id, j > 0);
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
  } else if (warp >= 4) {
    // ---------------- epilogue ----------------
    const int ew = warp - 4, quarter = ew & 3, half = ew >> 2;
    const int f = quarter * 32 + lane;  // feature of the accumulator
    float* s_scale = reinterpret_cast<float*>(smem + kOffScale) + ew * 2 * kTokens;
    const uint32_t lane_addr = tmem_base + (static_cast<uint32_t>(quarter * 32) << 16) + half * kTokens;
    uint32_t g = 0;
    Piece pc;
    bool dead = false;  // a wait gave up: keep every barrier, write zeros
    griddep_wait();
    for (int i = 0; piece_first(sched, p.kb, i, pc); ++i) {
      const Unit u = k7::find_unit<kTokens>(p, s_tiles, s_first, pc.unit);
      // lane l holds the scales of tokens l and l + 32
      const float* sx0 = p.sx + (static_cast<size_t>(u.row0) + min(lane, u.rows - 1)) * p.kb;
      const float* sx1 = p.sx + (static_cast<size_t>(u.row0) + min(lane + 32, u.rows - 1)) * p.kb;
      const int nb = min(GATED ? (half ? p.I / 128 : 0) + u.n : 2 * u.n + half, p.nb - 1);
      const float* sw = p.sw + (static_cast<size_t>(u.e) * p.nb + nb) * p.kb;
      float acc[kTokens];
#pragma unroll
      for (int c = 0; c < kTokens; ++c) acc[c] = 0.0f;
      // the scales of a block are in shared memory before its products are waited for: stored while the
      // block in front is read, loaded one block earlier
      float x0 = __ldg(sx0 + pc.k0), x1 = __ldg(sx1 + pc.k0), w = __ldg(sw + pc.k0);
      auto next_scales = [&](int b) {  // of block b, and the loads of block b + 1
        float* s = s_scale + (b & 1) * kTokens;
        s[lane] = x0 * w;
        s[lane + 32] = x1 * w;
        if (b + 1 < pc.k1) {
          x0 = __ldg(sx0 + b + 1);
          x1 = __ldg(sx1 + b + 1);
          w = __ldg(sw + b + 1);
        }
      };
      __syncwarp();
      next_scales(pc.k0);
      __syncwarp();
      for (int b = pc.k0; b < pc.k1; ++b, ++g) {
        const int t = g % kAccStages;
        if (!k7::warp_wait(&acc_full[t], (g / kAccStages) & 1, abort_flag)) {
          dead = true;
        } else {
          k5::tc_fence_after();
          const float* s = s_scale + (b & 1) * kTokens;
#pragma unroll
          for (int c0 = 0; c0 < kTokens; c0 += 16)
            if (c0 < u.rows) {
              uint32_t v[16];
              tmem_ld16(lane_addr + t * 2 * kTokens + c0, v);
              if (c0 == 0 && b + 1 < pc.k1) next_scales(b + 1);
              tmem_wait16(v);
#pragma unroll
              for (int c = 0; c < 16; c += 4) {
                const float4 q = *reinterpret_cast<const float4*>(s + c0 + c);
                acc[c0 + c] = fmaf(__uint_as_float(v[c]), q.x, acc[c0 + c]);
                acc[c0 + c + 1] = fmaf(__uint_as_float(v[c + 1]), q.y, acc[c0 + c + 1]);
                acc[c0 + c + 2] = fmaf(__uint_as_float(v[c + 2]), q.z, acc[c0 + c + 2]);
                acc[c0 + c + 3] = fmaf(__uint_as_float(v[c + 3]), q.w, acc[c0 + c + 3]);
              }
            }
        }
        k5::tc_fence_before();
        __syncwarp();
        if (lane == 0) mbar_arrive(&acc_empty[t]);
      }
      if (dead) {
#pragma unroll
        for (int c = 0; c < kTokens; ++c) acc[c] = 0.0f;
      }
      if (pc.count > 1) {
        // partials to the workspace, [token][256]; the last piece to arrive adds all in piece order
        const size_t slot_floats = static_cast<size_t>(kRows) * p.rcap;
        float* d = p.part + blockIdx.x * slot_floats + half * 128 + f;
#pragma unroll
        for (int c = 0; c < kTokens; ++c)
          if (c < u.rows) __stcg(d + c * kRows, acc[c]);
        const int j = pc.unit - sched.waves * static_cast<int>(gridDim.x);
        if (!k7::last_piece(p.counter + j, pc.count, s_last)) continue;
#pragma unroll
        for (int c0 = 0; c0 < kTokens; c0 += 16)
          if (c0 < u.rows) {
#pragma unroll
            for (int c = 0; c < 16; ++c) acc[c0 + c] = 0.0f;
            constexpr int Q = 3;  // pieces loaded at once (a unit of the usual cut has two or three)
            for (int q0 = pc.first; q0 < pc.first + pc.count; q0 += Q) {
              float v[Q][16];
#pragma unroll
              for (int q = 0; q < Q; ++q) {
                const bool in = q0 + q < pc.first + pc.count;
                const float* src = p.part + (q0 + q) * slot_floats + half * 128 + f;
#pragma unroll
                for (int c = 0; c < 16; ++c)
                  v[q][c] = in && c0 + c < u.rows ? __ldcg(src + (c0 + c) * kRows) : 0.0f;
              }
#pragma unroll
              for (int q = 0; q < Q; ++q)
#pragma unroll
                for (int c = 0; c < 16; ++c) acc[c0 + c] += v[q][c];
            }
          }
      }
      if constexpr (GATED) {
        // sixteen tokens at a time: up half -> shared memory -> SiLU(gate) * up of the gate half ->
        // shared memory -> every warp quantises two tokens, four features a lane
#pragma unroll
        for (int c0 = 0; c0 < kTokens; c0 += 16) {
          if (c0 >= u.rows) break;
          named_sync(k7::kEpiBarrier, kEpiThreads);  // the buffer is read
          if (half == 1) {
#pragma unroll
            for (int c = 0; c < 16; ++c) s_ex[c * 128 + f] = acc[c0 + c];
          }
          named_sync(k7::kEpiBarrier, kEpiThreads);
          if (half == 0) {
#pragma unroll
            for (int c = 0; c < 16; ++c) s_ex[c * 128 + f] = k7::gated(acc[c0 + c], s_ex[c * 128 + f]);
          }
          named_sync(k7::kEpiBarrier, kEpiThreads);
#pragma unroll
          for (int q = 0; q < 2; ++q) {
            const int c = 2 * ew + q;
            const float4 v = *reinterpret_cast<const float4*>(s_ex + c * 128 + lane * 4);
            float m = fmaxf(fmaxf(finite_abs(v.x), finite_abs(v.y)), fmaxf(finite_abs(v.z), finite_abs(v.w)));
#pragma unroll
            for (int o = 16; o > 0; o >>= 1) m = fmaxf(m, __shfl_xor_sync(0xffffffffu, m, o));
            const int ex = scale_exponent(m);
            const float inv = pow2(-ex);
            if (c0 + c < u.rows) {
              const size_t row = static_cast<size_t>(u.row0) + c0 + c;
              if (lane == 0) p.hs[row * (p.I / 128) + u.n] = pow2(ex);
              *reinterpret_cast<uint32_t*>(p.hq + row * p.I + u.n * 128 + lane * 4) =
                  e4m3_pair(v.x * inv, v.y * inv) | (e4m3_pair(v.z * inv, v.w * inv) << 16);
            }
          }
        }
      } else {
        const int n = u.n * kRows + half * 128 + f;
        constexpr int S = ElemSize<TO>::value;
        if (n < p.N) {
#pragma unroll
          for (int c = 0; c < kTokens; ++c)
            if (c < u.rows) {
              const float v[1] = {acc[c]};
              store_elems<TO, 1>(elem_at(p.y, (static_cast<size_t>(u.row0) + c) * p.ld_y + n, S), v);
            }
        }
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

}  // namespace k8
}  // namespace pw
