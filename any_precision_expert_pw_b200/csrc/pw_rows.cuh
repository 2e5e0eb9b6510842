// K6: token rows sorted by expert and back (the mixture of LYNX, 1: each token's k experts), for
// batches of up to 2^24 slots, with the gradients of both movements.
//
//   sort      row order = (expert, token, slot): pos[t][s] = row of a slot, src[row] = slot
//   dispatch  xs[pos[t][s]] = x[t]                      gradient: dx[t] = sum_s dxs[pos[t][s]]
//   combine   y[t] = sum_s g[t][s] o[pos[t][s]]         gradient: do[pos] = g dy[t],
//                                                       dg[t][s] = <dy[t], o[pos[t][s]]>
//
// All but the sort are bound by the rows' bytes: every kernel walks tokens, so a token's own row is
// read (or written) once and only the k sorted rows move besides.  No atomics: every sum has one
// owner and runs in slot order, so results repeat bit for bit.
#pragma once
#include <cuda_bf16.h>

#include "pw_common.cuh"

namespace pw {

// ---- element types (PW_TYPE_*) ----
template <int TY>
struct ElemSize {
  static constexpr int value = TY == PW_TYPE_F32 ? 4 : 2;
};

// V consecutive elements at p as they lie in memory (one load; half the registers of fp32 for 16-bit
// types: what bounds the row kernels is loads in flight), and their values.
template <int TY, int V>
struct Raw {
  uint32_t w[V * ElemSize<TY>::value / 4 > 0 ? V * ElemSize<TY>::value / 4 : 1];
};
template <int TY, int V>
__device__ __forceinline__ void load_raw(const void* p, Raw<TY, V>& r) {
  constexpr int B = V * ElemSize<TY>::value;
  static_assert(B == 2 || B == 4 || B == 16, "one load");
  if constexpr (B == 16) {
    const uint4 a = __ldg(static_cast<const uint4*>(p));
    r.w[0] = a.x, r.w[1] = a.y, r.w[2] = a.z, r.w[3] = a.w;
  } else if constexpr (B == 4) {
    r.w[0] = __ldg(static_cast<const unsigned int*>(p));
  } else {
    r.w[0] = __ldg(static_cast<const unsigned short*>(p));
  }
}
template <int TY, int V>
__device__ __forceinline__ float raw_value(const Raw<TY, V>& r, int i) {
  if constexpr (TY == PW_TYPE_F32) {
    return __uint_as_float(r.w[i]);
  } else if constexpr (TY == PW_TYPE_BF16) {
    return __uint_as_float(i & 1 ? r.w[i / 2] & 0xffff0000u : r.w[i / 2] << 16);
  } else {
    return f16_to_f32(static_cast<uint16_t>(r.w[i / 2] >> (16 * (i & 1))));
  }
}

template <int TY>
__device__ __forceinline__ uint16_t to_bits16(float f) {
  if constexpr (TY == PW_TYPE_BF16) return __bfloat16_as_ushort(__float2bfloat16_rn(f));
  return __half_as_ushort(__float2half_rn(f));
}

// V consecutive elements, rounded once to the type (to nearest even).  p is aligned to V elements
// (at most 16 bytes).
template <int TY, int V>
__device__ __forceinline__ void store_elems(void* p, const float (&v)[V]) {
  if constexpr (TY == PW_TYPE_F32) {
    if constexpr (V == 1) {
      *static_cast<float*>(p) = v[0];
    } else {
#pragma unroll
      for (int i = 0; i < V / 4; ++i)
        static_cast<float4*>(p)[i] = make_float4(v[4 * i], v[4 * i + 1], v[4 * i + 2], v[4 * i + 3]);
    }
  } else if constexpr (V == 1) {
    *static_cast<uint16_t*>(p) = to_bits16<TY>(v[0]);
  } else {
    uint32_t w[V / 2];
#pragma unroll
    for (int i = 0; i < V / 2; ++i)
      w[i] = static_cast<uint32_t>(to_bits16<TY>(v[2 * i])) |
             (static_cast<uint32_t>(to_bits16<TY>(v[2 * i + 1])) << 16);
    if constexpr (V == 8)
      *static_cast<uint4*>(p) = make_uint4(w[0], w[1], w[2], w[3]);
    else
      *static_cast<uint2*>(p) = make_uint2(w[0], w[1]);
  }
}

__device__ __forceinline__ const void* elem_at(const void* base, size_t i, int size) {
  return static_cast<const uint8_t*>(base) + i * size;
}
__device__ __forceinline__ void* elem_at(void* base, size_t i, int size) {
  return static_cast<uint8_t*>(base) + i * size;
}

// The row behind a slot, or -1: an empty slot, or a value that no sort of n slots gives (recorded).
__device__ __forceinline__ int checked_row(const int32_t* pos, long long slot, int n) {
  const int r = pos[slot];
  if (r >= n || r < -1) {
    set_status(PW_ERR_BOUNDS);
    return -1;
  }
  return r;
}

// ---- sort ----
// A CTA owns a contiguous run of slots, each of its 32 warps a contiguous part of it, so "earlier in
// the run" is "earlier warp, then earlier step, then lower lane" and a stable order needs no
// sorting network: count per (warp, expert), prefix over warps, CTAs and experts, then each warp
// walks its part again and takes places in order.  Equal ids inside a step of 32 are ranked with one
// warp match.  With more than one CTA a first launch leaves each CTA's counts in the workspace and
// every CTA sums the ones before its own (one CTA per SM, 257 for the largest batch, so at most 257 x
// E values from L2).  A warp's counts, and its first places within the CTA's run, are 16 bits: a run
// has at most kSortMaxRun slots, whatever its ids.  Latency bound: two walks over the ids and three
// block-wide steps (131072 slots of 64 experts: 14 us in two launches; 160 slots of 512 experts: 5 us).
constexpr int kSortThreads = 1024;
constexpr int kSortWarps = kSortThreads / 32;
constexpr int kSortMaxRun = 65535;  // slots of a CTA's run
constexpr int kSortAhead = 4;       // steps whose ids are loaded before the first is used

// Warps that share a run of n slots: whole steps of 32 each, no more warps than steps (fewer rows of
// the count table to clear and to sum).
__device__ __forceinline__ int sort_warps(int n) { return min(kSortWarps, max(1, (n + 31) / 32)); }

__device__ __forceinline__ int slot_expert(const int32_t* idx, int i, int end, int E) {
  if (i >= end) return -1;
  const int e = __ldg(idx + i);
  return e;
}

// Counts of this warp's part into cnt[E] (its own row of the table).
__device__ __forceinline__ void sort_count(const int32_t* idx, int a, int b, int E, uint16_t* cnt,
                                           int lane) {
  for (int i0 = a; i0 < b; i0 += 32 * kSortAhead) {
    int e[kSortAhead];
#pragma unroll
    for (int u = 0; u < kSortAhead; ++u) e[u] = slot_expert(idx, i0 + 32 * u + lane, b, E);
#pragma unroll
    for (int u = 0; u < kSortAhead; ++u) {
      if (i0 + 32 * u >= b) break;
      if (e[u] < -1 || e[u] >= E) {
        set_status(PW_ERR_BAD_EXPERT);
        e[u] = -1;
      }
      const uint32_t same = __match_any_sync(0xffffffffu, e[u]);
      if (e[u] >= 0 && (same & ((1u << lane) - 1u)) == 0)
        cnt[e[u]] = static_cast<uint16_t>(cnt[e[u]] + __popc(same));
      __syncwarp();
    }
  }
}

__device__ __forceinline__ void run_of(int n, int parts, int part, int& a, int& b) {
  a = static_cast<int>(static_cast<long long>(n) * part / parts);
  b = static_cast<int>(static_cast<long long>(n) * (part + 1) / parts);
}

// First launch of a sort over several CTAs: part[cta][e] = assignments of the CTA's run.
__global__ void __launch_bounds__(kSortThreads) sort_count_kernel(const int32_t* idx, int n, int E,
                                                                  int32_t* part) {
  extern __shared__ __align__(16) uint8_t sort_smem[];
  uint16_t* cnt = reinterpret_cast<uint16_t*>(sort_smem);
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  int a, b, wa, wb;
  run_of(n, gridDim.x, blockIdx.x, a, b);
  const int warps = sort_warps(b - a);
  for (int i = threadIdx.x; i < warps * E; i += kSortThreads) cnt[i] = 0;
  __syncthreads();
  griddep_wait();
  griddep_launch();
  if (warp < warps) {
    run_of(b - a, warps, warp, wa, wb);
    sort_count(idx, a + wa, a + wb, E, cnt + warp * E, lane);
  }
  __syncthreads();
  for (int e = threadIdx.x; e < E; e += kSortThreads) {
    int s = 0;
    for (int w = 0; w < warps; ++w) s += cnt[w * E + e];
    part[static_cast<size_t>(blockIdx.x) * E + e] = s;
  }
}

// Inclusive sum over the block of one value per thread.
__device__ __forceinline__ int block_inclusive(int v, int* warp_sum) {
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
#pragma unroll
  for (int d = 1; d < 32; d <<= 1) {
    const int o = __shfl_up_sync(0xffffffffu, v, d);
    if (lane >= d) v += o;
  }
  if (lane == 31) warp_sum[warp] = v;
  __syncthreads();
  if (warp == 0) {
    int s = warp_sum[lane];
#pragma unroll
    for (int d = 1; d < 32; d <<= 1) {
      const int o = __shfl_up_sync(0xffffffffu, s, d);
      if (lane >= d) s += o;
    }
    warp_sum[lane] = s;
  }
  __syncthreads();
  return v + (warp ? warp_sum[warp - 1] : 0);
}

// part: counts of every CTA's run (NULL with one CTA).  src may be NULL.  zero: n_zero words set to zero.
__global__ void __launch_bounds__(kSortThreads) sort_place_kernel(const int32_t* idx, int n, int E,
                                                                  const int32_t* part, int32_t* pos,
                                                                  int32_t* src, int32_t* offsets,
                                                                  int32_t* zero, int n_zero) {
  extern __shared__ __align__(16) uint8_t sort_smem[];
  __shared__ int warp_sum[kSortWarps];
  __shared__ int s_before[kSortThreads], s_all[kSortThreads];
  int* base = reinterpret_cast<int*>(sort_smem);                    // [E] first row of the CTA
  uint16_t* cnt = reinterpret_cast<uint16_t*>(base + E);            // [warps][E]
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  int a, b, wa = 0, wb = 0;
  run_of(n, gridDim.x, blockIdx.x, a, b);
  const int warps = sort_warps(b - a);
  for (int i = threadIdx.x; i < warps * E; i += kSortThreads) cnt[i] = 0;
  __syncthreads();
  griddep_wait();
  griddep_launch();
  if (blockIdx.x == 0)
    for (int i = threadIdx.x; i < n_zero; i += kSortThreads) zero[i] = 0;
  if (part) {
    // counts of the CTAs before this one, and of all: `groups` threads an expert, each over its share
    // of the CTAs
    const int groups = kSortThreads / E, g = threadIdx.x / E, e = threadIdx.x - g * E;
    int before = 0, all = 0;
    if (g < groups) {
      const int ctas = gridDim.x, me = blockIdx.x;
      int c0, c1;
      run_of(ctas, groups, g, c0, c1);
#pragma unroll 8
      for (int c = c0; c < c1; ++c) {
        const int v = __ldcg(part + static_cast<size_t>(c) * E + e);
        before += c < me ? v : 0;
        all += v;
      }
    }
    s_before[threadIdx.x] = before;
    s_all[threadIdx.x] = all;
  }
  if (warp < warps) {
    run_of(b - a, warps, warp, wa, wb);
    wa += a, wb += a;
    sort_count(idx, wa, wb, E, cnt + warp * E, lane);
  }
  __syncthreads();
  // thread e: prefix over the warps; E <= 1024 = the block
  const int e = threadIdx.x;
  int run = 0;
  if (e < E)
    for (int w = 0; w < warps; ++w) {
      const int c = cnt[w * E + e];
      cnt[w * E + e] = static_cast<uint16_t>(run);
      run += c;
    }
  int before = 0, all = e < E ? run : 0;
  if (part && e < E) {
    all = 0;
    for (int g = 0; g < kSortThreads / E; ++g) {
      before += s_before[g * E + e];
      all += s_all[g * E + e];
    }
  }
  const int incl = block_inclusive(all, warp_sum);
  if (e < E) {
    base[e] = incl - all + before;
    if (blockIdx.x == 0) {
      offsets[e + 1] = incl;
      if (e == 0) offsets[0] = 0;
    }
  }
  __syncthreads();
  uint16_t* mine = cnt + warp * E;
  for (int i0 = wa; i0 < wb; i0 += 32 * kSortAhead) {
    int id[kSortAhead];
#pragma unroll
    for (int u = 0; u < kSortAhead; ++u) id[u] = slot_expert(idx, i0 + 32 * u + lane, wb, E);
#pragma unroll
    for (int u = 0; u < kSortAhead; ++u) {
      if (i0 + 32 * u >= wb) break;
      const int i = i0 + 32 * u + lane;
      const bool live = id[u] >= 0 && id[u] < E;
      const int x = live ? id[u] : -1;
      const uint32_t same = __match_any_sync(0xffffffffu, x);
      const uint32_t lower = same & ((1u << lane) - 1u);
      const int first = live ? mine[x] : 0;
      __syncwarp();
      if (live && lower == 0) mine[x] = static_cast<uint16_t>(first + __popc(same));
      __syncwarp();
      if (i < wb) {
        const int row = live ? base[x] + first + __popc(lower) : -1;
        pos[i] = row;
        if (live && src) src[row] = i;
      }
    }
  }
}

__global__ void zero_words_kernel(int32_t* p, int n) {
  griddep_wait();
  griddep_launch();
  for (int i = threadIdx.x; i < n; i += blockDim.x) p[i] = 0;
}

// ---- dispatch ----
// One warp: token t, 32 x U units of 16 bytes or of one element (2 or 4 bytes), read once and written
// to the token's k rows.  Bound by the bytes written (16384 tokens x 8 x 3584 bf16, 1.03 GB: 162 us,
// 6.3 TB/s).
template <typename UNIT, int U>
__global__ void __launch_bounds__(256) dispatch_kernel(const UNIT* x, int T, int k, int units,
                                                       size_t ld_x, const int32_t* pos, UNIT* xs,
                                                       size_t ld_xs, int groups) {
  const int lane = threadIdx.x & 31;
  const long long w = static_cast<long long>(blockIdx.x) * 8 + (threadIdx.x >> 5);
  griddep_wait();
  griddep_launch();
  const long long t = w / groups;
  if (t >= T) return;
  const int c0 = static_cast<int>(w - t * groups) * 32 * U + lane;
  int row = -1;
  if (lane < k) row = checked_row(pos, t * k + lane, T * k);
  UNIT v[U];
#pragma unroll
  for (int u = 0; u < U; ++u)
    if (c0 + 32 * u < units) v[u] = __ldg(x + t * ld_x + c0 + 32 * u);
  for (int j = 0; j < k; ++j) {
    const int r = __shfl_sync(0xffffffffu, row, j);
    if (r < 0) continue;
    UNIT* d = xs + static_cast<size_t>(r) * ld_xs;
#pragma unroll
    for (int u = 0; u < U; ++u)
      if (c0 + 32 * u < units) d[c0 + 32 * u] = v[u];
  }
}

// ---- combine, and the gradient of dispatch (gate = NULL: weights of one) ----
// One warp: token t, 32 x U vectors of V elements; four sorted rows in flight, as they lie in memory;
// fp32 sums in slot order.  Bound by the bytes read (8192 tokens x 4 x 2048 fp32, 332 MB: 53 us; 4096 x
// 8 x 3584 bf16, 264 MB: 41 us; with the rows converted as they arrive the latter took 66, registers).
template <int TI, int TO, int V, int U>
__global__ void __launch_bounds__(256) combine_rows_kernel(const void* o, int T, int k, int H,
                                                           size_t ld_o, const int32_t* pos,
                                                           const float* gate, void* y, size_t ld_y,
                                                           int groups) {
  const int lane = threadIdx.x & 31;
  const long long w = static_cast<long long>(blockIdx.x) * 8 + (threadIdx.x >> 5);
  griddep_wait();
  griddep_launch();
  const long long t = w / groups;
  if (t >= T) return;
  const int c0 = (static_cast<int>(w - t * groups) * 32 * U + lane) * V;
  int row = -1;
  float g = 0.0f;
  if (lane < k) {
    row = checked_row(pos, t * k + lane, T * k);
    g = gate ? __ldg(gate + t * k + lane) : 1.0f;
  }
  float acc[U][V];
#pragma unroll
  for (int u = 0; u < U; ++u)
#pragma unroll
    for (int i = 0; i < V; ++i) acc[u][i] = 0.0f;
  constexpr int J = 4;
  for (int j0 = 0; j0 < k; j0 += J) {
    Raw<TI, V> v[J][U];
    int r[J];
#pragma unroll
    for (int j = 0; j < J; ++j) {
      r[j] = j0 + j < k ? __shfl_sync(0xffffffffu, row, j0 + j) : -1;
      if (r[j] < 0) continue;
#pragma unroll
      for (int u = 0; u < U; ++u)
        if (c0 + 32 * V * u < H)
          load_raw<TI, V>(elem_at(o, static_cast<size_t>(r[j]) * ld_o + c0 + 32 * V * u,
                                  ElemSize<TI>::value), v[j][u]);
    }
#pragma unroll
    for (int j = 0; j < J; ++j) {
      if (r[j] < 0) continue;
      const float gj = __shfl_sync(0xffffffffu, g, j0 + j);
#pragma unroll
      for (int u = 0; u < U; ++u)
        if (c0 + 32 * V * u < H) {
#pragma unroll
          for (int i = 0; i < V; ++i) acc[u][i] = fmaf(gj, raw_value<TI, V>(v[j][u], i), acc[u][i]);
        }
    }
  }
#pragma unroll
  for (int u = 0; u < U; ++u)
    if (c0 + 32 * V * u < H)
      store_elems<TO, V>(elem_at(y, static_cast<size_t>(t) * ld_y + c0 + 32 * V * u,
                                 ElemSize<TO>::value), acc[u]);
}

// ---- gradient of combine ----
// One CTA per token: dy[t] is read once; per column vector the k rows of o are read, their products
// with dy summed per slot (fp32, then a fixed tree over the block), and g dy written to the k rows.
// Bound by the bytes (4096 x 8 x 3584 bf16, 499 MB: 77 us, 6.5 TB/s; 512 threads 97, 128 84).
constexpr int kGradThreads = 256;

template <int TY, int V, int KM>
__global__ void __launch_bounds__(kGradThreads) combine_grad_kernel(
    const void* dy, const void* o, int T, int k, int H, size_t ld_dy, size_t ld_o,
    const int32_t* pos, const float* gate, void* d_o, size_t ld_do, float* d_gate) {
  __shared__ int s_row[KM];
  __shared__ float s_gate[KM];
  __shared__ float s_sum[kGradThreads / 32][KM];
  griddep_wait();
  griddep_launch();
  const int t = blockIdx.x, lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  constexpr int S = ElemSize<TY>::value;
  if (static_cast<int>(threadIdx.x) < KM) {
    const bool in = static_cast<int>(threadIdx.x) < k;
    const long long slot = static_cast<long long>(t) * k + threadIdx.x;
    s_row[threadIdx.x] = in ? checked_row(pos, slot, T * k) : -1;
    s_gate[threadIdx.x] = in ? gate[slot] : 0.0f;
  }
  __syncthreads();
  float acc[KM];
#pragma unroll
  for (int j = 0; j < KM; ++j) acc[j] = 0.0f;
  // columns (vectors) of a thread in flight: four where they are single elements (rows of odd sizes,
  // 4096 x 8 x 3583 bf16: one 180 us, four 158)
  constexpr int U = V == 1 ? 4 : 1;
  constexpr int J = 4;               // rows of o in flight (more cost occupancy)
  for (int c0 = threadIdx.x * V; c0 < H; c0 += kGradThreads * V * U) {
    Raw<TY, V> d[U];
#pragma unroll
    for (int u = 0; u < U; ++u) {
      const int c = c0 + u * kGradThreads * V;
      if (c < H) load_raw<TY, V>(elem_at(dy, static_cast<size_t>(t) * ld_dy + c, S), d[u]);
    }
#pragma unroll
    for (int j0 = 0; j0 < KM; j0 += J) {
      if (j0 >= k) break;
      Raw<TY, V> v[J][U];
      if (d_gate) {
#pragma unroll
        for (int j = 0; j < J; ++j)
          if (s_row[j0 + j] >= 0) {
#pragma unroll
            for (int u = 0; u < U; ++u) {
              const int c = c0 + u * kGradThreads * V;
              if (c < H)
                load_raw<TY, V>(elem_at(o, static_cast<size_t>(s_row[j0 + j]) * ld_o + c, S), v[j][u]);
            }
          }
      }
#pragma unroll
      for (int j = 0; j < J; ++j) {
        const int r = s_row[j0 + j];
        if (r < 0) continue;
#pragma unroll
        for (int u = 0; u < U; ++u) {
          const int c = c0 + u * kGradThreads * V;
          if (c >= H) break;
          if (d_gate) {
#pragma unroll
            for (int i = 0; i < V; ++i)
              acc[j0 + j] = fmaf(raw_value<TY, V>(d[u], i), raw_value<TY, V>(v[j][u], i), acc[j0 + j]);
          }
          if (d_o) {
            float w[V];
#pragma unroll
            for (int i = 0; i < V; ++i) w[i] = s_gate[j0 + j] * raw_value<TY, V>(d[u], i);
            store_elems<TY, V>(elem_at(d_o, static_cast<size_t>(r) * ld_do + c, S), w);
          }
        }
      }
    }
  }
  if (!d_gate) return;
#pragma unroll
  for (int j = 0; j < KM; ++j) {
    if (j >= k) break;
    float s = acc[j];
#pragma unroll
    for (int off = 16; off > 0; off >>= 1) s += __shfl_xor_sync(0xffffffffu, s, off);
    if (lane == 0) s_sum[warp][j] = s;
  }
  __syncthreads();
  if (static_cast<int>(threadIdx.x) < k) {
    float s = 0.0f;
#pragma unroll
    for (int w = 0; w < kGradThreads / 32; ++w) s += s_sum[w][threadIdx.x];
    d_gate[static_cast<size_t>(t) * k + threadIdx.x] = s;
  }
}

// ---- quantisation to e4m3 ----
// Power-of-two scale of a block with largest finite magnitude m: the smallest 2^e (e >= -126) with
// m <= 448 * 2^e; 1 for a block of zeros.  448 = 1.75 * 2^8, so e is the exponent of m less 8, and
// one more where the mantissa of m is above 1.75.  With such a scale x / scale is exact, so the only
// rounding is the one to e4m3.
__device__ __forceinline__ int scale_exponent(float m) {
  if (m == 0.0f) return 0;
  const uint32_t b = __float_as_uint(m);
  const int ex = static_cast<int>(b >> 23) - 127;  // subnormals: -127, below the limit anyway
  const int e = ex - 8 + ((b & 0x7fffffu) > 0x600000u ? 1 : 0);
  return e < -126 ? -126 : e;
}
__device__ __forceinline__ float pow2(int e) {  // -126 <= e <= 127
  return __uint_as_float(static_cast<uint32_t>(e + 127) << 23);
}
__device__ __forceinline__ float finite_abs(float x) {
  const float a = fabsf(x);
  return a <= 3.402823466e38f ? a : 0.0f;  // inf and NaN do not set a scale
}

// Two values, |v| <= 448, to e4m3 (nearest even); an infinity (of x, not representable) becomes NaN.
__device__ __forceinline__ uint32_t e4m3_pair(float lo, float hi) {
  const float n = __uint_as_float(0x7fffffffu);
  lo = fabsf(lo) <= 3.402823466e38f ? lo : n;
  hi = fabsf(hi) <= 3.402823466e38f ? hi : n;
  uint16_t r;
  asm("cvt.rn.satfinite.e4m3x2.f32 %0, %1, %2;" : "=h"(r) : "f"(hi), "f"(lo));
  return r;
}

// Four values to a word of e4m3, |v| <= 448 or NaN.
__device__ __forceinline__ uint32_t e4m3_word(float a, float b, float c, float d) {
  uint16_t lo, hi;
  asm("cvt.rn.satfinite.e4m3x2.f32 %0, %1, %2;" : "=h"(lo) : "f"(b), "f"(a));
  asm("cvt.rn.satfinite.e4m3x2.f32 %0, %1, %2;" : "=h"(hi) : "f"(d), "f"(c));
  return static_cast<uint32_t>(lo) | (static_cast<uint32_t>(hi) << 16);
}

// One half-warp per (row, 128-column block), 8 columns a lane, U rows in flight; a CTA's sixteen
// half-warps take up to 16 blocks of a row (blockIdx.y: the next 16), and rp rows side by side where a
// row has fewer.  pos == NULL: to row t of q; else to the rows of the token's k slots (quantise and
// dispatch in one pass).  4096 x 3584 bf16: 11.8 us (44 MB; 16.4 with fp32 values throughout), to 8 rows
// each 30 us (150 MB).
template <int TY, bool VEC, int U>
__global__ void __launch_bounds__(256) quantize_rows_kernel(const void* x, long long rows, int cols,
                                                            size_t ld_x, int k, const int32_t* pos,
                                                            uint8_t* q, size_t ld_q, float* scale,
                                                            int blocks) {
  constexpr int S = ElemSize<TY>::value;
  const int lane = threadIdx.x & 31, sub = lane & 15, hw = threadIdx.x >> 4;
  griddep_wait();
  griddep_launch();
  const int nb = min(16, blocks), rp = 16 / nb, r_in = hw / nb;
  const int b = blockIdx.y * 16 + hw - r_in * nb, c = b * 128 + sub * 8;
  const long long t0 = static_cast<long long>(blockIdx.x) * rp * U + r_in;
  const bool in = r_in < rp && b < blocks;
  // The loads of all U rows first, without a branch (a lane beyond the matrix repeats its last values
  // and counts for nothing below).  Issue slots (77 % in use) and the integer pipe (66 %) bound this kernel
  // before DRAM (24 %) does, so values stay packed as long as they can.
  constexpr int W = TY == PW_TYPE_F32 ? 4 : 8;  // elements of 16 bytes
  Raw<TY, W> raw[U][8 / W];
  const int cc = min(c, cols - 8);
#pragma unroll
  for (int u = 0; u < U; ++u) {
    const long long t = min(t0 + u * rp, rows - 1);
#pragma unroll
    for (int i = 0; i < 8 / W; ++i) {
      if (VEC) {  // cols % 8 == 0
        load_raw<TY, W>(elem_at(x, static_cast<size_t>(t) * ld_x + cc + i * W, S), raw[u][i]);
      } else {
#pragma unroll
        for (int j = 0; j < 4; ++j) raw[u][i].w[j] = 0;
#pragma unroll
        for (int j = 0; j < W; ++j)
          if (c + i * W + j < cols) {
            Raw<TY, 1> one;
            load_raw<TY, 1>(elem_at(x, static_cast<size_t>(t) * ld_x + c + i * W + j, S), one);
            if (TY == PW_TYPE_F32) raw[u][i].w[j & 3] = one.w[0];
            else raw[u][i].w[j / 2] |= one.w[0] << (16 * (j & 1));
          }
      }
    }
  }
#pragma unroll
  for (int u = 0; u < U; ++u) {
    const long long t = t0 + u * rp;
    const bool here = in && t < rows;
    // rows of the token's slots, one a lane (k <= 16)
    int row = -1;
    if (pos && here && sub < k) row = checked_row(pos, t * k + sub, static_cast<int>(rows * k));
    // largest magnitude by its bits: infinities and NaN come out on top and are looked at apart
    uint32_t top = 0;
#pragma unroll
    for (int i = 0; i < 8 / W; ++i)
#pragma unroll
      for (int j = 0; j < 4; ++j)
        top = TY == PW_TYPE_F32 ? max(top, raw[u][i].w[j] & 0x7fffffffu)
                                : __vmaxu2(top, raw[u][i].w[j] & 0x7fff7fffu);
    if (!here || c >= cols) top = 0;
    if (TY != PW_TYPE_F32) top = max(top & 0xffffu, top >> 16);
#pragma unroll
    for (int off = 8; off > 0; off >>= 1) top = max(top, __shfl_xor_sync(0xffffffffu, top, off));
    if (TY == PW_TYPE_BF16) top <<= 16;
    if (TY == PW_TYPE_F16) top = __float_as_uint(f16_to_f32(static_cast<uint16_t>(top)));
    float v[8];
#pragma unroll
    for (int i = 0; i < 8; ++i) v[i] = raw_value<TY, W>(raw[u][i / W], i % W);
    if (__any_sync(0xffffffffu, top >= 0x7f800000u)) {
      float m = 0.0f;
#pragma unroll
      for (int i = 0; i < 8; ++i) {
        m = fmaxf(m, finite_abs(v[i]));
        if (fabsf(v[i]) > 3.402823466e38f) v[i] = __uint_as_float(0x7fffffffu);  // NaN
      }
      if (!here || c >= cols) m = 0.0f;
#pragma unroll
      for (int off = 8; off > 0; off >>= 1) m = fmaxf(m, __shfl_xor_sync(0xffffffffu, m, off));
      top = __float_as_uint(m);
    }
    const int e = scale_exponent(__uint_as_float(top));
    const float inv = pow2(-e);
    const uint32_t w0 = e4m3_word(v[0] * inv, v[1] * inv, v[2] * inv, v[3] * inv);
    const uint32_t w1 = e4m3_word(v[4] * inv, v[5] * inv, v[6] * inv, v[7] * inv);
    const int slots = pos ? k : 1;
    for (int j = 0; j < slots; ++j) {
      const long long r = pos ? __shfl_sync(0xffffffffu, row, (lane & 16) + j) : (here ? t : -1);
      if (r < 0) continue;
      if (sub == 0) scale[r * blocks + b] = pow2(e);
      uint8_t* d = q + static_cast<size_t>(r) * ld_q + c;
      if (VEC ? c < cols : c + 8 <= cols) {
        *reinterpret_cast<uint2*>(d) = make_uint2(w0, w1);
      } else if (!VEC) {
#pragma unroll
        for (int i = 0; i < 8; ++i)
          if (c + i < cols) d[i] = static_cast<uint8_t>((i < 4 ? w0 >> (8 * i) : w1 >> (8 * (i - 4))) & 0xffu);
      }
    }
  }
}

// One CTA per 128 x 128 block (weights; done once): the largest magnitude, then the values.
template <int TY>
__global__ void __launch_bounds__(256) quantize_blocks_kernel(const void* x, long long rows, int cols,
                                                              size_t ld_x, uint8_t* q, size_t ld_q,
                                                              float* scale, int blocks) {
  constexpr int S = ElemSize<TY>::value;
  __shared__ float s_max[8];
  const long long rb = blockIdx.x / blocks;
  const int b = static_cast<int>(blockIdx.x - rb * blocks);
  const long long r0 = rb * 128;
  const int nr = static_cast<int>(rows - r0 < 128 ? rows - r0 : 128);
  const int c = b * 128 + (threadIdx.x & 127), half = threadIdx.x >> 7;
  float m = 0.0f;
  if (c < cols)
    for (int r = half; r < nr; r += 2) {
      Raw<TY, 1> v;
      load_raw<TY, 1>(elem_at(x, static_cast<size_t>(r0 + r) * ld_x + c, S), v);
      m = fmaxf(m, finite_abs(raw_value<TY, 1>(v, 0)));
    }
#pragma unroll
  for (int off = 16; off > 0; off >>= 1) m = fmaxf(m, __shfl_xor_sync(0xffffffffu, m, off));
  if ((threadIdx.x & 31) == 0) s_max[threadIdx.x >> 5] = m;
  __syncthreads();
  m = s_max[0];
#pragma unroll
  for (int w = 1; w < 8; ++w) m = fmaxf(m, s_max[w]);
  const int e = scale_exponent(m);
  const float inv = pow2(-e);
  if (threadIdx.x == 0) scale[rb * blocks + b] = pow2(e);
  if (c < cols)
    for (int r = half; r < nr; r += 2) {
      Raw<TY, 1> v;
      load_raw<TY, 1>(elem_at(x, static_cast<size_t>(r0 + r) * ld_x + c, S), v);
      q[static_cast<size_t>(r0 + r) * ld_q + c] =
          static_cast<uint8_t>(e4m3_pair(raw_value<TY, 1>(v, 0) * inv, 0.0f) & 0xffu);
    }
}

}  // namespace pw
