// Host side of the expert-row calls and the scaled (e4m3) products of include/pw.h.  Included once,
// by pw_lib.cu, after its launch helpers.
#pragma once

namespace {

constexpr int kScaledMaxGrid = 160;  // CTAs of a scaled product the workspace is sized for

inline bool type_ok(int t) { return t == PW_TYPE_F32 || t == PW_TYPE_BF16 || t == PW_TYPE_F16; }
inline int type_size(int t) { return t == PW_TYPE_F32 ? 4 : 2; }
inline bool aligned(const void* p, size_t a) { return reinterpret_cast<uintptr_t>(p) % a == 0; }

// T tokens of k slots: the sizes every row call takes.
inline bool slots_ok(int T, int k) {
  return T >= 1 && k >= 1 && k <= PW_MAX_TOPK && static_cast<long long>(T) * k <= PW_MAX_ROWS;
}
// H columns with row stride ld (elements), at p: not NULL, aligned to its elements.
inline bool rows_ok(const void* p, int type, int H, long long ld) {
  return p && type_ok(type) && H >= 1 && H <= PW_MAX_COLS && ld >= H && ld <= PW_MAX_COLS &&
         aligned(p, type_size(type));
}
// 16-byte accesses: whole vectors in a row, rows that start on 16 bytes.
inline bool vec_ok(const void* p, int size, int H, long long ld) {
  return aligned(p, 16) && H * static_cast<long long>(size) % 16 == 0 && ld * size % 16 == 0;
}

// A sort of n slots uses one CTA up to kSortOne (both measured: there a second launch costs more
// than the longer walk), then one per kSortRun slots, at most one per SM; more than that only where a
// CTA's run would pass what its 16-bit places hold (pw::kSortMaxRun: from 9.7 million slots on).
constexpr int kSortOne = 8192;
constexpr int kSortRun = 1024;
static_assert(kSortOne <= pw::kSortMaxRun && kSortRun <= pw::kSortMaxRun, "16-bit places");
int sort_ctas(int n, int sms) {
  if (n <= kSortOne) return 1;
  return std::max(std::min(sms, (n + kSortRun - 1) / kSortRun), (n + pw::kSortMaxRun - 1) / pw::kSortMaxRun);
}

struct ScaledDevice {
  bool ready = false;
};
ScaledDevice g_scaled_dev[kMaxDevices];
std::mutex g_scaled_mu;

template <typename F>
bool shared_ready(F* kernel, int bytes) {
  return cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, bytes) == cudaSuccess;
}
template <typename F>
bool scaled_kernel_ready(F* kernel) {
  cudaFuncAttributes a;
  if (!shared_ready(kernel, pw::k7::smem_bytes(PW_MAX_EXPERTS)) ||
      cudaFuncGetAttributes(&a, kernel) != cudaSuccess)
    return false;
  // the register split of the warpgroups has to fit what the block is launched with
  return a.numRegs * pw::k7::kThreads >= pw::k7::kSplitRegs;
}

// Once per device: shared memory opt-ins of the kernels here.
pw_status scaled_device(DeviceInfo** di) {
  int dev = 0;
  if (device_info(di) != PW_OK) return PW_ERR_CUDA;
  if (cudaGetDevice(&dev) != cudaSuccess) return PW_ERR_CUDA;
  std::lock_guard<std::mutex> lk(g_scaled_mu);
  if (g_scaled_dev[dev].ready) return PW_OK;
  const int few = pw::k8::smem_bytes(PW_MAX_EXPERTS);
  if (!shared_ready(pw::sort_count_kernel, 2 * pw::kSortWarps * PW_MAX_EXPERTS) ||
      !shared_ready(pw::sort_place_kernel, (4 + 2 * pw::kSortWarps) * PW_MAX_EXPERTS) ||
      !shared_ready(pw::k8::few_kernel<true, PW_TYPE_F32>, few) ||
      !shared_ready(pw::k8::few_kernel<false, PW_TYPE_F32>, few) ||
      !shared_ready(pw::k8::few_kernel<false, PW_TYPE_BF16>, few) ||
      !shared_ready(pw::k8::few_kernel<false, PW_TYPE_F16>, few))
    return PW_ERR_CUDA;
  if (!scaled_kernel_ready(pw::k7::scaled_kernel<true, PW_TYPE_F32>) ||
      !scaled_kernel_ready(pw::k7::scaled_kernel<false, PW_TYPE_F32>) ||
      !scaled_kernel_ready(pw::k7::scaled_kernel<false, PW_TYPE_BF16>) ||
      !scaled_kernel_ready(pw::k7::scaled_kernel<false, PW_TYPE_F16>))
    return PW_ERR_CUDA;
  g_scaled_dev[dev].ready = true;
  return PW_OK;
}

typedef CUresult (*EncodeTiled)(CUtensorMap*, CUtensorMapDataType, cuuint32_t, void*, const cuuint64_t*,
                                const cuuint64_t*, const cuuint32_t*, const cuuint32_t*,
                                CUtensorMapInterleave, CUtensorMapSwizzle, CUtensorMapL2promotion,
                                CUtensorMapFloatOOBfill);

EncodeTiled encode_tiled() {
  static std::atomic<EncodeTiled> fn{nullptr};
  EncodeTiled f = fn.load();
  if (f) return f;
  void* p = nullptr;
  cudaDriverEntryPointQueryResult q;
  if (cudaGetDriverEntryPointByVersion("cuTensorMapEncodeTiled", &p, 12000, cudaEnableDefault, &q) !=
          cudaSuccess ||
      q != cudaDriverEntryPointSuccess)
    return nullptr;
  f = reinterpret_cast<EncodeTiled>(p);
  fn.store(f);
  return f;
}

// Tensor map of bytes [d2][d1][d0] with row stride ld, box 128 columns x `box` rows, 128-byte
// swizzle, zeros outside.
bool byte_map(CUtensorMap* m, const void* p, uint64_t d0, uint64_t d1, uint64_t d2, uint64_t ld, int rank,
              int box) {
  const cuuint64_t dims[3] = {d0, d1, d2};
  const cuuint64_t strides[2] = {ld, ld * d1};
  const cuuint32_t boxes[3] = {128, static_cast<cuuint32_t>(box), 1};
  const cuuint32_t ones[3] = {1, 1, 1};
  EncodeTiled f = encode_tiled();
  return f && f(m, CU_TENSOR_MAP_DATA_TYPE_UINT8, rank, const_cast<void*>(p), dims, strides, boxes, ones,
                CU_TENSOR_MAP_INTERLEAVE_NONE, CU_TENSOR_MAP_SWIZZLE_128B,
                CU_TENSOR_MAP_L2_PROMOTION_L2_256B, CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) == CUDA_SUCCESS;
}

// One launch of a scaled product; the counters are zero before it runs.
struct ScaledCall {
  const uint8_t* xq;
  const float* xs;
  int M, K;
  long long ldx;
  const uint8_t* wq;
  const float* ws;
  int E, N;
  long long ldw;
  const int32_t* offsets;
  void* y;
  int y_type;
  long long ld_y;
  uint8_t* hq;  // gated (then N = 2 I and y is unused)
  float* hs;
  int I;
  float* part;
  int32_t* counter;
};

// Rows per expert, on average over the experts that can have one, up to which the few-rows kernel is
// used.  With even loads it is ahead up to there (64 experts of 8, 16 and 32 rows, 5120 x 3584: 180, 190 and
// 198 us against 201, 206 and 213; one matrix, 32 rows: 16.7 against 20.6), with 64 even or behind (64 x
// 28672 x 4096: 36 against 31), and ragged groups of 50 rows on average, many above 64, take 96 against 80.
// The host does not know the loads: M counts empty slots, and rows on few of the experts (a remap to a
// critical set, a skewed router) are more to each than this average.  What counts is the rows of an
// expert in use: 2048 rows on 64, 32, 16 and 4 of 64 experts take 198, 144, 117 and 102 us here and 213, 133,
// 80 and 58 with the large-rows kernel, 512 rows 180, 105, 68 and 41 against 201, 119, 73 and 25; loads
// falling as 1 / rank, 2048 rows: 237 against 229, 512 rows: 189 against 217.
constexpr int kFewRows = 32;

int part_rows(int M) { return static_cast<int>(align_up(std::min(M, pw::k7::kTileM), 32)); }
size_t part_bytes(int M) {
  return sizeof(float) * kScaledMaxGrid * pw::k7::kTileN * static_cast<size_t>(part_rows(M));
}

pw_status launch_scaled(const ScaledCall& c, int sms, cudaStream_t st) {
  pw::k7::Params p;
  const bool gated = c.hq != nullptr;
  const bool few = c.M <= kFewRows * std::min(c.E, c.M);
  if (!byte_map(&p.xmap, c.xq, c.K, c.M, 1, c.ldx, 2, pw::k7::kTileM) ||
      !byte_map(&p.xsmall, c.xq, c.K, c.M, 1, c.ldx, 2, pw::k7::kSmallRows) ||
      !byte_map(&p.wmap, c.wq, c.K, c.N, c.E, c.ldw, 3, gated ? (few ? 128 : 64) : pw::k7::kTileN))
    return PW_ERR_CUDA;
  p.sx = c.xs;
  p.sw = c.ws;
  p.offsets = c.offsets;
  p.M = c.M;
  p.N = c.N;
  p.K = c.K;
  p.E = c.E;
  p.kb = (c.K + 127) / 128;
  p.nb = (c.N + 127) / 128;
  p.nt = gated ? c.I / 128 : (c.N + pw::k7::kTileN - 1) / pw::k7::kTileN;
  p.y = c.y;
  p.ld_y = static_cast<size_t>(c.ld_y);
  p.vec = !gated && aligned(c.y, 16) && c.ld_y * type_size(c.y_type) % 16 == 0;
  p.hq = c.hq;
  p.hs = c.hs;
  p.I = c.I;
  p.part = c.part;
  p.rcap = part_rows(c.M);
  p.counter = c.counter;
  const dim3 grid(std::min(sms, kScaledMaxGrid)), block(few ? pw::k8::kThreads : pw::k7::kThreads);
  if (few) {
    const size_t smem = pw::k8::smem_bytes(c.E);
    if (gated) return launch_dependent(pw::k8::few_kernel<true, PW_TYPE_F32>, grid, block, smem, st, p);
    if (c.y_type == PW_TYPE_F32)
      return launch_dependent(pw::k8::few_kernel<false, PW_TYPE_F32>, grid, block, smem, st, p);
    if (c.y_type == PW_TYPE_BF16)
      return launch_dependent(pw::k8::few_kernel<false, PW_TYPE_BF16>, grid, block, smem, st, p);
    return launch_dependent(pw::k8::few_kernel<false, PW_TYPE_F16>, grid, block, smem, st, p);
  }
  const size_t smem = pw::k7::smem_bytes(c.E);
  if (gated) return launch_dependent(pw::k7::scaled_kernel<true, PW_TYPE_F32>, grid, block, smem, st, p);
  if (c.y_type == PW_TYPE_F32)
    return launch_dependent(pw::k7::scaled_kernel<false, PW_TYPE_F32>, grid, block, smem, st, p);
  if (c.y_type == PW_TYPE_BF16)
    return launch_dependent(pw::k7::scaled_kernel<false, PW_TYPE_BF16>, grid, block, smem, st, p);
  return launch_dependent(pw::k7::scaled_kernel<false, PW_TYPE_F16>, grid, block, smem, st, p);
}

pw_status launch_sort(const int32_t* idx, int T, int k, int E, int32_t* pos, int32_t* src,
                      int32_t* offsets, int32_t* part, int32_t* zero, int n_zero, int sms,
                      cudaStream_t st) {
  const int n = T * k, ctas = sort_ctas(n, std::min(sms, kScaledMaxGrid));
  const dim3 block(pw::kSortThreads);
  if (ctas > 1 &&
      launch_dependent(pw::sort_count_kernel, dim3(ctas), block,
                       2 * pw::kSortWarps * static_cast<size_t>(E), st, idx, n, E, part) != PW_OK)
    return PW_ERR_CUDA;
  return launch_dependent(pw::sort_place_kernel, dim3(ctas), block,
                          (4 + 2 * pw::kSortWarps) * static_cast<size_t>(E), st, idx, n, E,
                          static_cast<const int32_t*>(ctas > 1 ? part : nullptr), pos, src, offsets, zero,
                          n_zero);
}

pw_status launch_quantize_rows(const void* x, int type, long long rows, int cols, long long ld, int k,
                               const int32_t* pos, uint8_t* q, long long ldq, float* scale,
                               cudaStream_t st) {
  const int blocks = (cols + 127) / 128;
  // rows in flight: two once enough half-warps are left (4096 x 3584 bf16: one 15.1 us, two 11.8, four
  // 12.1)
  const int per = rows * blocks >= 65536 ? 2 : 1;
  const long long side = static_cast<long long>(16 / std::min(16, blocks)) * per;
  const dim3 grid(static_cast<unsigned>((rows + side - 1) / side), static_cast<unsigned>((blocks + 15) / 16));
  const bool vec = cols % 8 == 0 && vec_ok(x, type_size(type), cols, ld);
#define PW_QUANT(TY)                                                                              \
  return launch_dependent(vec ? (per == 1 ? pw::quantize_rows_kernel<TY, true, 1>                 \
                                          : pw::quantize_rows_kernel<TY, true, 2>)             \
                              : (per == 1 ? pw::quantize_rows_kernel<TY, false, 1>                \
                                          : pw::quantize_rows_kernel<TY, false, 2>),           \
                          grid, dim3(256), 0, st, x, rows, cols,                                  \
                          static_cast<size_t>(ld), k, pos, q, static_cast<size_t>(ldq), scale, blocks)
  if (type == PW_TYPE_F32) PW_QUANT(PW_TYPE_F32);
  if (type == PW_TYPE_BF16) PW_QUANT(PW_TYPE_BF16);
  PW_QUANT(PW_TYPE_F16);
#undef PW_QUANT
}

template <int TI, int TO>
pw_status launch_combine_types(const void* o, int T, int k, int H, long long ld_o, const int32_t* pos,
                               const float* gate, void* y, long long ld_y, cudaStream_t st) {
  constexpr int VI = 16 / pw::ElemSize<TI>::value;  // elements of one 16-byte load
  const bool vec = vec_ok(o, pw::ElemSize<TI>::value, H, ld_o) && aligned(y, 16) &&
                   ld_y * pw::ElemSize<TO>::value % 16 == 0;
  // vectors (single elements) of a lane; 16-bit types take one of 8 (4096 x 8 rows of 3584 bf16: 41.6
  // us, two 44.3), fp32 two of 4 (8192 x 4 rows of 2048: 53.9 us, one 57.6)
  constexpr int UV = 8 / VI, US = 8;
  const int cols = vec ? 32 * UV * VI : 32 * US;  // columns of one warp
  const int groups = (H + cols - 1) / cols;
  const long long grid = (static_cast<long long>(T) * groups + 7) / 8;
  if (grid > 0x7fffffffLL) return PW_ERR_UNSUPPORTED;
  const dim3 g(static_cast<unsigned>(grid)), b(256);
  if (vec)
    return launch_dependent(pw::combine_rows_kernel<TI, TO, VI, UV>, g, b, 0, st, o, T, k, H,
                            static_cast<size_t>(ld_o), pos, gate, y, static_cast<size_t>(ld_y), groups);
  return launch_dependent(pw::combine_rows_kernel<TI, TO, 1, US>, g, b, 0, st, o, T, k, H,
                          static_cast<size_t>(ld_o), pos, gate, y, static_cast<size_t>(ld_y), groups);
}

pw_status launch_combine(const void* o, int o_type, int T, int k, int H, long long ld_o,
                         const int32_t* pos, const float* gate, void* y, int y_type, long long ld_y,
                         cudaStream_t st) {
#define PW_COMBINE(TI, TO) \
  if (o_type == TI && y_type == TO) return launch_combine_types<TI, TO>(o, T, k, H, ld_o, pos, gate, y, ld_y, st)
  PW_COMBINE(PW_TYPE_F32, PW_TYPE_F32);
  PW_COMBINE(PW_TYPE_F32, PW_TYPE_BF16);
  PW_COMBINE(PW_TYPE_F32, PW_TYPE_F16);
  PW_COMBINE(PW_TYPE_BF16, PW_TYPE_F32);
  PW_COMBINE(PW_TYPE_BF16, PW_TYPE_BF16);
  PW_COMBINE(PW_TYPE_BF16, PW_TYPE_F16);
  PW_COMBINE(PW_TYPE_F16, PW_TYPE_F32);
  PW_COMBINE(PW_TYPE_F16, PW_TYPE_BF16);
  PW_COMBINE(PW_TYPE_F16, PW_TYPE_F16);
#undef PW_COMBINE
  return PW_ERR_INVALID_ARG;
}

template <int TY, int V>
pw_status launch_combine_grad(const void* dy, const void* o, int T, int k, int H, long long ld_dy,
                              long long ld_o, const int32_t* pos, const float* gate, void* d_o,
                              long long ld_do, float* d_gate, cudaStream_t st) {
  auto kernel = k <= 4   ? pw::combine_grad_kernel<TY, V, 4>
                : k <= 8 ? pw::combine_grad_kernel<TY, V, 8>
                         : pw::combine_grad_kernel<TY, V, 16>;
  return launch_dependent(kernel, dim3(T), dim3(pw::kGradThreads), 0, st, dy, o, T, k, H,
                          static_cast<size_t>(ld_dy), static_cast<size_t>(ld_o), pos, gate, d_o,
                          static_cast<size_t>(ld_do), d_gate);
}

// Workspace of pw_moe_scaled_forward.
struct ScaledWorkspace {
  size_t pos, offsets, sort, counter, xq, xs, hq, hs, o, part, total;
};
ScaledWorkspace scaled_ws(int T, int k, int E, int H, int I) {
  ScaledWorkspace w;
  const size_t n = static_cast<size_t>(T) * k;
  size_t at = 0;
  auto take = [&](size_t bytes) {
    const size_t a = at;
    at = align_up(at + bytes, 256);
    return a;
  };
  w.offsets = take(4 * static_cast<size_t>(E + 1));
  w.pos = take(4 * n);
  w.sort = take(pw_expert_sort_workspace_bytes(T, k, E));
  w.counter = take(4 * 2 * kScaledMaxGrid);  // one set for each product, both zeroed by the sort
  w.xq = take(n * H);
  w.xs = take(4 * n * (H / 128));
  w.hq = take(n * I);
  w.hs = take(4 * n * (I / 128));
  w.o = take(4 * n * H);
  // partials of either product: the second writes its own only when the first has ended
  w.part = take(part_bytes(static_cast<int>(n)));
  w.total = at;
  return w;
}

}  // namespace

extern "C" {

size_t pw_expert_sort_workspace_bytes(int T, int k, int E) {
  if (!slots_ok(T, k) || E < 1 || E > PW_MAX_EXPERTS) return 0;
  // counts of every CTA (none up to kSortOne slots), at least one word
  const int ctas = sort_ctas(T * k, kScaledMaxGrid);
  return align_up(4 * static_cast<size_t>(ctas > 1 ? ctas : 1) * E, 256);
}

pw_status pw_expert_sort(const int32_t* idx, int T, int k, int E, int32_t* pos, int32_t* src,
                         int32_t* offsets, void* workspace, size_t ws_bytes, pw_stream_t stream) {
  if (!idx || !pos || !src || !offsets || !workspace) return PW_ERR_INVALID_ARG;
  if (!slots_ok(T, k) || E < 1 || E > PW_MAX_EXPERTS) return PW_ERR_INVALID_ARG;
  if (!aligned(idx, 4) || !aligned(pos, 4) || !aligned(src, 4) || !aligned(offsets, 4) ||
      !aligned(workspace, 256) || ws_bytes < pw_expert_sort_workspace_bytes(T, k, E))
    return PW_ERR_INVALID_ARG;
  DeviceInfo* di = nullptr;
  if (scaled_device(&di) != PW_OK) return PW_ERR_CUDA;
  return launch_sort(idx, T, k, E, pos, src, offsets, static_cast<int32_t*>(workspace), nullptr, 0,
                     di->sms, as_cuda(stream));
}

pw_status pw_expert_dispatch(const void* x, int type, int T, int k, int H, long long x_stride,
                             const int32_t* pos, void* xs, long long xs_stride, pw_stream_t stream) {
  if (!slots_ok(T, k) || !rows_ok(x, type, H, x_stride) || !rows_ok(xs, type, H, xs_stride) || !pos ||
      !aligned(pos, 4))
    return PW_ERR_INVALID_ARG;
  const int size = type_size(type);
  const size_t lx = static_cast<size_t>(x_stride), ls = static_cast<size_t>(xs_stride);
  constexpr int U = 4;
  auto groups = [&](int units) { return (units + 32 * U - 1) / (32 * U); };
  auto grid = [&](int units) {
    return dim3(static_cast<unsigned>((static_cast<long long>(T) * groups(units) + 7) / 8));
  };
  if (static_cast<long long>(T) * groups(H) > 0x7fffffffLL) return PW_ERR_UNSUPPORTED;
  cudaStream_t st = as_cuda(stream);
  if (vec_ok(x, size, H, x_stride) && vec_ok(xs, size, H, xs_stride)) {
    const int per = 16 / size, units = H / per;
    return launch_dependent(pw::dispatch_kernel<uint4, U>, grid(units), dim3(256), 0, st,
                            static_cast<const uint4*>(x), T, k, units, lx / per, pos,
                            static_cast<uint4*>(xs), ls / per, groups(units));
  }
  if (size == 4)
    return launch_dependent(pw::dispatch_kernel<uint32_t, U>, grid(H), dim3(256), 0, st,
                            static_cast<const uint32_t*>(x), T, k, H, lx, pos,
                            static_cast<uint32_t*>(xs), ls, groups(H));
  return launch_dependent(pw::dispatch_kernel<unsigned short, U>, grid(H), dim3(256), 0, st,
                          static_cast<const unsigned short*>(x), T, k, H, lx, pos,
                          static_cast<unsigned short*>(xs), ls, groups(H));
}

pw_status pw_expert_dispatch_grad(const void* d_xs, int type, int T, int k, int H, long long d_xs_stride,
                                  const int32_t* pos, void* d_x, long long d_x_stride,
                                  pw_stream_t stream) {
  if (!slots_ok(T, k) || !rows_ok(d_xs, type, H, d_xs_stride) || !rows_ok(d_x, type, H, d_x_stride) ||
      !pos || !aligned(pos, 4))
    return PW_ERR_INVALID_ARG;
  return launch_combine(d_xs, type, T, k, H, d_xs_stride, pos, nullptr, d_x, type, d_x_stride,
                        as_cuda(stream));
}

pw_status pw_expert_combine(const void* o, int o_type, int T, int k, int H, long long o_stride,
                            const int32_t* pos, const float* gate, void* y, int y_type,
                            long long y_stride, pw_stream_t stream) {
  if (!slots_ok(T, k) || !rows_ok(o, o_type, H, o_stride) || !rows_ok(y, y_type, H, y_stride) || !pos ||
      !aligned(pos, 4) || !gate || !aligned(gate, 4))
    return PW_ERR_INVALID_ARG;
  return launch_combine(o, o_type, T, k, H, o_stride, pos, gate, y, y_type, y_stride, as_cuda(stream));
}

pw_status pw_expert_combine_grad(const void* d_y, const void* o, int type, int T, int k, int H,
                                 long long d_y_stride, long long o_stride, const int32_t* pos,
                                 const float* gate, void* d_o, long long d_o_stride, float* d_gate,
                                 pw_stream_t stream) {
  if (!d_o && !d_gate) return PW_ERR_INVALID_ARG;
  if (!slots_ok(T, k) || !rows_ok(d_y, type, H, d_y_stride) || !pos || !aligned(pos, 4) || !gate ||
      !aligned(gate, 4))
    return PW_ERR_INVALID_ARG;
  if (d_gate && (!rows_ok(o, type, H, o_stride) || !aligned(d_gate, 4))) return PW_ERR_INVALID_ARG;
  if (d_o && !rows_ok(d_o, type, H, d_o_stride)) return PW_ERR_INVALID_ARG;
  const int size = type_size(type);
  const bool vec = vec_ok(d_y, size, H, d_y_stride) && (!d_gate || vec_ok(o, size, H, o_stride)) &&
                   (!d_o || vec_ok(d_o, size, H, d_o_stride));
  cudaStream_t st = as_cuda(stream);
#define PW_GRAD(TY, V) \
  return launch_combine_grad<TY, V>(d_y, o, T, k, H, d_y_stride, o_stride, pos, gate, d_o, d_o_stride, d_gate, st)
  if (type == PW_TYPE_F32) {
    if (vec) PW_GRAD(PW_TYPE_F32, 4);
    PW_GRAD(PW_TYPE_F32, 1);
  }
  if (type == PW_TYPE_BF16) {
    if (vec) PW_GRAD(PW_TYPE_BF16, 8);
    PW_GRAD(PW_TYPE_BF16, 1);
  }
  if (vec) PW_GRAD(PW_TYPE_F16, 8);
  PW_GRAD(PW_TYPE_F16, 1);
#undef PW_GRAD
}

pw_status pw_scaled_quantize(const void* x, int type, int rows, int cols, long long x_stride,
                             int block_rows, uint8_t* q, long long q_stride, float* scale,
                             pw_stream_t stream) {
  if (rows < 1 || rows > PW_MAX_ROWS || (block_rows != 1 && block_rows != 128)) return PW_ERR_INVALID_ARG;
  if (!rows_ok(x, type, cols, x_stride) || !q || !scale || !aligned(scale, 4) || !aligned(q, 16) ||
      q_stride < cols || q_stride % 16 || q_stride > PW_MAX_COLS)
    return PW_ERR_INVALID_ARG;
  cudaStream_t st = as_cuda(stream);
  if (block_rows == 1)
    return launch_quantize_rows(x, type, rows, cols, x_stride, 1, nullptr, q, q_stride, scale, st);
  const int blocks = (cols + 127) / 128;
  const long long grid = static_cast<long long>((rows + 127) / 128) * blocks;
  if (grid > 0x7fffffffLL) return PW_ERR_UNSUPPORTED;
  auto kernel = type == PW_TYPE_F32    ? pw::quantize_blocks_kernel<PW_TYPE_F32>
                : type == PW_TYPE_BF16 ? pw::quantize_blocks_kernel<PW_TYPE_BF16>
                                       : pw::quantize_blocks_kernel<PW_TYPE_F16>;
  kernel<<<static_cast<unsigned>(grid), 256, 0, st>>>(x, rows, cols, static_cast<size_t>(x_stride), q,
                                                      static_cast<size_t>(q_stride), scale, blocks);
  return launch_status();
}

size_t pw_scaled_gemm_workspace_bytes(int M, int N, int K, int E) {
  if (M < 1 || M > PW_MAX_ROWS || N < 1 || N > PW_MAX_COLS || K < 1 || K > PW_MAX_COLS || E < 1 ||
      E > PW_MAX_EXPERTS)
    return 0;
  return align_up(4 * kScaledMaxGrid, 256) + part_bytes(M);
}

pw_status pw_scaled_gemm(const uint8_t* x_q, const float* x_scale, int M, int K, long long x_stride,
                         const uint8_t* w_q, const float* w_scale, int E, int N, long long w_stride,
                         const int32_t* offsets, void* y, int y_type, long long y_stride,
                         void* workspace, size_t ws_bytes, pw_stream_t stream) {
  const size_t need = pw_scaled_gemm_workspace_bytes(M, N, K, E);
  if (!need || !x_q || !x_scale || !w_q || !w_scale || !workspace) return PW_ERR_INVALID_ARG;
  if (!offsets && E != 1) return PW_ERR_INVALID_ARG;
  if (!aligned(x_q, 16) || !aligned(w_q, 16) || !aligned(x_scale, 4) || !aligned(w_scale, 4) ||
      !aligned(offsets, 4) || x_stride % 16 || w_stride % 16 || x_stride < K || w_stride < K ||
      x_stride > PW_MAX_COLS || w_stride > PW_MAX_COLS)
    return PW_ERR_INVALID_ARG;
  if (!rows_ok(y, y_type, N, y_stride)) return PW_ERR_INVALID_ARG;
  if (!aligned(workspace, 256) || ws_bytes < need) return PW_ERR_INVALID_ARG;
  DeviceInfo* di = nullptr;
  if (scaled_device(&di) != PW_OK) return PW_ERR_CUDA;
  cudaStream_t st = as_cuda(stream);
  ScaledCall c = {};
  c.xq = x_q;
  c.xs = x_scale;
  c.M = M;
  c.K = K;
  c.ldx = x_stride;
  c.wq = w_q;
  c.ws = w_scale;
  c.E = E;
  c.N = N;
  c.ldw = w_stride;
  c.offsets = offsets;
  c.y = y;
  c.y_type = y_type;
  c.ld_y = y_stride;
  c.counter = static_cast<int32_t*>(workspace);
  c.part = reinterpret_cast<float*>(static_cast<uint8_t*>(workspace) + align_up(4 * kScaledMaxGrid, 256));
  if (launch_dependent(pw::zero_words_kernel, dim3(1), dim3(256), 0, st, c.counter, kScaledMaxGrid) != PW_OK)
    return PW_ERR_CUDA;
  return launch_scaled(c, di->sms, st);
}

size_t pw_moe_scaled_workspace_bytes(int T, int k, int E, int H, int I) {
  if (!slots_ok(T, k) || E < 1 || E > PW_MAX_EXPERTS || H < 128 || H > PW_MAX_COLS || H % 128 || I < 128 ||
      2 * static_cast<long long>(I) > PW_MAX_COLS || I % 128)
    return 0;
  return scaled_ws(T, k, E, H, I).total;
}

pw_status pw_moe_scaled_forward(const pw_scaled_experts* ex, const void* x, int x_type, int T, int k,
                                const int32_t* idx, const float* gate, void* y, int y_type,
                                void* workspace, size_t ws_bytes, pw_stream_t stream) {
  if (!ex || !idx || !gate || !workspace) return PW_ERR_INVALID_ARG;
  const int E = ex->E, H = ex->H, I = ex->I;
  const size_t need = pw_moe_scaled_workspace_bytes(T, k, E, H, I);
  if (!need || ws_bytes < need || !aligned(workspace, 256)) return PW_ERR_INVALID_ARG;
  if (!ex->gate_up || !ex->gate_up_scale || !ex->down || !ex->down_scale || !aligned(ex->gate_up, 16) ||
      !aligned(ex->down, 16) || !aligned(ex->gate_up_scale, 4) || !aligned(ex->down_scale, 4))
    return PW_ERR_INVALID_ARG;
  if (!rows_ok(x, x_type, H, H) || !rows_ok(y, y_type, H, H) || !aligned(idx, 4) || !aligned(gate, 4))
    return PW_ERR_INVALID_ARG;
  DeviceInfo* di = nullptr;
  if (scaled_device(&di) != PW_OK) return PW_ERR_CUDA;
  const ScaledWorkspace w = scaled_ws(T, k, E, H, I);
  uint8_t* base = static_cast<uint8_t*>(workspace);
  int32_t* pos = reinterpret_cast<int32_t*>(base + w.pos);
  int32_t* offsets = reinterpret_cast<int32_t*>(base + w.offsets);
  int32_t* counter = reinterpret_cast<int32_t*>(base + w.counter);
  uint8_t* xq = base + w.xq;
  float* xs = reinterpret_cast<float*>(base + w.xs);
  uint8_t* hq = base + w.hq;
  float* hs = reinterpret_cast<float*>(base + w.hs);
  float* o = reinterpret_cast<float*>(base + w.o);
  cudaStream_t st = as_cuda(stream);
  pw_status s = launch_sort(idx, T, k, E, pos, nullptr, offsets, reinterpret_cast<int32_t*>(base + w.sort),
                            counter, 2 * kScaledMaxGrid, di->sms, st);
  if (s != PW_OK) return s;
  s = launch_quantize_rows(x, x_type, T, H, H, k, pos, xq, H, xs, st);
  if (s != PW_OK) return s;
  ScaledCall c = {};
  c.xq = xq;
  c.xs = xs;
  c.M = T * k;
  c.K = H;
  c.ldx = H;
  c.wq = ex->gate_up;
  c.ws = ex->gate_up_scale;
  c.E = E;
  c.N = 2 * I;
  c.ldw = H;
  c.offsets = offsets;
  c.hq = hq;
  c.hs = hs;
  c.I = I;
  c.counter = counter;
  c.part = reinterpret_cast<float*>(base + w.part);
  s = launch_scaled(c, di->sms, st);
  if (s != PW_OK) return s;
  ScaledCall d = {};
  d.xq = hq;
  d.xs = hs;
  d.M = T * k;
  d.K = I;
  d.ldx = I;
  d.wq = ex->down;
  d.ws = ex->down_scale;
  d.E = E;
  d.N = H;
  d.ldw = I;
  d.offsets = offsets;
  d.y = o;
  d.y_type = PW_TYPE_F32;
  d.ld_y = H;
  d.counter = counter + kScaledMaxGrid;
  d.part = c.part;
  s = launch_scaled(d, di->sms, st);
  if (s != PW_OK) return s;
  return launch_combine(o, PW_TYPE_F32, T, k, H, H, pos, gate, y, y_type, H, st);
}

}  // extern "C"
