// Host side of linear_gate: checks, the choice of a kernel, tensor maps, launches.
#include <cudaTypedefs.h>

#include <atomic>
#include <cstring>
#include <new>

#include "host_checks.h"
#include "linear_gate_kernel.cuh"

using namespace block_ops;

struct linear_gate_s {
  lg_config cfg;
};

namespace {

constexpr int64_t kMaxWidth = 1 << 20;

int element_size(const lg_config& c) { return c.dtype == BO_E4M3 ? 1 : 2; }

fn_status validate(const linear_gate_s* h, const lg_args* a) {
  if (!h || !a) return FN_ERR_INVALID_ARG;
  const lg_config& c = h->cfg;
  const int64_t B = a->B, L = a->L, tpf = a->tokens_per_frame, K = c.K, N = c.N;
  const bool fp8 = c.dtype == BO_E4M3;
  const int size = element_size(c), unit = 16 / size;
  if (B < 0 || L < 0 || tpf < 0) return FN_ERR_INVALID_ARG;
  if (B == 0 || L == 0) return FN_OK;
  if (B > kMaxRows || L > kMaxRows || B * L > kMaxRows - 256) return FN_ERR_INVALID_ARG;  // tiles of 256 rows stay in 31 bits
  if ((__int128)B * L * (K > N ? K : N) > kMaxExtent) return FN_ERR_INVALID_ARG;
  if (tpf > 0 && L % tpf != 0) return FN_ERR_INVALID_ARG;
  const int64_t F = tpf > 0 ? L / tpf : 1;

  Findings f;
  f.require(a->x.ptr && a->weight && a->out, FN_ERR_INVALID_ARG);
  f.require((a->bias != nullptr) == (c.has_bias != 0) && (a->gate.ptr != nullptr) == (c.has_gate != 0) &&
                (a->residual.ptr != nullptr) == (c.has_residual != 0),
            FN_ERR_INVALID_ARG);
  f.require((a->x_scale != nullptr) == fp8 && (a->weight_scale != nullptr) == fp8, FN_ERR_INVALID_ARG);
  f.require(a->x.stride_b >= 0 && a->x.stride_l >= 0 && a->x.stride_f == 0, FN_ERR_INVALID_ARG);
  f.require(aligned16(a->x.ptr) && a->x.stride_b % unit == 0 && a->x.stride_l % unit == 0, FN_ERR_MISALIGNED);
  f.require(a->weight_stride >= (N > 1 ? K : 0), FN_ERR_INVALID_ARG);
  f.require(aligned16(a->weight) && a->weight_stride % unit == 0, FN_ERR_MISALIGNED);
  f.require(aligned16(a->bias) && aligned16(a->weight_scale), FN_ERR_MISALIGNED);
  f.require(reinterpret_cast<uintptr_t>(a->x_scale) % 4 == 0, FN_ERR_MISALIGNED);
  if (a->gate.ptr) check_operand(a->gate, tpf > 0, f);
  if (a->residual.ptr) {
    check_operand(a->residual, false, f);
    f.require((L == 1 || a->residual.stride_l > 0) && (B == 1 || a->residual.stride_b > 0), FN_ERR_INVALID_ARG);
  }
  check_output(a->out, a->out_stride_b, a->out_stride_l, B, L, N, 8, f);
  if (f.status != FN_OK) return f.status;
  // what a tensor map holds: no row that several tokens share, strides below 2^40 bytes
  if (B * L > kTokens && ((L > 1 && a->x.stride_l == 0) || (B > 1 && a->x.stride_b == 0))) return FN_ERR_UNSUPPORTED;
  if (a->x.stride_b * size >= (int64_t)1 << 39 || a->x.stride_l * size >= (int64_t)1 << 39 ||
      a->weight_stride * size >= (int64_t)1 << 39 || a->out_stride_b >= (int64_t)1 << 38 || a->out_stride_l >= (int64_t)1 << 38 ||
      a->residual.stride_b >= (int64_t)1 << 38 || a->residual.stride_l >= (int64_t)1 << 38)
    return FN_ERR_INVALID_ARG;

  const int64_t n[2] = {B, L}, os[2] = {a->out_stride_b, a->out_stride_l}, xs[2] = {a->x.stride_b, a->x.stride_l};
  const int64_t wn[1] = {N}, ws[1] = {a->weight_stride};
  const int64_t oe = extent_of(n, os, N), xe = extent_of(n, xs, K), we = extent_of(wn, ws, K);
  if (oe < 0 || xe < 0 || we < 0) return FN_ERR_INVALID_ARG;
  const Span out = bytes_at(a->out, (uint64_t)oe * 2);
  if (overlaps(out, bytes_at(a->x.ptr, (uint64_t)xe * size)) || overlaps(out, bytes_at(a->weight, (uint64_t)we * size)))
    return FN_ERR_INVALID_ARG;
  if (a->bias && overlaps(out, bytes_at(a->bias, (uint64_t)N * 2))) return FN_ERR_INVALID_ARG;
  if (fp8 && (overlaps(out, bytes_at(a->x_scale, (uint64_t)B * L * 4)) || overlaps(out, bytes_at(a->weight_scale, (uint64_t)N * 4))))
    return FN_ERR_INVALID_ARG;
  const bool in_place = same_rows(a->residual, a->out, a->out_stride_b, a->out_stride_l, B, L);
  for (const fn_operand* o : {&a->gate, &a->residual}) {
    if (!o->ptr) continue;
    Span s;
    if (!operand_span(*o, B, F, L, N, 2, &s)) return FN_ERR_INVALID_ARG;
    if (overlaps(out, s) && !(o == &a->residual && in_place)) return FN_ERR_INVALID_ARG;
  }
  return FN_OK;
}

// Where the matrix kernels say that a wait ran out: four bytes of host memory that every device
// maps, for the life of the process. The first call may be captured, or come from two threads.
cudaError_t gave_up_word(int** word) {
  static std::atomic<int*> known{nullptr};
  if ((*word = known.load(std::memory_order_acquire))) return cudaSuccess;
  void* at = nullptr;
  cudaStreamCaptureMode mode = cudaStreamCaptureModeRelaxed;
  cudaError_t e = cudaThreadExchangeStreamCaptureMode(&mode);
  if (e != cudaSuccess) return e;
  e = cudaHostAlloc(&at, sizeof(int), cudaHostAllocPortable | cudaHostAllocMapped);
  if (e == cudaSuccess) {
    *(*word = static_cast<int*>(at)) = 0;
    int* other = nullptr;
    if (!known.compare_exchange_strong(other, *word, std::memory_order_acq_rel)) {
      *word = other;
      cudaFreeHost(at);
    }
  }
  cudaThreadExchangeStreamCaptureMode(&mode);
  return e;
}

LinearOperand operand_of(const fn_operand& o) {
  return LinearOperand{static_cast<const uint16_t*>(o.ptr), o.stride_b, o.stride_f, o.stride_l};
}

LinearParams make_params(const linear_gate_s* h, const lg_args* a) {
  LinearParams p;
  std::memset(&p, 0, sizeof(p));
  p.x = a->x.ptr, p.weight = a->weight;
  p.x_sb = a->x.stride_b, p.x_sl = a->x.stride_l, p.weight_stride = a->weight_stride;
  p.rows = (uint32_t)(a->B * a->L), p.L = (uint32_t)a->L, p.tpf = (uint32_t)a->tokens_per_frame;
  p.div_L = fused_norm_impl::make_div_u32(p.L);
  p.div_tpf = fused_norm_impl::make_div_u32(p.tpf ? p.tpf : 1u);
  p.N = (uint32_t)h->cfg.N, p.K = (uint32_t)h->cfg.K;
  p.act = h->cfg.act;
  p.bias = static_cast<const uint16_t*>(a->bias);
  p.gate = operand_of(a->gate), p.residual = operand_of(a->residual);
  p.has_residual = h->cfg.has_residual;
  p.x_scale = a->x_scale, p.weight_scale = a->weight_scale;
  p.out = static_cast<uint16_t*>(a->out);
  p.out_sb = a->out_stride_b, p.out_sl = a->out_stride_l;
  return p;
}

// ---- a few tokens ---------------------------------------------------------------------------

template <int PARTS, bool FP8, bool FP16>
void* token_kernel(int M) {
  if constexpr (PARTS == 4) {  // one part is for three and four tokens only
    if (M == 1) return (void*)linear_gate_tokens<1, PARTS, FP8, FP16>;
    if (M == 2) return (void*)linear_gate_tokens<2, PARTS, FP8, FP16>;
  }
  return M == 3 ? (void*)linear_gate_tokens<3, PARTS, FP8, FP16> : (void*)linear_gate_tokens<4, PARTS, FP8, FP16>;
}
template <int PARTS>
void* token_kernel(int dtype, int M) {
  return dtype == BO_E4M3 ? token_kernel<PARTS, true, false>(M) : dtype == BO_FP16 ? token_kernel<PARTS, false, true>(M) : token_kernel<PARTS, false, false>(M);
}

// Four warps share K, except for three and four tokens where N keeps the GPU busy with a warp to
// its columns (four tokens, 5120 -> 30720 65.5 against 70.7 us, -> 5120 20.5 against 15.0; one
// token, -> 30720 52.4 against 48.0, -> 5120 16.5 against 10.2).
constexpr uint32_t kBusyColumns = 16384;

fn_status launch_tokens(const linear_gate_s* h, LinearParams& p, cudaStream_t stream) {
  const int parts = p.rows > 2 && p.N >= kBusyColumns ? 1 : 4, per_cta = kTokenThreads / 32 / parts * kTokenColumns;
  void* kernel = parts == 1 ? token_kernel<1>(h->cfg.dtype, p.rows) : token_kernel<4>(h->cfg.dtype, p.rows);
  void* args[] = {&p};
  return launch_status(cudaLaunchKernel(kernel, dim3((p.N + per_cta - 1) / per_cta), dim3(kTokenThreads), args, 0, stream));
}

// ---- many rows --------------------------------------------------------------------------------

struct Variant {
  int cg, bn, shared, stages, received[9];  // received: bytes of sums by the parts of K, of a split tile
  void* kernel[3];  // by dtype: bf16, fp16, e4m3
  int rows() const { return kTileM * cg; }
};
template <int CG, int BN>
Variant variant() {
  using S = MatrixShape<CG, BN>;
  return Variant{CG, BN, S::kShared, S::kStages, {},
                 {(void*)linear_gate_tiles<CG, BN, false, false>, (void*)linear_gate_tiles<CG, BN, false, true>,
                  (void*)linear_gate_tiles<CG, BN, true, false>}};
}
const Variant kVariants[] = {variant<2, 256>(), variant<2, 192>(), variant<2, 128>(), variant<1, 256>(), variant<1, 128>(), variant<1, 64>()};

template <int CG, int BN>
Variant split_variant() {
  using S = SplitShape<CG, BN>;
  Variant v{CG, BN, S::kShared, S::kStages, {},
            {(void*)linear_gate_split<CG, BN, false, false>, (void*)linear_gate_split<CG, BN, false, true>,
             (void*)linear_gate_split<CG, BN, true, false>}};
  for (int n = 1; n <= 8; ++n) v.received[n] = S::received(n);
  return v;
}
const Variant kSplitVariants[] = {split_variant<2, 256>(), split_variant<1, 128>(), split_variant<1, 64>()};

// Cycles of a step of K: the products, or the operands' way into an SM: 80 bytes a cycle, and
// less where rows of 128 bytes start between lines (999 x 2048 x 1288 12.2 us, K = 2080 13.5,
// 2064 14.9, 2056 19.1); and no step is shorter than its share of a load's 2500 cycles (16 x 5120
// x 5120 as 80 CTAs of 8 stages: 335 cycles a step).
int64_t step_cycles(const Variant& v, int64_t rows, int64_t row_bytes) {
  const int64_t products = 2 * v.bn;
  const int64_t x = rows < kTileM ? rows : kTileM;  // rows past the last are not read
  const int percent = row_bytes % 128 == 0 ? 100 : row_bytes % 64 == 0 ? 120 : row_bytes % 32 == 0 ? 140 : 200;
  const int64_t bytes = (x + v.bn / v.cg) * kStepBytes * percent / 8000;
  const int64_t least = 2500 / v.stages, most = products > bytes ? products : bytes;
  return most > least ? most : least;
}
// What a tile takes besides: its way through the epilogue, which the next tile hides or not.
int64_t drain_cycles(const Variant& v) { return 1500 + v.bn * 16; }

// A matrix of `rows` rows of `width` elements per batch, as a tensor map of boxes.
struct Matrix {
  const void* ptr;
  int64_t width, rows, row_stride, batches, batch_stride;
};
fn_status encode(CUtensorMap* m, int dtype, const Matrix& a, int box_width, int box_rows, CUtensorMapSwizzle swizzle) {
  static const auto fn = []() -> PFN_cuTensorMapEncodeTiled_v12000 {
    void* f = nullptr;
    cudaDriverEntryPointQueryResult found;
    if (cudaGetDriverEntryPointByVersion("cuTensorMapEncodeTiled", &f, 12000, cudaEnableDefault, &found) != cudaSuccess ||
        found != cudaDriverEntryPointSuccess)
      return nullptr;
    return reinterpret_cast<PFN_cuTensorMapEncodeTiled_v12000>(f);
  }();
  if (!fn) return launch_status(cudaErrorNotSupported);
  const int size = dtype == BO_E4M3 ? 1 : 2;
  const cuuint64_t dims[3] = {(cuuint64_t)a.width, (cuuint64_t)a.rows, (cuuint64_t)a.batches};
  // a single row or batch is never stepped over: any valid stride serves
  const cuuint64_t strides[2] = {(cuuint64_t)(a.rows > 1 ? a.row_stride * size : 16),
                                 (cuuint64_t)(a.batches > 1 ? a.batch_stride * size : 16)};
  const cuuint32_t box[3] = {(cuuint32_t)box_width, (cuuint32_t)box_rows, 1}, unit[3] = {1, 1, 1};
  const CUtensorMapDataType type = dtype == BO_E4M3   ? CU_TENSOR_MAP_DATA_TYPE_UINT8
                                   : dtype == BO_FP16 ? CU_TENSOR_MAP_DATA_TYPE_FLOAT16
                                                      : CU_TENSOR_MAP_DATA_TYPE_BFLOAT16;
  const CUresult r = fn(m, type, 3, const_cast<void*>(a.ptr), dims, strides, box, unit, CU_TENSOR_MAP_INTERLEAVE_NONE, swizzle,
                        CU_TENSOR_MAP_L2_PROMOTION_L2_256B, CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE);
  return r == CUDA_SUCCESS ? FN_OK : launch_status(cudaErrorInvalidValue);
}

// How many clusters of n parts of K run at once; asked once per variant (devices of one kind).
fn_status clusters_at_once(const Variant& v, int n, int dtype, int* count) {
  static std::atomic<int> known[3][9][3];
  std::atomic<int>& k = known[&v - kSplitVariants][n][dtype];
  *count = k.load(std::memory_order_relaxed);
  if (*count) return FN_OK;
  cudaError_t e = cudaFuncSetAttribute(v.kernel[dtype], cudaFuncAttributeMaxDynamicSharedMemorySize, v.shared);
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3(n * v.cg), cfg.blockDim = dim3(kMatrixThreads), cfg.dynamicSmemBytes = v.shared;
  cudaLaunchAttribute cluster;
  cluster.id = cudaLaunchAttributeClusterDimension;
  cluster.val.clusterDim.x = n * v.cg, cluster.val.clusterDim.y = 1, cluster.val.clusterDim.z = 1;
  cfg.attrs = &cluster, cfg.numAttrs = 1;
  if (e == cudaSuccess) e = cudaOccupancyMaxActiveClusters(count, v.kernel[dtype], &cfg);
  if (e != cudaSuccess) return launch_status(e);
  k.store(*count, std::memory_order_relaxed);
  return FN_OK;
}

fn_status launch_tiles(const linear_gate_s* h, const lg_args* a, LinearParams& p, cudaStream_t stream) {
  const lg_config& c = h->cfg;
  int device = 0, sms = 0;
  cudaError_t e = cudaGetDevice(&device);
  if (e == cudaSuccess) e = cudaDeviceGetAttribute(&sms, cudaDevAttrMultiProcessorCount, device);
  if (e != cudaSuccess) return launch_status(e);

  // Rows at one distance from each other are one batch; otherwise a tile stays inside a batch.
  auto even = [&](int64_t sb, int64_t sl) { return sb == a->L * sl; };
  const bool flat = a->B == 1 || a->L == 1 ||
                    (even(a->x.stride_b, a->x.stride_l) && even(a->out_stride_b, a->out_stride_l) &&
                     (!c.has_residual || even(a->residual.stride_b, a->residual.stride_l)));
  const int64_t batches = flat ? 1 : a->B, rows = flat ? a->B * a->L : a->L;
  auto matrix = [&](const void* ptr, int64_t width, int64_t sb, int64_t sl) {
    return Matrix{ptr, width, rows, a->L == 1 ? sb : sl, batches, sb};
  };

  const int64_t steps = (c.K * element_size(c) + kStepBytes - 1) / kStepBytes;
  const int64_t row_bytes = (a->L > 1 ? a->x.stride_l : a->x.stride_b) * element_size(c) | a->weight_stride * element_size(c);
  const Variant* best = nullptr;
  int64_t best_cost = 0, parts = 1;
  for (const Variant& v : kVariants) {
    const int64_t tm = (rows + v.rows() - 1) / v.rows() * batches, tn = (c.N + v.bn - 1) / v.bn;
    const int64_t waves = (tm * tn + sms / v.cg - 1) / (sms / v.cg);
    const int64_t cost = waves * steps * step_cycles(v, rows, row_bytes) + drain_cycles(v);
    if (!best || cost < best_cost) best = &v, best_cost = cost;
  }
  // Few tiles: K split over a cluster, where its CTAs all run at once. Exchanging the sums takes
  // some 8500 cycles for 128 columns, 13000 for 256.
  for (const Variant& v : kSplitVariants) {
    const int64_t tiles = (rows + v.rows() - 1) / v.rows() * batches * ((c.N + v.bn - 1) / v.bn);
    for (int n = 2; n * v.cg <= 8 && n * 2 <= steps; ++n) {
      if (tiles * n * v.cg > sms || v.received[n] > v.shared - 1024) continue;
      const int64_t cost = (steps + n - 1) / n * step_cycles(v, rows, row_bytes) + 4000 + 35 * v.bn + drain_cycles(v) / n;
      if (cost >= best_cost) continue;
      int resident = 0;
      const fn_status s = clusters_at_once(v, n, c.dtype, &resident);
      if (s != FN_OK) return s;
      if (tiles <= resident) best = &v, best_cost = cost, parts = n;
    }
  }
  const Variant& v = *best;
  const int size = element_size(c);
  p.batch_rows = (uint32_t)rows, p.batches = (uint32_t)batches;
  p.tiles_m = (uint32_t)((rows + v.rows() - 1) / v.rows()), p.tiles_n = (uint32_t)((c.N + v.bn - 1) / v.bn);
  const int64_t tiles = (int64_t)p.tiles_m * p.batches * p.tiles_n;
  if (tiles > kMaxRows) return FN_ERR_INVALID_ARG;
  p.tiles = (uint32_t)tiles;
  p.group = 8;
  p.div_band = fused_norm_impl::make_div_u32(p.group * p.tiles_n);
  p.div_tiles_m = fused_norm_impl::make_div_u32(p.tiles_m);
  p.steps = (uint32_t)steps;
  // fp32 sums (bit 4), operand types (fp16 0, bf16 1; e4m3 0), N / 8 at bit 17, M / 16 at bit 24
  const uint32_t type = c.dtype == BO_BF16 ? 1u : 0u;
  p.idesc = 1u << 4 | type << 7 | type << 10 | (uint32_t)(v.bn / 8) << 17 | (uint32_t)(kTileM * v.cg / 16) << 24;

  const int out_type = c.dtype == BO_FP16 ? BO_FP16 : BO_BF16, per_step = kStepBytes / size;
  CUtensorMap mx, mw, mo = {}, mr;
  fn_status s = encode(&mx, c.dtype, matrix(a->x.ptr, c.K, a->x.stride_b, a->x.stride_l), per_step, kTileM, CU_TENSOR_MAP_SWIZZLE_128B);
  if (s == FN_OK)
    s = encode(&mw, c.dtype, Matrix{a->weight, c.K, c.N, a->weight_stride, 1, 0}, per_step, v.bn / v.cg, CU_TENSOR_MAP_SWIZZLE_128B);
  if (s == FN_OK && parts == 1)
    s = encode(&mo, out_type, matrix(a->out, c.N, a->out_stride_b, a->out_stride_l), kBox, kBox, CU_TENSOR_MAP_SWIZZLE_64B);
  mr = mo;
  if (s == FN_OK && parts == 1 && c.has_residual)
    s = encode(&mr, out_type, matrix(a->residual.ptr, c.N, a->residual.stride_b, a->residual.stride_l), kBox, kBox,
               CU_TENSOR_MAP_SWIZZLE_64B);
  if (s != FN_OK) return s;

  void* kernel = v.kernel[c.dtype];
  e = cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, v.shared);
  if (e != cudaSuccess) return launch_status(e);
  const int64_t resident = sms / v.cg;  // a split tile's CTAs are not persistent
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3((unsigned)((tiles < resident || parts > 1 ? tiles : resident) * v.cg * parts));
  cfg.blockDim = dim3(kMatrixThreads);
  cfg.dynamicSmemBytes = v.shared;
  cfg.stream = stream;
  cudaLaunchAttribute cluster;
  cluster.id = cudaLaunchAttributeClusterDimension;
  cluster.val.clusterDim.x = v.cg * parts, cluster.val.clusterDim.y = 1, cluster.val.clusterDim.z = 1;
  cfg.attrs = &cluster;
  cfg.numAttrs = v.cg * parts > 1 ? 1 : 0;
  void* args[] = {&p, &mx, &mw, &mo, &mr};  // the first three where K is split
  return launch_status(cudaLaunchKernelExC(&cfg, kernel, args));
}

}  // namespace

extern "C" {

fn_status linear_gate_create(linear_gate_t* out, const lg_config* cfg) {
  if (!out || !cfg) return FN_ERR_INVALID_ARG;
  const lg_config& c = *cfg;
  for (int v : {c.has_bias, c.has_gate, c.has_residual})
    if (!is_flag(v)) return FN_ERR_INVALID_ARG;
  if (c.act < BO_ACT_NONE || c.act > BO_ACT_GELU_TANH) return FN_ERR_INVALID_ARG;
  if (c.dtype != BO_BF16 && c.dtype != BO_FP16 && c.dtype != BO_E4M3) return FN_ERR_UNSUPPORTED;
  if (c.K < 8 || c.N < 8 || c.K > kMaxWidth || c.N > kMaxWidth || c.N % 8 || c.K % (16 / element_size(c))) return FN_ERR_UNSUPPORTED;
  linear_gate_s* h = new (std::nothrow) linear_gate_s;
  if (!h) return FN_ERR_INVALID_ARG;
  h->cfg = c;
  *out = h;
  return FN_OK;
}

fn_status linear_gate_validate(linear_gate_t h, const lg_args* a) { return validate(h, a); }

fn_status linear_gate_launch(linear_gate_t h, const lg_args* a, fn_stream_t stream) {
  const fn_status s = validate(h, a);
  if (s != FN_OK || a->B == 0 || a->L == 0) return s;
  LinearParams p = make_params(h, a);
  const cudaError_t e = gave_up_word(&p.gave_up);
  if (e != cudaSuccess) return launch_status(e);
  const fn_status before = wait_status(p.gave_up);
  if (before != FN_OK) return before;
  if (p.rows <= (uint32_t)kTokens) return launch_tokens(h, p, reinterpret_cast<cudaStream_t>(stream));
  return launch_tiles(h, a, p, reinterpret_cast<cudaStream_t>(stream));
}

fn_status linear_gate_timeouts(int* count) {
  if (!count) return FN_ERR_INVALID_ARG;
  return launch_status(cudaMemcpyFromSymbol(count, linear_gate_gave_up, sizeof(int)));
}

fn_status linear_gate_destroy(linear_gate_t h) {
  delete h;
  return FN_OK;
}

}  // extern "C"
