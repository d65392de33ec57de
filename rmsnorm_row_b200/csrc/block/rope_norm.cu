// Host side of rope_norm (checks, shapes, launches) and the sum of dweight's partials.
#include <atomic>
#include <cmath>
#include <cstring>
#include <new>
#include <utility>

#include "host_checks.h"
#include "rope_norm_kernel.cuh"

namespace block_ops {
namespace {

// dweight[c] = the partials' sum over CTAs, in fp64, in a fixed order: kSlices slices of the CTAs
// per column, then the slices.
constexpr int kSlices = 32;
__global__ void __launch_bounds__(32 * kSlices) sum_partials(const float* partial, int parts, int n, float* out) {
  __shared__ double slices[kSlices][32];
  const int c = blockIdx.x * 32 + threadIdx.x;
  double s = 0.0;
  if (c < n)
#pragma unroll 8
    for (int i = threadIdx.y; i < parts; i += kSlices) s += (double)__ldcg(partial + (size_t)i * n + c);
  slices[threadIdx.y][threadIdx.x] = s;
  __syncthreads();
  if (threadIdx.y == 0 && c < n) {
#pragma unroll
    for (int i = 1; i < kSlices; ++i) s += slices[i][threadIdx.x];
    out[c] = (float)s;
  }
}

struct RopeShape {
  int W, T, G, nh, rows_per_cta;
  RopeKernel kernel;
  size_t smem;
  int stages;
};
constexpr size_t kMaxShared = 227 * 1024;  // of a CTA

int lanes_of(int hd) {
  int W = 1;
  while (W < hd / 16) W *= 2;
  return W;
}
RopeShape shared_warps(int H, int W) {  // a row of up to 32 lanes
  int T = 1;
  while (T < H * W) T *= 2;
  return RopeShape{W, T, T / W, 1, kSharedRows / T, nullptr, 0, 0};
}

// Forward: a warp to a row where a lane can hold its part of it (10 heads, 80 registers), or in
// the case of a norm that is not over all heads, in passes of four; CTAs of several warps for
// longer rows. With `few` rows, the warps of a CTA share a row two heads to a lane; both add up
// squares in the same order.
RopeShape forward_shape(int H, int hd, int norm, bool few) {
  const int W = lanes_of(hd), G = 32 / W, need = (H + G - 1) / G;
  if (H * W <= 32) return shared_warps(H, W);
  RopeShape s{W, 32, G, 2, kSharedRows / 32, nullptr, 0, 0};
  int P = 1;
  if (norm == BO_NORM_ALL && need > 10) {
    P = 0;
    for (int nh : {10, 6, 4}) {
      const int n = (need + nh - 1) / nh;
      if (P == 0 || (n <= kForwardThreads / 32 && n * nh < P * s.nh)) P = n, s.nh = nh;
    }
  } else if (few) {
    P = (need + 1) / 2 < kForwardThreads / 32 ? (need + 1) / 2 : kForwardThreads / 32;
  } else if (norm == BO_NORM_ALL) {
    s.nh = need <= 2 ? 2 : need <= 4 ? 4 : need <= 6 ? 6 : 10;
  } else {
    s.nh = need <= 2 ? 2 : 4;
  }
  s.T = 32 * P;
  if (P > 1) s.rows_per_cta = 1;
  return s;
}

// Gradient: rows of more than 32 lanes take the number of heads per thread (1, 2 or 4) that
// leaves the fewest idle lanes, 2 where it is even.
RopeShape backward_shape(int H, int hd) {
  const int W = lanes_of(hd);
  if (H * W <= 32) return shared_warps(H, W);
  RopeShape s{W, 0, 0, 0, 0, nullptr, 0, 0};
  for (int nh : {2, 1, 4}) {
    const int T = ((H + nh - 1) / nh * W + 31) / 32 * 32;
    if (T <= kRopeThreads && (s.T == 0 || T * nh < s.T * s.nh)) s.T = T, s.nh = nh;
  }
  s.G = s.T / W;
  s.rows_per_cta = s.T > 32 ? 1 : kSharedRows / s.T;
  return s;
}

}  // namespace
}  // namespace block_ops

using namespace block_ops;

struct rope_norm_s {
  rn_config cfg;
  RopeShape shape[3];  // kForward, kFew, kGradient
  RopeParams base;  // the parts of the launch parameters that the configuration settles
  mutable std::atomic<int> resident[3] = {{0}, {0}, {0}};  // CTAs per SM of the kernels, once known
};

namespace {

int weight_values(const rn_config& c) { return c.norm == BO_NORM_ALL ? c.heads * c.head_dim : c.head_dim; }
enum { kForward = 0, kFew = 1, kGradient = 2 };
// Rows up to which the warps of a CTA share one (40 heads of 128: 296 rows 6.0 against 8.4 us, 592
// rows 7.9 against 8.7; the same from 1184 to 2368, slower beyond: 9472 rows 50 against 43).
constexpr int kFewPerSm = 4;
bool sums_dweight(const rn_config& c) { return c.has_weight != 0; }

bool rows_extent(const rn_rows& r, int64_t B, int64_t L, const rn_config& c, Span* out) {
  const int64_t n[3] = {B, L, c.heads}, s[3] = {r.stride_b, r.stride_l, r.stride_h};
  const int64_t e = extent_of(n, s, c.head_dim);
  if (e < 0) return false;
  *out = bytes_at(r.ptr, (uint64_t)e * 2);
  return true;
}

void check_rows(const rn_rows& r, Findings& f) {
  f.require(r.stride_b >= 0 && r.stride_l >= 0 && r.stride_h >= 0, FN_ERR_INVALID_ARG);
  f.require(aligned16(r.ptr) && r.stride_b % 8 == 0 && r.stride_l % 8 == 0 && r.stride_h % 8 == 0, FN_ERR_MISALIGNED);
}

// Output rows: no two (b, l, h) share a byte, whichever of the three strides is the largest.
void check_out(const rn_rows& r, int64_t B, int64_t L, const rn_config& c, Findings& f) {
  check_rows(r, f);
  int64_t n[3] = {B, L, c.heads}, s[3] = {r.stride_b, r.stride_l, r.stride_h};
  __int128 width = c.head_dim;  // of what the dimensions so far span
  for (int done = 0; done < 3; ++done) {
    int at = done;
    for (int i = done + 1; i < 3; ++i)
      if (n[at] == 1 || (n[i] > 1 && s[i] < s[at])) at = i;
    std::swap(n[at], n[done]);
    std::swap(s[at], s[done]);
    if (n[done] == 1) continue;
    f.require((__int128)s[done] >= width, FN_ERR_INVALID_ARG);
    width += (__int128)(n[done] - 1) * s[done];
  }
}

bool same_places(const rn_rows& a, const rn_rows& b, int64_t B, int64_t L, int H) {
  return a.ptr == b.ptr && (B == 1 || a.stride_b == b.stride_b) && (L == 1 || a.stride_l == b.stride_l) &&
         (H == 1 || a.stride_h == b.stride_h);
}

// What both directions check: sizes, positions, weight, the inputs against the output.
fn_status check(const rope_norm_s* h, int64_t B, int64_t L, const rn_rows* const (&ins)[2], const rn_rows& out,
                const void* positions, int64_t psb, int64_t psl, const void* weight, const Span& dweight, const Span& work) {
  const rn_config& c = h->cfg;
  Findings f;
  f.require(positions && out.ptr, FN_ERR_INVALID_ARG);
  f.require((weight != nullptr) == (c.has_weight != 0), FN_ERR_INVALID_ARG);
  f.require(psb >= 0 && psl >= 0, FN_ERR_INVALID_ARG);
  f.require(reinterpret_cast<uintptr_t>(positions) % (c.index64 ? 8 : 4) == 0, FN_ERR_MISALIGNED);
  f.require(aligned16(weight), FN_ERR_MISALIGNED);
  for (const rn_rows* r : ins)
    if (r) check_rows(*r, f);
  check_out(out, B, L, c, f);
  if (f.status != FN_OK) return f.status;

  Span o;
  if (!rows_extent(out, B, L, c, &o)) return FN_ERR_INVALID_ARG;
  const int64_t n[2] = {B, L}, ps[2] = {psb, psl};
  const int64_t pe = extent_of(n, ps, c.axes);
  if (pe < 0) return FN_ERR_INVALID_ARG;
  const Span pos = bytes_at(positions, (uint64_t)pe * (c.index64 ? 8 : 4));
  const Span w = bytes_at(weight, weight ? (uint64_t)weight_values(c) * (c.weight_fp32 ? 4 : 2) : 0);
  const Span written[3] = {o, dweight, work};
  for (int i = 0; i < 3; ++i) {
    if (overlaps(written[i], pos) || overlaps(written[i], w)) return FN_ERR_INVALID_ARG;
    for (int j = 0; j < i; ++j)
      if (overlaps(written[i], written[j])) return FN_ERR_INVALID_ARG;
  }
  for (const rn_rows* r : ins) {
    if (!r) continue;
    Span s;
    if (!rows_extent(*r, B, L, c, &s)) return FN_ERR_INVALID_ARG;
    if (overlaps(o, s) && !same_places(*r, out, B, L, c.heads)) return FN_ERR_INVALID_ARG;
    if (overlaps(dweight, s) || overlaps(work, s)) return FN_ERR_INVALID_ARG;
  }
  return FN_OK;
}

// Sizes alone: FN_OK with *empty set when there is nothing to do.
fn_status check_sizes(const rope_norm_s* h, int64_t B, int64_t L, bool* empty) {
  if (B < 0 || L < 0) return FN_ERR_INVALID_ARG;
  *empty = B == 0 || L == 0;
  if (*empty) return FN_OK;
  if (B > kMaxRows || L > kMaxRows || B * L > kMaxRows) return FN_ERR_INVALID_ARG;
  if ((__int128)B * L * h->cfg.heads * h->cfg.head_dim > kMaxExtent) return FN_ERR_INVALID_ARG;
  return FN_OK;
}

fn_status validate(const rope_norm_s* h, const rn_args* a, bool* empty) {
  if (!h || !a) return FN_ERR_INVALID_ARG;
  const fn_status s = check_sizes(h, a->B, a->L, empty);
  if (s != FN_OK || *empty) return s;
  if (!a->x.ptr) return FN_ERR_INVALID_ARG;
  const rn_rows* ins[2] = {&a->x, nullptr};
  return check(h, a->B, a->L, ins, a->y, a->positions, a->pos_stride_b, a->pos_stride_l, a->weight, Span{}, Span{});
}

int64_t ctas(const RopeShape& s, int64_t rows) { return (rows + s.rows_per_cta - 1) / s.rows_per_cta; }

uint64_t workspace_bytes(const rope_norm_s* h, int64_t rows) {
  if (!sums_dweight(h->cfg) || rows == 0) return 0;
  const int64_t n = ctas(h->shape[kGradient], rows);
  return (uint64_t)(n < kMaxPartials ? n : kMaxPartials) * weight_values(h->cfg) * sizeof(float);
}

fn_status validate(const rope_norm_s* h, const rn_backward_args* a, bool* empty) {
  if (!h || !a) return FN_ERR_INVALID_ARG;
  const rn_config& c = h->cfg;
  const fn_status s = check_sizes(h, a->B, a->L, empty);
  if (s != FN_OK) return s;
  if ((a->dweight != nullptr) != sums_dweight(c)) return FN_ERR_INVALID_ARG;
  if (reinterpret_cast<uintptr_t>(a->dweight) % 4) return FN_ERR_MISALIGNED;
  if (*empty) return FN_OK;
  if (!a->grad.ptr || (a->x.ptr != nullptr) != (c.norm != BO_NORM_NONE)) return FN_ERR_INVALID_ARG;
  const uint64_t need = workspace_bytes(h, a->B * a->L);
  if (need && (!a->workspace || a->workspace_bytes < need)) return FN_ERR_INVALID_ARG;
  if (need && !aligned16(a->workspace)) return FN_ERR_MISALIGNED;
  const rn_rows* ins[2] = {&a->grad, c.norm != BO_NORM_NONE ? &a->x : nullptr};
  return check(h, a->B, a->L, ins, a->dx, a->positions, a->pos_stride_b, a->pos_stride_l, a->weight,
               bytes_at(a->dweight, a->dweight ? 4 * (uint64_t)weight_values(c) : 0), bytes_at(a->workspace, need));
}

RopeRows rows_of(const rn_rows& r) {
  return RopeRows{static_cast<const uint16_t*>(r.ptr), r.stride_b, r.stride_l, r.stride_h};
}

// Above 48 KB a kernel's shared memory is asked for: all there is, whatever the handle needs, since
// another host thread may be launching the same kernel for a handle that needs more.
cudaError_t allow_shared(const RopeShape& s) {
  if (s.smem <= 48 * 1024) return cudaSuccess;
  return cudaFuncSetAttribute(s.kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, (int)kMaxShared);
}

fn_status sms_of(int* sms) {
  int device = 0;
  cudaError_t e = cudaGetDevice(&device);
  if (e == cudaSuccess) e = cudaDeviceGetAttribute(sms, cudaDevAttrMultiProcessorCount, device);
  return e == cudaSuccess ? FN_OK : launch_status(e);
}

// The number of CTAs: what the current device holds at once, at most one per rows_per_cta rows.
fn_status grid_of(const rope_norm_s* h, int which, int64_t rows, int sms, int* grid) {
  const RopeShape& s = h->shape[which];
  int per_sm = h->resident[which].load(std::memory_order_relaxed);
  if (per_sm == 0) {
    cudaError_t e = allow_shared(s);
    if (e == cudaSuccess) e = cudaOccupancyMaxActiveBlocksPerMultiprocessor(&per_sm, s.kernel, s.T * s.rows_per_cta, s.smem);
    if (e != cudaSuccess) return launch_status(e);
    if (per_sm < 1) per_sm = 1;
    h->resident[which].store(per_sm, std::memory_order_relaxed);
  }
  int64_t g = (int64_t)per_sm * sms;
  if (which == kGradient && g > kMaxPartials) g = kMaxPartials;
  const int64_t n = ctas(s, rows);
  *grid = (int)(g < n ? g : n);
  return FN_OK;
}

fn_status run(const rope_norm_s* h, int which, RopeParams& p, int64_t B, int64_t L, const void* positions, int64_t psb,
              int64_t psl, const void* weight, const rn_rows& out, int sms, cudaStream_t stream, int* grid) {
  const RopeShape& s = h->shape[which];
  fn_status st = grid_of(h, which, B * L, sms, grid);
  if (st != FN_OK) return st;
  p.W = s.W, p.T = s.T, p.G = s.G, p.stages = s.stages;
  p.out = rows_of(out);
  p.positions = positions, p.pos_sb = psb, p.pos_sl = psl;
  p.weight = weight;
  p.L = (uint32_t)L;
  p.div_L = fused_norm_impl::make_div_u32(p.L);
  const cudaError_t e = allow_shared(s);
  if (e != cudaSuccess) return launch_status(e);
  cudaLaunchConfig_t cfg = {};
  cfg.blockDim = dim3(s.T * s.rows_per_cta);
  cfg.dynamicSmemBytes = s.smem;
  cfg.stream = stream;
  // A thread sums dweight in fp32 over its rows: a launch goes over so many that the sum's error
  // does not grow with the tokens, and the parts of several launches are added up (227,000 tokens of
  // 40 heads of 128 are the most of one; flushing the sums every 64 rows inside the kernel cost it
  // registers, 757 against 580 us at 90000 tokens).
  const int64_t rows = B * L, turn = (int64_t)*grid * s.rows_per_cta, turns = (rows + turn - 1) / turn;
  const int64_t launches = which == kGradient && p.partial ? (turns + kMaxTurns - 1) / kMaxTurns : 1;
  const int64_t each = (turns + launches - 1) / launches * turn;
  for (int64_t first = 0; first < rows; first += each) {
    const int64_t n = rows - first < each ? rows - first : each, own = ctas(s, n);
    p.first = (uint32_t)first, p.rows = (uint32_t)(first + n), p.add = first > 0;
    cfg.gridDim = dim3((unsigned)(own < *grid ? own : *grid));
    st = launch_status(cudaLaunchKernelEx(&cfg, s.kernel, p));
    if (st != FN_OK) return st;
  }
  return FN_OK;
}

// The forward kernel over x, which also turns a gradient back (SIGN -1) where there is no norm.
fn_status run_forward(const rope_norm_s* h, const rn_rows& x, float sign, int64_t B, int64_t L, const void* positions, int64_t psb,
                      int64_t psl, const void* weight, const rn_rows& out, cudaStream_t stream) {
  int sms, grid;
  const fn_status s = sms_of(&sms);
  if (s != FN_OK) return s;
  RopeParams p = h->base;
  p.x = rows_of(x);
  p.sign = sign;
  return run(h, B * L <= (int64_t)kFewPerSm * sms ? kFew : kForward, p, B, L, positions, psb, psl, weight, out, sms, stream, &grid);
}

}  // namespace

extern "C" {

fn_status rope_norm_create(rope_norm_t* out, const rn_config* cfg) {
  if (!out || !cfg) return FN_ERR_INVALID_ARG;
  const rn_config& c = *cfg;
  for (int v : {c.has_weight, c.weight_fp32, c.half_pairs, c.shared_frequencies, c.index64})
    if (!is_flag(v)) return FN_ERR_INVALID_ARG;
  if (c.norm < BO_NORM_NONE || c.norm > BO_NORM_ALL) return FN_ERR_INVALID_ARG;
  if (c.has_weight && c.norm == BO_NORM_NONE) return FN_ERR_INVALID_ARG;
  if (c.weight_fp32 && !c.has_weight) return FN_ERR_INVALID_ARG;
  if (!std::isfinite(c.theta) || c.theta <= 0.0 || !std::isfinite(c.eps) || c.eps < 0.0 || c.eps > 0x1p100) return FN_ERR_INVALID_ARG;
  if (c.axes < 1 || c.axes > 4 || c.heads < 1 || c.head_dim < 1) return FN_ERR_INVALID_ARG;
  int64_t pairs = 0;
  for (int a = 0; a < c.axes; ++a) {
    if (c.section[a] < 1) return FN_ERR_INVALID_ARG;
    pairs += c.section[a];
  }
  if (pairs > c.head_dim / 2) return FN_ERR_INVALID_ARG;
  if (c.dtype != BO_BF16 && c.dtype != BO_FP16) return FN_ERR_UNSUPPORTED;
  if (c.head_dim % 16 || c.head_dim > 2 * kMaxPairs || (int64_t)c.heads * c.head_dim > 16384) return FN_ERR_UNSUPPORTED;
  if (c.half_pairs && pairs % 8) return FN_ERR_UNSUPPORTED;
  rope_norm_s* h = new (std::nothrow) rope_norm_s;
  if (!h) return FN_ERR_INVALID_ARG;
  h->cfg = c;
  const bool pass = 2 * pairs < c.head_dim;
  const int units = c.norm != BO_NORM_NONE ? weight_values(c) / 16 : 0, weights = weight_floats(units);
  for (int i : {kForward, kFew, kGradient}) {
    RopeShape& s = h->shape[i];
    s = i == kGradient ? backward_shape(c.heads, c.head_dim) : forward_shape(c.heads, c.head_dim, c.norm, i == kFew);
    if (i != kGradient) {
      s.kernel = c.dtype == BO_FP16 ? pick_rope<true>(s.nh, c.norm, c.half_pairs, pass) : pick_rope<false>(s.nh, c.norm, c.half_pairs, pass);
      s.smem = forward_shared_bytes(s.rows_per_cta, c.head_dim, weights);
    } else if (c.norm != BO_NORM_NONE) {
      s.kernel = c.dtype == BO_FP16 ? pick_rope_gradient<true>(s.nh, c.norm, c.half_pairs, sums_dweight(c), pass)
                                    : pick_rope_gradient<false>(s.nh, c.norm, c.half_pairs, sums_dweight(c), pass);
      for (s.stages = 2; s.stages >= 1; --s.stages) {
        s.smem = backward_shared_bytes(s.rows_per_cta, c.head_dim, weights, s.T * s.rows_per_cta, s.nh, s.stages);
        if (s.smem <= kMaxShared) break;
      }
    }
  }
  RopeParams& p = h->base;
  std::memset(&p, 0, sizeof(p));
  p.H = c.heads, p.hd = c.head_dim, p.units = c.head_dim / 16, p.pairs = (int)pairs;
  p.sign = 1.0f;
  p.index64 = c.index64, p.weight_fp32 = c.weight_fp32;
  p.weight_sh = c.norm == BO_NORM_ALL ? c.head_dim / 16 : 0;
  p.weight_units = units;
  p.inv_n64 = 1.0 / (c.norm == BO_NORM_ALL ? c.heads * c.head_dim : c.head_dim), p.eps64 = c.eps;
  p.inv_n = (float)p.inv_n64, p.eps = (float)c.eps;
  int i = 0;
  for (int a = 0; a < c.axes; ++a)
    for (int k = 0; k < c.section[a]; ++k, ++i) {
      const double part = c.shared_frequencies ? (double)i / (double)pairs : (double)k / c.section[a];
      p.turns[i] = std::pow(c.theta, -part) / 6.283185307179586476925;
      p.axis[i] = (uint8_t)a;
    }
  *out = h;
  return FN_OK;
}

fn_status rope_norm_validate(rope_norm_t h, const rn_args* a) {
  bool empty;
  return validate(h, a, &empty);
}

fn_status rope_norm_launch(rope_norm_t h, const rn_args* a, fn_stream_t stream) {
  bool empty;
  const fn_status s = validate(h, a, &empty);
  if (s != FN_OK || empty) return s;
  return run_forward(h, a->x, 1.0f, a->B, a->L, a->positions, a->pos_stride_b, a->pos_stride_l, a->weight, a->y,
                     reinterpret_cast<cudaStream_t>(stream));
}

fn_status rope_norm_backward_workspace(rope_norm_t h, int64_t B, int64_t L, uint64_t* bytes) {
  if (!h || !bytes) return FN_ERR_INVALID_ARG;
  bool empty;
  const fn_status s = check_sizes(h, B, L, &empty);
  if (s == FN_OK) *bytes = empty ? 0 : workspace_bytes(h, B * L);
  return s;
}

fn_status rope_norm_backward_validate(rope_norm_t h, const rn_backward_args* a) {
  bool empty;
  return validate(h, a, &empty);
}

fn_status rope_norm_backward_launch(rope_norm_t h, const rn_backward_args* a, fn_stream_t stream_) {
  bool empty;
  fn_status s = validate(h, a, &empty);
  if (s != FN_OK) return s;
  const cudaStream_t stream = reinterpret_cast<cudaStream_t>(stream_);
  const int n = weight_values(h->cfg);
  if (empty)
    return a->dweight ? launch_status(cudaMemsetAsync(a->dweight, 0, (size_t)n * 4, stream)) : FN_OK;
  if (h->cfg.norm == BO_NORM_NONE)
    return run_forward(h, a->grad, -1.0f, a->B, a->L, a->positions, a->pos_stride_b, a->pos_stride_l, nullptr, a->dx, stream);
  int sms, grid;
  s = sms_of(&sms);
  if (s != FN_OK) return s;
  RopeParams p = h->base;
  p.x = rows_of(a->x), p.dy = rows_of(a->grad);
  p.partial = static_cast<float*>(a->workspace);
  s = run(h, kGradient, p, a->B, a->L, a->positions, a->pos_stride_b, a->pos_stride_l, a->weight, a->dx, sms, stream, &grid);
  if (s != FN_OK || !a->dweight) return s;
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3((n + 31) / 32);
  cfg.blockDim = dim3(32, kSlices);
  cfg.stream = stream;
  return launch_status(cudaLaunchKernelEx(&cfg, sum_partials, (const float*)p.partial, grid, n, a->dweight));
}

fn_status rope_norm_destroy(rope_norm_t h) {
  delete h;
  return FN_OK;
}

}  // extern "C"
