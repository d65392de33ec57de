// Residual / gate / norm / modulation rows with an e4m3 output and one scale per row
// (contract: include/block_ops.h, norm_quant).
//
// Mathematics, per row of D channels: r = bf16(residual + gate x); n = (r - mu) rho (mu = 0
// for RMSNorm), rho = 1 / sqrt(var + eps); y = (n w + b)(1 + scale) + shift; a = max |y|;
// row_scale = a / 448; q = e4m3(y 448 / a).
//
// Bound: HBM. A row moves 2 (x) + 2 (residual) + 2 (r) + 1 (q) bytes per element, plus 4 with
// per-token modulation, against ~15 fp32 operations. The row therefore stays in registers
// from its only read to its only write: as packed bf16 for the statistics, as fp32 from the
// norm to the quantisation (the scale needs the whole row's maximum first).
//
// Layout: thread t of the row's T threads owns the 16-byte vectors t, t + T, ... (every warp
// access is 512 contiguous bytes). Rows of up to 1024 channels take one warp each, eight rows
// to a CTA, and reduce through shuffles alone; longer rows take one CTA of T threads with NV
// vectors each and one barrier per reduction (statistics, then the maximum).
#include <cuda_fp8.h>

#include <cmath>
#include <cstring>
#include <new>

#include "../fused_norm_kernel.cuh"
#include "host_checks.h"

namespace block_ops {
namespace {

using namespace fused_norm_impl;  // row addressing, 16-byte loads, bf16 and paired-fp32 arithmetic

struct QuantParams {
  const uint16_t *x, *res, *gate, *scale, *shift;
  const void *weight, *bias;
  uint8_t* q;
  float* row_scale;
  uint16_t* r;
  int64_t x_sb, x_sf, x_sl, res_sb, res_sf, res_sl, gate_sb, gate_sf, gate_sl;
  int64_t scale_sb, scale_sf, scale_sl, shift_sb, shift_sf, shift_sl;
  int64_t q_sb, q_sl, r_sb, r_sl;
  uint32_t rows, L, tpf;
  DivU32 div_L, div_tpf;
  uint32_t vecs;  // D / 8
  uint32_t stream_mask;
  uint32_t affine_fp32;
  double inv_d;  // 1 / D
  double eps;
};

constexpr int kMaxWarps = 16;  // of a row: T <= 512
constexpr int kRowsPerCta = 8;  // rows of one warp each

// Sums over the row's threads, the same value in each of them. `slot` is shared memory of a
// CTA-wide row that nothing else has used since the last barrier.
template <bool WARP_ROW>
__device__ __forceinline__ double row_sum(double v, double* slot) {
#pragma unroll
  for (int o = 16; o >= 1; o >>= 1) v += __shfl_xor_sync(0xFFFFFFFFu, v, o);
  if (WARP_ROW) return v;
  const int warps = blockDim.x >> 5;
  if ((threadIdx.x & 31) == 0) slot[threadIdx.x >> 5] = v;
  __syncthreads();
  double t = slot[0];
  for (int w = 1; w < warps; ++w) t += slot[w];
  return t;
}

// Bits of the largest |y| over the row's threads. Magnitudes order as unsigned integers, and
// a NaN's lie above infinity's: a NaN anywhere makes the row's maximum a NaN.
template <bool WARP_ROW>
__device__ __forceinline__ uint32_t row_max(uint32_t v, uint32_t* slot) {
  v = __reduce_max_sync(0xFFFFFFFFu, v);
  if (WARP_ROW) return v;
  const int warps = blockDim.x >> 5;
  if ((threadIdx.x & 31) == 0) slot[threadIdx.x >> 5] = v;
  __syncthreads();
  uint32_t t = slot[0];
  for (int w = 1; w < warps; ++w) t = max(t, slot[w]);
  return t;
}

__device__ __forceinline__ uint64_t widen(uint32_t pair) { return pk2(lo_f(pair), hi_f(pair)); }

// Eight affine values as four fp32 pairs.
__device__ __forceinline__ void load_affine(const void* p, bool fp32, int j, uint64_t (&out)[4]) {
  if (fp32) {
    const float4* f = reinterpret_cast<const float4*>(p) + 2 * j;
    const float4 a = __ldg(f), c = __ldg(f + 1);
    out[0] = pk2(a.x, a.y), out[1] = pk2(a.z, a.w), out[2] = pk2(c.x, c.y), out[3] = pk2(c.z, c.w);
  } else {
    const uint4 a = __ldg(reinterpret_cast<const uint4*>(p) + j);
#pragma unroll
    for (int i = 0; i < 4; ++i) out[i] = widen(word(a, i));
  }
}

template <int NV, bool IS_RMS, bool ROW_MOD, bool WARP_ROW>
__global__ void __launch_bounds__(WARP_ROW ? 32 * kRowsPerCta : 512)
norm_quant_rows(const QuantParams p) {
  __shared__ double sums[4][kMaxWarps];
  __shared__ uint32_t tops[kMaxWarps];
  const uint32_t row = WARP_ROW ? blockIdx.x * kRowsPerCta + threadIdx.y : blockIdx.x;
  if (WARP_ROW && row >= p.rows) return;  // whole warps
  const int tid = threadIdx.x, T = WARP_ROW ? 32 : blockDim.x;
  const uint32_t b = div_u32(row, p.div_L), l = row - b * p.L;
  const uint32_t f = p.tpf > 0 ? div_u32(l, p.div_tpf) : 0u;
  auto has = [&](int k) { return (uint32_t)(tid + k * T) < p.vecs; };

  // ---- the row: r = residual + gate x, or x; packed bf16 in v -------------------------
  const uint16_t* xr = p.x + (b * p.x_sb + f * p.x_sf + l * p.x_sl);
  uint4 v[NV];
#pragma unroll
  for (int k = 0; k < NV; ++k)
    v[k] = has(k) ? load_vec(xr, tid + k * T, p.stream_mask & kX) : make_uint4(0, 0, 0, 0);
  if (p.res) {
    const uint16_t* rr = p.res + (b * p.res_sb + f * p.res_sf + l * p.res_sl);
    uint16_t* ro = p.r + (b * p.r_sb + l * p.r_sl);
    uint4 rv[NV];
#pragma unroll
    for (int k = 0; k < NV; ++k)
      rv[k] = has(k) ? load_vec(rr, tid + k * T, p.stream_mask & kRes) : make_uint4(0, 0, 0, 0);
    if (p.gate) {
      const uint16_t* gr = p.gate + (b * p.gate_sb + f * p.gate_sf + l * p.gate_sl);
#pragma unroll
      for (int k = 0; k < NV; ++k)
        if (has(k)) v[k] = residual_vec<true>(rv[k], v[k], load_vec(gr, tid + k * T, p.stream_mask & kGate));
    } else {
#pragma unroll
      for (int k = 0; k < NV; ++k) v[k] = residual_vec<false>(rv[k], v[k], v[k]);
    }
#pragma unroll
    for (int k = 0; k < NV; ++k)
      if (has(k)) __stcs(reinterpret_cast<uint4*>(ro) + tid + k * T, v[k]);
  }

  // Modulation that changes from token to token is requested here, so that the statistics
  // hide its latency; broadcast rows come from L1 where they are used.
  const uint16_t* sr = p.scale ? p.scale + (b * p.scale_sb + f * p.scale_sf + l * p.scale_sl) : nullptr;
  const uint16_t* tr = p.scale ? p.shift + (b * p.shift_sb + f * p.shift_sf + l * p.shift_sl) : nullptr;
  uint4 sv[ROW_MOD ? NV : 1], tv[ROW_MOD ? NV : 1];
  if (ROW_MOD) {
#pragma unroll
    for (int k = 0; k < NV; ++k)
      if (has(k)) {
        sv[k] = load_vec(sr, tid + k * T, p.stream_mask & kScale);
        tv[k] = load_vec(tr, tid + k * T, p.stream_mask & kShift);
      }
  }

  // ---- statistics: fp32 within a thread (at most 40 elements), fp64 across threads ------
  // LayerNorm sums squares around the thread's own mean m, so nothing cancels in fp32:
  // sum r^2 = sum (r - m)^2 + m (2 S - n m), joined in fp64. An error of S enters the
  // variance only through its product with m - mu.
  double mu = 0.0, var;
  if (IS_RMS) {
    uint64_t acc[2] = {0, 0};
#pragma unroll
    for (int k = 0; k < NV; ++k)  // vectors past the row's end are zero
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        const uint64_t e = widen(word(v[k], i));
        acc[i & 1] = fma2(e, e, acc[i & 1]);
      }
    float a0, a1;
    upk2(add2(acc[0], acc[1]), a0, a1);
    var = row_sum<WARP_ROW>((double)a0 + (double)a1, sums[0]) * p.inv_d;
  } else {
    uint64_t acc[2] = {0, 0};
    int n = 0;
#pragma unroll
    for (int k = 0; k < NV; ++k) {
      n += has(k) ? 8 : 0;
#pragma unroll
      for (int i = 0; i < 4; ++i) acc[i & 1] = add2(acc[i & 1], widen(word(v[k], i)));
    }
    float a0, a1;
    upk2(add2(acc[0], acc[1]), a0, a1);
    const float S = a0 + a1, m = n ? S / (float)n : 0.0f;
    acc[0] = acc[1] = 0;
#pragma unroll
    for (int k = 0; k < NV; ++k)
      if (has(k)) {
#pragma unroll
        for (int i = 0; i < 4; ++i) {
          const uint64_t d = add2(widen(word(v[k], i)), pk2(-m, -m));
          acc[i & 1] = fma2(d, d, acc[i & 1]);
        }
      }
    upk2(add2(acc[0], acc[1]), a0, a1);
    double s1 = S, s2 = ((double)a0 + (double)a1) + (double)m * (2.0 * S - (double)n * m);
#pragma unroll
    for (int o = 16; o >= 1; o >>= 1) {
      s1 += __shfl_xor_sync(0xFFFFFFFFu, s1, o);
      s2 += __shfl_xor_sync(0xFFFFFFFFu, s2, o);
    }
    if (!WARP_ROW) {
      if ((tid & 31) == 0) sums[0][tid >> 5] = s1, sums[1][tid >> 5] = s2;
      __syncthreads();
      s1 = sums[0][0], s2 = sums[1][0];
      for (int w = 1; w < (T >> 5); ++w) s1 += sums[0][w], s2 += sums[1][w];
    }
    mu = s1 * p.inv_d;
    var = s2 * p.inv_d - mu * mu;
  }
  // Rows that fp32 does not serve (squares near its limits, a spread below 1/32 of the
  // mean, zeros, infinities, NaN) take their statistics from fp64, around the exact mean.
  // The branch is the same for all threads of a row. The thread reads its vectors again (its
  // own r stores, or x) in rolled loops: walking the registers here would set the register
  // allocation of the whole kernel (118-128 registers with spills, against 80).
  if (!(var >= 0x1p-80 && var <= 0x1p+100 && mu * mu <= 1024.0 * var)) {
    const uint4* again = reinterpret_cast<const uint4*>(p.res ? p.r + (b * p.r_sb + l * p.r_sl) : xr);
    double c = 0.0;
    if (!IS_RMS) {
#pragma unroll 1
      for (int j = tid; j < (int)p.vecs; j += T) {
        const uint4 u = __ldcg(again + j);
#pragma unroll
        for (int i = 0; i < 4; ++i) c += bf16_f64<0>(word(u, i)) + bf16_f64<1>(word(u, i));
      }
      mu = row_sum<WARP_ROW>(c, sums[2]) * p.inv_d;
      c = 0.0;
    }
#pragma unroll 1
    for (int j = tid; j < (int)p.vecs; j += T) {
      const uint4 u = __ldcg(again + j);
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        const double d0 = bf16_f64<0>(word(u, i)) - mu, d1 = bf16_f64<1>(word(u, i)) - mu;
        c = fma(d1, d1, fma(d0, d0, c));
      }
    }
    var = row_sum<WARP_ROW>(c, sums[3]) * p.inv_d;
  }
  const float rho = (float)rsqrt(var + p.eps);
  const float mu_hi = (float)mu, mu_lo = (float)(mu - (double)mu_hi);  // r - mu keeps fp32's precision

  // ---- y in fp32, and the row's largest magnitude ---------------------------------------
  uint64_t y[NV][4];
  uint32_t top = 0;
#pragma unroll
  for (int k = 0; k < NV; ++k) {
    const int j = tid + k * T;
    if (!has(k)) continue;
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      uint64_t d = widen(word(v[k], i));
      if (!IS_RMS) d = add2(add2(d, pk2(-mu_hi, -mu_hi)), pk2(-mu_lo, -mu_lo));
      y[k][i] = mul2(d, pk2(rho, rho));
    }
    if (p.weight) {
      uint64_t w[4];
      load_affine(p.weight, p.affine_fp32, j, w);
#pragma unroll
      for (int i = 0; i < 4; ++i) y[k][i] = mul2(y[k][i], w[i]);
    }
    if (p.bias) {
      uint64_t w[4];
      load_affine(p.bias, p.affine_fp32, j, w);
#pragma unroll
      for (int i = 0; i < 4; ++i) y[k][i] = add2(y[k][i], w[i]);
    }
    if (ROW_MOD || p.scale) {
      const uint4 s = ROW_MOD ? sv[k] : __ldg(reinterpret_cast<const uint4*>(sr) + j);
      const uint4 t = ROW_MOD ? tv[k] : __ldg(reinterpret_cast<const uint4*>(tr) + j);
#pragma unroll
      for (int i = 0; i < 4; ++i)
        y[k][i] = fma2(y[k][i], add2(widen(word(s, i)), pk2(1.0f, 1.0f)), widen(word(t, i)));
    }
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      float a0, a1;
      upk2(y[k][i], a0, a1);
      top = max(top, max(__float_as_uint(a0) & 0x7FFFFFFFu, __float_as_uint(a1) & 0x7FFFFFFFu));
    }
  }
  const float a = __uint_as_float(row_max<WARP_ROW>(top, tops));

  // ---- scale and quantise ------------------------------------------------------------------
  // The product with 448 / a stands for the quotient by row_scale: one rounding less than
  // dividing by the rounded row_scale. fmaxf would drop a NaN, so the floor is a comparison.
  const float a1 = a < 0x1p-100f ? 0x1p-100f : a;
  if (tid == 0) p.row_scale[row] = a == 0.0f ? 1.0f : a1 / 448.0f;
  const float inv = 448.0f / a1;
  uint8_t* qo = p.q + (b * p.q_sb + l * p.q_sl);
#pragma unroll
  for (int k = 0; k < NV; ++k) {
    if (!has(k)) continue;
    uint32_t h[4];
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      float2 e;
      upk2(mul2(y[k][i], pk2(inv, inv)), e.x, e.y);
      h[i] = __nv_cvt_float2_to_fp8x2(e, __NV_SATFINITE, __NV_E4M3);
    }
    __stcs(reinterpret_cast<uint2*>(qo) + tid + k * T, make_uint2(h[0] | h[1] << 16, h[2] | h[3] << 16));
  }
}

struct Shape {
  int nv, threads;
  bool warp_row;
};

// One warp per row up to 1024 channels; beyond, four or five vectors per thread, whichever
// leaves fewer lanes without a vector (five where both fit).
Shape shape_of(int D) {
  const int V = D / 8;
  if (V <= 128) return Shape{(V + 31) / 32, 32, true};
  const int t4 = (V + 127) / 128 * 32, t5 = (V + 159) / 160 * 32;
  return t5 * 5 <= t4 * 4 ? Shape{5, t5, false} : Shape{4, t4, false};
}

using Kernel = void (*)(QuantParams);

template <bool RMS, bool MOD>
Kernel pick(const Shape& s) {
  if (s.warp_row) {
    switch (s.nv) {
      case 1: return norm_quant_rows<1, RMS, MOD, true>;
      case 2: return norm_quant_rows<2, RMS, MOD, true>;
      case 3: return norm_quant_rows<3, RMS, MOD, true>;
      default: return norm_quant_rows<4, RMS, MOD, true>;
    }
  }
  return s.nv == 4 ? norm_quant_rows<4, RMS, MOD, false> : norm_quant_rows<5, RMS, MOD, false>;
}

}  // namespace
}  // namespace block_ops

using namespace block_ops;

struct norm_quant_s {
  nq_config cfg;
  Shape shape;
  Kernel kernel, kernel_row_mod;
};

namespace {

fn_status validate(const norm_quant_s* h, const nq_args* a) {
  if (!h || !a) return FN_ERR_INVALID_ARG;
  const nq_config& c = h->cfg;
  const int64_t B = a->B, L = a->L, D = c.D, tpf = a->tokens_per_frame;
  if (B < 0 || L < 0 || tpf < 0) return FN_ERR_INVALID_ARG;
  if (B == 0 || L == 0) return FN_OK;
  if (B > kMaxRows || L > kMaxRows || B * L > kMaxRows || (__int128)B * L * D > kMaxExtent) return FN_ERR_INVALID_ARG;
  if (tpf > 0 && L % tpf != 0) return FN_ERR_INVALID_ARG;
  const int64_t F = tpf > 0 ? L / tpf : 1;

  Findings f;
  f.require(a->x.ptr && a->q && a->row_scale, FN_ERR_INVALID_ARG);
  f.require((a->residual.ptr != nullptr) == (c.has_residual != 0) && (a->r != nullptr) == (c.has_residual != 0),
            FN_ERR_INVALID_ARG);
  f.require((a->gate.ptr != nullptr) == (c.has_gate != 0), FN_ERR_INVALID_ARG);
  f.require((a->scale.ptr != nullptr) == (c.has_modulation != 0), FN_ERR_INVALID_ARG);
  f.require((a->shift.ptr != nullptr) == (c.has_modulation != 0), FN_ERR_INVALID_ARG);
  f.require((a->weight != nullptr) == (c.has_weight != 0) && (a->bias != nullptr) == (c.has_bias != 0),
            FN_ERR_INVALID_ARG);
  const fn_operand* ins[5] = {&a->x, &a->residual, &a->gate, &a->scale, &a->shift};
  for (const fn_operand* o : ins)
    if (o->ptr) check_operand(*o, tpf > 0, f);
  f.require(aligned16(a->weight) && aligned16(a->bias), FN_ERR_MISALIGNED);
  f.require(reinterpret_cast<uintptr_t>(a->row_scale) % 4 == 0, FN_ERR_MISALIGNED);
  check_output(a->q, a->q_stride_b, a->q_stride_l, B, L, D, 16, f);
  if (c.has_residual) check_output(a->r, a->r_stride_b, a->r_stride_l, B, L, D, 8, f);
  if (f.status != FN_OK) return f.status;

  const int64_t n[2] = {B, L}, qs[2] = {a->q_stride_b, a->q_stride_l}, rs[2] = {a->r_stride_b, a->r_stride_l};
  const int64_t qe = extent_of(n, qs, D), re = c.has_residual ? extent_of(n, rs, D) : 0;
  if (qe < 0 || re < 0) return FN_ERR_INVALID_ARG;
  const Span outs[3] = {bytes_at(a->q, qe), bytes_at(a->row_scale, (uint64_t)B * L * 4), bytes_at(a->r, (uint64_t)re * 2)};
  for (int i = 0; i < 3; ++i)
    for (int j = 0; j < i; ++j)
      if (overlaps(outs[i], outs[j])) return FN_ERR_INVALID_ARG;
  const bool in_place = c.has_residual && same_rows(a->residual, a->r, a->r_stride_b, a->r_stride_l, B, L);
  for (const fn_operand* o : ins) {
    if (!o->ptr) continue;
    Span s;
    if (!operand_span(*o, B, F, L, D, 2, &s)) return FN_ERR_INVALID_ARG;
    for (int i = 0; i < 3; ++i)
      if (overlaps(outs[i], s) && !(i == 2 && o == &a->residual && in_place)) return FN_ERR_INVALID_ARG;
  }
  for (const void* v : {a->weight, a->bias})
    for (int i = 0; i < 3 && v; ++i)
      if (overlaps(outs[i], bytes_at(v, (uint64_t)D * (c.affine_fp32 ? 4 : 2)))) return FN_ERR_INVALID_ARG;
  return FN_OK;
}

QuantParams make_params(const norm_quant_s* h, const nq_args* a) {
  QuantParams p;
  std::memset(&p, 0, sizeof(p));
  auto u16 = [](const void* v) { return static_cast<const uint16_t*>(v); };
  p.x = u16(a->x.ptr), p.res = u16(a->residual.ptr), p.gate = u16(a->gate.ptr);
  p.scale = u16(a->scale.ptr), p.shift = u16(a->shift.ptr);
  p.weight = a->weight, p.bias = a->bias;
  p.q = static_cast<uint8_t*>(a->q), p.row_scale = a->row_scale, p.r = static_cast<uint16_t*>(a->r);
  p.x_sb = a->x.stride_b, p.x_sf = a->x.stride_f, p.x_sl = a->x.stride_l;
  p.res_sb = a->residual.stride_b, p.res_sf = a->residual.stride_f, p.res_sl = a->residual.stride_l;
  p.gate_sb = a->gate.stride_b, p.gate_sf = a->gate.stride_f, p.gate_sl = a->gate.stride_l;
  p.scale_sb = a->scale.stride_b, p.scale_sf = a->scale.stride_f, p.scale_sl = a->scale.stride_l;
  p.shift_sb = a->shift.stride_b, p.shift_sf = a->shift.stride_f, p.shift_sl = a->shift.stride_l;
  p.q_sb = a->q_stride_b, p.q_sl = a->q_stride_l, p.r_sb = a->r_stride_b, p.r_sl = a->r_stride_l;
  p.rows = (uint32_t)(a->B * a->L), p.L = (uint32_t)a->L, p.tpf = (uint32_t)a->tokens_per_frame;
  p.div_L = make_div_u32(p.L);
  p.div_tpf = make_div_u32(p.tpf ? p.tpf : 1u);
  p.vecs = (uint32_t)h->cfg.D / 8;
  // operands that change from token to token are read once: streamed past the caches
  p.stream_mask = (a->x.stride_l ? kX : 0u) | (a->residual.stride_l ? kRes : 0u) | (a->gate.stride_l ? kGate : 0u) |
                  (a->scale.stride_l ? kScale : 0u) | (a->shift.stride_l ? kShift : 0u);
  p.affine_fp32 = (uint32_t)h->cfg.affine_fp32;
  p.inv_d = 1.0 / h->cfg.D;
  p.eps = h->cfg.eps;
  return p;
}

}  // namespace

extern "C" {

fn_status norm_quant_create(norm_quant_t* out, const nq_config* cfg) {
  if (!out || !cfg) return FN_ERR_INVALID_ARG;
  const nq_config& c = *cfg;
  for (int v : {c.is_rms, c.has_residual, c.has_gate, c.has_weight, c.has_bias, c.affine_fp32, c.has_modulation})
    if (!is_flag(v)) return FN_ERR_INVALID_ARG;
  if (c.has_gate && !c.has_residual) return FN_ERR_INVALID_ARG;
  if (c.affine_fp32 && !c.has_weight && !c.has_bias) return FN_ERR_INVALID_ARG;
  if (!std::isfinite(c.eps) || c.eps < 0.0) return FN_ERR_INVALID_ARG;
  if (c.D < 16 || c.D > 16384 || c.D % 16) return FN_ERR_UNSUPPORTED;
  norm_quant_s* h = new (std::nothrow) norm_quant_s;
  if (!h) return FN_ERR_INVALID_ARG;
  h->cfg = c;
  h->shape = shape_of(c.D);
  h->kernel = c.is_rms ? pick<true, false>(h->shape) : pick<false, false>(h->shape);
  h->kernel_row_mod = c.is_rms ? pick<true, true>(h->shape) : pick<false, true>(h->shape);
  *out = h;
  return FN_OK;
}

fn_status norm_quant_validate(norm_quant_t h, const nq_args* a) { return validate(h, a); }

fn_status norm_quant_launch(norm_quant_t h, const nq_args* a, fn_stream_t stream) {
  const fn_status s = validate(h, a);
  if (s != FN_OK || a->B == 0 || a->L == 0) return s;
  const QuantParams p = make_params(h, a);
  const bool row_mod = a->scale.stride_l != 0 || a->shift.stride_l != 0;
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3(h->shape.warp_row ? (p.rows + kRowsPerCta - 1) / kRowsPerCta : p.rows);
  cfg.blockDim = dim3(h->shape.threads, h->shape.warp_row ? kRowsPerCta : 1);
  cfg.stream = reinterpret_cast<cudaStream_t>(stream);
  return launch_status(cudaLaunchKernelEx(&cfg, row_mod ? h->kernel_row_mod : h->kernel, p));
}

fn_status norm_quant_destroy(norm_quant_t h) {
  delete h;
  return FN_OK;
}

}  // extern "C"
