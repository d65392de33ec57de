// Residual / gate / norm / modulation rows with an e4m3 output and one scale per row
// (contract: include/block_ops.h, norm_quant).
//
// Mathematics, per row of D channels: r = bf16(residual + gate x); n = (r - mu) rho (mu = 0
// for RMSNorm), rho = 1 / sqrt(var + eps); y = (n w + b)(1 + scale) + shift; a = max |y|;
// row_scale = a / 448; q = e4m3(y 448 / a).
//
// Bound: HBM. A row moves 2 (x) + 2 (residual) + 2 (r) + 1 (q) bytes per element, plus 4 with
// per-token modulation. At the copy rate an SM has some 6000 instruction slots for a row of 5120
// channels without modulation of its own, so instructions count too: arithmetic on fp32 pairs,
// and what rows share is prepared once. The row stays in registers from its only read to its
// only write, as fp32 (the scale needs the whole row's maximum before anything is quantised).
//
// Layout: thread t of the row's T threads owns the 16-byte vectors t, t + T, ... (every warp
// access is 512 contiguous bytes), at most five, in 128 registers (LayerNorm with modulation per
// token, which keeps row, scale and shift, spills 100 bytes). A row meets at two barriers, for its
// statistics and its maximum; rows of one warp reduce through shuffles alone.
//
// Where no operand changes from token to token, CTAs are persistent (one per SM, its threads as
// groups of T with a row each) and keep gate, weight (1 + scale) and bias (1 + scale) + shift of
// their frame or batch in shared memory; the next row's vectors are requested as soon as this
// one's are used. Otherwise, and for few rows, a group of T threads takes one row and reads its
// operands with it. Both compute the same values in the same order.
//
// B200: 176400 rows of 5120 with frame gate and modulation 995 us, 6.4 TB/s of the 6.6 of a plain
// copy (2850 instructions a row, issue 48% busy; one row per CTA reading its operands 1382 us and
// 5360); 90000 rows of 10240 with modulation per token 1614 to 1705 us, 6.0 TB/s and more.
#include <cuda_fp8.h>

#include <cmath>
#include <cstring>
#include <new>

#include "elements.cuh"
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
  uint32_t chunk;    // rows of a CTA
  uint32_t segment;  // rows with the same gate, scale and shift, from row 0 on
  DivU32 div_segment;
  uint32_t stream_mask;
  uint32_t affine_fp32;
  double inv_d;  // 1 / D
  double eps;
};

constexpr int kMaxWarps = 16;  // of a CTA
constexpr int kMaxThreads = 32 * kMaxWarps;
constexpr int kMaxVectors = 5;   // of a thread

// The largest of three magnitudes; a NaN stays.
__device__ __forceinline__ float max_abs(float top, float a, float b) {
  asm("max.NaN.abs.f32 %0, %0, %1, %2;" : "+f"(top) : "f"(a), "f"(b));
  return top;
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

// y = n a + b of a vector: a = weight (1 + scale), b = bias (1 + scale) + shift. Where there is
// neither bias nor modulation b is -0, which leaves every n a as it is, a zero's sign too: the
// kernels that have no b give the same.
__device__ __forceinline__ void coefficients(const QuantParams& p, int j, bool modulated, const uint4& scale, const uint4& shift,
                                             uint64_t (&a)[4], uint64_t (&b)[4]) {
  const uint64_t one = pk2(1.0f, 1.0f);
#pragma unroll
  for (int i = 0; i < 4; ++i) a[i] = one, b[i] = modulated ? 0 : pk2(-0.0f, -0.0f);
  if (p.weight) load_affine(p.weight, p.affine_fp32, j, a);
  if (p.bias) load_affine(p.bias, p.affine_fp32, j, b);
  if (modulated) {
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      const uint64_t s = add2(widen(word(scale, i)), one);
      a[i] = mul2(a[i], s);
      b[i] = fma2(b[i], s, widen(word(shift, i)));
    }
  }
}

struct RowAt {
  uint32_t b, l, f;
};
__device__ __forceinline__ RowAt row_at(const QuantParams& p, uint32_t row) {
  const uint32_t b = div_u32(row, p.div_L), l = row - b * p.L;
  return RowAt{b, l, p.tpf > 0 ? div_u32(l, p.div_tpf) : 0u};
}
__device__ __forceinline__ const uint16_t* at_row(const uint16_t* base, int64_t sb, int64_t sf, int64_t sl, const RowAt& r) {
  return base + (r.b * sb + r.f * sf + r.l * sl);
}

// Shared memory of a group: its warps' sums and maxima, of this row and the next by turns.
struct GroupShared {
  double sums[2][2][kMaxWarps];
  double again[2][kMaxWarps];
  float tops[2][kMaxWarps];
};

// A row's threads: T of them, in warps of their own.
struct Group {
  GroupShared* sh;
  int id, tid, T;

  __device__ __forceinline__ void meet() const {
    if (T > 32) asm volatile("bar.sync %0, %1;" ::"r"(id + 1), "r"(T) : "memory");
    else __syncwarp();
  }
  // The sum over the row's threads, the same value in each of them.
  __device__ __forceinline__ double sum(double v, double* slot) const {
#pragma unroll
    for (int o = 16; o >= 1; o >>= 1) v += __shfl_xor_sync(0xFFFFFFFFu, v, o);
    if (T == 32) return v;
    if ((tid & 31) == 0) slot[tid >> 5] = v;
    meet();
    v = slot[0];
    for (int w = 1; w < (T >> 5); ++w) v += slot[w];
    return v;
  }
  // Magnitudes order as unsigned integers, a NaN's above infinity's.
  __device__ __forceinline__ float max(float v, float* slot) const {
    uint32_t t = __reduce_max_sync(0xFFFFFFFFu, __float_as_uint(v));
    if (T == 32) return __uint_as_float(t);
    if ((tid & 31) == 0) slot[tid >> 5] = __uint_as_float(t);
    meet();
    t = __float_as_uint(slot[0]);
    for (int w = 1; w < (T >> 5); ++w) t = ::max(t, __float_as_uint(slot[w]));
    return __uint_as_float(t);
  }
};

struct Stats {
  float rho, mu_hi, mu_lo;  // r - mu keeps fp32's precision
};

// fp32 within a thread (at most 40 elements), fp64 across threads. v(k, i): pair i of the thread's
// vector k in fp32, zeros where it has none; `full`: it has its last one. `again`: the row in memory.
// LayerNorm sums squares around the thread's own mean m, so nothing cancels in fp32:
// sum r^2 = sum (r - m)^2 + m (2 S - n m), joined in fp64. An error of S enters the variance
// only through its product with m - mu.
template <int NV, bool IS_RMS, typename Values>
__device__ __forceinline__ Stats statistics(const QuantParams& p, const Group& g, int parity, Values v, bool full, const uint4* again) {
  double mu = 0.0, var;
  uint64_t acc[2] = {0, 0};
  float a0, a1;
  if (IS_RMS) {
#pragma unroll
    for (int k = 0; k < NV; ++k)
#pragma unroll
      for (int i = 0; i < 4; ++i) acc[i & 1] = fma2(v(k, i), v(k, i), acc[i & 1]);
    upk2(add2(acc[0], acc[1]), a0, a1);
    var = g.sum((double)a0 + (double)a1, g.sh->sums[parity][0]) * p.inv_d;
  } else {
#pragma unroll
    for (int k = 0; k < NV; ++k)
#pragma unroll
      for (int i = 0; i < 4; ++i) acc[i & 1] = add2(acc[i & 1], v(k, i));
    upk2(add2(acc[0], acc[1]), a0, a1);
    const float n = full ? 8.0f * NV : 8.0f * (NV - 1);
    const float S = a0 + a1, m = S * (full ? 1.0f / (8.0f * NV) : NV > 1 ? 1.0f / (8.0f * (NV - 1)) : 0.0f);
    acc[0] = acc[1] = 0;
#pragma unroll
    for (int k = 0; k < NV; ++k) {
      const float c = k < NV - 1 || full ? -m : 0.0f;  // zeros stay zeros
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        const uint64_t d = add2(v(k, i), pk2(c, c));
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
    if (g.T > 32) {
      double(&sums)[2][kMaxWarps] = g.sh->sums[parity];
      if ((g.tid & 31) == 0) sums[0][g.tid >> 5] = s1, sums[1][g.tid >> 5] = s2;
      g.meet();
      s1 = sums[0][0], s2 = sums[1][0];
      for (int w = 1; w < (g.T >> 5); ++w) s1 += sums[0][w], s2 += sums[1][w];
    }
    mu = s1 * p.inv_d;
    var = s2 * p.inv_d - mu * mu;
  }
  // Rows that fp32 does not serve (squares near its limits, a spread below 1/32 of the
  // mean, zeros, infinities, NaN) take their statistics from fp64, around the exact mean.
  // The branch is the same for all threads of a row. The thread reads its vectors again (its
  // own r stores, or x) in rolled loops: walking the registers here would set the register
  // allocation of the whole kernel.
  if (!(var >= 0x1p-80 && var <= 0x1p+100 && mu * mu <= 1024.0 * var)) {
    double c = 0.0;
    if (!IS_RMS) {
#pragma unroll 1
      for (int j = g.tid; j < (int)p.vecs; j += g.T) {
        const uint4 u = __ldcg(again + j);
#pragma unroll
        for (int i = 0; i < 4; ++i) c += bf16_f64<0>(word(u, i)) + bf16_f64<1>(word(u, i));
      }
      // 1 / D is rounded: one correction gives the rounded quotient, so that the mean of equal values is
      // that value and their row is zero.
      c = g.sum(c, g.sh->again[0]);
      mu = c * p.inv_d;
      mu = fma(fma(-mu, 8.0 * p.vecs, c), p.inv_d, mu);
      c = 0.0;
    }
#pragma unroll 1
    for (int j = g.tid; j < (int)p.vecs; j += g.T) {
      const uint4 u = __ldcg(again + j);
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        const double d0 = bf16_f64<0>(word(u, i)) - mu, d1 = bf16_f64<1>(word(u, i)) - mu;
        c = fma(d1, d1, fma(d0, d0, c));
      }
    }
    var = g.sum(c, g.sh->again[1]) * p.inv_d;
  }
  const float hi = (float)mu;
  return Stats{(float)rsqrt(var + p.eps), hi, (float)(mu - (double)hi)};
}

// SHARED: the operands come from shared memory, rows one after another; otherwise one row per
// group, with its operands (MOD: scale and shift are read with the row and wait in registers).
// ADD: y = n a + b has a b.
template <int NV, bool IS_RMS, bool SHARED, bool MOD, bool ADD>
__global__ void __launch_bounds__(kMaxThreads, 1) norm_quant_rows(const __grid_constant__ QuantParams p) {
  __shared__ GroupShared groups[kMaxWarps];
  extern __shared__ __align__(16) uint4 kept[];  // SHARED: a and b in halves of a vector's eight, the gate
  const Group g{&groups[threadIdx.y], (int)threadIdx.y, (int)threadIdx.x, (int)blockDim.x};
  const int T = g.T, tid = g.tid;
  const bool full = (uint32_t)(tid + (NV - 1) * T) < p.vecs;
  auto has = [&](int k) { return k < NV - 1 || full; };
  const uint32_t begin = blockIdx.x * p.chunk, end = min(begin + p.chunk, p.rows);
  uint32_t row = begin + threadIdx.y;

  uint4 xv[NV], rv[NV];
  auto load = [&](const RowAt& at) {
    const uint4* x = reinterpret_cast<const uint4*>(at_row(p.x, p.x_sb, p.x_sf, p.x_sl, at)) + tid;
#pragma unroll
    for (int k = 0; k < NV; ++k, x += T)
      if (has(k)) xv[k] = p.stream_mask & kX ? __ldcs(x) : *x;
    if (p.res) {
      const uint4* r = reinterpret_cast<const uint4*>(at_row(p.res, p.res_sb, p.res_sf, p.res_sl, at)) + tid;
#pragma unroll
      for (int k = 0; k < NV; ++k, r += T)
        if (has(k)) rv[k] = p.stream_mask & kRes ? __ldcs(r) : *r;
    }
  };
#pragma unroll
  for (int k = 0; k < NV; ++k) xv[k] = rv[k] = make_uint4(0, 0, 0, 0);
  RowAt at = row_at(p, row);
  if (row < end) load(at);

  int parity = 0;
  for (uint32_t seg = SHARED ? div_u32(begin, p.div_segment) : 0u;; ++seg) {
    const uint32_t seg_end = SHARED ? (uint32_t)min((uint64_t)end, (uint64_t)(seg + 1) * p.segment) : end;
    if (SHARED) {
      // The operands of the rows up to seg_end; NV T vectors, zeros past the row's end.
      const RowAt first = row_at(p, min(seg * p.segment, p.rows - 1));
      const uint4* sr = reinterpret_cast<const uint4*>(at_row(p.scale, p.scale_sb, p.scale_sf, 0, first));
      const uint4* tr = reinterpret_cast<const uint4*>(at_row(p.shift, p.shift_sb, p.shift_sf, 0, first));
      const uint4* gr = reinterpret_cast<const uint4*>(at_row(p.gate, p.gate_sb, p.gate_sf, 0, first));
      __syncthreads();
      const int all = NV * T;
      for (int j = threadIdx.y * T + tid; j < all; j += T * blockDim.y) {
        uint64_t a[4] = {0, 0, 0, 0}, b[4] = {0, 0, 0, 0};
        uint4 gate = make_uint4(0, 0, 0, 0);
        if ((uint32_t)j < p.vecs) {
          uint4 s = gate, t = gate;
          if (p.scale) s = __ldg(sr + j), t = __ldg(tr + j);
          coefficients(p, j, p.scale != nullptr, s, t, a, b);
          if (p.gate) gate = __ldg(gr + j);
        }
        ulonglong2* to = reinterpret_cast<ulonglong2*>(kept);
        to[j] = make_ulonglong2(a[0], a[1]), to[j + all] = make_ulonglong2(a[2], a[3]);
        if (p.gate) kept[j + 2 * all] = gate;
        if (ADD) to[j + 3 * all] = make_ulonglong2(b[0], b[1]), to[j + 4 * all] = make_ulonglong2(b[2], b[3]);
      }
      __syncthreads();
    }
    for (; row < seg_end; row += blockDim.y, parity ^= 1) {
      // ---- r = residual + gate x, or x ----------------------------------------------------
      uint64_t y[NV][4];
      const uint4* again = reinterpret_cast<const uint4*>(at_row(p.x, p.x_sb, p.x_sf, p.x_sl, at));
      if (p.res) {
        if (p.gate) {
          const uint4* gr = SHARED ? kept + 2 * NV * T : reinterpret_cast<const uint4*>(at_row(p.gate, p.gate_sb, p.gate_sf, p.gate_sl, at));
          gr += tid;
#pragma unroll
          for (int k = 0; k < NV; ++k, gr += T)
            if (SHARED || has(k)) xv[k] = residual_vec<true>(rv[k], xv[k], SHARED ? *gr : p.stream_mask & kGate ? __ldcs(gr) : __ldg(gr));
        } else {
#pragma unroll
          for (int k = 0; k < NV; ++k) xv[k] = residual_vec<false>(rv[k], xv[k], xv[k]);
        }
        uint4* ro = reinterpret_cast<uint4*>(p.r + (at.b * p.r_sb + at.l * p.r_sl));
        again = ro;
        ro += tid;
#pragma unroll
        for (int k = 0; k < NV; ++k, ro += T)
          if (has(k)) __stcs(ro, xv[k]);
      }
      // Its values in fp32: kept where the next row's vectors take their place, otherwise widened
      // when they are used (modulation waits in registers meanwhile).
      if (SHARED) {
#pragma unroll
        for (int k = 0; k < NV; ++k)
#pragma unroll
          for (int i = 0; i < 4; ++i) y[k][i] = widen(has(k) ? word(xv[k], i) : 0u);
      }
      auto value = [&](int k, int i) { return SHARED ? y[k][i] : widen(word(xv[k], i)); };

      uint4 sv[MOD ? NV : 1], tv[MOD ? NV : 1];
      if (MOD) {  // the statistics hide its latency
        const uint4* sr = reinterpret_cast<const uint4*>(at_row(p.scale, p.scale_sb, p.scale_sf, p.scale_sl, at)) + tid;
        const uint4* tr = reinterpret_cast<const uint4*>(at_row(p.shift, p.shift_sb, p.shift_sf, p.shift_sl, at)) + tid;
#pragma unroll
        for (int k = 0; k < NV; ++k, sr += T, tr += T)
          if (has(k)) {
            sv[k] = p.stream_mask & kScale ? __ldcs(sr) : __ldg(sr);
            tv[k] = p.stream_mask & kShift ? __ldcs(tr) : __ldg(tr);
          }
      }
      const RowAt next = row_at(p, row + blockDim.y);
      if (SHARED && row + blockDim.y < end) load(next);

      const Stats st = statistics<NV, IS_RMS>(p, g, parity, value, full, again);

      if (!SHARED) {
#pragma unroll
        for (int k = 0; k < NV; ++k) xv[k] = here(xv[k]);
      }

      // ---- y in fp32, and the row's largest magnitude -------------------------------------
      float top = 0.0f;
#pragma unroll
      for (int k = 0; k < NV; ++k) {
        uint64_t a[4], b[4];
        if (SHARED) {
          const ulonglong2* from = reinterpret_cast<const ulonglong2*>(kept) + (tid + k * T);
          const ulonglong2 a0 = from[0], a1 = from[NV * T];
          a[0] = a0.x, a[1] = a0.y, a[2] = a1.x, a[3] = a1.y;
          if (ADD) {
            const ulonglong2 b0 = from[3 * NV * T], b1 = from[4 * NV * T];
            b[0] = b0.x, b[1] = b0.y, b[2] = b1.x, b[3] = b1.y;
          }
        } else if (has(k)) {
          coefficients(p, tid + k * T, MOD, sv[MOD ? k : 0], tv[MOD ? k : 0], a, b);
        } else {
#pragma unroll
          for (int i = 0; i < 4; ++i) a[i] = b[i] = 0;
        }
#pragma unroll
        for (int i = 0; i < 4; ++i) {
          uint64_t d = value(k, i);
          if (!IS_RMS) d = add2(add2(d, pk2(-st.mu_hi, -st.mu_hi)), pk2(-st.mu_lo, -st.mu_lo));
          d = mul2(d, pk2(st.rho, st.rho));
          y[k][i] = ADD ? fma2(d, a[i], b[i]) : mul2(d, a[i]);
          float a0, a1;
          upk2(y[k][i], a0, a1);
          if (has(k)) top = max_abs(top, a0, a1);  // 0 - mu, times rho, may be an infinity
        }
      }
      const float a = g.max(top, g.sh->tops[parity]);

      // ---- scale and quantise --------------------------------------------------------------
      // The product with 448 / a stands for the quotient by row_scale: one rounding less than
      // dividing by the rounded row_scale. fmaxf would drop a NaN, so the floor is a comparison.
      const float a1 = a < 0x1p-100f ? 0x1p-100f : a;
      if (tid == 0) p.row_scale[row] = a == 0.0f ? 1.0f : a1 / 448.0f;
      const float inv = 448.0f / a1;
      uint2* qo = reinterpret_cast<uint2*>(p.q + (at.b * p.q_sb + at.l * p.q_sl)) + tid;
#pragma unroll
      for (int k = 0; k < NV; ++k, qo += T) {
        uint32_t h[4];
#pragma unroll
        for (int i = 0; i < 4; ++i) {
          float2 e;
          upk2(mul2(y[k][i], pk2(inv, inv)), e.x, e.y);
          h[i] = __nv_cvt_float2_to_fp8x2(e, __NV_SATFINITE, __NV_E4M3);
        }
        if (has(k)) __stcs(qo, make_uint2(h[0] | h[1] << 16, h[2] | h[3] << 16));
      }
      at = next;
    }
    if (seg_end >= end) return;
  }
}

// As few threads as five vectors each allow.
struct Shape {
  int nv, threads;
};
Shape shape_of(int D) {
  const int V = D / 8, T = (V + 32 * kMaxVectors - 1) / (32 * kMaxVectors) * 32;
  return Shape{(V + T - 1) / T, T};
}

// Shared memory that the widest rows keep. A kernel's limit is set to that, whatever the handle: handles
// of several widths share a kernel, and another host thread may be between its limit and its launch.
constexpr int kMaxKept = 5 * 16 * kMaxVectors * 416;
static_assert(16384 / 8 <= kMaxVectors * 416 && kMaxKept + sizeof(GroupShared) * kMaxWarps <= 227 * 1024, "rows of 16384 channels fit");

using Kernel = void (*)(QuantParams);

template <bool RMS, bool SHARED, bool MOD, bool ADD>
Kernel pick(int nv) {
  switch (nv) {
    case 1: return norm_quant_rows<1, RMS, SHARED, MOD, ADD>;
    case 2: return norm_quant_rows<2, RMS, SHARED, MOD, ADD>;
    case 3: return norm_quant_rows<3, RMS, SHARED, MOD, ADD>;
    case 4: return norm_quant_rows<4, RMS, SHARED, MOD, ADD>;
    default: return norm_quant_rows<5, RMS, SHARED, MOD, ADD>;
  }
}

}  // namespace
}  // namespace block_ops

using namespace block_ops;

struct norm_quant_s {
  nq_config cfg;
  Shape shape;
  Kernel each, each_mod, shared;  // a row per group, the same with modulation, persistent
  size_t kept;                    // bytes of shared memory of the last
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
  const int nv = h->shape.nv;
  const bool add = c.has_bias || c.has_modulation;
  if (c.is_rms) {
    h->each = pick<true, false, false, true>(nv), h->each_mod = pick<true, false, true, true>(nv);
    h->shared = add ? pick<true, true, false, true>(nv) : pick<true, true, false, false>(nv);
  } else {
    h->each = pick<false, false, false, true>(nv), h->each_mod = pick<false, false, true, true>(nv);
    h->shared = add ? pick<false, true, false, true>(nv) : pick<false, true, false, false>(nv);
  }
  h->kept = (size_t)nv * h->shape.threads * 16 * (add ? 5 : 3);
  *out = h;
  return FN_OK;
}

fn_status norm_quant_validate(norm_quant_t h, const nq_args* a) { return validate(h, a); }

fn_status norm_quant_launch(norm_quant_t h, const nq_args* a, fn_stream_t stream) {
  const fn_status s = validate(h, a);
  if (s != FN_OK || a->B == 0 || a->L == 0) return s;
  QuantParams p = make_params(h, a);
  int device = 0, sms = 0;
  cudaError_t e = cudaGetDevice(&device);
  if (e == cudaSuccess) e = cudaDeviceGetAttribute(&sms, cudaDevAttrMultiProcessorCount, device);
  if (e != cudaSuccess) return launch_status(e);

  // Rows that share gate, scale and shift, and the rows of a CTA.
  const fn_operand* by_row[3] = {&a->gate, &a->scale, &a->shift};
  bool own = false, by_batch = false, by_frame = false;
  for (const fn_operand* o : by_row) own |= o->stride_l != 0, by_batch |= o->stride_b != 0, by_frame |= o->stride_f != 0;
  p.segment = by_frame ? p.tpf : by_batch ? p.L : p.rows;
  const int T = h->shape.threads, groups = kMaxThreads / T;
  // The persistent kernel is ahead once every group has a row (D = 5120: 1184 rows 9.3 against
  // 12.8 us, 9472 rows 62 against 94; below that a CTA to a row spreads wider) and an operand
  // serves a row of each group (frames of 16 rows 67 against 100 us, of 2 164 against 112).
  const bool shared = !own && p.rows >= (uint32_t)(sms * groups) && p.segment >= (uint32_t)(groups > 4 ? groups : 4);
  cudaLaunchConfig_t cfg = {};
  Kernel kernel;
  if (shared) {
    kernel = h->shared;
    p.chunk = (p.rows + sms - 1) / sms;
    p.div_segment = make_div_u32(p.segment);
    cfg.blockDim = dim3(T, groups);
    cfg.dynamicSmemBytes = h->kept;
    e = cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, kMaxKept);
    if (e != cudaSuccess) return launch_status(e);
  } else {
    kernel = p.scale ? h->each_mod : h->each;
    p.chunk = T > 32 ? 1 : 8;
    cfg.blockDim = dim3(T, p.chunk);
  }
  cfg.gridDim = dim3((p.rows + p.chunk - 1) / p.chunk);
  cfg.stream = reinterpret_cast<cudaStream_t>(stream);
  return launch_status(cudaLaunchKernelEx(&cfg, kernel, p));
}

fn_status norm_quant_destroy(norm_quant_t h) {
  delete h;
  return FN_OK;
}

}  // extern "C"
