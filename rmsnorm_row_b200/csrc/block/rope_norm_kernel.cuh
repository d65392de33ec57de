// RMS norm of q or k and rotary positions over several axes, and the gradient
// (contract: include/block_ops.h, rope_norm).
//
// Mathematics, per token of H heads of hd channels: rho = 1 / sqrt(mean(x^2) + eps) over the
// head or the token, n = x rho w, and pair i of each head turned by position[axis(i)] freq(i).
// The gradient turns grad back (dn), then dx = rho (w dn - x rho^2 mean(w dn x)) and
// dw = sum dn x rho.
//
// Bound: HBM. A token moves 2 + 2 bytes per channel (gradient: 2 + 2 + 2) against ~10 fp32
// operations (~25). The angle of a pair is shared by all heads of a token: one thread reduces
// it in fp64 and leaves cos and sin in shared memory, one token ahead of its use.
//
// Layout: a thread owns "units" of 16 channels of a head as two 16-byte vectors A and B, the
// same unit u in each of its heads h = g, g + G, ... (g: its lane group of W lanes, W the
// power of two from hd / 16 up). Half pairing puts the 8 partners of A in B, so every pair is
// inside one thread; adjacent pairing has A in the head's first half and B in its second, so
// that neighbouring lanes touch neighbouring vectors. A norm over the head is a shuffle inside
// W lanes. Rows of up to 32 lanes share warps; longer rows are a CTA with one barrier per
// token. CTAs are persistent; each thread copies its own vectors of the
// next two tokens to shared memory while it works on the present one, so no registers wait
// for loads and nobody else has to be waited for.
#pragma once

#include <cuda_bf16.h>
#include <cuda_fp16.h>
#include <cuda_runtime.h>
#include <stdint.h>

#include "../fused_norm_kernel.cuh"
#include "../../../include/block_ops.h"

namespace block_ops {

using fused_norm_impl::DivU32;
using fused_norm_impl::div_u32;

constexpr int kMaxPairs = 256;      // of a head
constexpr int kRopeThreads = 512;   // of a CTA, at most
constexpr int kSharedRows = 128;    // threads of a CTA whose rows take 32 lanes or fewer
constexpr int kMaxPartials = 1024;  // CTAs that sum dweight

struct RopeRows {
  const uint16_t* ptr;
  int64_t sb, sl, sh;
};

struct RopeParams {
  RopeRows x, dy;
  RopeRows out;
  const void* positions;
  int64_t pos_sb, pos_sl;
  const void* weight;
  float* partial;
  uint32_t rows, L;
  DivU32 div_L;
  int H, hd, units, pairs;  // units of a head (hd / 16), pairs that turn
  int W, T, G;              // lanes of a head, threads of a row, T / W
  int index64, weight_fp32, weight_sh;  // weight's step from head to head (0: one head's)
  float inv_n, eps;
  double inv_n64, eps64;
  double turns[kMaxPairs];    // freq / 2 pi
  uint8_t axis[kMaxPairs];
};

// ---- element types --------------------------------------------------------------------------

template <bool FP16>
__device__ __forceinline__ float2 widen16(uint32_t u) {
  if (FP16) {
    __half2 h;
    memcpy(&h, &u, 4);
    return __half22float2(h);
  }
  return make_float2(fused_norm_impl::lo_f(u), fused_norm_impl::hi_f(u));
}

template <bool FP16>
__device__ __forceinline__ uint32_t pack16(float a, float b) {
  if (FP16) {
    const __half2 h = __floats2half2_rn(a, b);
    uint32_t u;
    memcpy(&u, &h, 4);
    return u;
  }
  return fused_norm_impl::pack_rn(a, b);
}

template <bool FP16>
__device__ __forceinline__ void widen8(const uint4& v, float (&f)[8]) {
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    const float2 e = widen16<FP16>(fused_norm_impl::word(v, i));
    f[2 * i] = e.x, f[2 * i + 1] = e.y;
  }
}

template <bool FP16>
__device__ __forceinline__ uint4 pack8(const float (&f)[8]) {
  return make_uint4(pack16<FP16>(f[0], f[1]), pack16<FP16>(f[2], f[3]), pack16<FP16>(f[4], f[5]),
                    pack16<FP16>(f[6], f[7]));
}

template <bool FP16>
__device__ __forceinline__ void load_weight8(const void* w, bool fp32, int at, float (&f)[8]) {
  if (fp32) {
    const float4* q = reinterpret_cast<const float4*>(static_cast<const float*>(w) + at);
    const float4 a = __ldg(q), b = __ldg(q + 1);
    f[0] = a.x, f[1] = a.y, f[2] = a.z, f[3] = a.w, f[4] = b.x, f[5] = b.y, f[6] = b.z, f[7] = b.w;
  } else {
    widen8<FP16>(__ldg(reinterpret_cast<const uint4*>(static_cast<const uint16_t*>(w) + at)), f);
  }
}

// ---- one thread's place in a row ---------------------------------------------------------------

struct Place {
  int u, g;        // unit, lane group
  int offA, offB;  // channels of the two vectors in the head
  bool owns;       // u is a unit of the head
};

template <bool HALF>
__device__ __forceinline__ Place place_of(const RopeParams& p, int t) {
  Place q;
  q.u = t & (p.W - 1);
  q.g = t / p.W;
  q.owns = q.u < p.units;
  if (!HALF) {
    q.offA = 8 * q.u, q.offB = p.hd / 2 + 8 * q.u;
  } else if (8 * q.u < p.pairs) {
    q.offA = 8 * q.u, q.offB = p.pairs + 8 * q.u;
  } else {
    q.offA = 16 * q.u, q.offB = 16 * q.u + 8;  // channels that pass
  }
  return q;
}

// The pairs of a unit turned by (cos, sin) from the table of this row; SIGN -1 turns back.
template <bool HALF, int SIGN>
__device__ __forceinline__ void turn(const RopeParams& p, const Place& q, const float2* cs, float (&a)[8], float (&b)[8]) {
  if (HALF) {
    if (8 * q.u >= p.pairs) return;
#pragma unroll
    for (int i = 0; i < 8; ++i) {
      const float2 e = cs[8 * q.u + i];
      const float s = SIGN * e.y, y0 = fmaf(a[i], e.x, -b[i] * s);
      b[i] = fmaf(a[i], s, b[i] * e.x);
      a[i] = y0;
    }
  } else {
#pragma unroll
    for (int side = 0; side < 2; ++side) {
      float(&v)[8] = side ? b : a;
      const int first = side ? p.hd / 4 + 4 * q.u : 4 * q.u;
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        if (first + i >= p.pairs) continue;
        const float2 e = cs[first + i];
        const float s = SIGN * e.y, y0 = fmaf(v[2 * i], e.x, -v[2 * i + 1] * s);
        v[2 * i + 1] = fmaf(v[2 * i], s, v[2 * i + 1] * e.x);
        v[2 * i] = y0;
      }
    }
  }
}

// Puts back the packed pairs that do not turn.
template <bool HALF>
__device__ __forceinline__ void keep_passing(const RopeParams& p, const Place& q, const uint4& a, const uint4& b, uint4& oa, uint4& ob) {
  if (HALF) {
    if (8 * q.u >= p.pairs) oa = a, ob = b;
    return;
  }
  const int ka = p.pairs - 4 * q.u, kb = ka - p.hd / 4;  // pairs of each vector that turn
  if (ka < 4) oa = make_uint4(ka > 0 ? oa.x : a.x, ka > 1 ? oa.y : a.y, ka > 2 ? oa.z : a.z, a.w);
  if (kb < 4) ob = make_uint4(kb > 0 ? ob.x : b.x, kb > 1 ? ob.y : b.y, kb > 2 ? ob.z : b.z, b.w);
}

struct RowAt {
  uint32_t b, l;
};
__device__ __forceinline__ RowAt row_at(const RopeParams& p, uint32_t row) {
  const uint32_t b = div_u32(row, p.div_L);
  return RowAt{b, row - b * p.L};
}
__device__ __forceinline__ const uint16_t* row_ptr(const RopeRows& r, const RowAt& at) {
  return r.ptr + (at.b * r.sb + at.l * r.sl);
}

// cos and sin of a row's pairs, by its T threads. The angle in turns is reduced in fp64 to
// [-1/2, 1/2]; what fp32 then adds is 2^-25 of a turn.
__device__ __forceinline__ void fill_table(const RopeParams& p, const double* turns, const uint8_t* axis, const RowAt& at,
                                           int t, float2* cs) {
  for (int i = t; i < p.pairs; i += p.T) {
    const int64_t o = at.b * p.pos_sb + at.l * p.pos_sl + axis[i];
    const double pos = p.index64 ? (double)__ldg(static_cast<const long long*>(p.positions) + o)
                                 : (double)__ldg(static_cast<const int*>(p.positions) + o);
    double a = pos * turns[i];
    a -= rint(a);
    float s, c;
    sincospif(2.0f * (float)a, &s, &c);
    cs[i] = make_float2(c, s);
  }
}

template <typename V>
__device__ __forceinline__ V lanes_sum(V v, int lanes) {
  for (int o = lanes >> 1; o >= 1; o >>= 1) v += __shfl_xor_sync(0xFFFFFFFFu, v, o);
  return v;
}

// fp32 sums of squares that are kept: outside, the sums are taken again in fp64.
__device__ __forceinline__ bool in_range(float ss) { return ss >= 0x1p-80f && ss <= 0x1p+100f; }

// A thread's own two vectors of a head, in shared memory: x's, then grad's where BACK. One
// stage holds all heads of a thread; vectors of neighbouring threads are neighbours.
template <bool BACK>
struct Stage {
  static constexpr int kVectors = BACK ? 4 : 2;
  uint4* mine;  // vector 0 of head 0
  int step;     // vectors from one to the next: the CTA's threads
  __device__ __forceinline__ uint4* at(int k, int v) const { return mine + (k * kVectors + v) * step; }
};

template <bool FP16>
__device__ __forceinline__ void load_weights(const RopeParams& p, const Place& q, int h, float (&wa)[8], float (&wb)[8]) {
  load_weight8<FP16>(p.weight, p.weight_fp32, h * p.weight_sh + q.offA, wa);
  load_weight8<FP16>(p.weight, p.weight_fp32, h * p.weight_sh + q.offB, wb);
}

// A head's sums of x^2 and of w dn x over this thread's channels.
template <typename Sum, bool FP16, bool HALF, bool BACK>
__device__ __forceinline__ void unit_sums(const RopeParams& p, const Place& q, const float2* cs, const Stage<BACK>& st, int k,
                                          Sum& xx, Sum& gx) {
  float xa[8], xb[8];
  widen8<FP16>(*st.at(k, 0), xa);
  widen8<FP16>(*st.at(k, 1), xb);
  Sum s0 = 0, s1 = 0;
#pragma unroll
  for (int i = 0; i < 8; ++i) s0 += (Sum)xa[i] * (Sum)xa[i], s1 += (Sum)xb[i] * (Sum)xb[i];
  xx += s0 + s1;
  if (BACK) {
    float a[8], b[8];
    widen8<FP16>(*st.at(k, 2), a);
    widen8<FP16>(*st.at(k, 3), b);
    turn<HALF, -1>(p, q, cs, a, b);
    if (p.weight) {
      float wa[8], wb[8];
      load_weights<FP16>(p, q, q.g + k * p.G, wa, wb);
#pragma unroll
      for (int i = 0; i < 8; ++i) a[i] *= wa[i], b[i] *= wb[i];
    }
    s0 = s1 = 0;
#pragma unroll
    for (int i = 0; i < 8; ++i) s0 += (Sum)a[i] * (Sum)xa[i], s1 += (Sum)b[i] * (Sum)xb[i];
    gx += s0 + s1;
  }
}

// The same in fp64, for the rare rows; out of line.
template <bool FP16, bool HALF, bool BACK>
__device__ __noinline__ double2 exact_sums(const RopeParams& p, const Place& q, const float2* cs, const Stage<BACK>& st, int k) {
  double2 r = make_double2(0.0, 0.0);
  unit_sums<double, FP16, HALF, BACK>(p, q, cs, st, k, r.x, r.y);
  return r;
}

__device__ __forceinline__ void copy_async(uint4* to, const uint16_t* from) {
  asm volatile("cp.async.cg.shared.global [%0], [%1], 16;" ::"r"((uint32_t)__cvta_generic_to_shared(to)), "l"(from) : "memory");
}

// Shared memory of a CTA: the frequency table, sums; then three tables of (cos, sin) per row
// slot; then three stages of rows. A row's table is written before the barrier of the row
// ahead of it and read up to the barrier of the row behind it, so its buffer comes round again
// at the third row.
constexpr int kStages = 3;
struct RopeShared {
  double turns[kMaxPairs];
  double sums64[2][kRopeThreads / 32];
  float2 sums[kStages][kRopeThreads / 32];
  uint8_t axis[kMaxPairs];
};
__host__ __device__ inline size_t rope_tables_bytes(int rows_per_cta, int pairs) {
  return ((size_t)kStages * rows_per_cta * pairs * sizeof(float2) + 15) / 16 * 16;
}
inline size_t rope_shared_bytes(int rows_per_cta, int pairs, int threads, int nh, bool back) {
  const size_t rows = (size_t)kStages * threads * nh * (back ? 4 : 2) * 16;
  return sizeof(RopeShared) + rope_tables_bytes(rows_per_cta, pairs) + rows;
}
static_assert(sizeof(RopeShared) % 16 == 0, "what follows is 16-byte aligned");

// BACK: the gradient. DW: it sums dweight's partials too (needs a norm).
template <bool FP16, int NH, int NORM, bool HALF, bool BACK, bool DW>
__global__ void __launch_bounds__(kRopeThreads, 1) rope_norm_rows(const __grid_constant__ RopeParams p) {
  extern __shared__ __align__(16) unsigned char raw[];
  RopeShared& sh = *reinterpret_cast<RopeShared*>(raw);
  float2* const tables = reinterpret_cast<float2*>(raw + sizeof(RopeShared));
  constexpr bool READ_X = !BACK || NORM != BO_NORM_NONE;
  const int T = p.T, R = blockDim.x / T;  // R > 1 only where T <= 32
  const int slot = threadIdx.x / T, t = threadIdx.x - slot * T;
  const bool wide = T > 32;
  const Place q = place_of<HALF>(p, t);
  uint4* const stages = reinterpret_cast<uint4*>(raw + sizeof(RopeShared) + rope_tables_bytes(R, p.pairs)) + threadIdx.x;
  for (int i = threadIdx.x; i < p.pairs; i += blockDim.x) sh.turns[i] = p.turns[i], sh.axis[i] = p.axis[i];
  __syncthreads();
  auto table = [&](int buf) { return tables + (size_t)(buf * R + slot) * p.pairs; };
  auto stage = [&](int buf) {
    return Stage<BACK>{stages + (size_t)buf * NH * Stage<BACK>::kVectors * blockDim.x, (int)blockDim.x};
  };
  auto has = [&](int k) { return q.owns && q.g + k * p.G < p.H; };
  auto fetch = [&](uint32_t row, int buf) {
    if (row < p.rows) {
      const RowAt at = row_at(p, row);
      const Stage<BACK> st = stage(buf);
#pragma unroll
      for (int k = 0; k < NH; ++k) {
        if (!has(k)) continue;
        const int h = q.g + k * p.G;
        if (READ_X) {
          const uint16_t* b = row_ptr(p.x, at) + h * p.x.sh;
          copy_async(st.at(k, 0), b + q.offA);
          copy_async(st.at(k, 1), b + q.offB);
        }
        if (BACK) {
          const uint16_t* b = row_ptr(p.dy, at) + h * p.dy.sh;
          copy_async(st.at(k, 2), b + q.offA);
          copy_async(st.at(k, 3), b + q.offB);
        }
      }
    }
    asm volatile("cp.async.commit_group;" ::: "memory");
  };

  constexpr int NACC = NORM == BO_NORM_ALL ? NH : 1;
  float acc[DW ? NACC : 1][16];
#pragma unroll
  for (int k = 0; k < (DW ? NACC : 1); ++k)
#pragma unroll
    for (int i = 0; i < 16; ++i) acc[k][i] = 0.0f;

  // The output of one head, and its part of dweight; m = mean(w dn x) rho.
  auto finish = [&](const float2* cs, const Stage<BACK>& st, uint16_t* ob, int k, float rho, float m) {
    const int h = q.g + k * p.G;
    float a[8], b[8];
    widen8<FP16>(*st.at(k, BACK ? 2 : 0), a);
    widen8<FP16>(*st.at(k, BACK ? 3 : 1), b);
    if (!BACK) {
      if (NORM != BO_NORM_NONE) {
#pragma unroll
        for (int i = 0; i < 8; ++i) a[i] *= rho, b[i] *= rho;
        if (p.weight) {
          float wa[8], wb[8];
          load_weights<FP16>(p, q, h, wa, wb);
#pragma unroll
          for (int i = 0; i < 8; ++i) a[i] *= wa[i], b[i] *= wb[i];
        }
      }
      turn<HALF, 1>(p, q, cs, a, b);
    } else {
      turn<HALF, -1>(p, q, cs, a, b);  // dn, the same values as in the sums
      if (NORM != BO_NORM_NONE) {
        float na[8], nb[8];
        widen8<FP16>(*st.at(k, 0), na);
        widen8<FP16>(*st.at(k, 1), nb);
#pragma unroll
        for (int i = 0; i < 8; ++i) na[i] *= rho, nb[i] *= rho;
        if (DW) {
          float(&s)[16] = acc[NORM == BO_NORM_ALL ? k : 0];
#pragma unroll
          for (int i = 0; i < 8; ++i) s[i] = fmaf(a[i], na[i], s[i]), s[8 + i] = fmaf(b[i], nb[i], s[8 + i]);
        }
        if (p.weight) {
          float wa[8], wb[8];
          load_weights<FP16>(p, q, h, wa, wb);
#pragma unroll
          for (int i = 0; i < 8; ++i) a[i] *= wa[i], b[i] *= wb[i];
        }
#pragma unroll
        for (int i = 0; i < 8; ++i) a[i] = rho * fmaf(-na[i], m, a[i]), b[i] = rho * fmaf(-nb[i], m, b[i]);
      }
    }
    uint4 va = pack8<FP16>(a), vb = pack8<FP16>(b);
    if (NORM == BO_NORM_NONE) {  // channels that pass keep their bits, a NaN's too
      keep_passing<HALF>(p, q, *st.at(k, BACK ? 2 : 0), *st.at(k, BACK ? 3 : 1), va, vb);
    }
    __stcs(reinterpret_cast<uint4*>(ob + (h * p.out.sh + q.offA)), va);
    __stcs(reinterpret_cast<uint4*>(ob + (h * p.out.sh + q.offB)), vb);
  };
  // Sums that fp32 does not hold.
  auto outside = [](float xx, float gx) { return !(in_range(xx) && (!BACK || fabsf(gx) <= 0x1p+100f)); };

  const uint32_t step = gridDim.x * R;
  uint32_t base = blockIdx.x * R;
  fetch(base + slot, 0);
  fetch(base + slot + step, 1);  // rows + 2 step < 2^32: the host bounds both
  if (base + slot < p.rows) fill_table(p, sh.turns, sh.axis, row_at(p, base + slot), t, table(0));
  if (wide) __syncthreads();
  else __syncwarp();

  for (int buf = 0, ahead = 1; base < p.rows; base += step, buf = ahead, ahead = ahead == kStages - 1 ? 0 : ahead + 1) {
    const uint32_t row = base + slot, next = row + step;
    const RowAt at = row_at(p, row);
    const bool live = row < p.rows;
    const float2* const cs = table(buf);
    const Stage<BACK> st = stage(buf);
    fetch(next + step, ahead == kStages - 1 ? 0 : ahead + 1);
    asm volatile("cp.async.wait_group 2;" ::: "memory");  // this row's vectors are here

    float2 all = make_float2(0.0f, 0.0f);
    if (NORM == BO_NORM_ALL) {
#pragma unroll
      for (int k = 0; k < NH; ++k)
        if (live && has(k)) unit_sums<float, FP16, HALF, BACK>(p, q, cs, st, k, all.x, all.y);
      all.x = lanes_sum(all.x, wide ? 32 : T);
      if (BACK) all.y = lanes_sum(all.y, wide ? 32 : T);
      if (wide && (t & 31) == 0) sh.sums[buf][t >> 5] = all;
    }
    if (next < p.rows) fill_table(p, sh.turns, sh.axis, row_at(p, next), t, table(ahead));
    if (wide) __syncthreads();
    else __syncwarp();

    uint16_t* const ob = const_cast<uint16_t*>(row_ptr(p.out, at));
    if (NORM == BO_NORM_NONE) {
#pragma unroll
      for (int k = 0; k < NH; ++k)
        if (live && has(k)) finish(cs, st, ob, k, 1.0f, 0.0f);
    } else if (NORM == BO_NORM_HEAD) {
#pragma unroll
      for (int k = 0; k < NH; ++k) {
        float2 s = make_float2(0.0f, 0.0f);
        const bool mine = live && has(k);
        if (mine) unit_sums<float, FP16, HALF, BACK>(p, q, cs, st, k, s.x, s.y);
        s.x = lanes_sum(s.x, p.W);
        if (BACK) s.y = lanes_sum(s.y, p.W);
        float rho = rsqrtf(fmaf(s.x, p.inv_n, p.eps)), m = s.y * p.inv_n * rho;
        if (__any_sync(0xFFFFFFFFu, mine && outside(s.x, s.y))) {
          double2 e = mine ? exact_sums<FP16, HALF, BACK>(p, q, cs, st, k) : make_double2(0.0, 0.0);
          e.x = lanes_sum(e.x, p.W);
          if (BACK) e.y = lanes_sum(e.y, p.W);
          if (outside(s.x, s.y)) {
            const double f = rsqrt(e.x * p.inv_n64 + p.eps64);
            rho = (float)f, m = (float)(e.y * p.inv_n64 * f);
          }
        }
        if (mine) finish(cs, st, ob, k, rho, m);
      }
    } else {
      if (wide) {
        all = sh.sums[buf][0];
        for (int w = 1; w < (T >> 5); ++w) {
          const float2 o = sh.sums[buf][w];
          all.x += o.x, all.y += o.y;
        }
      }
      float rho = rsqrtf(fmaf(all.x, p.inv_n, p.eps)), m = all.y * p.inv_n * rho;
      const bool odd = live && outside(all.x, all.y);
      if (wide ? odd : (bool)__any_sync(0xFFFFFFFFu, odd)) {  // the same for all threads that meet below
        double2 e = make_double2(0.0, 0.0);
        for (int k = 0; k < NH; ++k)
          if (live && has(k)) {
            const double2 one = exact_sums<FP16, HALF, BACK>(p, q, cs, st, k);
            e.x += one.x, e.y += one.y;
          }
        e.x = lanes_sum(e.x, wide ? 32 : T);
        if (BACK) e.y = lanes_sum(e.y, wide ? 32 : T);
        if (wide) {
          if ((t & 31) == 0) sh.sums64[0][t >> 5] = e.x, sh.sums64[1][t >> 5] = e.y;
          __syncthreads();
          e = make_double2(0.0, 0.0);
          for (int w = 0; w < (T >> 5); ++w) e.x += sh.sums64[0][w], e.y += sh.sums64[1][w];
          __syncthreads();
        }
        if (odd) {
          const double f = rsqrt(e.x * p.inv_n64 + p.eps64);
          rho = (float)f, m = (float)(e.y * p.inv_n64 * f);
        }
      }
#pragma unroll
      for (int k = 0; k < NH; ++k)
        if (live && has(k)) finish(cs, st, ob, k, rho, m);
    }
  }

  if (!DW) return;
  // ---- this CTA's part of dweight --------------------------------------------------------------
  float* const part = p.partial + (size_t)blockIdx.x * (NORM == BO_NORM_ALL ? p.H * p.hd : p.hd);
  if (NORM == BO_NORM_ALL && wide) {  // every channel of the token has one thread
#pragma unroll
    for (int k = 0; k < NACC; ++k) {
      if (!has(k)) continue;
      float* o = part + (q.g + k * p.G) * p.hd;
#pragma unroll
      for (int i = 0; i < 8; ++i) o[q.offA + i] = acc[k][i], o[q.offB + i] = acc[k][8 + i];
    }
    return;
  }
  // Threads with the same channels: lanes of a warp through shuffles, then warps in turn,
  // through the first stage (every thread is past its rows, and its copies have landed).
  asm volatile("cp.async.wait_all;" ::: "memory");
  const int span = NORM == BO_NORM_ALL ? T : p.W;
#pragma unroll
  for (int i = 0; i < 16; ++i)
    for (int o = span; o < 32; o <<= 1) acc[0][i] += __shfl_xor_sync(0xFFFFFFFFu, acc[0][i], o);
  float* const sums = reinterpret_cast<float*>(stages - threadIdx.x);  // 16 values of `span` lanes
  for (int w = 0; w < (int)(blockDim.x >> 5); ++w) {
    __syncthreads();
    if ((int)(threadIdx.x >> 5) == w && (int)(threadIdx.x & 31) < span) {
#pragma unroll
      for (int i = 0; i < 16; ++i) {
        float& s = sums[i * 32 + (threadIdx.x & 31)];
        s = (w ? s : 0.0f) + acc[0][i];
      }
    }
  }
  __syncthreads();
  if ((int)threadIdx.x < span && has(0)) {
    float* o = part + (NORM == BO_NORM_ALL ? q.g * p.hd : 0);
#pragma unroll
    for (int i = 0; i < 8; ++i) o[q.offA + i] = sums[i * 32 + threadIdx.x], o[q.offB + i] = sums[(8 + i) * 32 + threadIdx.x];
  }
}

using RopeKernel = void (*)(RopeParams);

// One kernel for (threads' heads, norm, pairing, gradient, dweight); the two element types are
// compiled in files of their own.
template <bool FP16>
RopeKernel pick_rope(int nh, int norm, bool half, bool back, bool dw);
extern template RopeKernel pick_rope<false>(int, int, bool, bool, bool);
extern template RopeKernel pick_rope<true>(int, int, bool, bool, bool);

template <bool FP16, int NH, int NORM, bool HALF>
RopeKernel pick_rope_pass(bool back, bool dw) {
  if (!back) return rope_norm_rows<FP16, NH, NORM, HALF, false, false>;
  if (NORM != BO_NORM_NONE && dw) return rope_norm_rows<FP16, NH, NORM, HALF, true, NORM != BO_NORM_NONE>;
  return rope_norm_rows<FP16, NH, NORM, HALF, true, false>;
}
template <bool FP16, int NH>
RopeKernel pick_rope_norm(int norm, bool half, bool back, bool dw) {
  switch (norm) {
    case BO_NORM_NONE:
      return half ? pick_rope_pass<FP16, NH, BO_NORM_NONE, true>(back, dw) : pick_rope_pass<FP16, NH, BO_NORM_NONE, false>(back, dw);
    case BO_NORM_HEAD:
      return half ? pick_rope_pass<FP16, NH, BO_NORM_HEAD, true>(back, dw) : pick_rope_pass<FP16, NH, BO_NORM_HEAD, false>(back, dw);
    default:
      return half ? pick_rope_pass<FP16, NH, BO_NORM_ALL, true>(back, dw) : pick_rope_pass<FP16, NH, BO_NORM_ALL, false>(back, dw);
  }
}
template <bool FP16>
RopeKernel pick_rope(int nh, int norm, bool half, bool back, bool dw) {
  return nh == 1   ? pick_rope_norm<FP16, 1>(norm, half, back, dw)
         : nh == 2 ? pick_rope_norm<FP16, 2>(norm, half, back, dw)
                   : pick_rope_norm<FP16, 4>(norm, half, back, dw);
}

}  // namespace block_ops
