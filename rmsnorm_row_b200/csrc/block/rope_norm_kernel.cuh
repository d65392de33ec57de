// RMS norm of q or k and rotary positions over several axes, and the gradient
// (contract: include/block_ops.h, rope_norm).
//
// Mathematics, per token of H heads of hd channels: rho = 1 / sqrt(mean(x^2) + eps) over the
// head or the token, n = x rho w, and pair i of each head turned by position[axis(i)] freq(i).
// The gradient turns grad back (dn), then dx = rho (w dn - x rho^2 mean(w dn x)) and
// dw = sum dn x rho.
//
// Bound: HBM. A token moves 2 + 2 bytes per channel (gradient: 2 + 2 + 2). At the copy rate an
// SM has about 3500 instruction slots for a forward row of 5120 channels and 5200 for a gradient
// row, so instructions count too: the arithmetic runs on pairs of fp32, a warp keeps a whole
// row, and the angles of a token, which all heads share, are reduced once (in fp64) and left
// as cos and sin in shared memory.
//
// Layout: a thread owns "units" of 16 channels of a head as two 16-byte vectors A and B, the
// same unit u in each of its heads (W lanes to a head, W the power of two from hd / 16 up).
// Half pairing puts the 8 partners of A in B, so every pair is inside one thread; adjacent
// pairing has A in the head's first half and B in its second, so that neighbouring lanes touch
// neighbouring vectors. A norm over the head is a shuffle inside W lanes.
//
// B200, 40 heads of 128: 176400 tokens forward 639 us, 5.7 TB/s of the 6.6 of a plain copy (1730
// instructions a row); gradient of 90000 tokens 553 to 597 us, 4.7 TB/s (4100 a row, issue 58% busy).
#pragma once

#include "../../../include/block_ops.h"
#include "elements.cuh"

namespace block_ops {

constexpr int kMaxPairs = 256;      // of a head
constexpr int kRopeThreads = 512;   // of a CTA, at most
constexpr int kForwardThreads = 384;  // of a forward CTA: a lane's ten heads in 168 registers, but for 52 bytes (half pairs 72)
constexpr int kSharedRows = 128;    // threads of a CTA whose rows take 32 lanes or fewer
constexpr int kMaxPartials = 1024;  // CTAs that sum dweight
constexpr int kMaxTurns = 512;      // rows (of each slot) that a CTA sums dweight over in a launch

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
  uint32_t rows, L;         // rows up to which the launch goes
  uint32_t first;           // the gradient: its first row
  int add;                  // the CTAs' parts of dweight are added to those of a launch before
  DivU32 div_L;
  int H, hd, units, pairs;  // units of a head (hd / 16), pairs that turn
  int W, T, G;              // lanes of a head, threads of a row, lane groups (of a warp, in the forward kernel)
  int stages;               // rows of the gradient kernel in shared memory: 2 or 1
  float sign;               // -1 turns the other way
  int index64, weight_fp32;
  int weight_sh, weight_units;  // units from a head's weights to the next (0: one head's); units of it (0: none)
  float inv_n, eps;
  double inv_n64, eps64;
  double turns[kMaxPairs];    // freq / 2 pi
  uint8_t axis[kMaxPairs];
};

// ---- one thread's place in a row ---------------------------------------------------------------

struct Place {
  int u, g;        // unit, lane group
  int offA, offB;  // channels of the two vectors in the head
  int pairA, pairB;  // first pairs of the two runs of four that the thread turns
  bool owns;       // u is a unit of the head
};

template <bool HALF>
__device__ __forceinline__ Place unit_place(const RopeParams& p, int u) {
  Place q;
  q.u = u, q.g = 0, q.owns = true;
  if (!HALF) {
    q.offA = 8 * q.u, q.offB = p.hd / 2 + 8 * q.u;
    q.pairA = 4 * q.u, q.pairB = p.hd / 4 + 4 * q.u;
  } else {
    q.offA = 8 * q.u, q.offB = p.pairs + 8 * q.u;
    if (8 * q.u >= p.pairs) q.offA = 16 * q.u, q.offB = 16 * q.u + 8;  // channels that pass
    q.pairA = 8 * q.u, q.pairB = 8 * q.u + 4;
  }
  return q;
}
// Thread t's unit and head group.
template <bool HALF>
__device__ __forceinline__ Place place_of(const RopeParams& p, int t) {
  const int u = t & (p.W - 1);
  Place q = unit_place<HALF>(p, u < p.units ? u : 0);  // without a unit it reads what it may, and stores nothing
  q.g = t / p.W;
  q.owns = u < p.units;
  return q;
}

// The unit's 16 values as fp32 pairs {first, second}[4]: element j of each holds two pairs'
// first (second) channels, so that one instruction works on two pairs. The four words of
// adjacent pairing hold a pair each; those of half pairing hold two pairs' same side.
template <bool FP16, bool HALF>
__device__ __forceinline__ void split(const uint4& a, const uint4& b, uint64_t (&first)[4], uint64_t (&second)[4]) {
  using namespace fused_norm_impl;
#pragma unroll
  for (int j = 0; j < 4; ++j) {
    if (HALF) {
      const float2 e = widen16<FP16>(word(a, j)), f = widen16<FP16>(word(b, j));
      first[j] = pk2(e.x, e.y), second[j] = pk2(f.x, f.y);
    } else {
      const uint4& v = j < 2 ? a : b;
      const float2 e = widen16<FP16>(word(v, 2 * (j & 1))), f = widen16<FP16>(word(v, 2 * (j & 1) + 1));
      first[j] = pk2(e.x, f.x), second[j] = pk2(e.y, f.y);
    }
  }
}
template <bool FP16, bool HALF>
__device__ __forceinline__ void join(const uint64_t (&first)[4], const uint64_t (&second)[4], uint4& a, uint4& b) {
  uint32_t wa[4], wb[4];
#pragma unroll
  for (int j = 0; j < 4; ++j) {
    float x0, x1, y0, y1;
    fused_norm_impl::upk2(first[j], x0, x1);
    fused_norm_impl::upk2(second[j], y0, y1);
    if (HALF) {
      wa[j] = pack16<FP16>(x0, x1), wb[j] = pack16<FP16>(y0, y1);
    } else {
      uint32_t(&w)[4] = j < 2 ? wa : wb;
      w[2 * (j & 1)] = pack16<FP16>(x0, y0), w[2 * (j & 1) + 1] = pack16<FP16>(x1, y1);
    }
  }
  a = make_uint4(wa[0], wa[1], wa[2], wa[3]), b = make_uint4(wb[0], wb[1], wb[2], wb[3]);
}
// Where element (j, half, side) of a split unit lies: channel of the head.
template <bool HALF>
__device__ __forceinline__ int channel_of(const Place& q, int j, int half, int side) {
  if (HALF) return (side ? q.offB : q.offA) + 2 * j + half;
  return (j < 2 ? q.offA : q.offB) + 4 * (j & 1) + 2 * half + side;
}

// The weights in shared memory as fp32 in the order of split units, which CTAs keep for all
// their rows (widening and addressing them in global memory took a fifth of a row's
// instructions), ones without a weight. The four quarters of eight units' values alternate, so that eight lanes read
// 128 bytes without bank conflicts.
__host__ __device__ constexpr int weight_floats(int units) { return (units + 7) / 8 * 128; }
__device__ __forceinline__ int weight_at(int unit) { return (unit >> 3) * 128 + (unit & 7) * 4; }

template <bool FP16, bool HALF>
__device__ __forceinline__ void fill_weights(const RopeParams& p, float* to) {
  for (int i = threadIdx.x; i < p.weight_units; i += blockDim.x) {
    const int h = i / p.units;
    const Place q = unit_place<HALF>(p, i - h * p.units);
#pragma unroll
    for (int e = 0; e < 16; ++e) {
      const int at = h * p.hd + channel_of<HALF>(q, e / 2 % 4, e & 1, e / 8);
      to[weight_at(i) + e / 4 * 32 + e % 4] = !p.weight       ? 1.0f
                                              : p.weight_fp32 ? __ldg(static_cast<const float*>(p.weight) + at)
                                                              : widen16<FP16>(__ldg(static_cast<const uint16_t*>(p.weight) + at)).x;
    }
  }
}
// x times the weights at w.
__device__ __forceinline__ void weigh(const float* w, uint64_t (&first)[4], uint64_t (&second)[4]) {
#pragma unroll
  for (int j = 0; j < 4; j += 2) {
    const ulonglong2 a = *reinterpret_cast<const ulonglong2*>(w + 16 * j), b = *reinterpret_cast<const ulonglong2*>(w + 64 + 16 * j);
    first[j] = fused_norm_impl::mul2(first[j], a.x), first[j + 1] = fused_norm_impl::mul2(first[j + 1], a.y);
    second[j] = fused_norm_impl::mul2(second[j], b.x), second[j + 1] = fused_norm_impl::mul2(second[j + 1], b.y);
  }
}

// cos and sin of the unit's eight pairs, in the order of a split unit.
struct Turn {
  uint64_t c[4], s[4];
};
// A row's table: cos of every pair of the head, then sin (1 and 0 for pairs that pass).
__device__ __forceinline__ Turn load_turn(const RopeParams& p, const Place& q, const float* table) {
  Turn t;
  const float* sides[2] = {table, table + p.hd / 2};
#pragma unroll
  for (int i = 0; i < 2; ++i) {
    uint64_t(&o)[4] = i ? t.s : t.c;
    const ulonglong2 a = *reinterpret_cast<const ulonglong2*>(sides[i] + q.pairA), b = *reinterpret_cast<const ulonglong2*>(sides[i] + q.pairB);
    o[0] = a.x, o[1] = a.y, o[2] = b.x, o[3] = b.y;
  }
  return t;
}
__device__ __forceinline__ uint64_t negated(uint64_t v) { return v ^ 0x8000000080000000ull; }

// The pairs turned by their angles (SIGN -1: turned back). PASS: some pairs of a head pass, and
// are put back, or a NaN would enter its partner.
template <bool HALF, bool PASS, int SIGN>
__device__ __forceinline__ void turn(const RopeParams& p, const Place& q, const Turn& t, uint64_t (&first)[4], uint64_t (&second)[4]) {
  using namespace fused_norm_impl;
  uint64_t x[4], y[4];
#pragma unroll
  for (int j = 0; j < 4; ++j) {
    const uint64_t n = negated(t.s[j]);
    x[j] = fma2(second[j], SIGN > 0 ? n : t.s[j], mul2(first[j], t.c[j]));
    y[j] = fma2(first[j], SIGN > 0 ? t.s[j] : n, mul2(second[j], t.c[j]));
  }
  if (PASS) {
#pragma unroll
    for (int j = 0; j < 4; ++j) {
      const int pair = (j < 2 ? q.pairA : q.pairB) + 2 * (j & 1);
      float x0, x1, y0, y1, a0, a1, b0, b1;
      upk2(first[j], x0, x1), upk2(second[j], y0, y1), upk2(x[j], a0, a1), upk2(y[j], b0, b1);
      if (pair >= p.pairs) a0 = x0, b0 = y0;
      if (pair + 1 >= p.pairs) a1 = x1, b1 = y1;
      x[j] = pk2(a0, a1), y[j] = pk2(b0, b1);
    }
  }
#pragma unroll
  for (int j = 0; j < 4; ++j) first[j] = x[j], second[j] = y[j];
}

// Puts back the packed pairs that do not turn.
template <bool HALF>
__device__ __forceinline__ void keep_passing(const RopeParams& p, const Place& q, const uint4& a, const uint4& b, uint4& oa, uint4& ob) {
  if (HALF) {
    if (8 * q.u >= p.pairs) oa = a, ob = b;
    return;
  }
  const int ka = p.pairs - q.pairA, kb = p.pairs - q.pairB;  // pairs of each vector that turn
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
// [-1/2, 1/2]; what fp32 then adds is 2^-25 of a turn. The position of a thread's first pair is
// read a row ahead (`ahead`): it would come from L2 right before a barrier. Pairs that pass have
// cos 1 and sin 0.
struct Angles {
  const double* turns;  // of the pairs, in shared memory
  const uint8_t* axis;
  int2 ahead;  // low and high half of a position

  __device__ __forceinline__ int2 position(const RopeParams& p, const RowAt& at, int i) const {
    const int64_t o = at.b * p.pos_sb + at.l * p.pos_sl + axis[i];
    if (p.index64) return __ldg(static_cast<const int2*>(p.positions) + o);
    return make_int2(__ldg(static_cast<const int*>(p.positions) + o), 0);
  }
  __device__ __forceinline__ void read_ahead(const RopeParams& p, const RowAt& at, int t) {
    if (t < p.pairs) ahead = position(p, at, t);
  }
  __device__ __forceinline__ void fill(const RopeParams& p, const RowAt& at, int t, float* table) const {
#pragma unroll 1
    for (int i = t; i < p.hd / 2; i += p.T) {
      float s = 0.0f, c = 1.0f;
      if (i < p.pairs) {
        const int2 v = i == t ? ahead : position(p, at, i);
        const double pos = p.index64 ? (double)((long long)((unsigned long long)(unsigned)v.y << 32 | (unsigned)v.x)) : (double)v.x;
        double a = pos * turns[i];
        a -= rint(a);
        sincospif(2.0f * (float)a, &s, &c);
      }
      table[i] = c, table[p.hd / 2 + i] = s * p.sign;
    }
  }
};

template <typename V>
__device__ __forceinline__ V lanes_sum(V v, int lanes) {
  if (lanes == 32) {
#pragma unroll
    for (int o = 16; o >= 1; o >>= 1) v += __shfl_xor_sync(0xFFFFFFFFu, v, o);
    return v;
  }
#pragma unroll 1
  for (int o = lanes >> 1; o >= 1; o >>= 1) v += __shfl_xor_sync(0xFFFFFFFFu, v, o);
  return v;
}

// fp32 sums of squares that are kept: outside, the sums are taken again in fp64.
__device__ __forceinline__ bool in_range(float ss) { return ss >= 0x1p-80f && ss <= 0x1p+100f; }

__device__ __forceinline__ float sum_of(uint64_t v) {
  float a, b;
  fused_norm_impl::upk2(v, a, b);
  return a + b;
}

// The sum of eight values' squares in fp64, for the rare rows. The values are read again, and
// the loop stays rolled: walking the registers would set the allocation of the whole kernel.
template <bool FP16>
__device__ __forceinline__ double exact_squares(const uint16_t* at) {
  double s = 0.0;
#pragma unroll 1
  for (int i = 0; i < 4; ++i) {
    const float2 e = widen16<FP16>(*(reinterpret_cast<const uint32_t*>(at) + i));
    s = fma((double)e.y, (double)e.y, fma((double)e.x, (double)e.x, s));
  }
  return s;
}

// ---- forward ---------------------------------------------------------------------------------
//
// A row belongs to one warp (or to fewer lanes, rows sharing warps; or to the P = T / 32 warps
// of a CTA, where there are few rows or the row is long), whose lanes hold all of it in
// registers as it was loaded: one barrier at most, and the lane's cos and sin serve all its
// heads. Each head's registers take the next row's vectors as soon as its output is stored, so
// loads are in flight while the row is worked on.

struct alignas(16) ForwardShared {
  double turns[kMaxPairs];
  float sums[2][kForwardThreads / 32][32];
  double sums64[kForwardThreads / 32];
  uint8_t axis[kMaxPairs];
};
static_assert(sizeof(ForwardShared) % 16 == 0, "the tables behind it are 16-byte aligned");
inline size_t forward_shared_bytes(int rows_per_cta, int hd, int weights) {
  return sizeof(ForwardShared) + ((size_t)2 * rows_per_cta * hd + weights) * sizeof(float);
}

template <bool FP16, int NH, int NORM, bool HALF, bool PASS>
__global__ void __launch_bounds__(kForwardThreads, 1) rope_norm_rows(const __grid_constant__ RopeParams p) {
  using namespace fused_norm_impl;
  extern __shared__ __align__(16) unsigned char raw[];
  ForwardShared& sh = *reinterpret_cast<ForwardShared*>(raw);
  const int T = p.T, R = blockDim.x / T;  // R > 1 only where T <= 32
  const int slot = threadIdx.x / T, t = threadIdx.x - slot * T;
  const bool wide = T > 32;
  const int lane = threadIdx.x & 31, warp = wide ? t >> 5 : 0, P = wide ? T >> 5 : 1;
  const Place q = place_of<HALF>(p, wide ? lane : t);
  float* const tables = reinterpret_cast<float*>(raw + sizeof(ForwardShared)) + (size_t)slot * p.hd;
  for (int i = threadIdx.x; i < p.pairs; i += blockDim.x) sh.turns[i] = p.turns[i], sh.axis[i] = p.axis[i];
  float* const weights = reinterpret_cast<float*>(raw + sizeof(ForwardShared)) + (size_t)2 * R * p.hd;
  if (NORM != BO_NORM_NONE) fill_weights<FP16, HALF>(p, weights);
  __syncthreads();

  // Heads of a pass over the row: NH of each lane group of each warp; a norm over all heads
  // takes one pass.
  const int per_pass = P * NH * p.G;
  const int head0 = warp * NH * p.G + q.g;
  // The number of the thread's heads in the pass that starts with its head h.
  auto heads_from = [&](int h) { return q.owns && h < p.H ? (p.H - h + p.G - 1) / p.G : 0; };
  const int apart = q.offB - q.offA;
  uint4 a[NH], b[NH];
  // One head's two vectors, A at `from`; on to the thread's next head.
  auto load = [&](const uint16_t*& from, int k, int n) {
    if (k < n) {
      a[k] = __ldcs(reinterpret_cast<const uint4*>(from));
      b[k] = __ldcs(reinterpret_cast<const uint4*>(from + apart));
    }
    from += p.G * p.x.sh;
  };
  const int n0 = heads_from(head0);
  const uint32_t step = gridDim.x * R;
  uint32_t row = blockIdx.x * R + slot;
  RowAt at = row_at(p, row);
#pragma unroll
  for (int k = 0; k < NH; ++k) a[k] = b[k] = make_uint4(0, 0, 0, 0);
  Angles angles{sh.turns, sh.axis, make_int2(0, 0)};
  if (row < p.rows) {
    angles.read_ahead(p, at, t);
    const uint16_t* from = row_ptr(p.x, at) + (head0 * p.x.sh + q.offA);
#pragma unroll
    for (int k = 0; k < NH; ++k) load(from, k, n0);
  }
  // the lanes of a warp go round together; step + rows < 2^32, the host bounds both
  for (int parity = 0; wide ? row < p.rows : __any_sync(0xFFFFFFFFu, row < p.rows); row += step, parity ^= 1) {
    const bool live = row < p.rows;
    const RowAt next = row_at(p, row + step);
    const bool more = live && row + step < p.rows;
    float* const table = tables + (size_t)parity * R * p.hd;
    if (live) angles.fill(p, at, t, table);
    if (more) angles.read_ahead(p, next, t);
    const uint16_t* const xr = row_ptr(p.x, at);
    float rho = 1.0f;
    float part = 0.0f;  // of the row's squares: pairs of heads, then the pairs in order, whatever NH is
    if (NORM == BO_NORM_ALL) {
#pragma unroll
      for (int k = 0; k < NH; k += 2) {
        uint64_t s[2] = {0, 0};
#pragma unroll
        for (int i = k; i < k + 2 && i < NH; ++i) {
          uint64_t x[4], y[4];
          split<FP16, HALF>(a[i], b[i], x, y);
#pragma unroll
          for (int j = 0; j < 4; ++j) s[0] = fma2(x[j], x[j], s[0]), s[1] = fma2(y[j], y[j], s[1]);
        }
        part += sum_of(add2(s[0], s[1]));
      }
      if (wide) sh.sums[parity][warp][lane] = part;
    }
    if (wide) __syncthreads();
    else __syncwarp();
    const Turn turns = load_turn(p, q, table);
    if (NORM == BO_NORM_ALL) {
      if (wide) {
        part = sh.sums[parity][0][lane];
        for (int w = 1; w < P; ++w) part += sh.sums[parity][w][lane];
      }
      const float ss = lanes_sum(part, wide ? 32 : T);
      rho = rsqrtf(fmaf(ss, p.inv_n, p.eps));
      const bool odd = live && !in_range(ss);
      if (__any_sync(0xFFFFFFFFu, odd)) {  // a wide row's threads agree
        double e = 0.0;
#pragma unroll 1
        for (int k = 0; k < NH; ++k)
          if (live && k < n0) {
            const uint16_t* v = xr + (head0 + k * p.G) * p.x.sh;
            e += exact_squares<FP16>(v + q.offA) + exact_squares<FP16>(v + q.offB);
          }
        e = lanes_sum(e, wide ? 32 : T);
        if (wide) {
          if (lane == 0) sh.sums64[warp] = e;
          __syncthreads();
          e = 0.0;
          for (int w = 0; w < P; ++w) e += sh.sums64[w];
          __syncthreads();
        }
        if (odd) rho = (float)rsqrt(e * p.inv_n64 + p.eps64);
      }
    }
    uint16_t* const out = const_cast<uint16_t*>(row_ptr(p.out, at));
    for (int base = 0; base < (NORM == BO_NORM_ALL ? 1 : p.H); base += per_pass) {
      const bool last = NORM == BO_NORM_ALL || base + per_pass >= p.H;
      const int first = here(base + head0);
      uint16_t* to = out + (first * p.out.sh + q.offA);
      const uint16_t* from = (last ? row_ptr(p.x, next) + head0 * p.x.sh : xr + (first + per_pass) * p.x.sh) + q.offA;
      int unit = first * p.weight_sh + q.u;
      const int n = live ? NORM == BO_NORM_ALL ? n0 : heads_from(first) : 0;
      const int n_next = last ? (more ? n0 : 0) : live ? heads_from(first + per_pass) : 0;
#pragma unroll
      for (int k = 0; k < NH; ++k) {
        // What a thread without this head computes is not stored.
        uint64_t x[4], y[4];
        if (NORM == BO_NORM_HEAD) {
          split<FP16, HALF>(a[k], b[k], x, y);
          uint64_t s[2] = {0, 0};
#pragma unroll
          for (int j = 0; j < 4; ++j) s[0] = fma2(x[j], x[j], s[0]), s[1] = fma2(y[j], y[j], s[1]);
          const float ss = lanes_sum(q.owns ? sum_of(add2(s[0], s[1])) : 0.0f, p.W);
          rho = rsqrtf(fmaf(ss, p.inv_n, p.eps));
          const bool odd = k < n && !in_range(ss);
          if (__any_sync(0xFFFFFFFFu, odd)) {
            double e = 0.0;
            const uint16_t* v = xr + (first + k * p.G) * p.x.sh;
            if (k < n) e = exact_squares<FP16>(v + q.offA) + exact_squares<FP16>(v + q.offB);
            e = lanes_sum(e, p.W);
            if (odd) rho = (float)rsqrt(e * p.inv_n64 + p.eps64);
          }
        }
        split<FP16, HALF>(here(a[k]), here(b[k]), x, y);
        if (NORM != BO_NORM_NONE) {
#pragma unroll
          for (int j = 0; j < 4; ++j) x[j] = mul2(x[j], pk2(rho, rho)), y[j] = mul2(y[j], pk2(rho, rho));
          weigh(weights + weight_at(min(unit, p.weight_units - 1)), x, y);
        }
        turn<HALF, PASS && NORM != BO_NORM_NONE, 1>(p, q, turns, x, y);
        uint4 oa, ob;
        join<FP16, HALF>(x, y, oa, ob);
        if (NORM == BO_NORM_NONE && PASS) keep_passing<HALF>(p, q, a[k], b[k], oa, ob);  // a NaN keeps its bits too
        if (k < n) {
          __stcs(reinterpret_cast<uint4*>(to), oa);
          __stcs(reinterpret_cast<uint4*>(to + apart), ob);
        }
        to += p.G * p.out.sh, unit += p.G * p.weight_sh;
        load(from, k, n_next);
      }
    }
    at = next;
  }
}

// ---- gradient --------------------------------------------------------------------------------
//
// One row per CTA turn (rows of 32 lanes or fewer share warps) with NH heads to a thread, since
// a thread also keeps dn between the sums and the output, and the sums of dweight over its rows.
// Each thread copies its own vectors of the next row to shared memory while it works on the
// present one, so no registers wait for loads and nobody else has to be waited for. 128 registers and two
// stages let three CTAs of a row of 5120 channels run side by side (two with 168 registers or a
// third stage): 1.08 against 1.24 ms over 176400 tokens. Two heads to a thread spill 4 bytes;
// four, taken where two leave more lanes idle, some 700 with dweight of all heads.

// A thread's own two vectors of a head, in shared memory: x's, then grad's. One stage holds all
// heads of a thread; vectors of neighbouring threads are neighbours.
struct Stage {
  uint4* mine;  // vector 0 of head 0
  int step;     // vectors from one to the next: the CTA's threads
  __device__ __forceinline__ uint4* at(int k, int v) const { return mine + (k * 4 + v) * step; }
};

// A head's sums of x^2 and of w dn x over this thread's channels in fp64, for the rare rows.
template <bool FP16, bool HALF, bool PASS>
__device__ __noinline__ double2 exact_sums(const RopeParams& p, const Place& q, const float* table, const Stage& st, int k, const float* weight) {
  uint64_t x[2][4], d[2][4];
  split<FP16, HALF>(*st.at(k, 0), *st.at(k, 1), x[0], x[1]);
  split<FP16, HALF>(*st.at(k, 2), *st.at(k, 3), d[0], d[1]);
  turn<HALF, PASS, -1>(p, q, load_turn(p, q, table), d[0], d[1]);
  double2 r = make_double2(0.0, 0.0);
  for (int i = 0; i < 2; ++i)
    for (int j = 0; j < 4; ++j) {
      float xe[2], de[2];
      fused_norm_impl::upk2(x[i][j], xe[0], xe[1]);
      fused_norm_impl::upk2(d[i][j], de[0], de[1]);
      for (int e = 0; e < 2; ++e) {
        r.x = fma((double)xe[e], (double)xe[e], r.x);
        r.y = fma((p.weight ? (double)weight[64 * i + j / 2 * 32 + j % 2 * 2 + e] : 1.0) * (double)de[e], (double)xe[e], r.y);
      }
    }
  return r;
}

// 16 bytes, or (bytes = 0) zeros without reading.
__device__ __forceinline__ void copy_async(uint4* to, const uint16_t* from, uint32_t bytes) {
  asm volatile("cp.async.cg.shared.global [%0], [%1], 16, %2;" ::"r"((uint32_t)__cvta_generic_to_shared(to)), "l"(from), "r"(bytes) : "memory");
}

// Shared memory of a CTA: the frequency table, sums; then three tables of cos and sin per row
// slot, the weights, and the stages of rows (two, or one where two do not fit). A row's table is
// written before the barrier of the row ahead of it and read up to the barrier of the row behind
// it, so its buffer comes round again at the third row.
constexpr int kTables = 3;
struct alignas(16) BackwardShared {
  double turns[kMaxPairs];
  double sums64[2][kRopeThreads / 32];
  float2 sums[kTables][kRopeThreads / 32];
  uint8_t axis[kMaxPairs];
};
__host__ __device__ inline size_t backward_tables_bytes(int rows_per_cta, int hd) {
  return (size_t)kTables * rows_per_cta * hd * sizeof(float);
}
inline size_t backward_shared_bytes(int rows_per_cta, int hd, int weights, int threads, int nh, int stages) {
  return sizeof(BackwardShared) + backward_tables_bytes(rows_per_cta, hd) + (size_t)weights * sizeof(float) + (size_t)stages * threads * nh * 4 * 16;
}
static_assert(sizeof(BackwardShared) % 16 == 0, "what follows is 16-byte aligned");

// NORM: over the head or over all. DW: there is a weight, whose gradient's partials the kernel
// sums. Heads that a thread does not have, and rows past the last, are zeros in shared memory:
// all arithmetic is unconditional, so that the heads' instructions mix.
template <bool FP16, int NH, int NORM, bool HALF, bool DW, bool PASS>
__global__ void __launch_bounds__(kRopeThreads, 1) rope_norm_gradient(const __grid_constant__ RopeParams p) {
  using namespace fused_norm_impl;
  extern __shared__ __align__(16) unsigned char raw[];
  BackwardShared& sh = *reinterpret_cast<BackwardShared*>(raw);
  float* const tables = reinterpret_cast<float*>(raw + sizeof(BackwardShared));
  const int T = p.T, R = blockDim.x / T;  // R > 1 only where T <= 32
  const int slot = threadIdx.x / T, t = threadIdx.x - slot * T;
  const bool wide = T > 32;
  const Place q = place_of<HALF>(p, t);
  float* const weights = tables + (size_t)kTables * R * p.hd;
  uint4* const stages = reinterpret_cast<uint4*>(weights + weight_floats(p.weight_units)) + threadIdx.x;
  for (int i = threadIdx.x; i < p.pairs; i += blockDim.x) sh.turns[i] = p.turns[i], sh.axis[i] = p.axis[i];
  // A slot without a row turns its zeros by what its table holds, and they are added to dweight:
  // what another kernel left there may be a NaN.
  if (!wide)
    for (int i = threadIdx.x; i < kTables * R * p.hd; i += blockDim.x) tables[i] = 0.0f;
  fill_weights<FP16, HALF>(p, weights);
  __syncthreads();
  const int apart = q.offB - q.offA;
  auto weight = [&](int k) { return weights + weight_at(min((q.g + k * p.G) * p.weight_sh + q.u, p.weight_units - 1)); };
  auto table = [&](int buf) { return tables + (size_t)(buf * R + slot) * p.hd; };
  auto stage = [&](int buf) { return Stage{stages + (size_t)buf * NH * 4 * blockDim.x, (int)blockDim.x}; };
  auto has = [&](int k) { return q.owns && q.g + k * p.G < p.H; };
  auto fetch = [&](const RowAt& at, bool live, int buf) {
    const Stage st = stage(buf);
    const uint16_t* x = live ? row_ptr(p.x, at) + (q.g * p.x.sh + q.offA) : p.x.ptr;
    const uint16_t* d = live ? row_ptr(p.dy, at) + (q.g * p.dy.sh + q.offA) : p.dy.ptr;
#pragma unroll
    for (int k = 0; k < NH; ++k) {
      const uint32_t bytes = live && has(k) ? 16 : 0;
      copy_async(st.at(k, 0), x, bytes);
      copy_async(st.at(k, 1), x + apart, bytes);
      copy_async(st.at(k, 2), d, bytes);
      copy_async(st.at(k, 3), d + apart, bytes);
      x += p.G * p.x.sh, d += p.G * p.dy.sh;
    }
    asm volatile("cp.async.commit_group;" ::: "memory");
  };

  constexpr int NACC = NORM == BO_NORM_ALL ? NH : 1;
  uint64_t acc[DW ? NACC : 1][8];
#pragma unroll
  for (int k = 0; k < (DW ? NACC : 1); ++k)
#pragma unroll
    for (int i = 0; i < 8; ++i) acc[k][i] = 0;

  uint64_t dx[NH][4], dy[NH][4];  // dn of the present row
  // dn of head k, and its sums of x^2 and w dn x.
  auto begin = [&](const Turn& turns, const Stage& st, int k) {
    uint64_t x[4], y[4], sx[2] = {0, 0}, sg[2] = {0, 0};
    split<FP16, HALF>(*st.at(k, 2), *st.at(k, 3), dx[k], dy[k]);
    turn<HALF, PASS, -1>(p, q, turns, dx[k], dy[k]);
    split<FP16, HALF>(*st.at(k, 0), *st.at(k, 1), x, y);
#pragma unroll
    for (int j = 0; j < 4; ++j) sx[0] = fma2(x[j], x[j], sx[0]), sx[1] = fma2(y[j], y[j], sx[1]);
    uint64_t gx[4], gy[4];
#pragma unroll
    for (int j = 0; j < 4; ++j) gx[j] = dx[k][j], gy[j] = dy[k][j];
    if (DW) weigh(weight(k), gx, gy);
#pragma unroll
    for (int j = 0; j < 4; ++j) sg[0] = fma2(gx[j], x[j], sg[0]), sg[1] = fma2(gy[j], y[j], sg[1]);
    return make_float2(sum_of(add2(sx[0], sx[1])), sum_of(add2(sg[0], sg[1])));
  };
  // The output of head k, and its part of dweight; m = mean(w dn x) rho.
  auto finish = [&](const Stage& st, uint16_t* ob, bool store, int k, float rho, float m) {
    const uint64_t rr = pk2(rho, rho), mm = pk2(-m, -m);
    uint64_t x[4], y[4];
    split<FP16, HALF>(*st.at(k, 0), *st.at(k, 1), x, y);
#pragma unroll
    for (int j = 0; j < 4; ++j) x[j] = mul2(x[j], rr), y[j] = mul2(y[j], rr);
    if (DW) {
      uint64_t(&s)[8] = acc[NORM == BO_NORM_ALL ? k : 0];
#pragma unroll
      for (int j = 0; j < 4; ++j) s[j] = fma2(dx[k][j], x[j], s[j]), s[4 + j] = fma2(dy[k][j], y[j], s[4 + j]);
    }
    if (DW) weigh(weight(k), dx[k], dy[k]);
#pragma unroll
    for (int j = 0; j < 4; ++j) x[j] = mul2(rr, fma2(x[j], mm, dx[k][j])), y[j] = mul2(rr, fma2(y[j], mm, dy[k][j]));
    uint4 va, vb;
    join<FP16, HALF>(x, y, va, vb);
    if (store && has(k)) {
      uint16_t* const to = ob + (here(q.g + k * p.G) * p.out.sh + q.offA);
      __stcs(reinterpret_cast<uint4*>(to), va);
      __stcs(reinterpret_cast<uint4*>(to + apart), vb);
    }
  };
  // Sums that fp32 does not hold.
  auto outside = [](float xx, float gx) { return !(in_range(xx) && fabsf(gx) <= 0x1p+100f); };

  const uint32_t step = gridDim.x * R;
  uint32_t base = p.first + blockIdx.x * R;
  RowAt at = row_at(p, base + slot), at1 = row_at(p, base + slot + step);  // rows + 2 step < 2^32: the host bounds both
  if (p.stages > 1) fetch(at, base + slot < p.rows, 0);
  Angles angles{sh.turns, sh.axis, make_int2(0, 0)};
  if (base + slot < p.rows) {
    angles.read_ahead(p, at, t);
    angles.fill(p, at, t, table(0));
  }
  if (base + slot + step < p.rows) angles.read_ahead(p, at1, t);
  if (wide) __syncthreads();
  else __syncwarp();

  for (int buf = 0, ahead = 1, now = 0; base < p.rows; base += step, buf = ahead, ahead = ahead == kTables - 1 ? 0 : ahead + 1,
           now = now == p.stages - 1 ? 0 : now + 1) {
    const uint32_t row = base + slot;
    const bool live = row < p.rows;
    const Stage st = stage(now);
    const RowAt at2 = row_at(p, row + 2 * step);
    const Turn turns = load_turn(p, q, table(buf));
    // the stage before this one is free; then this row's vectors are here
    if (p.stages == 2) {
      fetch(at1, row + step < p.rows, now ^ 1);
      asm volatile("cp.async.wait_group 1;" ::: "memory");
    } else {
      fetch(at, live, 0);
      asm volatile("cp.async.wait_group 0;" ::: "memory");
    }

    float2 all = make_float2(0.0f, 0.0f);
    if (NORM == BO_NORM_ALL) {
#pragma unroll
      for (int k = 0; k < NH; ++k) {
        const float2 s = begin(turns, st, k);
        all.x += s.x, all.y += s.y;
      }
      all.x = lanes_sum(all.x, wide ? 32 : T);
      all.y = lanes_sum(all.y, wide ? 32 : T);
      if (wide && (t & 31) == 0) sh.sums[buf][t >> 5] = all;
    }
    if (row + step < p.rows) angles.fill(p, at1, t, table(ahead));
    if (row + 2 * step < p.rows) angles.read_ahead(p, at2, t);
    if (wide) __syncthreads();
    else __syncwarp();

    uint16_t* const ob = const_cast<uint16_t*>(row_ptr(p.out, at));
    if (NORM == BO_NORM_HEAD) {
#pragma unroll
      for (int k = 0; k < NH; ++k) {
        float2 s = begin(turns, st, k);
        const bool mine = live && has(k);
        s.x = lanes_sum(s.x, p.W);
        s.y = lanes_sum(s.y, p.W);
        float rho = rsqrtf(fmaf(s.x, p.inv_n, p.eps)), m = s.y * p.inv_n * rho;
        if (__any_sync(0xFFFFFFFFu, mine && outside(s.x, s.y))) {
          double2 e = make_double2(0.0, 0.0);
          if (mine) e = exact_sums<FP16, HALF, PASS>(p, q, table(buf), st, k, weight(k));
          e.x = lanes_sum(e.x, p.W);
          e.y = lanes_sum(e.y, p.W);
          if (outside(s.x, s.y)) {
            const double f = rsqrt(e.x * p.inv_n64 + p.eps64);
            rho = (float)f, m = (float)(e.y * p.inv_n64 * f);
          }
        }
        finish(st, ob, live, k, mine ? rho : 0.0f, mine ? m : 0.0f);
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
#pragma unroll 1
        for (int k = 0; k < NH; ++k)
          if (live && has(k)) {
            const double2 one = exact_sums<FP16, HALF, PASS>(p, q, table(buf), st, k, weight(k));
            e.x += one.x, e.y += one.y;
          }
        e.x = lanes_sum(e.x, wide ? 32 : T);
        e.y = lanes_sum(e.y, wide ? 32 : T);
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
      if (!live) rho = m = 0.0f;  // zeros over zero
#pragma unroll
      for (int k = 0; k < NH; ++k) finish(st, ob, live, k, rho, m);
    }
    at = at1, at1 = at2;
  }

  if (!DW) return;
  // ---- this CTA's part of dweight --------------------------------------------------------------
  float* const part = p.partial + (size_t)blockIdx.x * (NORM == BO_NORM_ALL ? p.H * p.hd : p.hd);
  // value i of a thread: side i / 8, element (i / 2) % 4, half i % 2
  auto value = [&](int k, int i) {
    float v[2];
    upk2(acc[k][i / 2], v[0], v[1]);
    return v[i & 1];
  };
  auto put = [&](const Place& at, int k, int i, float v) {
    float& to = part[(NORM == BO_NORM_ALL ? (at.g + k * p.G) * p.hd : 0) + channel_of<HALF>(at, (i / 2) % 4, i & 1, i / 8)];
    to = p.add ? to + v : v;
  };
  if (NORM == BO_NORM_ALL && wide) {  // every channel of the token has one thread
#pragma unroll
    for (int k = 0; k < NACC; ++k) {
      if (!has(k)) continue;
#pragma unroll
      for (int i = 0; i < 16; ++i) put(q, k, i, value(k, i));
    }
    return;
  }
  // Threads with the same channels, `span` apart, are summed in fp64 and in their order, from shared
  // memory (the first stage: every thread is past its rows, and its copies have landed). Rolled: what
  // the loops keep in registers here would set the allocation of the rows' loop.
  asm volatile("cp.async.wait_all;" ::: "memory");
  const int span = NORM == BO_NORM_ALL ? T : p.W, threads = blockDim.x;
  float* const sums = reinterpret_cast<float*>(stages - threadIdx.x);
#pragma unroll
  for (int k = 0; k < NACC; ++k) {
    __syncthreads();
#pragma unroll
    for (int i = 0; i < 16; ++i) sums[i * threads + threadIdx.x] = value(k, i);
    __syncthreads();
#pragma unroll 1
    for (int j = threadIdx.x; j < 16 * span; j += threads) {
      const int i = j / span;
      const Place at = place_of<HALF>(p, j - i * span);
      double s = 0.0;
#pragma unroll 1
      for (int from = j - i * span; from < threads; from += span) s += (double)sums[i * threads + from];
      if (at.owns && at.g + k * p.G < p.H) put(at, k, i, (float)s);
    }
  }
}

using RopeKernel = void (*)(RopeParams);

// Kernels for (threads' heads, norm, pairing); the two element types are compiled in files of
// their own. Forward: 1, 2 or 4 heads, and 6 or 10 for a norm over all; gradient: 1, 2 or 4.
template <bool FP16>
RopeKernel pick_rope(int nh, int norm, bool half, bool pass);
template <bool FP16>
RopeKernel pick_rope_gradient(int nh, int norm, bool half, bool dw, bool pass);
extern template RopeKernel pick_rope<false>(int, int, bool, bool);
extern template RopeKernel pick_rope<true>(int, int, bool, bool);
extern template RopeKernel pick_rope_gradient<false>(int, int, bool, bool, bool);
extern template RopeKernel pick_rope_gradient<true>(int, int, bool, bool, bool);

template <bool FP16, int NORM, bool HALF, bool PASS>
RopeKernel pick_rope_heads(int nh) {
  if constexpr (NORM == BO_NORM_ALL) {
    if (nh == 6) return rope_norm_rows<FP16, 6, NORM, HALF, PASS>;
    if (nh == 10) return rope_norm_rows<FP16, 10, NORM, HALF, PASS>;
  }
  return nh == 1   ? rope_norm_rows<FP16, 1, NORM, HALF, PASS>
         : nh == 2 ? rope_norm_rows<FP16, 2, NORM, HALF, PASS>
                   : rope_norm_rows<FP16, 4, NORM, HALF, PASS>;
}
template <bool FP16, int NORM>
RopeKernel pick_rope_norm(int nh, bool half, bool pass) {
  if (half) return pass ? pick_rope_heads<FP16, NORM, true, true>(nh) : pick_rope_heads<FP16, NORM, true, false>(nh);
  return pass ? pick_rope_heads<FP16, NORM, false, true>(nh) : pick_rope_heads<FP16, NORM, false, false>(nh);
}
template <bool FP16>
RopeKernel pick_rope(int nh, int norm, bool half, bool pass) {
  return norm == BO_NORM_NONE   ? pick_rope_norm<FP16, BO_NORM_NONE>(nh, half, pass)
         : norm == BO_NORM_HEAD ? pick_rope_norm<FP16, BO_NORM_HEAD>(nh, half, pass)
                                : pick_rope_norm<FP16, BO_NORM_ALL>(nh, half, pass);
}

template <bool FP16, int NORM, bool HALF, bool DW, bool PASS>
RopeKernel pick_rope_gradient_heads(int nh) {
  return nh == 1   ? rope_norm_gradient<FP16, 1, NORM, HALF, DW, PASS>
         : nh == 2 ? rope_norm_gradient<FP16, 2, NORM, HALF, DW, PASS>
                   : rope_norm_gradient<FP16, 4, NORM, HALF, DW, PASS>;
}
template <bool FP16, int NORM, bool HALF>
RopeKernel pick_rope_gradient_half(int nh, bool dw, bool pass) {
  if (dw) return pass ? pick_rope_gradient_heads<FP16, NORM, HALF, true, true>(nh) : pick_rope_gradient_heads<FP16, NORM, HALF, true, false>(nh);
  return pass ? pick_rope_gradient_heads<FP16, NORM, HALF, false, true>(nh) : pick_rope_gradient_heads<FP16, NORM, HALF, false, false>(nh);
}
template <bool FP16>
RopeKernel pick_rope_gradient(int nh, int norm, bool half, bool dw, bool pass) {
  if (norm == BO_NORM_HEAD)
    return half ? pick_rope_gradient_half<FP16, BO_NORM_HEAD, true>(nh, dw, pass) : pick_rope_gradient_half<FP16, BO_NORM_HEAD, false>(nh, dw, pass);
  return half ? pick_rope_gradient_half<FP16, BO_NORM_ALL, true>(nh, dw, pass) : pick_rope_gradient_half<FP16, BO_NORM_ALL, false>(nh, dw, pass);
}

}  // namespace block_ops
