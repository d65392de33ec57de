// Matrix product with bias, activation, gate and residual in its epilogue
// (contract: include/block_ops.h, linear_gate).
//
// out = residual + gate * act(x W^T + bias). Many rows are bound by the tensor cores
// (2 M N K operations against (M + N) K + 2 M N elements), a few tokens by reading W once.
//
// Many rows: persistent CTAs or CTA pairs (CG = 2) of ten warps. One thread loads 128-byte
// wide tiles of x and W by TMA into a ring of shared-memory stages, one thread issues the
// tcgen05 products of a 128 CG x BN tile into TMEM, eight warps read the sums back, a row per
// thread, and finish them. TMEM holds two tiles, so the epilogue of one runs under the products
// of the next. A pair shares W's tile: each CTA loads half of it. Residual and output pass
// through shared memory in boxes of 32 x 32: TMA brings a warp's next residual box while the
// present one is worked on in place, and stores it. The tensor pipe is 95% busy at 18944 x 5120 x
// 5120; over seconds the power that the chip may draw sets the clock instead (176400 rows with
// residual: 6.3 ms at first, 7.2 to 8.0 sustained at 1.0 to 1.1 GHz; cuBLAS without epilogue 5.7
// and 6.6). Tiles of 512 x 256 move a quarter less through L2 but leave TMEM no second tile: 7.4
// against 7.2 ms.
//
// A few tokens: every warp streams rows of W past the tokens with 16-byte loads; one token against
// 30720 rows of 5120 takes 48 to 50 us, 97% of the copy rate.
#pragma once

#include <cuda_fp8.h>

#include "../../../include/block_ops.h"
#include "elements.cuh"
#include "tcgen05.cuh"

namespace block_ops {

struct LinearOperand {
  const uint16_t* ptr;
  int64_t sb, sf, sl;
};

struct LinearParams {
  const void* x;       // few tokens: x and W by pointer
  const void* weight;
  int64_t x_sb, x_sl, weight_stride;
  uint32_t rows, L, tpf;           // B * L < 2^31
  DivU32 div_L, div_tpf;
  uint32_t batch_rows;             // rows of a tile map's batch: L, or all rows
  uint32_t tiles_m, tiles_n, batches;  // tiles of a batch
  uint32_t tiles, group;           // all tiles; tiles of m that take turns over n
  DivU32 div_band, div_tiles_m;
  uint32_t N, K, steps;            // steps of 128 bytes over K
  uint32_t idesc;
  int act;
  const uint16_t* bias;
  LinearOperand gate, residual;
  int has_residual;
  const float *x_scale, *weight_scale;
  uint16_t* out;
  int64_t out_sb, out_sl;
  int* gave_up;  // host memory: set when a wait ran out
};

// ---- the epilogue -----------------------------------------------------------------------------

// z sigmoid(s z') forms: the quotient of a huge |z| and e^|z| is 0, of an infinity NaN.
__device__ __forceinline__ float logistic_times(float z, float e) { return __fdividef(z, 1.0f + __expf(-e)); }

// GELU z Phi(z) of two values. Phi(-|z|) = erfc(|z| / sqrt 2) / 2 = e^(-z^2 / 2) s Q(s) with
// s = 1 / (1 + 0.212 |z|): Q is the polynomial of degree 8 with the least largest relative error, 2e-8,
// over |z| <= 13.5 (fitted by reweighted least squares). 1 + erf(z / sqrt 2) loses the value where
// z < 0, and erfcf, as good, takes longer: 50000 x 2048 x 4096 555 us, with erff 568, with erfcf 698.
// e^(-z^2 / 2) below 2^-126 (z < -13.2) is 0.
__device__ __forceinline__ uint64_t gelu(uint64_t z) {
  using namespace fused_norm_impl;
  auto both = [](float v) { return pk2(v, v); };
  float z0, z1, a0, a1, e0, e1;
  upk2(z, z0, z1);
  upk2(fma2(pk2(fabsf(z0), fabsf(z1)), both(0.212132037f), both(1.0f)), a0, a1);
  const uint64_t s = pk2(__fdividef(1.0f, a0), __fdividef(1.0f, a1));
  uint64_t h = both(-0.064728424f);
  h = fma2(h, s, both(0.242608264f));
  h = fma2(h, s, both(-0.255749017f));
  h = fma2(h, s, both(0.273369312f));
  h = fma2(h, s, both(-0.0469483174f));
  h = fma2(h, s, both(0.107282139f));
  h = fma2(h, s, both(0.0742224231f));
  h = fma2(h, s, both(0.0853490382f));
  h = fma2(h, s, both(0.0845945925f));
  upk2(mul2(mul2(z, z), both(-0.72134752f)), e0, e1);  // z^2 log2(e) / 2
  asm("ex2.approx.ftz.f32 %0, %0;" : "+f"(e0));
  asm("ex2.approx.ftz.f32 %0, %0;" : "+f"(e1));
  upk2(mul2(mul2(h, s), pk2(e0, e1)), a0, a1);
  return mul2(z, pk2(z0 > 0.0f ? 1.0f - a0 : a0, z1 > 0.0f ? 1.0f - a1 : a1));
}

// SiLU and GELU's tanh form.
template <int N>
__device__ __forceinline__ void activate(int act, float (&v)[N]) {
  if (act == BO_ACT_SILU) {
#pragma unroll
    for (int i = 0; i < N; ++i) v[i] = logistic_times(v[i], v[i]);
  } else {  // 1/2 (1 + tanh t) = 1 / (1 + e^-2t)
#pragma unroll
    for (int i = 0; i < N; ++i) {
      const float t = v[i] * fmaf(v[i] * v[i], 1.5957691216057308f * 0.044715f, 1.5957691216057308f);
      v[i] = logistic_times(v[i], t);
    }
  }
}

// A row's token, gate and scale.
struct RowOut {
  uint32_t b, l;
  const uint16_t* gate;
  float x_scale;
};
__device__ __forceinline__ RowOut row_out(const LinearParams& p, uint32_t row) {
  RowOut r;
  const uint32_t b = div_u32(row, p.div_L), l = row - b * p.L;
  const uint32_t f = p.tpf ? div_u32(l, p.div_tpf) : 0u;
  r.b = b, r.l = l;
  r.gate = p.gate.ptr ? p.gate.ptr + (b * p.gate.sb + f * p.gate.sf + l * p.gate.sl) : nullptr;
  r.x_scale = p.x_scale ? __ldg(p.x_scale + row) : 1.0f;
  return r;
}

// A row's 32 columns from n on. What they need is requested first (`load`), so that it comes
// while the sums do; columns past N take the last eight's values and are not stored. The
// options are decided once for the 32, and the arithmetic runs two elements per instruction:
// per element it left 22 instructions, which set the pace at small K.
template <bool FP8, bool FP16>
struct Columns {
  uint4 bias[4], gate[4];
  float4 scale[FP8 ? 8 : 1];

  __device__ __forceinline__ void load(const LinearParams& p, const RowOut& r, uint32_t n) {
    const uint32_t last = p.N - 8;
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      const uint32_t at = min(n + 8 * i, last);
      if (p.bias) bias[i] = __ldg(reinterpret_cast<const uint4*>(p.bias + at));
      if (r.gate) gate[i] = __ldg(reinterpret_cast<const uint4*>(r.gate + at));
      if (FP8) {
        scale[2 * i] = __ldg(reinterpret_cast<const float4*>(p.weight_scale + at));
        scale[2 * i + 1] = __ldg(reinterpret_cast<const float4*>(p.weight_scale + at) + 1);
      }
    }
  }
  __device__ __forceinline__ static uint64_t pair(const uint4& v, int i) {
    const float2 e = widen16<FP16>(fused_norm_impl::word(v, i));
    return fused_norm_impl::pk2(e.x, e.y);
  }
  // v: the sums of columns [8 i, 8 i + 8) in its i-th part; e: the residual, packed; out in its place.
  __device__ __forceinline__ void finish(const LinearParams& p, const RowOut& r, float (&v)[32], uint4 (&e)[4]) const {
    using namespace fused_norm_impl;
    uint64_t z[16];
#pragma unroll
    for (int i = 0; i < 16; ++i) z[i] = pk2(v[2 * i], v[2 * i + 1]);
    if (FP8) {
      const uint64_t s = pk2(r.x_scale, r.x_scale);
#pragma unroll
      for (int i = 0; i < 8; ++i) {
        z[2 * i] = mul2(z[2 * i], mul2(s, pk2(scale[i].x, scale[i].y)));
        z[2 * i + 1] = mul2(z[2 * i + 1], mul2(s, pk2(scale[i].z, scale[i].w)));
      }
    }
    if (p.bias) {
#pragma unroll
      for (int i = 0; i < 16; ++i) z[i] = add2(z[i], pair(bias[i >> 2], i & 3));
    }
    if (p.act == BO_ACT_GELU) {
      // In two halves: sixteen pairs' instructions at once cost the other activations up to 2% where a
      // tile's epilogue runs once (999 x 2056 x 1288 with SiLU 19.0 against 18.7 us).
#pragma unroll 1
      for (int r = 0; r < 2; ++r) {
        uint64_t t[8];
#pragma unroll
        for (int i = 0; i < 8; ++i) t[i] = gelu(z[i]);
#pragma unroll
        for (int i = 0; i < 8; ++i) z[i] = z[i + 8];
#pragma unroll
        for (int i = 0; i < 8; ++i) z[8 + i] = t[i];
      }
    } else if (p.act != BO_ACT_NONE) {
#pragma unroll
      for (int i = 0; i < 16; ++i) upk2(z[i], v[2 * i], v[2 * i + 1]);
      activate(p.act, v);
#pragma unroll
      for (int i = 0; i < 16; ++i) z[i] = pk2(v[2 * i], v[2 * i + 1]);
    }
    if (r.gate) {
      if (p.has_residual) {
#pragma unroll
        for (int i = 0; i < 16; ++i) z[i] = fma2(pair(gate[i >> 2], i & 3), z[i], pair(e[i >> 2], i & 3));
      } else {
#pragma unroll
        for (int i = 0; i < 16; ++i) z[i] = mul2(z[i], pair(gate[i >> 2], i & 3));
      }
    } else if (p.has_residual) {
#pragma unroll
      for (int i = 0; i < 16; ++i) z[i] = add2(z[i], pair(e[i >> 2], i & 3));
    }
    uint32_t o[16];
#pragma unroll
    for (int i = 0; i < 16; ++i) {
      float a, b;
      upk2(z[i], a, b);
      o[i] = pack16<FP16>(a, b);
    }
#pragma unroll
    for (int i = 0; i < 4; ++i) e[i] = make_uint4(o[4 * i], o[4 * i + 1], o[4 * i + 2], o[4 * i + 3]);
  }
};

// ---- many rows ----------------------------------------------------------------------------------

constexpr int kTileM = 128;          // rows of a CTA
constexpr int kStepBytes = 128;      // of K, per row and stage
constexpr int kMaxStages = 8;
constexpr int kEpilogueWarps = 8;    // two to each quarter of the rows, each half of the columns
constexpr int kMatrixThreads = 32 * (2 + kEpilogueWarps);
constexpr int kBox = 32;             // rows and columns of an output box
constexpr int kBoxBytes = kBox * kBox * 2;

// CG CTAs work on a tile together, each on kTileM rows and all BN columns of it.
template <int CG, int BN>
struct MatrixShape {
  static constexpr int kABytes = kTileM * kStepBytes, kBBytes = BN / CG * kStepBytes;
  static constexpr int kStageBytes = kABytes + kBBytes;
  static constexpr int kBoxes = 4;  // of a warp: two being brought, one worked on, one being stored
  static constexpr int kBoxesBytes = kEpilogueWarps * kBoxes * kBoxBytes;
  static constexpr int kFit = (226 * 1024 - 1024 - kBoxesBytes) / kStageBytes;
  static constexpr int kStages = kFit < kMaxStages ? kFit : kMaxStages;
  static constexpr int kColumns = BN == 192 ? 512 : 2 * BN;  // TMEM, a power of two: two blocks of sums
  static constexpr int kShared = kStages * kStageBytes + kBoxesBytes + 1024;  // 1024: alignment
};

struct Tile {
  uint32_t batch, m, n;
};
// Tile t: bands of `group` tiles of m, n outside m within a band, so that the tiles in flight
// together share rows of x and of W in L2.
__device__ __forceinline__ Tile tile_at(const LinearParams& p, uint32_t t) {
  const uint32_t band = div_u32(t, p.div_band), in = t - band * p.group * p.tiles_n;
  const uint32_t all = p.tiles_m * p.batches, left = all - band * p.group;
  const uint32_t height = left < p.group ? left : p.group;
  const uint32_t n = in / height, m = band * p.group + (in - n * height);
  const uint32_t b = div_u32(m, p.div_tiles_m);
  return Tile{b, m - b * p.tiles_m, n};
}

__device__ int linear_gate_gave_up = 0;  // CTAs in which a wait ran out (this file is included once)

// A wait of this CTA ran out (one thread): counted here, and said to the host's next call.
__device__ __forceinline__ void say_gave_up(const LinearParams& p) {
  atomicAdd(&linear_gate_gave_up, 1);
  *(volatile int*)p.gave_up = 1;
  __threadfence_system();
}

template <int CG, int BN, bool FP8, bool FP16>
__global__ void __launch_bounds__(kMatrixThreads, 1)
linear_gate_tiles(const __grid_constant__ LinearParams p, const __grid_constant__ CUtensorMap map_x,
                  const __grid_constant__ CUtensorMap map_w, const __grid_constant__ CUtensorMap map_out,
                  const __grid_constant__ CUtensorMap map_residual) {
  using S = MatrixShape<CG, BN>;
  constexpr int kBoxes = S::kBoxes, kAhead = kBoxes / 2;
  extern __shared__ unsigned char raw[];
  __shared__ __align__(8) uint64_t full[S::kStages], empty[S::kStages], sums_full[2], sums_empty[2];
  __shared__ __align__(8) uint64_t box_full[kEpilogueWarps][kBoxes];
  __shared__ uint32_t tmem_at;
  __shared__ int failed;
  const uint32_t stages = (smem_u32(raw) + 1023u) & ~1023u;
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const uint32_t rank = CG == 2 ? cluster_rank() : 0u;

  if (threadIdx.x == 0) {
    for (int i = 0; i < S::kStages; ++i) mbar_init(smem_u32(&full[i]), 1), mbar_init(smem_u32(&empty[i]), 1);
    for (int i = 0; i < 2; ++i) mbar_init(smem_u32(&sums_full[i]), 1), mbar_init(smem_u32(&sums_empty[i]), kEpilogueWarps * CG);
    for (int i = 0; i < kBoxes * kEpilogueWarps; ++i) mbar_init(smem_u32(&box_full[i / kBoxes][i % kBoxes]), 1);
    failed = 0;
    mbar_init_fence();
  }
  if (threadIdx.x == 64) {
    prefetch_map(&map_x);
    prefetch_map(&map_w);
    prefetch_map(&map_out);
    if (p.has_residual) prefetch_map(&map_residual);
  }
  if (warp == 1) tmem_alloc<CG>(smem_u32(&tmem_at), S::kColumns);
  __syncthreads();
  if (CG == 2) cluster_sync();
  tc_fence_after();
  const uint32_t tmem = *(volatile uint32_t*)&tmem_at;

  const uint32_t first = blockIdx.x / CG, step = gridDim.x / CG;
  if (warp == 0) {
    if (elect_one()) {
      constexpr int kElems = FP8 ? 128 : 64;  // of K, per step
      uint32_t stage = 0, parity = 0;
      bool ok = true;
      for (uint32_t t = first; ok && t < p.tiles; t += step) {
        const Tile at = tile_at(p, t);
        const int row = (int)((at.m * CG + rank) * kTileM), col = (int)(at.n * BN + rank * (BN / CG));
        for (uint32_t k = 0; k < p.steps; ++k) {
          if (!(ok = mbar_wait(smem_u32(&empty[stage]), parity ^ 1, &failed))) break;
          uint32_t bar = smem_u32(&full[stage]);
          if (rank == 0) mbar_expect(bar, CG * S::kStageBytes);
          if (CG == 2) bar = map_to(bar, 0);
          const uint32_t a = stages + stage * S::kStageBytes;
          tma_load<CG == 2>(a, &map_x, (int)k * kElems, row, (int)at.batch, bar);
          tma_load<CG == 2>(a + S::kABytes, &map_w, (int)k * kElems, col, 0, bar);
          if (++stage == S::kStages) stage = 0, parity ^= 1;
        }
      }
      // The last copies have landed when their stages are free again.
      for (int i = 0; ok && i < S::kStages; ++i) {
        ok = mbar_wait(smem_u32(&empty[stage]), parity ^ 1, &failed);
        if (++stage == S::kStages) stage = 0, parity ^= 1;
      }
    }
  } else if (warp == 1) {
    if (rank == 0 && elect_one()) {
      uint32_t stage = 0, parity = 0, n = 0;
      bool ok = true;
      for (uint32_t t = first; ok && t < p.tiles; t += step, ++n) {
        const uint32_t buf = n & 1, round = (n >> 1) & 1;
        if (!(ok = mbar_wait(smem_u32(&sums_empty[buf]), round ^ 1, &failed))) break;
        tc_fence_after();
        for (uint32_t k = 0; k < p.steps; ++k) {
          if (!(ok = mbar_wait(smem_u32(&full[stage]), parity, &failed))) break;
          tc_fence_after();
          const uint32_t a = stages + stage * S::kStageBytes;
          const uint64_t da = operand_desc(a), db = operand_desc(a + S::kABytes);
#pragma unroll
          for (int i = 0; i < kStepBytes / 32; ++i)  // 32 bytes of K each
            mma<CG, FP8>(tmem + buf * BN, da + 2 * i, db + 2 * i, p.idesc, k > 0 || i > 0);
          mma_commit<CG>(smem_u32(&empty[stage]));
          if (++stage == S::kStages) stage = 0, parity ^= 1;
        }
        if (ok) mma_commit<CG>(smem_u32(&sums_full[buf]));
      }
    }
  } else {
    const int mine = warp - 2, quarter = warp & 3;  // quarter: the TMEM lanes that this warp may read
    constexpr uint32_t kHalf = BN / 2, kChunks = kHalf / kBox;
    const uint32_t half = (mine >> 2) * kHalf;           // its columns of a tile
    const uint32_t boxes = stages + S::kStages * S::kStageBytes + mine * kBoxes * kBoxBytes;
    const uint32_t bars = smem_u32(&box_full[mine][0]);
    // The residual boxes of this warp's chunks, brought in order, kAhead ahead; lane 0 only.
    uint32_t next_t = first, next_c = 0, next_box = 0;
    auto row_of = [&](const Tile& at) { return (at.m * CG + rank) * kTileM + quarter * 32; };
    auto fetch = [&]() {
      if (next_t >= p.tiles) return;
      const Tile at = tile_at(p, next_t);
      mbar_expect(bars + 8 * next_box, kBoxBytes);
      tma_load<false>(boxes + next_box * kBoxBytes, &map_residual, (int)(at.n * BN + half + next_c * kBox),
                      (int)row_of(at), (int)at.batch, bars + 8 * next_box);
      next_box = (next_box + 1) % kBoxes;
      if (++next_c == kChunks) next_c = 0, next_t += step;
    };
    if (p.has_residual && lane == 0)
      for (int i = 0; i < kAhead; ++i) fetch();
    uint32_t n = 0, chunk = 0;
    bool ok = true;
    for (uint32_t t = first; ok && t < p.tiles; t += step, ++n) {
      const uint32_t acc = n & 1, round = (n >> 1) & 1;
      if (!(ok = warp_wait(smem_u32(&sums_full[acc]), round, &failed))) break;
      tc_fence_after();
      const Tile at = tile_at(p, t);
      const uint32_t row0 = row_of(at);
      const bool live = row0 + lane < p.batch_rows;
      const RowOut r = row_out(p, live ? at.batch * p.batch_rows + row0 + lane : 0u);
      const uint32_t n0 = at.n * BN + half;
#pragma unroll 1
      for (uint32_t c = 0; c < kChunks; ++c, ++chunk) {
        const uint32_t buf = chunk % kBoxes;
        Columns<FP8, FP16> columns;
        columns.load(p, r, n0 + c * kBox);
        float v[kBox];
        tmem_load32(tmem + ((uint32_t)(quarter * 32) << 16) + acc * BN + half + c * kBox, v);
        if (lane == 0) {
          if (p.has_residual) {
            tma_stores_read<kBoxes - kAhead - 1>();  // of the box that takes the residual kAhead ahead
            fetch();
          } else {
            tma_stores_read<kBoxes - 1>();  // of this box
          }
        }
        tmem_wait();
        if (c + 1 == kChunks) {  // the sums are in registers: the next tile may have their place
          tc_fence_before();
          __syncwarp();
          if (lane == 0) mbar_arrive_cluster(map_to(smem_u32(&sums_empty[acc]), 0));
        }
        if (p.has_residual && !(ok = warp_wait(bars + 8 * buf, (chunk / kBoxes) & 1, &failed))) break;
        __syncwarp();
        // row `lane` of the box: 64 bytes, 16-byte pieces swizzled as TMA's 64-byte mode has them
        const uint32_t row = boxes + buf * kBoxBytes + lane * 64;
        auto piece = [&](int i) { return row + ((i ^ ((lane >> 1) & 3)) << 4); };
        uint4 e[4];
        if (p.has_residual) {
#pragma unroll
          for (int i = 0; i < 4; ++i)
            asm volatile("ld.shared.v4.u32 {%0, %1, %2, %3}, [%4];" : "=r"(e[i].x), "=r"(e[i].y), "=r"(e[i].z), "=r"(e[i].w) : "r"(piece(i)) : "memory");
        }
        columns.finish(p, r, v, e);
#pragma unroll
        for (int i = 0; i < 4; ++i)
          asm volatile("st.shared.v4.u32 [%0], {%1, %2, %3, %4};" ::"r"(piece(i)), "r"(e[i].x), "r"(e[i].y), "r"(e[i].z), "r"(e[i].w) : "memory");
        fence_for_tma();
        __syncwarp();
        if (lane == 0) {
          if (row0 < p.batch_rows && n0 + c * kBox < p.N)
            tma_store(&map_out, boxes + buf * kBoxBytes, (int)(n0 + c * kBox), (int)row0, (int)at.batch);
          tma_stores_commit();  // a group to every box, stored or not
        }
      }
    }
    if (lane == 0) tma_stores_read<0>();  // shared memory stays until then; the writes end with the grid
  }
  if (failed && threadIdx.x % 32 == 0) {  // leave copies in flight the time to land
    const uint64_t start = now_ns();
    while (now_ns() - start < 1000000000ull) __nanosleep(1000000);
  }
  __syncwarp();
  tc_fence_before();
  __syncthreads();
  if (CG == 2) cluster_sync();
  if (threadIdx.x == 0 && failed) say_gave_up(p);
  if (warp == 1) {
    tc_fence_after();
    tmem_free<CG>(tmem, S::kColumns);
  }
}

// ---- few tiles: the sum over K split over a cluster ------------------------------------------
//
// Where there are fewer tiles than SMs, reading x and W through the few that have one sets the
// pace (an SM takes some 80 bytes a cycle). S groups of CG CTAs, a cluster, take a tile together,
// each an S-th of K; then each group finishes an S-th of the tile's 32-column chunks, to which
// the others add their sums: they write them to its shared memory, over the stages.

template <int CG, int BN>
struct SplitShape {
  static constexpr int kStageBytes = (kTileM + BN / CG) * kStepBytes;
  static constexpr int kFit = 225 * 1024 / kStageBytes, kStages = kFit < kMaxStages ? kFit : kMaxStages;
  static constexpr int kShared = kStages * kStageBytes + 1024;
  static constexpr int kChunks = BN / kBox;
  // Sums that a CTA receives: from each other group, for each of its chunks.
  static constexpr int received(int S) { return (S - 1) * ((kChunks + S - 1) / S) * kTileM * kBox * 4; }
};

template <int CG, int BN, bool FP8, bool FP16>
__global__ void __launch_bounds__(kMatrixThreads, 1)
linear_gate_split(const __grid_constant__ LinearParams p, const __grid_constant__ CUtensorMap map_x, const __grid_constant__ CUtensorMap map_w) {
  using Shape = SplitShape<CG, BN>;
  extern __shared__ unsigned char raw[];
  __shared__ __align__(8) uint64_t full[Shape::kStages], empty[Shape::kStages], sums_full;
  __shared__ uint32_t tmem_at;
  __shared__ int failed;
  const uint32_t stages = (smem_u32(raw) + 1023u) & ~1023u;
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const uint32_t rank = cluster_rank(), size = cluster_size();
  const uint32_t S = size / CG, mine = rank / CG, side = rank % CG, leader = rank - side;

  if (threadIdx.x == 0) {
    for (int i = 0; i < Shape::kStages; ++i) mbar_init(smem_u32(&full[i]), 1), mbar_init(smem_u32(&empty[i]), 1);
    mbar_init(smem_u32(&sums_full), 1);
    failed = 0;
    mbar_init_fence();
  }
  if (threadIdx.x == 64) {
    prefetch_map(&map_x);
    prefetch_map(&map_w);
  }
  if (warp == 1) tmem_alloc<CG>(smem_u32(&tmem_at), BN);
  __syncthreads();
  if (CG == 2) cluster_sync();
  tc_fence_after();
  const uint32_t tmem = *(volatile uint32_t*)&tmem_at;

  const Tile at = tile_at(p, blockIdx.x / size);
  const uint32_t k0 = mine * p.steps / S, k1 = (mine + 1) * p.steps / S;  // S <= steps
  if (warp == 0) {
    if (elect_one()) {
      constexpr int kElems = FP8 ? 128 : 64;
      const int row = (int)((at.m * CG + side) * kTileM), col = (int)(at.n * BN + side * (BN / CG));
      uint32_t stage = 0, parity = 0;
      for (uint32_t k = k0; k < k1; ++k) {
        if (!mbar_wait(smem_u32(&empty[stage]), parity ^ 1, &failed)) break;
        uint32_t bar = smem_u32(&full[stage]);
        if (side == 0) mbar_expect(bar, CG * Shape::kStageBytes);
        if (CG == 2) bar = map_to(bar, leader);
        const uint32_t a = stages + stage * Shape::kStageBytes;
        tma_load<CG == 2>(a, &map_x, (int)k * kElems, row, (int)at.batch, bar);
        tma_load<CG == 2>(a + kTileM * kStepBytes, &map_w, (int)k * kElems, col, 0, bar);
        if (++stage == Shape::kStages) stage = 0, parity ^= 1;
      }
    }
  } else if (warp == 1) {
    if (side == 0 && elect_one()) {
      uint32_t stage = 0, parity = 0;
      bool ok = true;
      for (uint32_t k = k0; k < k1; ++k) {
        if (!(ok = mbar_wait(smem_u32(&full[stage]), parity, &failed))) break;
        tc_fence_after();
        const uint32_t a = stages + stage * Shape::kStageBytes;
        const uint64_t da = operand_desc(a), db = operand_desc(a + kTileM * kStepBytes);
#pragma unroll
        for (int i = 0; i < kStepBytes / 32; ++i) mma<CG, FP8>(tmem, da + 2 * i, db + 2 * i, p.idesc, k > k0 || i > 0);
        mma_commit<CG>(smem_u32(&empty[stage]), leader);
        if (++stage == Shape::kStages) stage = 0, parity ^= 1;
      }
      if (ok) mma_commit<CG>(smem_u32(&sums_full), leader);
    }
  } else {
    warp_wait(smem_u32(&sums_full), 0, &failed);  // every product is done, and every copy has been used
    tc_fence_after();
  }
  // A wait that ran out in one CTA leaves copies in flight and sums undone: the whole cluster is told,
  // and neither exchanges nor stores.
  __syncwarp();
  if (*(volatile int*)&failed && lane < (int)size) set_remote(map_to(smem_u32(&failed), lane), 1);
  __syncwarp();
  cluster_sync();  // now no stage of the cluster is in use, unless `gave_up`
  const bool gave_up = *(volatile int*)&failed;

  constexpr uint32_t kHalf = Shape::kChunks / 2;
  const int quarter = warp & 3;
  const uint32_t first = warp >= 2 ? (uint32_t)(warp - 2) / 4 * kHalf : 0u;  // this warp's chunks
  const uint32_t each = (Shape::kChunks + S - 1) / S;                       // chunks of a group, at most
  auto owner_of = [&](uint32_t j) { return j * S / Shape::kChunks; };
  auto first_of = [&](uint32_t o) { return (o * Shape::kChunks + S - 1) / S; };
  auto slot = [&](uint32_t from, uint32_t to, uint32_t j) {  // of sums for chunk j, from one group to another
    return stages + ((((from < to ? from : from - 1) * each + (j - first_of(to))) * 4 + quarter) * 8 * 32 + lane) * 16;
  };
  const uint32_t lanes = tmem + ((uint32_t)(quarter * 32) << 16);
  if (warp >= 2 && !gave_up) {
    for (uint32_t j = first; j < first + kHalf; ++j) {
      const uint32_t to = owner_of(j);
      if (to == mine) continue;
      float v[kBox];
      tmem_load32(lanes + j * kBox, v);
      const uint32_t there = map_to(slot(mine, to, j), to * CG + side);
      tmem_wait();
#pragma unroll
      for (int i = 0; i < 8; ++i) store_remote(there + i * 512, v[4 * i], v[4 * i + 1], v[4 * i + 2], v[4 * i + 3]);
    }
  }
  cluster_sync();
  if (warp >= 2 && !gave_up) {
    const uint32_t row0 = (at.m * CG + side) * kTileM + quarter * 32;
    const bool live = row0 + lane < p.batch_rows;
    const RowOut r = row_out(p, live ? at.batch * p.batch_rows + row0 + lane : 0u);
    const uint16_t* res = p.residual.ptr + (r.b * p.residual.sb + r.l * p.residual.sl);
    uint16_t* out = p.out + (r.b * p.out_sb + r.l * p.out_sl);
    for (uint32_t j = first; j < first + kHalf; ++j) {
      if (owner_of(j) != mine) continue;
      const uint32_t n0 = at.n * BN + j * kBox;
      Columns<FP8, FP16> columns;
      columns.load(p, r, n0);
      uint4 e[4];
      auto here_too = [&](int i) { return live && n0 + 8 * i < p.N; };
#pragma unroll
      for (int i = 0; i < 4; ++i)
        if (p.has_residual && here_too(i)) e[i] = *reinterpret_cast<const uint4*>(res + n0 + 8 * i);
      float v[kBox];
      tmem_load32(lanes + j * kBox, v);
      tmem_wait();
      for (uint32_t from = 0; from < S; ++from) {  // in the order of K's parts, after its own
        if (from == mine) continue;
        const uint32_t here = slot(from, mine, j);
#pragma unroll
        for (int i = 0; i < 8; ++i) {
          float a, b, c, d;
          asm volatile("ld.shared.v4.f32 {%0, %1, %2, %3}, [%4];" : "=f"(a), "=f"(b), "=f"(c), "=f"(d) : "r"(here + i * 512) : "memory");
          v[4 * i] += a, v[4 * i + 1] += b, v[4 * i + 2] += c, v[4 * i + 3] += d;
        }
      }
      columns.finish(p, r, v, e);
#pragma unroll
      for (int i = 0; i < 4; ++i)
        if (here_too(i)) *reinterpret_cast<uint4*>(out + n0 + 8 * i) = e[i];
    }
  }
  if (failed && lane == 0) {  // leave copies in flight the time to land
    const uint64_t start = now_ns();
    while (now_ns() - start < 1000000000ull) __nanosleep(1000000);
  }
  __syncwarp();
  tc_fence_before();
  __syncthreads();
  if (CG == 2) cluster_sync();
  if (threadIdx.x == 0 && failed) say_gave_up(p);
  if (warp == 1) {
    tc_fence_after();
    tmem_free<CG>(tmem, BN);
  }
}

// ---- a few tokens ------------------------------------------------------------------------------

constexpr int kTokens = 4;        // tokens of a launch, at most
constexpr int kTokenThreads = 128;
constexpr int kTokenColumns = 4;  // rows of W that a warp streams together

// Sixteen bytes of codes or 16-bit values as products with x, added to acc.
template <bool FP8, bool FP16>
__device__ __forceinline__ void widen_vector(const uint4& v, float (&f)[FP8 ? 16 : 8]) {
  if constexpr (FP8) {
#pragma unroll
    for (int i = 0; i < 8; ++i) {
      const uint32_t w = fused_norm_impl::word(v, i >> 1);
      const __half2_raw h = __nv_cvt_fp8x2_to_halfraw2((__nv_fp8x2_storage_t)(w >> (16 * (i & 1))), __NV_E4M3);
      const float2 e = __half22float2(__half2(h));
      f[2 * i] = e.x, f[2 * i + 1] = e.y;
    }
  } else {
    widen8<FP16>(v, f);
  }
}

// PARTS warps of a CTA share K of the same columns: one, or four.
template <int M, int PARTS, bool FP8, bool FP16>
__global__ void __launch_bounds__(kTokenThreads) linear_gate_tokens(const __grid_constant__ LinearParams p) {
  constexpr int kPer = FP8 ? 16 : 8, kSize = FP8 ? 1 : 2;  // elements of a vector, bytes of one
  constexpr int kGroups = kTokenThreads / 32 / PARTS;
  __shared__ float sums[kTokenThreads / 32][M * kTokenColumns];
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5, part = warp % PARTS;
  const uint32_t n0 = (blockIdx.x * kGroups + warp / PARTS) * kTokenColumns;
  const bool any = n0 < p.N;  // N % 8 == 0: then the warp's columns all exist
  const unsigned char* w = static_cast<const unsigned char*>(p.weight) + (size_t)n0 * p.weight_stride * kSize;
  const unsigned char* x[M];
#pragma unroll
  for (int m = 0; m < M; ++m) {
    const uint32_t b = div_u32(m, p.div_L), l = m - b * p.L;
    x[m] = static_cast<const unsigned char*>(p.x) + (b * p.x_sb + l * p.x_sl) * kSize;
  }
  float acc[M][kTokenColumns];
#pragma unroll
  for (int m = 0; m < M; ++m)
#pragma unroll
    for (int c = 0; c < kTokenColumns; ++c) acc[m][c] = 0.0f;
  // 16 loads in flight where the registers allow it (one token, 5120 -> 30720, a warp to all of K:
  // 50.5 us against 55.6 with 8; four e4m3 tokens 75 against 53)
  constexpr int kUnroll = M * kPer <= 16 ? 4 : 2;
#pragma unroll(kUnroll)
  for (uint32_t k = (part * 32 + lane) * kPer; k < (any ? p.K : 0u); k += PARTS * 32 * kPer) {
    uint4 wv[kTokenColumns];
#pragma unroll
    for (int c = 0; c < kTokenColumns; ++c)
      wv[c] = __ldcs(reinterpret_cast<const uint4*>(w + ((size_t)c * p.weight_stride + k) * kSize));
    float xf[M][kPer];
#pragma unroll
    for (int m = 0; m < M; ++m) widen_vector<FP8, FP16>(__ldg(reinterpret_cast<const uint4*>(x[m] + (size_t)k * kSize)), xf[m]);
#pragma unroll
    for (int c = 0; c < kTokenColumns; ++c) {
      float wf[kPer];
      widen_vector<FP8, FP16>(wv[c], wf);
#pragma unroll
      for (int m = 0; m < M; ++m)
#pragma unroll
        for (int i = 0; i < kPer; ++i) acc[m][c] = fmaf(wf[i], xf[m][i], acc[m][c]);
    }
  }
#pragma unroll
  for (int m = 0; m < M; ++m)
#pragma unroll
    for (int c = 0; c < kTokenColumns; ++c)
#pragma unroll
      for (int o = 16; o >= 1; o >>= 1) acc[m][c] += __shfl_xor_sync(0xFFFFFFFFu, acc[m][c], o);
  // lane (m, c) finishes its value
  float v = 0.0f;
#pragma unroll
  for (int m = 0; m < M; ++m)
#pragma unroll
    for (int c = 0; c < kTokenColumns; ++c)
      if (lane == m * kTokenColumns + c) v = acc[m][c];
  if (PARTS > 1) {
    if (lane < M * kTokenColumns) sums[warp][lane] = v;
    __syncthreads();
    if (part > 0) return;
    if (lane < M * kTokenColumns)
#pragma unroll
      for (int i = 1; i < PARTS; ++i) v += sums[warp + i][lane];
  }
  if (!any || lane >= M * kTokenColumns) return;
  const RowOut r = row_out(p, lane / kTokenColumns);
  const uint32_t n = n0 + lane % kTokenColumns;
  if (p.weight_scale) v *= r.x_scale * __ldg(p.weight_scale + n);
  auto one = [](const uint16_t* at) { return widen16<FP16>((uint32_t)*at).x; };
  if (p.bias) v += one(p.bias + n);
  float a[1] = {v};
  if (p.act == BO_ACT_GELU) {
    float same;
    fused_norm_impl::upk2(gelu(fused_norm_impl::pk2(v, v)), a[0], same);
  } else if (p.act != BO_ACT_NONE) {
    activate(p.act, a);
  }
  v = a[0];
  const uint16_t* e = p.residual.ptr + (r.b * p.residual.sb + r.l * p.residual.sl) + n;
  if (r.gate && p.has_residual) v = fmaf(one(r.gate + n), v, one(e));
  else if (r.gate) v *= one(r.gate + n);
  else if (p.has_residual) v += one(e);
  p.out[r.b * p.out_sb + r.l * p.out_sl + n] = (uint16_t)pack16<FP16>(v, 0.0f);
}

}  // namespace block_ops
