// Matrix product with bias, activation, gate and residual in its epilogue
// (contract: include/block_ops.h, linear_gate).
//
// out = residual + gate * act(x W^T + bias). Many rows are bound by the tensor cores
// (2 M N K operations against (M + N) K + 2 M N elements), a few tokens by reading W once.
//
// Many rows: persistent CTAs or CTA pairs (CG = 2) of six warps. One thread loads 128-byte
// wide tiles of x and W by TMA into a ring of shared-memory stages, one thread issues the
// tcgen05 products of a 128 CG x BN tile into TMEM, four warps read the sums back, a row per
// thread, and finish them. TMEM holds two tiles, so the epilogue of one runs under the
// products of the next. A pair shares W's tile: each CTA loads half of it.
//
// A few tokens: every warp streams rows of W past the tokens with 16-byte loads.
#pragma once

#include <cuda_fp8.h>

#include "rope_norm_kernel.cuh"
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
  const float *x_scale, *weight_scale;
  uint16_t* out;
  int64_t out_sb, out_sl;
};

// ---- the epilogue -----------------------------------------------------------------------------

// z sigmoid(s z') forms: the quotient of a huge |z| and e^|z| is 0, of an infinity NaN.
__device__ __forceinline__ float logistic_times(float z, float e) { return __fdividef(z, 1.0f + __expf(-e)); }

template <int N>
__device__ __forceinline__ void activate(int act, float (&v)[N]) {
  if (act == BO_ACT_SILU) {
#pragma unroll
    for (int i = 0; i < N; ++i) v[i] = logistic_times(v[i], v[i]);
  } else if (act == BO_ACT_GELU) {
#pragma unroll
    for (int i = 0; i < N; ++i) v[i] = 0.5f * v[i] * (1.0f + erff(v[i] * 0.70710678118654752f));
  } else if (act == BO_ACT_GELU_TANH) {  // 1/2 (1 + tanh t) = 1 / (1 + e^-2t)
#pragma unroll
    for (int i = 0; i < N; ++i) {
      const float t = 1.5957691216057308f * fmaf(0.044715f * v[i] * v[i], v[i], v[i]);
      v[i] = logistic_times(v[i], t);
    }
  }
}

// Where a row's operands lie.
struct RowOut {
  uint16_t* out;
  const uint16_t *gate, *residual;
  float x_scale;
};
__device__ __forceinline__ RowOut row_out(const LinearParams& p, uint32_t row) {
  RowOut r;
  const uint32_t b = div_u32(row, p.div_L), l = row - b * p.L;
  const uint32_t f = p.tpf ? div_u32(l, p.div_tpf) : 0u;
  r.out = p.out + (b * p.out_sb + l * p.out_sl);
  r.gate = p.gate.ptr ? p.gate.ptr + (b * p.gate.sb + f * p.gate.sf + l * p.gate.sl) : nullptr;
  r.residual = p.residual.ptr ? p.residual.ptr + (b * p.residual.sb + f * p.residual.sf + l * p.residual.sl) : nullptr;
  r.x_scale = p.x_scale ? __ldg(p.x_scale + row) : 1.0f;
  return r;
}

// Eight columns from n on (n % 8 == 0, n < N): sums to outputs.
template <bool FP16>
__device__ __forceinline__ void finish8(const LinearParams& p, const RowOut& r, uint32_t n, float (&v)[8]) {
  if (p.weight_scale) {
    const float4* s = reinterpret_cast<const float4*>(p.weight_scale + n);
    const float4 a = __ldg(s), b = __ldg(s + 1);
    const float w[8] = {a.x, a.y, a.z, a.w, b.x, b.y, b.z, b.w};
#pragma unroll
    for (int i = 0; i < 8; ++i) v[i] *= r.x_scale * w[i];
  }
  if (p.bias) {
    float b[8];
    widen8<FP16>(__ldg(reinterpret_cast<const uint4*>(p.bias + n)), b);
#pragma unroll
    for (int i = 0; i < 8; ++i) v[i] += b[i];
  }
  activate(p.act, v);
  float g[8], e[8];
  if (r.gate) widen8<FP16>(__ldg(reinterpret_cast<const uint4*>(r.gate + n)), g);
  if (r.residual) widen8<FP16>(*reinterpret_cast<const uint4*>(r.residual + n), e);  // may be out itself
#pragma unroll
  for (int i = 0; i < 8; ++i) {
    if (r.gate && r.residual) v[i] = fmaf(g[i], v[i], e[i]);
    else if (r.gate) v[i] *= g[i];
    else if (r.residual) v[i] += e[i];
  }
  *reinterpret_cast<uint4*>(r.out + n) = pack8<FP16>(v);
}

// ---- many rows ----------------------------------------------------------------------------------

constexpr int kTileM = 128;          // rows of a CTA
constexpr int kStepBytes = 128;      // of K, per row and stage
constexpr int kMaxStages = 8;
constexpr int kMatrixThreads = 192;  // TMA, products, four warps of epilogue

template <int CG, int BN>
struct MatrixShape {
  static constexpr int kABytes = kTileM * kStepBytes, kBBytes = BN / CG * kStepBytes;
  static constexpr int kStageBytes = kABytes + kBBytes;
  static constexpr int kFit = 200 * 1024 / kStageBytes;
  static constexpr int kStages = kFit < kMaxStages ? kFit : kMaxStages;
  static constexpr int kColumns = 2 * BN;  // TMEM: two tiles of sums
  static constexpr int kShared = kStages * kStageBytes + 1024;  // 1024: alignment of the stages
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

__device__ int linear_gate_gave_up = 0;  // launches in which a wait ran out (this file is included once)

template <int CG, int BN, bool FP8, bool FP16>
__global__ void __launch_bounds__(kMatrixThreads, 1)
linear_gate_tiles(const __grid_constant__ LinearParams p, const __grid_constant__ CUtensorMap map_x,
                  const __grid_constant__ CUtensorMap map_w) {
  using S = MatrixShape<CG, BN>;
  extern __shared__ unsigned char raw[];
  __shared__ __align__(8) uint64_t full[S::kStages], empty[S::kStages], sums_full[2], sums_empty[2];
  __shared__ uint32_t tmem_at;
  __shared__ int failed;
  const uint32_t stages = (smem_u32(raw) + 1023u) & ~1023u;
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const uint32_t rank = CG == 2 ? cluster_rank() : 0u;

  if (threadIdx.x == 0) {
    for (int i = 0; i < S::kStages; ++i) mbar_init(smem_u32(&full[i]), 1), mbar_init(smem_u32(&empty[i]), 1);
    for (int i = 0; i < 2; ++i) mbar_init(smem_u32(&sums_full[i]), 1), mbar_init(smem_u32(&sums_empty[i]), 4 * CG);
    failed = 0;
    mbar_init_fence();
  }
  if (warp == 1) tmem_alloc<CG>(smem_u32(&tmem_at), S::kColumns);
  __syncthreads();
  if (CG == 2) cluster_sync();
  tc_fence_after();
  const uint32_t tmem = *(volatile uint32_t*)&tmem_at;

  const uint32_t first = blockIdx.x / CG, step = gridDim.x / CG;
  if (warp == 0) {
    if (elect_one()) {
      prefetch_map(&map_x);
      prefetch_map(&map_w);
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
      if (!ok) {  // leave copies in flight the time to land
        const uint64_t start = now_ns();
        while (now_ns() - start < 1000000000ull) __nanosleep(1000000);
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
    const int quarter = warp & 3;  // the TMEM lanes that this warp may read
    uint32_t n = 0;
    for (uint32_t t = first; t < p.tiles; t += step, ++n) {
      const uint32_t buf = n & 1, round = (n >> 1) & 1;
      if (!mbar_wait(smem_u32(&sums_full[buf]), round, &failed)) break;
      __syncwarp();
      tc_fence_after();
      const Tile at = tile_at(p, t);
      const uint32_t in_batch = (at.m * CG + rank) * kTileM + quarter * 32 + lane;
      const bool live = in_batch < p.batch_rows;
      const RowOut r = row_out(p, live ? at.batch * p.batch_rows + in_batch : 0u);
      const uint32_t n0 = at.n * BN;
#pragma unroll 1
      for (int c = 0; c < BN; c += 32) {
        if (n0 + c >= p.N) break;
        float v[32];
        tmem_load32(tmem + ((uint32_t)(quarter * 32) << 16) + buf * BN + c, v);
        tmem_wait();
#pragma unroll
        for (int i = 0; i < 4; ++i)
          if (live && n0 + c + 8 * i < p.N) finish8<FP16>(p, r, n0 + c + 8 * i, reinterpret_cast<float(&)[8]>(v[8 * i]));
      }
      tc_fence_before();
      __syncwarp();
      if (lane == 0) mbar_arrive_cluster(map_to(smem_u32(&sums_empty[buf]), 0));
    }
  }
  __syncwarp();
  tc_fence_before();
  __syncthreads();
  if (CG == 2) cluster_sync();
  if (threadIdx.x == 0 && failed) atomicAdd(&linear_gate_gave_up, 1);
  if (warp == 1) {
    tc_fence_after();
    tmem_free<CG>(tmem, S::kColumns);
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

template <int M, bool FP8, bool FP16>
__global__ void __launch_bounds__(kTokenThreads) linear_gate_tokens(const __grid_constant__ LinearParams p) {
  constexpr int kPer = FP8 ? 16 : 8, kSize = FP8 ? 1 : 2;  // elements of a vector, bytes of one
  const int lane = threadIdx.x & 31;
  const uint32_t n0 = (blockIdx.x * (kTokenThreads / 32) + (threadIdx.x >> 5)) * kTokenColumns;
  if (n0 >= p.N) return;  // N % 8 == 0: the warp's columns all exist
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
#pragma unroll 2
  for (uint32_t k = lane * kPer; k < p.K; k += 32 * kPer) {
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
  if (lane >= M * kTokenColumns) return;
  const RowOut r = row_out(p, lane / kTokenColumns);
  const uint32_t n = n0 + lane % kTokenColumns;
  if (p.weight_scale) v *= r.x_scale * __ldg(p.weight_scale + n);
  auto one = [](const uint16_t* at) { return widen16<FP16>((uint32_t)*at).x; };
  if (p.bias) v += one(p.bias + n);
  float a[1] = {v};
  activate(p.act, a);
  v = a[0];
  if (r.gate && r.residual) v = fmaf(one(r.gate + n), v, one(r.residual + n));
  else if (r.gate) v *= one(r.gate + n);
  else if (r.residual) v += one(r.residual + n);
  r.out[n] = (uint16_t)pack16<FP16>(v, 0.0f);
}

}  // namespace block_ops
