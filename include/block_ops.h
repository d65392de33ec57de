/*
 * block_ops.h -- C ABI of the operators that stand next to the fused norm rows in a
 * transformer block (libfused_norm.so, B200 sm_100a):
 *
 *   norm_quant   residual / gate / norm / modulation rows with an e4m3 output and one
 *                scale per row, the input of an 8-bit matrix product;
 *   rope_norm    RMS norm of q or k (per head, over all heads, or none) and rotary
 *                positions over up to four axes (time, height, width, ...), with its
 *                gradient;
 *   linear_gate  matrix product with bias, activation, gate and residual in its epilogue,
 *                from bf16, fp16 or (with row and channel scales) e4m3.
 *
 * They share the conventions of fused_norm.h: status codes and fn_operand, host-only
 * immutable handles that several threads and streams may use at once, launches that are
 * asynchronous on the caller's stream and go to the calling thread's current device (the
 * one that owns the stream and the buffers), argument errors found on the host before
 * anything is launched, outputs untouched on an error, no allocation, no synchronisation,
 * no fallback. All buffers are the caller's. Sizes with a zero are valid and launch
 * nothing. A non-zero stride need not be larger than the extent it steps over on inputs
 * (rows may overlap); output rows must not overlap each other or an input, except where a
 * call says so.
 */
#ifndef BLOCK_OPS_H_
#define BLOCK_OPS_H_

#include "fused_norm.h"

#ifdef __cplusplus
extern "C" {
#endif

/* Static text for a status of these operators; never NULL. */
const char* block_ops_status_string(fn_status s);

/* cudaError_t (as int) of the last launch of these operators that ended in FN_ERR_CUDA on
 * this host thread; 0 if none. */
int block_ops_last_cuda_error(void);

/* Element types of the calls below. */
typedef enum { BO_BF16 = 0, BO_FP16 = 1, BO_E4M3 = 2, BO_FP32 = 3 } bo_dtype;

/* ---- norm_quant -----------------------------------------------------------------------
 *
 *   r = residual + gate * x      (has_residual; rounded once to bf16, stored; gate = 1 when
 *                                 absent; without has_residual, r below is x)
 *   n = LayerNorm(r) or RMSNorm(r), eps inside the square root
 *   n = n * weight + bias        (each optional; bf16 or, with affine_fp32, fp32)
 *   y = n * (1 + scale) + shift  (has_modulation; y = n otherwise)
 *   a = max |y| over the row
 *   row_scale = a / 448, q = e4m3(y / row_scale)
 *
 * y is not rounded before q: it is an fp32 value (statistics in fp32 per thread, joined in
 * fp64; rows whose sums leave fp32's comfortable range, or whose spread vanishes in it, are
 * taken again in fp64). q is rounded once to nearest even. A row with a = 0 has row_scale 1;
 * a below 2^-100 is taken as 2^-100. A NaN or infinity in y leaves a NaN or infinite
 * row_scale: q is then NaN where y was not finite, and NaN everywhere in a NaN row.
 * 1 / sqrt(variance + eps) has to be below 2^127 (it is for any eps >= 2^-250).
 */
typedef struct norm_quant_s* norm_quant_t;

typedef struct {
  int D;             /* channels per row: a multiple of 16, 16 .. 16384 */
  int is_rms;        /* 0: LayerNorm, 1: RMSNorm */
  int has_residual;  /* 1: r = residual + gate * x is formed and stored */
  int has_gate;      /* needs has_residual */
  int has_weight, has_bias;
  int affine_fp32;   /* weight and bias are fp32; needs one of them */
  int has_modulation; /* scale and shift are given */
  double eps;        /* finite, >= 0 */
} nq_config;

typedef struct {
  int64_t B, L;
  int64_t tokens_per_frame;  /* as in fn_args */
  fn_operand x, residual, gate, scale, shift; /* bf16; ptr NULL where the config has none */
  const void* weight;        /* (D) */
  const void* bias;          /* (D) */
  void* q;                   /* (B, L, D) e4m3, 16-byte aligned rows: strides in elements, multiples of 16 */
  int64_t q_stride_b, q_stride_l;
  float* row_scale;          /* (B, L) contiguous */
  void* r;                   /* (B, L, D) bf16; NULL without has_residual; may be residual, element for element */
  int64_t r_stride_b, r_stride_l;
} nq_args;

fn_status norm_quant_create(norm_quant_t* out, const nq_config* cfg);
/* Every rule norm_quant_launch applies, on the host: the rules of fused_norm_validate. */
fn_status norm_quant_validate(norm_quant_t h, const nq_args* a);
/* One kernel launch. */
fn_status norm_quant_launch(norm_quant_t h, const nq_args* a, fn_stream_t stream);
fn_status norm_quant_destroy(norm_quant_t h);

#ifdef __cplusplus
}
#endif

#endif /* BLOCK_OPS_H_ */
