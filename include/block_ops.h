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
 * anything is launched, outputs untouched on an error, no allocation (but four bytes of host
 * memory that linear_gate's first launch takes for good), no synchronisation, no fallback. All
 * buffers are the caller's. Sizes with a zero are valid and launch nothing. A non-zero stride need not be larger than the extent it steps over on inputs
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

/* Element types of the calls below. BO_FP32 is that of scales and fp32 weights, which have arguments
 * of their own: no configuration takes it as its dtype (FN_ERR_UNSUPPORTED). */
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
 * 1 / sqrt(variance + eps) has to be below 2^127 (it is for any eps >= 2^-250), and r - mean,
 * weight (1 + scale) and bias (1 + scale) + shift, which are formed first, within fp32.
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
  const void* weight;        /* (D), 16-byte aligned, as bias */
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

/* ---- rope_norm --------------------------------------------------------------------------
 *
 * Rows are tokens: x is (B, L, H, hd), a token has one position per axis.
 *
 *   n = x * rho * weight         rho = 1 / sqrt(mean(x^2) + eps) over the head's hd channels
 *                                (BO_NORM_HEAD; weight of hd values) or over all H * hd of the
 *                                token (BO_NORM_ALL; weight of H * hd); n = x (BO_NORM_NONE)
 *   P = section[0] + ... pairs of every head turn, the other hd - 2 P channels pass:
 *   (y0, y1) = (n0 cos a - n1 sin a, n0 sin a + n1 cos a)
 *   a = position[axis of the pair] * freq(pair)
 *
 * Pair i is channels (2 i, 2 i + 1), or (i, P + i) with half_pairs. The first section[0] pairs
 * follow axis 0, the next section[1] axis 1, and so on. The i-th of a section's m pairs has
 * freq = theta^(-i / m); with shared_frequencies pair i of all P has theta^(-i / P).
 * Angles are reduced in fp64 (an error of at most |position| 2^-52 turns), all else is fp32,
 * each output is rounded once. A mean square that fp32 does not hold is taken again in fp64;
 * rho has to be below 2^127 (it is for any eps >= 2^-250).
 *
 * The gradient, of the same handle: with dn the grad turned back,
 *   dx = rho (w dn - x rho^2 mean(w dn x)),  dweight = sum over tokens (and heads, for
 * BO_NORM_HEAD) of dn x rho, in a fixed order: in fp32 over runs of at most 512 tokens of a thread
 * (up to 4 heads of each for BO_NORM_HEAD, so an error of at most 2048 2^-24 of the terms'
 * magnitudes), in fp64 across threads; a CTA's runs are added in fp32.
 * Terms w dn x below fp32's normal numbers are lost: x and grad of a row are to have a product above
 * 2^-100.
 */
typedef struct rope_norm_s* rope_norm_t;

typedef enum { BO_NORM_NONE = 0, BO_NORM_HEAD = 1, BO_NORM_ALL = 2 } bo_norm;

typedef struct {
  int dtype;       /* x, grad, y, dx: BO_BF16 or BO_FP16 */
  int heads, head_dim; /* head_dim: a multiple of 16 up to 512; heads * head_dim <= 16384 */
  int axes;        /* 1 .. 4 */
  int section[4];  /* pairs of each axis, >= 1 each; their sum P <= head_dim / 2, and P % 8 == 0
                      with half_pairs */
  int norm;        /* bo_norm */
  int has_weight;  /* needs a norm */
  int weight_fp32; /* weight is fp32 (otherwise dtype) */
  int half_pairs, shared_frequencies;
  int index64;     /* positions are int64_t (otherwise int32_t) */
  double theta;    /* finite, > 0 */
  double eps;      /* 0 .. 2^100 */
} rn_config;

/* Element (b, l, h, c) lies at ptr[b * stride_b + l * stride_l + h * stride_h + c]; strides are
 * multiples of 8 elements, pointers 16-byte aligned, and so is the weight. */
typedef struct {
  const void* ptr;
  int64_t stride_b, stride_l, stride_h;
} rn_rows;

typedef struct {
  int64_t B, L;
  rn_rows x;
  const void* positions;     /* (b, l, axis) at [b * stride_b + l * stride_l + axis] */
  int64_t pos_stride_b, pos_stride_l;
  const void* weight;
  rn_rows y;                 /* written; may be x, element for element */
} rn_args;

typedef struct {
  int64_t B, L;
  rn_rows grad, x;           /* x.ptr NULL for BO_NORM_NONE */
  const void* positions;
  int64_t pos_stride_b, pos_stride_l;
  const void* weight;
  rn_rows dx;                /* written; may be grad or x, element for element */
  float* dweight;            /* has_weight: written whole, zeros when there are no tokens */
  void* workspace;           /* 16-byte aligned, rope_norm_backward_workspace bytes, needed until
                                the launch has run; NULL when that is 0 */
  uint64_t workspace_bytes;
} rn_backward_args;

fn_status rope_norm_create(rope_norm_t* out, const rn_config* cfg);
fn_status rope_norm_validate(rope_norm_t h, const rn_args* a);
fn_status rope_norm_launch(rope_norm_t h, const rn_args* a, fn_stream_t stream);
/* Bytes of workspace for a backward launch over B * L tokens, on any device. */
fn_status rope_norm_backward_workspace(rope_norm_t h, int64_t B, int64_t L, uint64_t* bytes);
fn_status rope_norm_backward_validate(rope_norm_t h, const rn_backward_args* a);
/* One kernel launch (with a weight, one for every 512 tokens of each of its threads), and one that
 * sums dweight. */
fn_status rope_norm_backward_launch(rope_norm_t h, const rn_backward_args* a, fn_stream_t stream);
fn_status rope_norm_destroy(rope_norm_t h);

/* ---- linear_gate ------------------------------------------------------------------------
 *
 *   out = residual + gate * act(x W^T + bias)      x (B, L, K), W (N, K), out (B, L, N)
 *
 * x and W are both bf16, both fp16 or both e4m3 (then x W^T is x_scale[row] * weight_scale[n]
 * times the product of the codes, and bias, gate, residual and out are bf16; otherwise they
 * have x's type). The sum over K and everything after it is fp32; out is rounded once. The
 * order of the sum depends on the sizes, the strides and the device, not on the run: a strided view
 * and its contiguous copy may differ in the last bit.
 *
 * Up to four tokens x may repeat rows (a stride of 0); from five on a stride of 0 along an extent
 * above 1 is FN_ERR_UNSUPPORTED (a tensor map does not hold it). residual has a row per token at any
 * size. x_scale * weight_scale, which is formed first, has to be within fp32's normal numbers.
 * Tokens at one distance throughout, in x, out and residual, are worked on in tiles of 128 or 256;
 * where batches lie apart (a part of longer rows) a tile stays inside its batch, so many batches of
 * a few tokens cost up to 128 / L times what the same tokens cost together. Copy them together first.
 * act is SiLU z / (1 + e^-z), GELU z Phi(z), its tanh form, or nothing.
 */
typedef struct linear_gate_s* linear_gate_t;

typedef enum { BO_ACT_NONE = 0, BO_ACT_SILU = 1, BO_ACT_GELU = 2, BO_ACT_GELU_TANH = 3 } bo_act;

typedef struct {
  int dtype;          /* BO_BF16, BO_FP16 or BO_E4M3 */
  int64_t K, N;       /* 8 .. 2^20; N and K multiples of 8, K of 16 for e4m3 */
  int act;            /* bo_act */
  int has_bias, has_gate, has_residual;
} lg_config;

typedef struct {
  int64_t B, L;
  int64_t tokens_per_frame;   /* of the gate; as in fn_args */
  fn_operand x;               /* stride_f 0; strides multiples of 16 bytes */
  const void* weight;         /* row n at weight + n * weight_stride elements, 16-byte aligned rows */
  int64_t weight_stride;
  const void* bias;           /* (N), 16-byte aligned */
  fn_operand gate, residual;  /* residual: one row per token, stride_f 0 */
  const float* x_scale;       /* (B, L) contiguous; e4m3 */
  const float* weight_scale;  /* (N), 16-byte aligned; e4m3 */
  void* out;                  /* strides in elements, multiples of 8; may be residual, element for element */
  int64_t out_stride_b, out_stride_l;
} lg_args;

fn_status linear_gate_create(linear_gate_t* out, const lg_config* cfg);
fn_status linear_gate_validate(linear_gate_t h, const lg_args* a);
/* One kernel launch. */
fn_status linear_gate_launch(linear_gate_t h, const lg_args* a, fn_stream_t stream);
/* The matrix kernel bounds its internal waits (ten seconds of wall clock, in which the device may
 * also have been busy with another process); a launch in which one ran out leaves its output
 * incomplete. The next linear_gate_launch of the process, on any device, then launches nothing and
 * returns FN_ERR_CUDA with cudaErrorLaunchTimeout (702) as the last error, once; and the CTAs in
 * which it happened are counted on their device, for replayed graphs too. This call reads the
 * current device's count (and synchronises with its default stream). */
fn_status linear_gate_timeouts(int* count);
fn_status linear_gate_destroy(linear_gate_t h);

#ifdef __cplusplus
}
#endif

#endif /* BLOCK_OPS_H_ */
