/*
 * fp8block -- the block-scaled FP8 operators of libfp4moe.so: RMS norm with
 * the residual's addition and a quantized output, SiLU(gate)*up with a
 * quantized output, and the matrix product with one scale per 1x128 block of
 * the activations and per 128x128 block of the weights, dense and per expert.
 * C ABI.
 *
 * The conventions of fp4moe.h hold for every call here: device pointers owned
 * by the caller, host-side validation before any launch, work enqueued on
 * `stream`, no allocation, no synchronization, FP4MOE_* status codes and
 * fp4moe_last_error().
 *
 * Data
 *   - Codes are OCP E4M3FN bytes; a value is its code times the float32 scale
 *     of its block.  Blocks are 128 wide along the row (K, or the output
 *     width); the last block of a row may be shorter.  KB = ceil(K/128).
 *   - Activation scales: element (row, block) at row*row_stride +
 *     block*blk_stride, any non-negative strides (of an output: that put no two
 *     elements in one place).  The kernels read the scales of
 *     consecutive rows of one block together, so row_stride 1 is the layout
 *     to prefer (what the Python binding allocates).
 *   - Weight scales: [ceil(N/128), KB], row stride given.
 *   - Quantization (both producers): per block s = max(amax/448, 2^-64) and
 *     code = E4M3(v/s), round to nearest even, from a v/s that carries more than
 *     float32 (but for quotients below 2^-6 and blocks of tiny or huge values):
 *     nearly always the formula's code, also where float32 arithmetic step by step
 *     would take its neighbour.  A block that holds a NaN has a NaN scale and NaN
 *     codes; one that holds an infinity has an infinite scale, NaN codes for
 *     the infinities and zero codes for the rest.
 */
#ifndef FP8BLOCK_H
#define FP8BLOCK_H

#include <stdint.h>

#ifdef __cplusplus
extern "C" {
#endif

/* Element types of unquantized inputs and outputs. */
enum {
  FP8BLOCK_BF16 = 0,
  FP8BLOCK_F16 = 1,
  FP8BLOCK_F32 = 2
};

/*
 * rms_norm_fp8 -- RMS norm of x + residual, quantized 1x128.
 *   v = x + residual (float32; residual NULL: v = x);
 *   residual_out = v rounded to `dtype` (optional);
 *   y = v * weight / sqrt(mean(v^2) + eps) in float32, from the unrounded v;
 *   y_out = y rounded to `dtype` (optional);
 *   codes, scales = the 1x128 quantization of the float32 y (both NULL: only
 *   the other outputs are written).
 * x, residual, residual_out, y_out: [M, K] of `dtype`, row strides in
 * elements (>= K).  weight [K] of `dtype`.  codes [M, K] bytes with row stride
 * ldc, scales [M, KB].  residual_out and y_out may each be x or residual itself (same
 * stride); other overlaps of an output with an input or another output are refused.  M >= 0,
 * 1 <= K <= 65536.
 * Any alignment of whole elements is accepted; rows whose pointers and strides
 * are all 16-byte multiples (codes: 8) are the fastest.
 */
typedef struct {
  int dtype;               /* FP8BLOCK_* of x, residual, weight, residual_out, y_out */
  int M, K;
  float eps;
  const void* x;
  int64_t ldx;
  const void* residual;    /* or NULL                                          */
  int64_t ldr;
  const void* weight;
  void* residual_out;      /* or NULL                                          */
  int64_t ldro;
  void* y_out;             /* or NULL                                          */
  int64_t ldy;
  uint8_t* codes;          /* or NULL together with scales                     */
  int64_t ldc;
  float* scales;
  int64_t scale_row, scale_blk;   /* strides of scales                         */
} fp8block_norm_args;

int rms_norm_fp8(const fp8block_norm_args* args, void* stream);

/*
 * swiglu_fp8 -- h = SiLU(gate) * up, quantized 1x128.
 * gate_up [M, 2I] of `dtype`, row stride ldg: gate in columns [0, I), up in
 * [I, 2I).  h is not rounded in between; SiLU of a gate below -108.67, less than half
 * of the smallest float32, is -0.  codes [M, I] bytes, row stride ldc; scales [M, ceil(I/128)].
 * row_count (device, NULL = M): rows at or past it are not written.  M >= 0, I >= 1, M * ceil(I/128) < 2^31.
 * codes and scales may not overlap gate_up or each other.
 */
int swiglu_fp8(int dtype, const void* gate_up, int M, int I, int64_t ldg,
               const int32_t* row_count, uint8_t* codes, int64_t ldc, float* scales,
               int64_t scale_row, int64_t scale_blk, void* stream);

/*
 * fp8_block_linear / fp8_block_grouped_gemm -- out = round(A . W^T) with
 *   (A . W^T)[m,n] = sum_b a_scale[m,b] * w_scale[n/128,b] *
 *                    sum_{k in block b} A[m,k] * W[n,k],
 * the sum over a block by the matrix unit into float32, before its scales; the
 * sum over blocks in float32.  The unit aligns the products of a block to the
 * largest and drops what lies some 2^-13 below it (about 1.5e-5 of a typical
 * result): far below the rounding to bfloat16 or float16, and the reason why
 * no float32 output is offered.
 *
 * Common: a [a_rows, K] codes, row stride lda (bytes); a_scale [a_rows, KB];
 * w [N, K] codes, row stride ldw (bytes); w_scale [ceil(N/128), KB], row
 * stride ld_ws; out [rows, N] of out_dtype (FP8BLOCK_BF16 or _F16), row
 * stride ldo (elements).
 * K % 16 == 0, lda and ldw multiples of 16, a and w 16-byte aligned; N and the
 * row counts are free.  out may not overlap an operand.
 *
 * fp8_block_linear: rows [0, M), M <= a_rows.  The grouped fields are ignored.
 *
 * fp8_block_grouped_gemm: w, w_scale hold n_experts matrices at strides
 * w_expert (bytes, a multiple of 16) and ws_expert (elements).  Rows are the
 * sorted pairs of moe_permute: expert e owns rows expert_offsets[e] ..
 * expert_offsets[e+1]-1 (M = rows of the sorted buffers); tiles, n_tiles and
 * max_tiles are moe_permute's for the same block_m, one of 16, 32, 64, 128
 * (max_tiles * block_m/16 below 2^31).
 * Row r reads activation row a_row_gather[r] / gather_div when a_row_gather is
 * given, else row r.  Rows outside every segment are not written.  Tiles that
 * name an expert out of range are skipped, segments are cut at M and gathered
 * rows are clamped to [0, a_rows), so no content of the index tensors makes
 * the call touch memory outside the given buffers.
 */
typedef struct {
  int M, N, K;
  int a_rows;
  const uint8_t* a;
  int64_t lda;
  const float* a_scale;
  int64_t as_row, as_blk;
  const uint8_t* w;
  int64_t ldw;
  const float* w_scale;
  int64_t ld_ws;
  int out_dtype;
  void* out;
  int64_t ldo;
  /* grouped */
  int n_experts, block_m, gather_div, max_tiles;
  int64_t w_expert, ws_expert;
  const int32_t* a_row_gather;
  const int32_t* expert_offsets;
  const int32_t* tiles;
  const int32_t* n_tiles;
} fp8block_gemm_args;

int fp8_block_linear(const fp8block_gemm_args* args, void* stream);
int fp8_block_grouped_gemm(const fp8block_gemm_args* args, void* stream);

#ifdef __cplusplus
}
#endif

#endif /* FP8BLOCK_H */
