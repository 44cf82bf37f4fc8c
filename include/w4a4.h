/*
 * libw4a4 -- SVDQuant W4A4 quantized linear layer for AMD Instinct MI355X (gfx950).
 *
 * Plain C ABI.  Every tensor argument is a device pointer on the current HIP
 * device, dense and row-major in the shape given; the caller owns every
 * buffer.  All work is enqueued on `stream` (a hipStream_t passed as void*;
 * NULL is the default stream).  No entry point allocates, frees or
 * synchronizes.  Validation happens before any launch: a call that returns an
 * error has launched nothing and written nothing.  Faults during execution
 * surface at the caller's next synchronization.  Calls are thread-safe (for
 * svdq_linear_noalloc see its note on overlapping calls); no call depends on an
 * earlier one.  The library caches, once per device and atomically, the CU count,
 * the occupancy of its persistent kernels and the address of the static buffer
 * of svdq_linear_noalloc.  Checks run in this order: sizes
 * (W4A4_ERR_SHAPE / W4A4_ERR_UNSUPPORTED), the empty call (M or N == 0 is
 * valid, launches nothing and may pass NULL pointers), NULL pointers
 * (W4A4_ERR_NULL), alignment (W4A4_ERR_ALIGN).
 *
 * Formats (from the "SVDQuant W4A4" page, section "Checkpoint contract",
 * configuration precision "nvfp4"):
 *   FP4      E2M1, two values per byte, the even-k element in the low nibble;
 *   scales   float8_e4m3fn bytes, one per 16 consecutive inputs along K;
 *   bf16     IEEE bfloat16.
 *
 * Method (same page, sections "Overview" and "Runtime support"; rotation from
 * the rotate notes, sections 2.1-2.2 and 3.3): y = x W^T is computed as
 *   x_s   = x / smooth_factor                            (float32, IEEE)
 *   v     = x_s @ H_B^T per B-block of K                 (optional rotation)
 *   qact, ascales = per-16 group FP4 quantization of v   (amax/6 -> e4m3)
 *   y     = bf16( (dequant(qact) @ dequant(qweight)^T) * wcscales * wtscale
 *                 + (x_s @ proj_down) @ proj_up^T )
 * with the weight-side smoothing and rotation folded into qweight offline.
 */
#ifndef W4A4_H_
#define W4A4_H_

#include <stddef.h>
#include <stdint.h>

#ifdef __cplusplus
extern "C" {
#endif

typedef enum {
  W4A4_OK = 0,
  W4A4_ERR_NULL = 1,        /* a required pointer is NULL                         */
  W4A4_ERR_SHAPE = 2,       /* a size is negative, K % 16 != 0, K % block != 0,
                               or the workspace is too small                      */
  W4A4_ERR_ALIGN = 3,       /* a pointer breaks its required alignment            */
  W4A4_ERR_UNSUPPORTED = 4, /* hadamard_block not in {0,16,32,64,128}, R > 64, or K > W4A4_MAX_K */
  W4A4_ERR_HIP = 5,         /* the HIP runtime reported an error at launch        */
  W4A4_ERR_SCRATCH = 6      /* svdq_linear_noalloc: the sizes need more workspace than its static
                               device buffer holds (W4A4_NOALLOC_SCRATCH_BYTES)   */
} w4a4_status;

/* Largest supported correction rank R. */
#define W4A4_MAX_RANK 64
/* Largest supported K (2^24 columns): the kernels address a tile's rows x K/2 code bytes with
   32-bit offsets. */
#define W4A4_MAX_K (1 << 24)

/* Human-readable name of a status code (static storage). */
const char* w4a4_status_string(int status);

/* Library version as 10000*major + 100*minor + patch. */
int w4a4_version(void);

/*
 * Online activation quantizer ("SVDQuant W4A4" page, "Runtime support": BF16
 * input; rotation: rotate notes 2.1 and 3.3, quantization fused with the
 * rotation in one pass).  One HBM pass over x computes, per row m:
 *   x_s  = float32(x) / float32(smooth_factor)                  (IEEE division)
 *   v    = x_s, or x_s @ H_B^T on every contiguous B-block when hadamard_block
 *          B > 0 (Sylvester order, butterfly spans 1,2,...,B/2, then one
 *          multiply by float32(1/sqrt(B)))
 *   per group g of 16:  s8 = e4m3(amax|v| / 6)  (round-nearest-even, saturating
 *          at 448);  code = e2m1(v / e4m3_value(s8))  (round-nearest-even,
 *          saturating at 6, sign of zero kept), all codes 0 when s8 == 0
 *   lora_act = x_s @ proj_down       (unrotated x_s, float32 result)
 *
 *   x             bf16 [M, K]           16-byte aligned
 *   smooth_factor bf16 [K]
 *   proj_down     bf16 [K, R]           may be NULL when R == 0
 *   M >= 0, K >= 16 with K % 16 == 0, 0 <= R <= 64
 *   hadamard_block  0 (none) or 16, 32, 64, 128 with K % hadamard_block == 0
 *   qact          u8   [M, K/2]  out    E2M1 pairs, 4-byte aligned
 *   ascales       u8   [K/16, M] out    e4m3 bytes (layout mirrors wscales)
 *   lora_act      f32  [M, R]    out    may be NULL when R == 0
 * M == 0 is a valid empty call (nothing is launched).
 */
w4a4_status svdq_quantize_act(const void* x, const void* smooth_factor, const void* proj_down,
                              int64_t M, int64_t K, int64_t R, int32_t hadamard_block,
                              void* qact, void* ascales, float* lora_act, void* stream);

/*
 * Offline weight quantizer producing the checkpoint tensors ("SVDQuant W4A4"
 * page, "Checkpoint contract": qweight (N, K/2) packed FP4, wscales (K/16, N)
 * e4m3; rotate notes 2.1: weights are rotated offline, W' = R W).  Per row n:
 *   w_s = float32(w) * float32(smooth_factor)    (exact for bf16 inputs)
 *   v   = w_s, or w_s @ H_B^T per B-block (as in svdq_quantize_act)
 *   per-16 group quantization exactly as in svdq_quantize_act.
 *
 *   w        bf16 [N, K]   16-byte aligned
 *   smooth_factor bf16 [K]
 *   qweight  u8   [N, K/2] out   4-byte aligned
 *   wscales  u8   [K/16, N] out
 */
w4a4_status svdq_quantize_weight(const void* w, const void* smooth_factor, int64_t N, int64_t K,
                                 int32_t hadamard_block, void* qweight, void* wscales, void* stream);

/*
 * Block-scaled FP4 GEMM with the low-rank correction fused in the epilogue
 * ("SVDQuant W4A4" page, "Runtime support": NVFP4 GEMM followed by the BF16
 * rank correction; "Checkpoint contract": proj_up, wcscales, wtscale):
 *   y[m,n] = bf16( sum_k e2m1(qact[m,k]) e4m3(ascales[k/16,m])
 *                        e2m1(qweight[n,k]) e4m3(wscales[k/16,n])
 *                  * wcscales[n] * wtscale
 *                  + sum_r lora_act[m,r] proj_up[n,r] )
 * The products are exact; the sum is accumulated in float32 (matrix cores).
 *
 *   qact     u8   [M, K/2]   16-byte aligned     ascales u8 [K/16, M]
 *   lora_act f32  [M, R]     may be NULL when R == 0
 *   qweight  u8   [N, K/2]   16-byte aligned     wscales u8 [K/16, N]
 *   proj_up  bf16 [N, R]     may be NULL when R == 0
 *   wcscales bf16 [N]
 *   wtscale  bf16 [1]        device scalar, read by the kernel
 *   y        bf16 [M, N] out
 */
w4a4_status svdq_gemm_lowrank(const void* qact, const void* ascales, const float* lora_act,
                              const void* qweight, const void* wscales, const void* proj_up,
                              const void* wcscales, const void* wtscale,
                              int64_t M, int64_t N, int64_t K, int64_t R, void* y, void* stream);

/* Bytes of workspace svdq_linear needs for these sizes (qact, ascales and
 * lora_act, each 256-byte aligned).  Returns 0 for invalid sizes. */
size_t svdq_linear_workspace_bytes(int64_t M, int64_t K, int64_t R);

/*
 * The whole layer: svdq_quantize_act into the workspace, then
 * svdq_gemm_lowrank.  Arguments are the checkpoint tensors of the "SVDQuant
 * W4A4" page's table plus the BF16 input x [M, K] and the output y [M, N].
 * `workspace` is device memory of at least svdq_linear_workspace_bytes(M, K, R)
 * bytes, 256-byte aligned; its contents need no initialisation and are
 * overwritten.
 */
w4a4_status svdq_linear(const void* x, const void* qweight, const void* wscales, const void* proj_down,
                        const void* proj_up, const void* smooth_factor, const void* wcscales,
                        const void* wtscale, int64_t M, int64_t N, int64_t K, int64_t R,
                        int32_t hadamard_block, void* y, void* workspace, size_t workspace_bytes,
                        void* stream);


/*
 * MXFP4 variant of the layer (rotate notes, section 3.3, FP-Quant:
 * hadamard_group_size 32, forward_dtype "mxfp4", forward_method "abs_max";
 * fused_quantize_mx then matmul_mxf4_bf16).  Smoothing, the optional rotation
 * and the low-rank branch are those of the entry points above; the
 * quantization works on blocks of 32 consecutive K-columns with one E8M0
 * (power-of-two) scale per block instead of 16-groups with e4m3 scales:
 *   e     = the least integer with 2^e >= f32(amax|v| / 6), clamped to [-127, 127]
 *   scale byte = e + 127  (E8M0: value 2^(byte - 127))
 *   code  = e2m1(v * 2^-e)   (round-to-nearest-even, saturating at 6, sign kept)
 * and the GEMM multiplies E2M1 codes scaled by 2^(byte - 127) per row and block
 * (matrix-core instruction with per-block power-of-two scales), fp32
 * accumulation, the same epilogue.  Inputs must be finite.
 *
 * svdq_quantize_act_mx: as svdq_quantize_act with K % 32 == 0 and
 *   hadamard_block 0 or 32;
 *   ascales  u8 [K/32, Mp] out   Mp = 4 * ceil(M / 4); columns M .. Mp-1 are written 0
 * svdq_quantize_weight_mx: as svdq_quantize_weight with K % 32 == 0 and
 *   hadamard_block 0 or 32;  wscales u8 [K/32, N] out
 * svdq_gemm_lowrank_mx: as svdq_gemm_lowrank with K % 128 == 0, N % 4 == 0;
 *   ascales u8 [K/32, Mp] and wscales u8 [K/32, N], both 4-byte aligned
 * svdq_linear_mx: svdq_quantize_act_mx into the workspace (at least
 *   svdq_linear_mx_workspace_bytes(M, K, R) bytes, 256-byte aligned), then
 *   svdq_gemm_lowrank_mx.
 * Other sizes return W4A4_ERR_SHAPE (K, N) or W4A4_ERR_UNSUPPORTED (hadamard_block).
 */
w4a4_status svdq_quantize_act_mx(const void* x, const void* smooth_factor, const void* proj_down,
                                 int64_t M, int64_t K, int64_t R, int32_t hadamard_block,
                                 void* qact, void* ascales, float* lora_act, void* stream);

w4a4_status svdq_quantize_weight_mx(const void* w, const void* smooth_factor, int64_t N, int64_t K,
                                    int32_t hadamard_block, void* qweight, void* wscales, void* stream);

w4a4_status svdq_gemm_lowrank_mx(const void* qact, const void* ascales, const float* lora_act,
                                 const void* qweight, const void* wscales, const void* proj_up,
                                 const void* wcscales, const void* wtscale,
                                 int64_t M, int64_t N, int64_t K, int64_t R, void* y, void* stream);

size_t svdq_linear_mx_workspace_bytes(int64_t M, int64_t K, int64_t R);

w4a4_status svdq_linear_mx(const void* x, const void* qweight, const void* wscales, const void* proj_down,
                           const void* proj_up, const void* smooth_factor, const void* wcscales,
                           const void* wtscale, int64_t M, int64_t N, int64_t K, int64_t R,
                           int32_t hadamard_block, void* y, void* workspace, size_t workspace_bytes,
                           void* stream);

/* ---- Optional bias -------------------------------------------------------------------------
 * Rotate notes, section 3.2: the linear-layer wrapper hands the layer's optional bias to the
 * quantized method (apply(layer, x, bias)).  These four entry points are the ones above with one
 * more argument, `bias`: bf16 [N] (2-byte aligned) or NULL for none.  It is added in float32 to
 * each output after the scaled quantized product and the low-rank term, before the single
 * rounding to bf16, and is not multiplied by wcscales or wtscale:
 *   y = bf16( acc * wcscales * wtscale + L @ proj_up^T + bias )
 * Validation and errors are those of the entry point without bias, plus W4A4_ERR_ALIGN for an
 * odd bias address. */
w4a4_status svdq_gemm_lowrank_bias(const void* qact, const void* ascales, const float* lora_act,
                                   const void* qweight, const void* wscales, const void* proj_up,
                                   const void* wcscales, const void* wtscale, const void* bias, int64_t M,
                                   int64_t N, int64_t K, int64_t R, void* y, void* stream);
w4a4_status svdq_linear_bias(const void* x, const void* qweight, const void* wscales, const void* proj_down,
                             const void* proj_up, const void* smooth_factor, const void* wcscales,
                             const void* wtscale, const void* bias, int64_t M, int64_t N, int64_t K, int64_t R,
                             int32_t hadamard_block, void* y, void* workspace, size_t workspace_bytes,
                             void* stream);
w4a4_status svdq_gemm_lowrank_mx_bias(const void* qact, const void* ascales, const float* lora_act,
                                      const void* qweight, const void* wscales, const void* proj_up,
                                      const void* wcscales, const void* wtscale, const void* bias, int64_t M,
                                      int64_t N, int64_t K, int64_t R, void* y, void* stream);
w4a4_status svdq_linear_mx_bias(const void* x, const void* qweight, const void* wscales, const void* proj_down,
                                const void* proj_up, const void* smooth_factor, const void* wcscales,
                                const void* wtscale, const void* bias, int64_t M, int64_t N, int64_t K, int64_t R,
                                int32_t hadamard_block, void* y, void* workspace, size_t workspace_bytes,
                                void* stream);

/* ---- The layer without allocation ---------------------------------------------------------
 * For callers that cannot allocate device memory: code under HIP graph capture, tight serving
 * loops, harnesses that forbid hipMalloc.  svdq_linear_bias (bias may be NULL) with its workspace
 * in a static device buffer of W4A4_NOALLOC_SCRATCH_BYTES bytes that the library holds on each GPU
 * it runs on until the process ends, instead of a caller-provided one.  Same kernels, same
 * results bit for bit.  Calls whose workspace (svdq_linear_workspace_bytes(M, K, R)) exceeds the
 * buffer return W4A4_ERR_SCRATCH before any HIP call; other errors as for svdq_linear_bias.  The
 * call allocates and frees nothing; the buffer's address is looked up once per device (on the
 * first call with that device current).  Every call on one GPU uses that GPU's one buffer, so
 * calls that may overlap on a GPU (concurrent streams, host threads) race and must be ordered by
 * the caller. */
#define W4A4_NOALLOC_SCRATCH_BYTES (64u << 20)
w4a4_status svdq_linear_noalloc(const void* x, const void* qweight, const void* wscales, const void* proj_down,
                                const void* proj_up, const void* smooth_factor, const void* wcscales,
                                const void* wtscale, const void* bias, int64_t M, int64_t N, int64_t K, int64_t R,
                                int32_t hadamard_block, void* y, void* stream);

/* ---- Offline low-rank split (host) ----------------------------------------------------------
 * "SVDQuant W4A4" page, "Overview" (four-bit weights and activations plus a small low-rank
 * branch that corrects part of the quantization error; checkpoints are quantized offline) and
 * "Checkpoint contract" (proj_down (K, R), proj_up (N, R)).  HOST memory throughout; no GPU
 * work.  With W_s = W * smooth_factor (float64) and its top-R singular triplets U_R S_R V_R:
 *   proj_up   = bf16(U_R sqrt(S_R))         [N, R] bf16
 *   proj_down = bf16(V_R sqrt(S_R))         [K, R] bf16
 *   residual  = bf16(W_s - proj_up proj_down^T)   [N, K] bf16 (smoothing already applied: quantize
 *               it with svdq_quantize_weight and a smooth_factor of ones to get qweight, wscales)
 *   singular_values  S_1 >= ... >= S_R as float (may be NULL)
 * The triplets come from a randomized range finder with R + oversample Gaussian columns (drawn
 * from `seed`) and `power_iters` power iterations; `threads` host threads (<= 0: all cores).
 * Sizes: 1 <= N, K <= 2^20, N * K <= 2^31, 0 <= R <= min(N, K, W4A4_MAX_RANK), oversample >= 0,
 * power_iters >= 0, else W4A4_ERR_SHAPE; NULL w, smooth_factor or residual (or factors with
 * R > 0): W4A4_ERR_NULL.  R == 0 writes the smoothed weight to residual. */
w4a4_status svdq_lowrank_split(const void* w, const void* smooth_factor, int64_t N, int64_t K, int64_t R,
                               int32_t oversample, int32_t power_iters, uint64_t seed, int32_t threads,
                               void* proj_down, void* proj_up, void* residual, float* singular_values);

/* ---- Standalone block Hadamard transform ------------------------------------------------
 * Rotate notes, section 3.1 (the Hadacore kernel behind hadacore_transform(x, inplace): the
 * Sylvester Hadamard transform applied through its recursion, symmetric and therefore its own
 * inverse, in place or not) and section 3.2 (applied per head_dim block, and to column
 * partitions [start, start + length) of a layer's output); the Sylvester recursion and the
 * 1/sqrt(n) normalisation from sections 2.1-2.2.
 *
 * For each of `rows` rows and each block of `block` consecutive columns of the first `cols`:
 *   y[r, blk] = round( float32(1/sqrt(block)) * FWHT(float32(x[r, blk])) )
 * with butterfly spans 1, 2, ..., block/2 in that order, each pair (a, b) -> (a + b, a - b) in
 * float32, one multiply, then one round to nearest even into the storage type (bf16 and f16;
 * f32 is stored as computed).  Results are bit-identical to that sequence of float32
 * operations (the quantizers' fused rotation uses the same one).
 *   x, y   device pointers to element (0, 0); row r starts ldx (ldy) elements after row r - 1,
 *          so a column partition is addressed as x + start with the full row stride.
 *   ldx, ldy  row strides in elements, >= cols.
 *   dtype  W4A4_DTYPE_BF16, W4A4_DTYPE_F16 or W4A4_DTYPE_F32 (both tensors).
 *   block  a power of two in [2, W4A4_HADAMARD_MAX_BLOCK]; cols % block == 0.
 * x == y (with ldx == ldy) transforms in place; any other overlap of x and y is undefined.
 * Columns at and past `cols` in each row are not touched.  Errors: W4A4_ERR_SHAPE (negative
 * sizes, cols % block, ld < cols, x == y with ldx != ldy), W4A4_ERR_UNSUPPORTED (block,
 * dtype), W4A4_ERR_NULL, W4A4_ERR_ALIGN (x or y not aligned to the element size).  rows == 0
 * or cols == 0 launches nothing.  16-byte aligned pointers, row strides and column counts that
 * are multiples of 8 take the vectorised path. */
#define W4A4_DTYPE_BF16 0
#define W4A4_DTYPE_F16 1
#define W4A4_DTYPE_F32 2
#define W4A4_HADAMARD_MAX_BLOCK 4096
w4a4_status w4a4_hadamard_transform(const void* x, int64_t ldx, void* y, int64_t ldy, int64_t rows, int64_t cols,
                                    int32_t block, int32_t dtype, void* stream);

/* ---- W8A8 layer -----------------------------------------------------------------------------
 * An 8-bit linear layer beside the 4-bit ones, for layers that four bits hurt (the modules a
 * checkpoint lists as not to convert): signed int8 weights with one scale per output channel,
 * activations quantized to int8 with one scale per token, the same smoothing, the same fused block
 * rotation, an optional bias.  Per row m of x:
 *   x_s  = float32(x) / float32(smooth_factor)   (round to nearest; below 2^-110 in magnitude within
 *          2^-133; no smooth_factor: x_s = x)
 *   u    = x_s, or the butterflies of svdq_quantize_act on every B-block, not yet normalised
 *   amax = max_k |u|,  ascales[m] = float32(float32(amax * norm) / 127), norm = float32(1/sqrt(B))
 *          (1 without rotation)
 *   qact = u * float32(127 / amax), the exact product rounded to the nearest integer, ties to even
 *          (within [-127, 127])
 *   y    = round( (float32(sum_k qact qweight) * ascales[m]) * wscales[n] + bias[n] )
 * The sum is exact (int32); the arithmetic after it is float32 with one rounding to y's type.
 * A row with amax * norm < 2^-100 gets scale 0 and codes 0; a row that holds an infinity or a NaN (or
 * whose smoothing or rotation overflows) gets scale NaN and codes 0, so its whole output row is
 * NaN.  float32(sum) * ascales[m] overflows to infinity for |v| of about 2^97 and more.
 *
 *   x      [M, K], row r at x + r ldx elements; x_dtype W4A4_DTYPE_BF16, _F16 or _F32; 16-byte
 *          aligned, ldx >= K, ldx % 8 == 0
 *   smooth_factor  bf16 [K], 16-byte aligned, or NULL for none
 *   K      >= 16, K % 16 == 0, at most W8A8_MAX_K (so that the int32 sum is exact)
 *   M, N   at most W8A8_MAX_ROWS, M * N at most 2^37; strides of several rows at most 2^32
 *   hadamard_block  0 (none) or 16, 32, 64, 128 with K % hadamard_block == 0
 *   qact   s8 [M, K], 16-byte aligned      ascales f32 [M]
 *   qweight s8 [N, K], 16-byte aligned     wscales f32 [N]     (codes -128 .. 127)
 *   bias   bf16 [N] or NULL
 *   y      [M, N], row r at y + r ldy elements (ldy >= N: a column partition of a wider matrix is
 *          fine, and nothing outside it is written); y_dtype as x_dtype
 * w8a8_quantize_weight is the offline counterpart: w * smooth_factor instead of the quotient, per
 * row n, the same rotation and codes; qweight and wscales are the layer's checkpoint tensors.
 * w8a8_linear is w8a8_quantize_act into the workspace (at least w8a8_linear_workspace_bytes(M, K)
 * bytes, 256-byte aligned, contents overwritten), then w8a8_gemm; projections of one input may
 * share one w8a8_quantize_act instead.  (Few tokens may be quantized and multiplied in one launch,
 * which leaves the workspace as it was: the same results, but no codes to read there.)  Results do
 * not depend on the batch a row is in (only the quotients below 2^-110 of a smoothing factor outside
 * [2^-32, 2^32] may round otherwise).
 * Outputs and the workspace share no element with an input or with each other (y == x is
 * refused); a call on another stream at the same time takes another workspace.
 * Errors: W4A4_ERR_UNSUPPORTED (hadamard_block, dtype, K > W8A8_MAX_K), W4A4_ERR_SHAPE (sizes,
 * strides, a workspace too small), W4A4_ERR_NULL, W4A4_ERR_ALIGN; sizes are checked first, then
 * the empty call (M or N == 0), then pointers, then alignment. */
#define W8A8_MAX_K 131056
#define W8A8_MAX_ROWS (1 << 28)
w4a4_status w8a8_quantize_act(const void* x, int64_t ldx, int32_t x_dtype, const void* smooth_factor, int64_t M,
                              int64_t K, int32_t hadamard_block, void* qact, float* ascales, void* stream);
w4a4_status w8a8_quantize_weight(const void* w, int64_t ldw, int32_t w_dtype, const void* smooth_factor, int64_t N,
                                 int64_t K, int32_t hadamard_block, void* qweight, float* wscales, void* stream);
w4a4_status w8a8_gemm(const void* qact, const float* ascales, const void* qweight, const float* wscales,
                      const void* bias, int64_t M, int64_t N, int64_t K, void* y, int64_t ldy, int32_t y_dtype,
                      void* stream);
size_t w8a8_linear_workspace_bytes(int64_t M, int64_t K);
w4a4_status w8a8_linear(const void* x, int64_t ldx, int32_t x_dtype, const void* qweight, const float* wscales,
                        const void* smooth_factor, const void* bias, int64_t M, int64_t N, int64_t K,
                        int32_t hadamard_block, void* y, int64_t ldy, int32_t y_dtype, void* workspace,
                        size_t workspace_bytes, void* stream);

/* ---- q / k head norm and rotary positions -----------------------------------------------------
 * What the q and k partitions of a projection's output go through before attention, in one pass and
 * one launch: per token and head of head_dim elements
 *   u = (x * (1 / sqrt(mean(x^2) + eps))) * weight       (with W4A4_ROPE_NORM; weight may be NULL)
 * then the rotation of the first rot = sum(axis_dims) elements in pairs: the rot / 2 pairs are
 * divided among the position axes in order, axis a taking axis_dims[a] / 2 of them, and number i of
 * axis a (pair p of all) turns by
 *   angle = positions[t, a] * theta^(-2 i / axis_dims[a])
 *   angle = positions[t, a] * theta^(-2 p / rot)         (with W4A4_ROPE_SHARED_FREQUENCIES)
 *   (u0, u1) -> (u0 cos - u1 sin, u0 sin + u1 cos)
 * These powers of theta are the only frequencies: ladders scaled per pair (a table of frequencies, a factor on
 * the cosines and sines) and axes that take the pairs in turn instead of in runs are not covered.  (One factor
 * on all of a ladder's frequencies cannot be given either; positions are integers.)
 * Elements rot .. head_dim - 1 are normed only.  Angles are formed and reduced in float64 (to
 * within 6 * 2^-53 of the token's largest angle, for any theta: from angles of about 2^28 on, this
 * shows in float32; positions past 2^53 are rounded to float64 first); each cosine and sine is then
 * within a few 2^-24 of its own size, next to 0 too (or within 4e-14); the rest is float32 with one
 * rounding to the tensors' type.  Squares that overflow float32 (|x| above about 2^63) give zeros; with eps = 0, a
 * head whose squares all underflow gives infinities, and one of zeros NaN.
 *
 * Elements (e0, e1) of pair p, number i of axis a whose first pair is s_a:
 *   W4A4_ROPE_INTERLEAVED  (2 p, 2 p + 1)
 *   W4A4_ROPE_HALF         (p, p + rot / 2)                           halves of the rotary span
 *   W4A4_ROPE_AXIS_HALF    (2 s_a + i, 2 s_a + i + axis_dims[a] / 2)  halves of each axis's slice
 *
 * q and k (k may be NULL) describe [tokens, heads, head_dim] tensors with a dense last dimension:
 * element (t, h, d) is at x + t x_token_stride + h x_head_stride + d, so partitions of a fused
 * projection's output and head-major outputs are addressed as they lie; q and k may have different
 * head counts.  x == y (with equal strides) works in place; any other overlap of an input and an
 * output, or of the two outputs, is undefined (one's y == the other's y or x is refused).  Only the addressed
 * elements are written.
 *   positions  [tokens, axes] int32 (int64 with W4A4_ROPE_POSITIONS_I64), dense; NULL when rot == 0
 *   axis_dims  HOST array of `axes` even sizes (0 allowed), sum at most head_dim; axes 0 ..
 *              W4A4_ROPE_MAX_AXES (0: norm only)
 *   head_dim   even, 2 .. W4A4_ROPE_MAX_HEAD_DIM
 *   dtype      W4A4_DTYPE_BF16, _F16 or _F32, of x, weight and y alike
 * Errors: W4A4_ERR_UNSUPPORTED (dtype, layout, flags, head_dim or axes above the maximum),
 * W4A4_ERR_SHAPE (sizes, a rotary span past head_dim, theta not positive and finite, eps negative,
 * negative strides or more than 2^40, offsets past 2^60, outputs whose elements share an address, in
 * place with other strides),
 * W4A4_ERR_NULL, W4A4_ERR_ALIGN (element size).  tokens == 0 or no heads launches nothing.
 * head_dim % 8 == 0, and in the split layouts axes of multiples of 8 elements, take the vectorised path
 * (at any alignment). */
#define W4A4_ROPE_INTERLEAVED 0
#define W4A4_ROPE_HALF 1
#define W4A4_ROPE_AXIS_HALF 2
#define W4A4_ROPE_NORM 1
#define W4A4_ROPE_SHARED_FREQUENCIES 2
#define W4A4_ROPE_POSITIONS_I64 4
#define W4A4_ROPE_MAX_HEAD_DIM 512
#define W4A4_ROPE_MAX_AXES 8
typedef struct {
  const void* x;
  int64_t x_token_stride, x_head_stride; /* elements */
  int64_t heads;
  const void* weight; /* [head_dim], or NULL */
  void* y;
  int64_t y_token_stride, y_head_stride;
} w4a4_heads;
w4a4_status w4a4_qk_norm_rope(const w4a4_heads* q, const w4a4_heads* k, const void* positions, int64_t tokens,
                              int32_t head_dim, int32_t axes, const int32_t* axis_dims, int32_t layout, int32_t flags,
                              double theta, float eps, int32_t dtype, void* stream);

#ifdef __cplusplus
}
#endif

#endif /* W4A4_H_ */
