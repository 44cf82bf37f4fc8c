// Internal kernel launchers of libw4a4 (not part of the public C ABI).
// Arguments are already validated by the entry points in api.cpp.
#pragma once

#include <hip/hip_runtime_api.h>
#include <stdint.h>
#include <stdlib.h>

namespace w4a4 {

// Launchers that a host-only build of the C-ABI layer (argument validation without kernels) may
// leave out: their references are weak, and an entry point whose launcher is missing returns
// W4A4_ERR_HIP.
#define W4A4_KERNELS __attribute__((weak))

// Kernel-path overrides.  Only the test build of the library (compiled with W4A4_TEST_HOOKS)
// reads them, from the environment, so that tests can force every kernel variant; in the
// product build every hook is absent and the automatic choice always applies.
#ifdef W4A4_TEST_HOOKS
inline const char* test_hook(const char* name) { return getenv(name); }
#else
inline const char* test_hook(const char*) { return nullptr; }
#endif

// Activation (act = true: divide by smooth_factor, low-rank down-projection)
// or weight (act = false: multiply by smooth_factor) quantizer over `rows` x K.
// With parts > 1, K is split across workgroups and lora receives `parts`
// partial sums, each [rows, R], laid out one after another.
// With mx, the scales are MXFP4 E8M0 bytes per 32 columns in rows of scale_stride bytes
// (scale_stride >= rows; entries rows .. scale_stride - 1 receive 0) and hadamard_block is 0 or 32.
hipError_t launch_quantize(bool act, const void* x, const void* lam, const void* pd, int64_t rows, int64_t K,
                           int64_t R, int hadamard_block, int parts, void* q, void* scales, float* lora,
                           hipStream_t stream, bool mx = false, int64_t scale_stride = 0);

// Batches up to this many rows use the weight-streaming GEMM.
constexpr int64_t SKINNY_MAX_M = 32;

// Number of K parts the activation quantizer uses for svdq_linear at these sizes.
int quantize_parts(int64_t M, int64_t K);

// Block-scaled FP4 GEMM with the fused epilogue.  `lora` holds `lora_parts` partial sums,
// each [M, R], added in order (lora_parts > 1 only for batches of at most SKINNY_MAX_M rows).
// `bias` (bf16 [N]) may be null.
hipError_t launch_gemm(const void* qact, const void* ascales, const float* lora, int lora_parts,
                       const void* qweight, const void* wscales, const void* proj_up, const void* wcscales,
                       const void* wtscale, const void* bias, int64_t M, int64_t N, int64_t K, int64_t R, void* y,
                       hipStream_t stream);

// MXFP4 GEMM (E8M0 scales per 32 columns; K % 128 == 0, N % 4 == 0; the activation scales
// are (K/32, ms) with ms = M rounded up to 4) with the same fused epilogue.
hipError_t launch_gemm_mx(const void* qact, const void* ascales, const float* lora, int lora_parts,
                          const void* qweight, const void* wscales, const void* proj_up, const void* wcscales,
                          const void* wtscale, const void* bias, int64_t M, int64_t N, int64_t K, int64_t R,
                          int64_t ms, void* y, hipStream_t stream);

// Weight-streaming variant for M <= SKINNY_MAX_M (called by launch_gemm).
hipError_t launch_gemm_skinny(const void* qact, const void* ascales, const float* lora, int lora_parts,
                              const void* qweight, const void* wscales, const void* proj_up, const void* wcscales,
                              const void* wtscale, const void* bias, int64_t M, int64_t N, int64_t K, int64_t R,
                              void* y, hipStream_t stream);

// MXFP4 weight-streaming variant for M <= 16, K <= 5120 a multiple of 512, R <= 64, at most 8
// low-rank parts (called by launch_gemm_mx; `ms` is the activation scale row stride).
bool skinny_mx_supported(int64_t M, int64_t K, int64_t R, int lora_parts);
hipError_t launch_gemm_skinny_mx(const void* qact, const void* ascales, const float* lora, int lora_parts,
                                 const void* qweight, const void* wscales, const void* proj_up, const void* wcscales,
                                 const void* wtscale, const void* bias, int64_t M, int64_t N, int64_t K, int64_t R,
                                 int64_t ms, void* y, hipStream_t stream);

// Standalone block Hadamard transform of rows x cols elements (row strides ldx, ldy in
// elements; dtype 0 bf16, 1 f16, 2 f32; block a power of two in [2, 4096] dividing cols);
// norm = float32(1 / sqrt(block)).  x == y (with ldx == ldy) transforms in place.
hipError_t launch_hadamard(const void* x, int64_t ldx, void* y, int64_t ldy, int64_t rows, int64_t cols, int block,
                           int dtype, float norm, hipStream_t stream);

// int8 quantizer of the W8A8 layer over rows x K (K a multiple of 16; x with a row stride of ldx
// elements, 16-byte aligned rows; dtype 0 bf16, 1 f16, 2 f32): divides by `lam` (act) or multiplies
// by it, `lam` may be null; block 0 or 16, 32, 64, 128 with norm = float32(1 / sqrt(block)).
hipError_t W4A4_KERNELS launch_quantize_i8(bool act, const void* x, int64_t ldx, const void* lam, int64_t rows,
                                           int64_t K, int block, int dtype, float norm, void* q, float* scales,
                                           hipStream_t stream);

// int8 GEMM with scales per row and column and an optional bias (bf16 [N], may be null); y has a
// row stride of ldy elements and the given type.
hipError_t W4A4_KERNELS launch_gemm_i8(const void* qact, const float* ascales, const void* qweight,
                                       const float* wscales, const void* bias, int64_t M, int64_t N, int64_t K, void* y,
                                       int64_t ldy, int ydtype, hipStream_t stream);

// The whole layer for a few tokens in one launch, for the sizes that linear_i8_one_launch accepts.
bool W4A4_KERNELS linear_i8_one_launch(int64_t M, int64_t N, int64_t K);
hipError_t W4A4_KERNELS launch_linear_i8_token(const void* x, int64_t ldx, int xdtype, const void* lam, int block,
                                               float norm, const void* qweight, const float* wscales,
                                               const void* bias, int64_t M, int64_t N, int64_t K, void* y, int64_t ldy,
                                               int ydtype, hipStream_t stream);

// Heads of one tensor of qk_norm_rope: element (token, head, d) at x + token ts + head hs + d.
struct RopeHeads {
  const void* x;
  int64_t ts, hs;
  int heads;
  const void* weight;
  void* y;
  int64_t yts, yhs;
};

constexpr int ROPE_MAX_AXES = 8;

// The frequencies of one axis's pairs, in turns per position: top * 2^(-step |p - origin|) for pair p.  The pair
// `origin` has the highest: the ladder's first pair, or its last where theta < 1.  (Axes that share one
// ladder have the same record.)
struct RopeLadder {
  double top, step;
  int origin;
};

struct RopeArgs {
  RopeHeads q, k;
  const void* pos;                // [tokens, axes], int32 or int64
  int tokens, D, axes;
  int rot2;                       // rotated pairs
  int start[ROPE_MAX_AXES + 1];   // first pair of every axis, then rot2
  int layout;                     // 0 interleaved, 1 halves of the span, 2 halves of each axis's slice
  bool norm, pos64;
  float eps, inv_d;
  RopeLadder ladder[ROPE_MAX_AXES];
  // set by the launcher: tokens and heads of a workgroup's pass, log2 of the lanes per head and of the pairs
  int tb, hb, log2g, log2p;
};

// RMS norm and rotary rotation of q and k heads; dtype 0 bf16, 1 f16, 2 f32.
hipError_t W4A4_KERNELS launch_qk_norm_rope(RopeArgs args, int dtype, hipStream_t stream);

// Device address of the static workspace of svdq_linear_noalloc on the current device (looked up
// once per device), or NULL when the lookup fails.
void* noalloc_scratch();

}  // namespace w4a4
