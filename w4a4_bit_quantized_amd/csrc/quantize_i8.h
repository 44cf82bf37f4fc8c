// Arithmetic of the W8A8 layer's int8 quantizer (gfx950), shared by the quantizer kernels and the one-launch
// layer for a few tokens.
//
//   v     = x / smooth_factor (activations, float32, round to nearest) or w * smooth_factor (weights)
//   u     = v, or the butterflies of v per contiguous B-block (spans 1, 2, ..., B/2)
//   amax  = max_k |u[row, k]|
//   code  = u * float32(127 / amax), the exact product rounded to the nearest integer, ties to even
//   scale = float32(float32(amax * norm) / 127),  norm = float32(1/sqrt(B)), 1 without rotation
// so that code * scale stands for the normalised rotation's value: the normalisation is one
// multiply per row instead of one per element.  A row with amax * norm < 2^-100 gets scale 0 and codes
// 0; a row that holds an infinity or a NaN gets scale NaN and codes 0, so that every output of that
// row is NaN.
//
// Two-part division.  With rh the hardware's 1/lambda (within one unit in the last place) and rl =
// RN((1 - lambda rh) rh), whose first factor is exact, the sum rh + rl is within 2^-45 of 1/lambda, and
// q = RN(x rh + RN(x rl)) (one multiply, one fused multiply-add) differs from the exact quotient by
// less than 2^-44 of it before its one rounding.  lambda has 8
// significant bits, so a quotient x / lambda is at least 2^-33 of its value away from every midpoint
// of two float32 values (a midpoint times lambda has more bits than x): q is the correctly rounded
// quotient as long as x rl stays a normal number, that is for |q| >= 2^-110.  A smaller quotient is
// within 2^-133 of x / lambda; in a row that does not count as zero its code is 0 either way.  This
// holds for bf16, f16 and f32 x and lambda in [2^-32, 2^32]; a wave with another lambda divides.
//
// Rounding.  fma(u, inv, 1.5 * 2^23) rounds the exact product to an integer (the sum's ulp is 1)
// whose two's complement low byte is the code.
//
// Rotation.  A lane holds 8 consecutive columns: spans 1, 2, 4 stay inside it.  The spans 8 .. 64 pair
// lanes of a 16-lane row, all by one DPP operand of a fused multiply-add: v + s * (partner's v) with
// s = +-1 is a + b in the lower lane and -(a - b) in the upper one, the rounding of the difference and
// the opposite sign.  The sign is the same for all values of a lane and stays with them (a partner
// differs in one lane bit only), so it is undone by the sign of the lane's inv.  DPP pairs lanes l ^ 1,
// l ^ 2, l ^ 7 and l ^ 8 in one operand but not l ^ 4, so the lanes 4 .. 7 of 8 hold their four chunks in
// reverse order, which makes l ^ 7 the partner of span 32.
#pragma once

#include "device_common.h"

namespace w4a4 {

namespace {

constexpr uint32_t ABS_MASK = 0x7FFFFFFFu;
constexpr uint32_t INF_BITS = 0x7F800000u;
constexpr float ROUND_MAGIC = 12582912.0f;  // 1.5 * 2^23
constexpr float TINY_ROW = 7.888609052210118e-31f;   // 2^-100

// Eight consecutive elements as loaded (storage types: 0 bf16, 1 f16, 2 f32).
template <int DT>
struct Raw8 {
  u32x4_t w[DT == 2 ? 2 : 1];
};

template <int DT>
__device__ __forceinline__ Raw8<DT> load_raw(const void* base, int64_t i) {
  Raw8<DT> r;
  if constexpr (DT == 2) {
    const u32x4_t* p = reinterpret_cast<const u32x4_t*>(static_cast<const float*>(base) + i);
    r.w[0] = p[0];
    r.w[1] = p[1];
  } else {
    r.w[0] = *reinterpret_cast<const u32x4_t*>(static_cast<const uint16_t*>(base) + i);
  }
  return r;
}

template <int DT>
__device__ __forceinline__ Raw8<DT> zero_raw() {
  Raw8<DT> r;
  r.w[0] = u32x4_t{0u, 0u, 0u, 0u};
  if constexpr (DT == 2) r.w[1] = r.w[0];
  return r;
}

template <int DT>
__device__ __forceinline__ void widen8(const Raw8<DT>& r, float (&v)[8]) {
  if constexpr (DT == 2) {
#pragma unroll
    for (int e = 0; e < 4; ++e) {
      v[e] = __uint_as_float(r.w[0][e]);
      v[4 + e] = __uint_as_float(r.w[1][e]);
    }
  } else if constexpr (DT == 1) {
    const half8_t h = __builtin_bit_cast(half8_t, r.w[0]);
#pragma unroll
    for (int e = 0; e < 8; ++e) v[e] = (float)h[e];
  } else {
#pragma unroll
    for (int e = 0; e < 4; ++e) {
      v[2 * e] = __uint_as_float(r.w[0][e] << 16);
      v[2 * e + 1] = __uint_as_float(r.w[0][e] & 0xFFFF0000u);
    }
  }
}

__device__ __forceinline__ void lambda8(const uint16_t* lam, int64_t col, float (&l)[8]) {
  const u32x4_t w = *reinterpret_cast<const u32x4_t*>(lam + col);
#pragma unroll
  for (int e = 0; e < 4; ++e) {
    l[2 * e] = __uint_as_float(w[e] << 16);
    l[2 * e + 1] = __uint_as_float(w[e] & 0xFFFF0000u);
  }
}

template <int CTRL>
__device__ __forceinline__ float dpp(float v) {
  return __int_as_float(__builtin_amdgcn_mov_dpp(__float_as_int(v), CTRL, 0xF, 0xF, true));
}
template <int CTRL>
__device__ __forceinline__ uint32_t dpp(uint32_t v) {
  return (uint32_t)__builtin_amdgcn_mov_dpp((int)v, CTRL, 0xF, 0xF, true);
}
constexpr int DPP_XOR1 = 0xB1, DPP_XOR2 = 0x4E, DPP_XOR7 = 0x141, DPP_XOR15 = 0x140;

// Which chunk of 8 columns thread t holds (see the top of the file).
__device__ __forceinline__ int chunk_of(int t) { return t ^ ((t & 4) ? 3 : 0); }

// Reciprocals of 8 smoothing factors in two parts; whether all of them are in the division's range.
__device__ __forceinline__ bool reciprocals8(const float (&l)[8], float (&rh)[8], float (&rl)[8]) {
  bool plain = true;
#pragma unroll
  for (int i = 0; i < 8; ++i) {
    const float m = fabsf(l[i]);
    plain = plain && m >= 2.3283064365386963e-10f && m <= 4294967296.0f;
    rh[i] = __builtin_amdgcn_rcpf(l[i]);
    rl[i] = fmaf(-l[i], rh[i], 1.0f) * rh[i];
  }
  return plain;
}

// Signs of a lane's values after the rotation, as a factor.
__device__ __forceinline__ float lane_sign(int lane, int block) {
  // bits of the lane's chunk index: spans 8, 16, 32, 64
  const int j = chunk_of(lane) & (block / 8 - 1);
  return (__popc(j) & 1) ? -1.0f : 1.0f;
}

// v + s * (partner's v) for 8 values: v_fmac_f32 with a DPP first operand, which the compiler does not
// form from a move and an fma.  The leading s_nop covers the two wait states between a vector
// instruction that writes a register and one that reads it through DPP.
#define W8A8_FMAC_DPP(CTRL)                                                                                   \
  asm("s_nop 1\n\t"                                                                                           \
      "v_fmac_f32_dpp %0, %0, %8 " CTRL " row_mask:0xf bank_mask:0xf\n\t"                                     \
      "v_fmac_f32_dpp %1, %1, %8 " CTRL " row_mask:0xf bank_mask:0xf\n\t"                                     \
      "v_fmac_f32_dpp %2, %2, %8 " CTRL " row_mask:0xf bank_mask:0xf\n\t"                                     \
      "v_fmac_f32_dpp %3, %3, %8 " CTRL " row_mask:0xf bank_mask:0xf\n\t"                                     \
      "v_fmac_f32_dpp %4, %4, %8 " CTRL " row_mask:0xf bank_mask:0xf\n\t"                                     \
      "v_fmac_f32_dpp %5, %5, %8 " CTRL " row_mask:0xf bank_mask:0xf\n\t"                                     \
      "v_fmac_f32_dpp %6, %6, %8 " CTRL " row_mask:0xf bank_mask:0xf\n\t"                                     \
      "v_fmac_f32_dpp %7, %7, %8 " CTRL " row_mask:0xf bank_mask:0xf"                                         \
      : "+v"(v[0]), "+v"(v[1]), "+v"(v[2]), "+v"(v[3]), "+v"(v[4]), "+v"(v[5]), "+v"(v[6]), "+v"(v[7])        \
      : "v"(s))
__device__ __forceinline__ void stage_xor1(float (&v)[8], float s) { W8A8_FMAC_DPP("quad_perm:[1,0,3,2]"); }
__device__ __forceinline__ void stage_xor2(float (&v)[8], float s) { W8A8_FMAC_DPP("quad_perm:[2,3,0,1]"); }
__device__ __forceinline__ void stage_xor7(float (&v)[8], float s) { W8A8_FMAC_DPP("row_half_mirror"); }
__device__ __forceinline__ void stage_xor8(float (&v)[8], float s) { W8A8_FMAC_DPP("row_ror:8"); }
#undef W8A8_FMAC_DPP

// Butterflies of C chunks of 8 columns per lane, up to the lane's sign.  `block` is 16, 32, 64 or 128 (the
// same for the whole launch).
template <int C>
__device__ __forceinline__ void rotate(float (&v)[C][8], int block, int lane) {
#pragma unroll
  for (int s = 1; s < 8; s *= 2)
#pragma unroll
    for (int c = 0; c < C; ++c)
#pragma unroll
      for (int i = 0; i < 8; ++i)
        if ((i & s) == 0) {
          const float a = v[c][i], b = v[c][i + s];
          v[c][i] = a + b;
          v[c][i + s] = a - b;
        }
  const int j = chunk_of(lane);
#pragma unroll
  for (int c = 0; c < C; ++c) {
    stage_xor1(v[c], (j & 1) ? -1.0f : 1.0f);
    if (block >= 32) stage_xor2(v[c], (j & 2) ? -1.0f : 1.0f);
    if (block >= 64) stage_xor7(v[c], (j & 4) ? -1.0f : 1.0f);
    if (block >= 128) stage_xor8(v[c], (j & 8) ? -1.0f : 1.0f);
  }
}

// Largest magnitude of C chunks as bits (a NaN above an infinity above every number).
template <int C>
__device__ __forceinline__ uint32_t chunk_max(const float (&v)[C][8]) {
  uint32_t m = 0;
#pragma unroll
  for (int c = 0; c < C; ++c)
#pragma unroll
    for (int i = 0; i < 8; ++i) m = max(m, __float_as_uint(v[c][i]) & ABS_MASK);
  return m;
}

// Maximum over a row of 16 lanes.
__device__ __forceinline__ uint32_t lanes16_max(uint32_t m) {
  m = max(m, dpp<DPP_XOR1>(m));
  m = max(m, dpp<DPP_XOR2>(m));
  m = max(m, dpp<DPP_XOR7>(m));
  return max(m, dpp<DPP_XOR15>(m));
}

// Maxima of m0 and of m1 over a wave: the first in the lower 32 lanes, the second in the upper.
__device__ __forceinline__ uint32_t wave_max2(uint32_t m0, uint32_t m1) {
  auto a = __builtin_amdgcn_permlane32_swap(m0, m1, false, false);
  uint32_t m = lanes16_max(max(a[0], a[1]));
  auto b = __builtin_amdgcn_permlane16_swap(m, m, false, false);
  return max(b[0], b[1]);
}

// 127 / amax of a row from the bits of its maximum magnitude; 0 where the codes are 0.
__device__ __forceinline__ float row_inv(uint32_t bits, float norm) {
  const float amax = __uint_as_float(bits), inv = 127.0f / amax;
  return bits >= INF_BITS || amax * norm < TINY_ROW ? 0.0f : inv;
}

__device__ __forceinline__ float row_scale(uint32_t bits, float norm) {
  const float amax = __uint_as_float(bits), scale = (amax * norm) / 127.0f;
  return bits >= INF_BITS ? __uint_as_float(0x7FC00000u) : amax * norm < TINY_ROW ? 0.0f : scale;
}

// Eight codes of one chunk, packed.  inv == 0 gives 0 for every finite or non-finite value.
__device__ __forceinline__ u32x2_t codes8(const float (&v)[8], float inv) {
  uint32_t b[8];
#pragma unroll
  for (int i = 0; i < 8; ++i) b[i] = __float_as_uint(fmaf(v[i], inv, ROUND_MAGIC));
  u32x2_t r;
#pragma unroll
  for (int h = 0; h < 2; ++h) {
    const uint32_t lo = __builtin_amdgcn_perm(b[4 * h + 1], b[4 * h], 0x0C0C0400u);
    const uint32_t hi = __builtin_amdgcn_perm(b[4 * h + 3], b[4 * h + 2], 0x04000C0Cu);
    r[h] = lo | hi;
  }
  return inv == 0.0f ? u32x2_t{0u, 0u} : r;
}

}  // namespace

}  // namespace w4a4
