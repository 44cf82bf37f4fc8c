// Per-token (activations) and per-channel (weights) int8 quantizer of the W8A8 layer (gfx950).
//
//   v     = x / smooth_factor (activations, float32, round to nearest) or w * smooth_factor (weights);
//           quotients of magnitude below 2^-110 count as 0
//   v     = v @ H_B^T per contiguous B-block (optional; butterfly spans 1, 2, ..., B/2, then one
//           multiply by float32(1/sqrt(B)), the rotation of the FP4 quantizer)
//   amax  = max_k |v[row, k]|,  scale[row] = float32(amax / 127)
//   code  = v * float32(127 / amax), the exact product rounded to the nearest integer, ties to even
// A row with amax < 2^-100 gets scale 0 and codes 0; a row that holds an infinity or a NaN gets
// scale NaN and codes 0, so that every output of that row is NaN.
//
// Two-part division.  With rh = RN(1/lambda) and rl = RN(RN(1 - lambda rh) rh) the sum rh + rl is
// within 2^-46 of 1/lambda, and q = RN(x rh + RN(x rl)) (one multiply, one fused multiply-add)
// differs from the exact quotient by less than 2^-45 before its one rounding.  lambda has 8
// significant bits, so a quotient x / lambda that is no midpoint of two float32 values is at least
// 2^-34 of its value away from every one, and none is a midpoint (midpoint * lambda would need
// more bits than x has): q is the correctly rounded quotient as long as x rl stays a normal
// number, that is for |q| >= 2^-110, and smaller quotients count as 0 on either path.  This holds
// for bf16, f16 and f32 x and lambda in [2^-32, 2^32]; a wave with another lambda divides.
//
// Rounding.  fma(v, inv, 1.5 * 2^23) rounds the exact product to an integer (the sum's ulp is 1)
// whose two's complement low byte is the code.
//
// Bound: HBM (x read once, codes written once).  A row stays in the registers of one workgroup
// between its maximum and its codes; the reciprocals of lambda are made once per workgroup and
// kept for all its rows, and the next row's loads are issued before the current row is reduced.
#include "device_common.h"
#include "launch.h"

namespace w4a4 {

namespace {

constexpr uint32_t ABS_MASK = 0x7FFFFFFFu;
constexpr uint32_t INF_BITS = 0x7F800000u;
constexpr float ROUND_MAGIC = 12582912.0f;  // 1.5 * 2^23
constexpr float TINY_ROW = 7.888609052210118e-31f;   // 2^-100
constexpr float TINY_QUOTIENT = 7.703719777548943e-34f;  // 2^-110

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

__device__ __forceinline__ float drop_tiny(float q) { return fabsf(q) < TINY_QUOTIENT ? 0.0f : q; }

// The value of lane l ^ D within 16 lanes, by DPP.
template <int D>
__device__ __forceinline__ float lane16_xor(float v) {
  const int b = __float_as_int(v);
  if constexpr (D == 1) return __int_as_float(__builtin_amdgcn_mov_dpp(b, 0xB1, 0xF, 0xF, true));
  if constexpr (D == 2) return __int_as_float(__builtin_amdgcn_mov_dpp(b, 0x4E, 0xF, 0xF, true));
  if constexpr (D == 4)  // l ^ 7 (row_half_mirror), then l ^ 3 (quad_perm [3,2,1,0])
    return __int_as_float(__builtin_amdgcn_mov_dpp(__builtin_amdgcn_mov_dpp(b, 0x141, 0xF, 0xF, true), 0x1B, 0xF, 0xF, true));
  return __int_as_float(__builtin_amdgcn_mov_dpp(b, 0x128, 0xF, 0xF, true));  // row_ror:8
}

// One butterfly stage between lanes l and l ^ D: the lower lane keeps a + b, the upper a - b.
template <int D, int C>
__device__ __forceinline__ void lane_stage(float (&v)[C][8], int lane) {
  const uint32_t flip = (lane & D) ? 0x80000000u : 0u;
#pragma unroll
  for (int c = 0; c < C; ++c)
#pragma unroll
    for (int i = 0; i < 8; ++i)
      v[c][i] = lane16_xor<D>(v[c][i]) + __uint_as_float(__float_as_uint(v[c][i]) ^ flip);
}

// Rotation of C chunks of 8 columns; consecutive lanes hold consecutive chunks.  `block` is 16, 32,
// 64 or 128 (the same for the whole launch).
template <int C>
__device__ __forceinline__ void rotate(float (&v)[C][8], int block, float norm, int lane) {
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
  lane_stage<1, C>(v, lane);
  if (block >= 32) lane_stage<2, C>(v, lane);
  if (block >= 64) lane_stage<4, C>(v, lane);
  if (block >= 128) lane_stage<8, C>(v, lane);
#pragma unroll
  for (int c = 0; c < C; ++c)
#pragma unroll
    for (int i = 0; i < 8; ++i) v[c][i] *= norm;
}

__device__ __forceinline__ uint32_t wave_max(uint32_t m) {
#pragma unroll
  for (int d = 1; d < 64; d *= 2) m = max(m, (uint32_t)__shfl_xor((int)m, d));
  return m;
}

// Scale and 127 / amax of a row from the bits of its maximum magnitude; inv is 0 where the codes are 0.
__device__ __forceinline__ void row_scale(uint32_t bits, float& scale, float& inv) {
  const float amax = __uint_as_float(bits);
  if (bits >= INF_BITS) {
    scale = __uint_as_float(0x7FC00000u);
    inv = 0.0f;
  } else if (amax < TINY_ROW) {
    scale = 0.0f;
    inv = 0.0f;
  } else {
    scale = amax / 127.0f;
    inv = 127.0f / amax;
  }
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

// Activations, one row per workgroup at a time (rows blockIdx, blockIdx + gridDim, ...): thread t
// holds columns 8 (c T + t) .. + 8 for c < C, C T 8 >= K.
template <int DT, bool ROT, int T, int C>
__global__ __launch_bounds__(T) void quant_i8_kernel(const void* __restrict__ x, int64_t ldx,
                                                     const uint16_t* __restrict__ lam, int rows, int K, int block,
                                                     float norm, int8_t* __restrict__ q, float* __restrict__ scales) {
  constexpr int NW = T / 64;
  __shared__ uint32_t red[2][NW];
  const int t = threadIdx.x, lane = t & 63, wave = t >> 6;
  const bool smooth = lam != nullptr;
  int row = blockIdx.x;
  Raw8<DT> raw[C];
  const size_t es = DT == 2 ? 4 : 2;
  auto load_row = [&](int r) {
    const void* xr = static_cast<const uint8_t*>(x) + (size_t)r * ldx * es;
#pragma unroll
    for (int c = 0; c < C; ++c) {
      const int col = 8 * (c * T + t);
      raw[c] = col < K ? load_raw<DT>(xr, col) : zero_raw<DT>();
    }
  };
  load_row(row);
  float rh[C][8], rl[C][8];
  bool plain = true;  // every lambda of this lane takes the two-part division
#pragma unroll
  for (int c = 0; c < C; ++c) {
    const int col = 8 * (c * T + t);
    float l[8];
#pragma unroll
    for (int i = 0; i < 8; ++i) l[i] = 1.0f;
    if (smooth && col < K) lambda8(lam, col, l);
#pragma unroll
    for (int i = 0; i < 8; ++i) {
      const float m = fabsf(l[i]);
      plain = plain && m >= 2.3283064365386963e-10f && m <= 4294967296.0f;
      rh[c][i] = 1.0f / l[i];
      rl[c][i] = fmaf(-l[i], rh[c][i], 1.0f) * rh[c][i];
    }
  }
  const bool wave_plain = __all(plain);
  int par = 0;
  while (true) {
    float v[C][8];
#pragma unroll
    for (int c = 0; c < C; ++c) widen8<DT>(raw[c], v[c]);
    if (smooth) {
      if (wave_plain) {
#pragma unroll
        for (int c = 0; c < C; ++c)
#pragma unroll
          for (int i = 0; i < 8; ++i) v[c][i] = fmaf(v[c][i], rh[c][i], v[c][i] * rl[c][i]);
      } else {
        for (int c = 0; c < C; ++c) {
          const int col = 8 * (c * T + t);
          float l[8];
          if (col < K) {
            lambda8(lam, col, l);
#pragma unroll
            for (int i = 0; i < 8; ++i) v[c][i] = v[c][i] / l[i];
          }
        }
      }
      if (ROT) {
#pragma unroll
        for (int c = 0; c < C; ++c)
#pragma unroll
          for (int i = 0; i < 8; ++i) v[c][i] = drop_tiny(v[c][i]);
      }
    }
    const int next = row + gridDim.x;
    if (next < rows) load_row(next);
    if (ROT) rotate<C>(v, block, norm, lane);
    uint32_t m = 0;
#pragma unroll
    for (int c = 0; c < C; ++c)
#pragma unroll
      for (int i = 0; i < 8; ++i) m = max(m, __float_as_uint(v[c][i]) & ABS_MASK);
    m = wave_max(m);
    if (lane == 0) red[par][wave] = m;
    __syncthreads();  // the other parity's slots are rewritten only after the next barrier
#pragma unroll
    for (int w = 0; w < NW; ++w) m = max(m, red[par][w]);
    float scale, inv;
    row_scale(m, scale, inv);
    int8_t* qr = q + (size_t)row * K;
#pragma unroll
    for (int c = 0; c < C; ++c) {
      const int col = 8 * (c * T + t);
      if (col < K) *reinterpret_cast<u32x2_t*>(qr + col) = codes8(v[c], inv);
    }
    if (t == 0) scales[row] = scale;
    row = next;
    if (row >= rows) break;
    par ^= 1;
  }
}

// Weights (ACT false) and activations with rows too long for the registers: two passes over the row.
template <int DT, bool ROT, bool ACT>
__global__ __launch_bounds__(256) void quant_i8_long_kernel(const void* __restrict__ x, int64_t ldx,
                                                            const uint16_t* __restrict__ lam, int rows, int K,
                                                            int block, float norm, int8_t* __restrict__ q,
                                                            float* __restrict__ scales) {
  __shared__ uint32_t red[4];
  const int t = threadIdx.x, lane = t & 63;
  const size_t es = DT == 2 ? 4 : 2;
  for (int row = blockIdx.x; row < rows; row += gridDim.x) {
    const void* xr = static_cast<const uint8_t*>(x) + (size_t)row * ldx * es;
    auto values = [&](int col, float (&v)[1][8]) {
      const bool in = col < K;
      widen8<DT>(in ? load_raw<DT>(xr, col) : zero_raw<DT>(), v[0]);
      if (lam != nullptr && in) {
        float l[8];
        lambda8(lam, col, l);
#pragma unroll
        for (int i = 0; i < 8; ++i) v[0][i] = ACT ? v[0][i] / l[i] : v[0][i] * l[i];
        if (ROT && ACT) {
#pragma unroll
          for (int i = 0; i < 8; ++i) v[0][i] = drop_tiny(v[0][i]);
        }
      }
      if (ROT) rotate<1>(v, block, norm, lane);
    };
    uint32_t m = 0;
    for (int c0 = 0; c0 < K; c0 += 2048) {
      float v[1][8];
      values(c0 + 8 * t, v);
#pragma unroll
      for (int i = 0; i < 8; ++i) m = max(m, __float_as_uint(v[0][i]) & ABS_MASK);
    }
    m = wave_max(m);
    if (lane == 0) red[t >> 6] = m;
    __syncthreads();
    m = max(max(red[0], red[1]), max(red[2], red[3]));
    __syncthreads();
    float scale, inv;
    row_scale(m, scale, inv);
    int8_t* qr = q + (size_t)row * K;
    for (int c0 = 0; c0 < K; c0 += 2048) {
      const int col = c0 + 8 * t;
      float v[1][8];
      values(col, v);
      if (col < K) *reinterpret_cast<u32x2_t*>(qr + col) = codes8(v[0], inv);
    }
    if (t == 0) scales[row] = scale;
  }
}

struct QArgs {
  const void* x;
  int64_t ldx;
  const uint16_t* lam;
  int rows, K, block;
  float norm;
  int8_t* q;
  float* scales;
  hipStream_t stream;
};

template <int DT, bool ROT, int T, int C>
hipError_t run_short(const QArgs& a, int grid) {
  quant_i8_kernel<DT, ROT, T, C><<<dim3((unsigned)(a.rows < grid ? a.rows : grid)), T, 0, a.stream>>>(
      a.x, a.ldx, a.lam, a.rows, a.K, a.block, a.norm, a.q, a.scales);
  return hipGetLastError();
}

template <int DT, bool ROT>
hipError_t run(const QArgs& a, bool act) {
  if (act && a.K <= 16384) {
    // few rows: as many threads per row as it has chunks, for latency; many rows: smaller
    // workgroups, several per CU, each keeping its reciprocals over several rows
    if (a.rows < 1024) return a.K <= 8192 ? run_short<DT, ROT, 1024, 1>(a, 1024) : run_short<DT, ROT, 1024, 2>(a, 1024);
    if (a.K <= 2048) return run_short<DT, ROT, 256, 1>(a, 2048);
    if (a.K <= 4096) return run_short<DT, ROT, 256, 2>(a, 1024);
    if (a.K <= 6144) return run_short<DT, ROT, 256, 3>(a, 1024);
    if (a.K <= 8192) return run_short<DT, ROT, 256, 4>(a, 1024);
    if (a.K <= 12288) return run_short<DT, ROT, 512, 3>(a, 512);
    return run_short<DT, ROT, 512, 4>(a, 512);
  }
  const dim3 grid((unsigned)(a.rows < 4096 ? a.rows : 4096));
  if (act)
    quant_i8_long_kernel<DT, ROT, true><<<grid, 256, 0, a.stream>>>(a.x, a.ldx, a.lam, a.rows, a.K, a.block, a.norm, a.q, a.scales);
  else
    quant_i8_long_kernel<DT, ROT, false><<<grid, 256, 0, a.stream>>>(a.x, a.ldx, a.lam, a.rows, a.K, a.block, a.norm, a.q, a.scales);
  return hipGetLastError();
}

}  // namespace

hipError_t launch_quantize_i8(bool act, const void* x, int64_t ldx, const void* lam, int64_t rows, int64_t K, int block,
                              int dtype, float norm, void* q, float* scales, hipStream_t stream) {
  const QArgs a{x, ldx, static_cast<const uint16_t*>(lam), (int)rows, (int)K, block, norm, static_cast<int8_t*>(q),
                scales, stream};
  switch (dtype) {
    case 0: return block ? run<0, true>(a, act) : run<0, false>(a, act);
    case 1: return block ? run<1, true>(a, act) : run<1, false>(a, act);
    default: return block ? run<2, true>(a, act) : run<2, false>(a, act);
  }
}

}  // namespace w4a4
