// Per-token (activations) and per-channel (weights) int8 quantizer of the W8A8 layer (gfx950); the
// arithmetic is in quantize_i8.h.
//
// Bound: HBM (x read once, codes written once).  A row stays in the registers of one workgroup
// between its maximum and its codes; the reciprocals of lambda are made once per workgroup and
// kept for all its rows, and the next row's loads are issued before the current row is reduced.
#include "quantize_i8.h"
#include "launch.h"

namespace w4a4 {

namespace {

// Activations, R rows per workgroup at a time (blockIdx R + 0 .. R - 1, then gridDim R rows further on):
// thread t holds the chunks c T + chunk_of(t) of 8 columns for c < C; T = blockDim, C T 8 >= K.
template <int DT, bool ROT, int C, int R>
__global__ __launch_bounds__(1024) void quant_i8_kernel(const void* __restrict__ x, int64_t ldx,
                                                        const uint16_t* __restrict__ lam, int rows, int K, int block,
                                                        float norm, int8_t* __restrict__ q,
                                                        float* __restrict__ scales) {
  __shared__ uint32_t red[2][R][16];
  const int t = threadIdx.x, lane = t & 63, wave = t >> 6, T = blockDim.x;
  const bool smooth = lam != nullptr;
  if (t < 32 * R) red[0][0][t] = 0;  // waves that do not exist
  int row = blockIdx.x * R;
  Raw8<DT> raw[R][C];
  const size_t es = DT == 2 ? 4 : 2;
  int col[C];
#pragma unroll
  for (int c = 0; c < C; ++c) col[c] = 8 * (c * T + (ROT ? chunk_of(t) : t));
  auto load_rows = [&](int row0) {
#pragma unroll
    for (int r = 0; r < R; ++r) {
      const void* xr = static_cast<const uint8_t*>(x) + (size_t)(row0 + r) * ldx * es;
#pragma unroll
      for (int c = 0; c < C; ++c) raw[r][c] = col[c] < K && row0 + r < rows ? load_raw<DT>(xr, col[c]) : zero_raw<DT>();
    }
  };
  load_rows(row);
  float rh[C][8], rl[C][8];
  bool plain = true;  // every lambda of this lane takes the two-part division
#pragma unroll
  for (int c = 0; c < C; ++c) {
    float l[8];
#pragma unroll
    for (int i = 0; i < 8; ++i) l[i] = 1.0f;
    if (smooth && col[c] < K) lambda8(lam, col[c], l);
    plain = reciprocals8(l, rh[c], rl[c]) && plain;
  }
  const bool wave_plain = __all(plain);
  const float sign = ROT ? lane_sign(lane, block) : 1.0f;
  __syncthreads();  // red is cleared
  int par = 0;
  while (true) {
    float v[R][C][8];
#pragma unroll
    for (int r = 0; r < R; ++r)
#pragma unroll
      for (int c = 0; c < C; ++c) {
        widen8<DT>(raw[r][c], v[r][c]);
        if (smooth) {
          if (wave_plain) {
#pragma unroll
            for (int i = 0; i < 8; ++i) v[r][c][i] = fmaf(v[r][c][i], rh[c][i], v[r][c][i] * rl[c][i]);
          } else {  // one element at a time (the values move through v[r][c][0]), to spend no registers on it
#pragma unroll 1
            for (int i = 0; i < 8; ++i) {
              const float f = col[c] < K ? v[r][c][0] / bf16_bits_to_f32(lam[col[c] + i]) : 0.0f;
#pragma unroll
              for (int e = 0; e < 7; ++e) v[r][c][e] = v[r][c][e + 1];
              v[r][c][7] = f;
            }
          }
        }
      }
    const int next = row + gridDim.x * R;
    if (next < rows) load_rows(next);
    uint32_t m[R];
#pragma unroll
    for (int r = 0; r < R; ++r) {
      if (ROT) rotate<C>(v[r], block, lane);
      m[r] = chunk_max<C>(v[r]);
    }
    // lanes 0 .. 31 go on with the first row, 32 .. 63 with the second (with R = 1, both with the one)
    const uint32_t mw = wave_max2(m[0], m[R - 1]);
    const int lr = R > 1 ? lane >> 5 : 0;
    if ((lane & 31) == 0) red[par][lr][wave] = mw;
    __syncthreads();  // the other parity's slots are rewritten only after the next barrier
    const uint32_t bits = lanes16_max(red[par][lr][lane & 15]);
    const float inv = row_inv(bits, norm);
    if (wave == 0 && (lane & 31) == 0 && row + lr < rows) scales[row + lr] = row_scale(bits, norm);
#pragma unroll
    for (int r = 0; r < R; ++r) {
      if (R > 1 && row + r >= rows) break;
      const float f = __uint_as_float(__builtin_amdgcn_readlane(__float_as_uint(inv), 32 * r));
      int8_t* qr = q + (size_t)(row + r) * K;
#pragma unroll
      for (int c = 0; c < C; ++c)
        if (col[c] < K) *reinterpret_cast<u32x2_t*>(qr + col[c]) = codes8(v[r][c], ROT ? f * sign : f);
    }
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
      }
      if (ROT) rotate<1>(v, block, lane);
    };
    uint32_t m = 0;
    const int tc = 8 * (ROT ? chunk_of(t) : t);
    for (int c0 = 0; c0 < K; c0 += 2048) {
      float v[1][8];
      values(c0 + tc, v);
      m = max(m, chunk_max<1>(v));
    }
    m = wave_max2(m, m);
    if (lane == 0) red[t >> 6] = m;
    __syncthreads();
    m = max(max(red[0], red[1]), max(red[2], red[3]));
    __syncthreads();
    float inv = row_inv(m, norm);
    if (ROT) inv *= lane_sign(lane, block);
    int8_t* qr = q + (size_t)row * K;
    for (int c0 = 0; c0 < K; c0 += 2048) {
      const int col = c0 + tc;
      float v[1][8];
      values(col, v);
      if (col < K) *reinterpret_cast<u32x2_t*>(qr + col) = codes8(v[0], inv);
    }
    if (t == 0) scales[row] = row_scale(m, norm);
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

template <int DT, bool ROT, int C, int R>
hipError_t run_short(const QArgs& a, int waves_per_cu) {
  // whole waves, just enough for the row's chunks; workgroups to fill the CUs once
  const int T = (a.K / 8 + 64 * C - 1) / (64 * C) * 64;
  const int grid = 256 * (waves_per_cu / (T / 64)), need = (a.rows + R - 1) / R;
  quant_i8_kernel<DT, ROT, C, R><<<dim3((unsigned)(need < grid ? need : grid)), T, 0, a.stream>>>(
      a.x, a.ldx, a.lam, a.rows, a.K, a.block, a.norm, a.q, a.scales);
  return hipGetLastError();
}

template <int DT, bool ROT>
hipError_t run(const QArgs& a, bool act) {
  if (act && a.K <= 8192) return a.rows >= 2048 ? run_short<DT, ROT, 1, 2>(a, 24) : run_short<DT, ROT, 1, 1>(a, 32);
  if (act && a.K <= 16384) return a.rows >= 2048 ? run_short<DT, ROT, 2, 2>(a, 16) : run_short<DT, ROT, 2, 1>(a, 16);
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
