// int8 GEMM of the W8A8 layer (gfx950): one scale per token and per output channel.
//
//   y[m, n] = store( (float32(sum_k qact[m, k] qweight[n, k]) * ascales[m]) * wscales[n] + bias[n] )
// The sum is exact in int32 (K <= 131056: |sum| <= K * 127 * 128 < 2^31); the conversion to
// float32, the two products and the sum round to nearest, then one rounding to the storage type.
//
// Both operands are K-contiguous bytes, so every 16-byte chunk is matrix-core operand data as it
// stands: v_mfma_i32_32x32x32_i8 takes 16 K-columns per lane (row l % 32, columns 16 (l / 32) ..).
// Weights are the first operand, activations the second: lane l then holds column m = l % 32 of
// the product and four consecutive n per accumulator quad.
//
// Chunks past K (K is a multiple of 16, a K-step has 128 columns) are read from a 16-byte block of
// zeros, rows past M or N repeat the last row and are not stored.
#include <cstring>

#include "device_common.h"
#include "gemm_common.h"
#include "launch.h"
#include "quantize_i8.h"

namespace w4a4 {

namespace {

typedef int i32x4_t __attribute__((ext_vector_type(4)));
typedef int i32x16_t __attribute__((ext_vector_type(16)));

__device__ __attribute__((aligned(16))) const uint32_t zero_chunk[4] = {0u, 0u, 0u, 0u};

// Storage types of y: 0 bf16, 1 f16, 2 f32.
template <int YT>
struct YType {
  static constexpr int ES = YT == 2 ? 4 : 2;
};

__device__ __forceinline__ uint32_t pack_f16x2(float a, float b) {
  typedef _Float16 f16x2_t __attribute__((ext_vector_type(2)));
  return __builtin_bit_cast(uint32_t, f16x2_t{(_Float16)a, (_Float16)b});  // round to nearest even
}

template <int YT>
__device__ __forceinline__ void store_one(void* y, size_t i, float v) {
  if constexpr (YT == 2) static_cast<float*>(y)[i] = v;
  else if constexpr (YT == 1) static_cast<_Float16*>(y)[i] = (_Float16)v;
  else static_cast<uint16_t*>(y)[i] = (uint16_t)pack_bf16x2(v, v);
}

// ---- tiled GEMM ----------------------------------------------------------------------------------

// KG groups of WAVES_M x WAVES_N waves split K (group k takes the K-steps k, k + KG, ...), each with a ring
// of S stages of its own; their partial sums meet in LDS.
//
// NL > 0: NL further waves do nothing but the direct loads.  A wave whose load waits for its turn issues no
// matrix instruction either, so with loads in every wave the two times add up where a wave has few matrix
// instructions per K-step (L2-resident operands, 128 x 128 x 128 per step: 217 ns of loads and 222 of matrix
// instructions take 418 together); with waves of their own the loads run beside them (1021 x 2050 x 4096 in
// 128 x 128 tiles: 24.8 to 21.1 us; 1024 x 4096 x 4096: 25.9 to 23.4; 256 x 5120 x 5120 in 64 x 128: 17.6 to
// 16.5).  Four loaders, one per SIMD: two of them cannot issue fast enough, eight measured as four.  They
// are a third wave per SIMD, which leaves 168 registers to each: the tiles of 256 rows need more.
//
// SHIFT: rows off 128-byte boundaries (K % 128 != 0, or such operands).  Read from its own start, every
// 128-byte chunk of a row would touch two lines of memory (1024 x 2048 x 4112: 20.2 us, x 4096: 15.8).  Instead
// a stage holds one aligned line of every row, its window: window w of a row that starts s 16-byte chunks into
// a line holds its chunks 8 w - s .. 8 w - s + 7, and K-step kt takes chunk 8 kt + c from place c + s of window kt
// or, past its end, of window kt + 1.  s depends on the row modulo 8 only (K % 16 == 0), so a lane's rows
// share it.  One more window is resident, and places before a row's start or past its end hold zeros.
template <int WAVES_M, int WAVES_N, int FM, int FN, int S, int KG, int NL, bool SHIFT>
struct TileI8 {
  static constexpr int WAVES = WAVES_M * WAVES_N;  // of a group
  static constexpr int LW = NL ? NL / KG : WAVES;  // waves that load (of a group)
  static constexpr int THREADS = 64 * (WAVES * KG + NL);
  static constexpr int BM = WAVES_M * FM * 32, BN = WAVES_N * FN * 32;
  static constexpr int ROWS = BM + BN;             // activation rows, then weight rows
  static constexpr int STEP = 128;                 // K columns (bytes) per stage: whole 128-byte lines
  static constexpr int STAGE = ROWS * STEP;
  static constexpr int ROUNDS = ROWS / (8 * LW);   // a wave's direct load fills 8 rows
  static constexpr int REGION = 32 * FN * 32 * 4;  // a wave's epilogue region: 32 rows of f32
  static constexpr int PART = (KG - 1) * BM * BN * 4;  // partial sums of the groups after the first
  static constexpr int EPI = WAVES * REGION + BN * 8 > PART ? WAVES * REGION + BN * 8 : PART;
  static constexpr int LDS = KG * S * STAGE > EPI ? KG * S * STAGE : EPI;
  static_assert(ROWS % (8 * LW) == 0 && BM % (8 * LW) == 0, "whole rounds per operand");
  static_assert(NL % KG == 0 && (KG == 1 || NL > 0), "groups have loaders, as many each");
  static_assert(!SHIFT || (NL > 0 && S >= 3), "two windows resident, one on its way");
  static_assert(LDS <= 160 * 1024, "LDS of one CU");
  static_assert(ROUNDS * S < 64, "vmcnt range");
};

// LDS slot of chunk c of row r: c ^ ((r >> 1) & 7).  16 consecutive rows reading one chunk then
// touch 16 distinct 16-byte columns of the 256 bytes of banks.
__device__ __forceinline__ int i8_swizzle(int row) { return (row >> 1) & 7; }

// 16 bytes per lane from `src` to LDS at dst + 16 lane (dst is the wave's).
__device__ __forceinline__ void load_lds16(const uint8_t* src, uint8_t* dst) {
  __builtin_amdgcn_global_load_lds(src, (lds_void*)dst, 16, 0, 0);
}

// Rounds R0 .. R1 - 1 of one K-step's direct loads into a stage (16 bytes per lane, 8 rows of 128 bytes
// per instruction).  off is the chunk's offset from abase or bbase + k0 (SHIFT: plus 112, so that it is not
// negative), col its K-column minus k0 (SHIFT: possibly negative; as unsigned numbers, columns before the row's
// start are past its end).
template <class T, bool SHIFT, int R0, int R1>
__device__ __forceinline__ void i8_issue(uint8_t* stage, int wave, uint32_t k0, uint32_t K, const uint8_t* abase,
                                         const uint8_t* bbase, const uint32_t* off, const uint32_t* col) {
  if ((!SHIFT || k0 >= T::STEP) && k0 + T::STEP <= K) {
#pragma unroll
    for (int r = R0; r < R1; ++r)
      load_lds16((r * T::LW * 8 < T::BM ? abase : bbase) + k0 - (SHIFT ? 112 : 0) + off[r],
                 stage + (r * T::LW + wave) * 1024);
  } else {
#pragma unroll
    for (int r = R0; r < R1; ++r) {
      const uint8_t* p = (r * T::LW * 8 < T::BM ? abase : bbase) + k0 - (SHIFT ? 112 : 0) + off[r];
      if (k0 + col[r] >= K) p = reinterpret_cast<const uint8_t*>(zero_chunk);
      load_lds16(p, stage + (r * T::LW + wave) * 1024);
    }
  }
}

// Operands of K-columns 32 ks .. + 32 of a stage.  Fragment and wave offsets are multiples of 32
// rows, so the swizzle depends on the lane's row within 32 only.
template <int FM, int FN>
__device__ __forceinline__ void i8_read(const uint8_t* stage, int ks, int ra, int rb, int h, i32x4_t (&a)[FM],
                                        i32x4_t (&b)[FN]) {
  const int c = 16 * ((2 * ks + h) ^ i8_swizzle(ra));
#pragma unroll
  for (int j = 0; j < FN; ++j) b[j] = *reinterpret_cast<const i32x4_t*>(stage + (rb + j * 32) * 128 + c);
#pragma unroll
  for (int i = 0; i < FM; ++i) a[i] = *reinterpret_cast<const i32x4_t*>(stage + (ra + i * 32) * 128 + c);
}

template <int FM, int FN>
__device__ __forceinline__ void i8_mma(i32x16_t (&acc)[FM][FN], const i32x4_t (&a)[FM], const i32x4_t (&b)[FN]) {
#pragma unroll
  for (int i = 0; i < FM; ++i)
#pragma unroll
    for (int j = 0; j < FN; ++j) acc[i][j] = __builtin_amdgcn_mfma_i32_32x32x32_i8(b[j], a[i], acc[i][j], 0, 0, 0);
}

// The same for Q quarters of a K-step from `ks` on, in windows cur and nxt where the lane's rows start sa
// and sb chunks into a line.
template <int Q, int FM, int FN>
struct I8Ops {
  i32x4_t a[Q][FM], b[Q][FN];
};

template <bool SHIFT, int Q, int FM, int FN>
__device__ __forceinline__ void i8_read(const uint8_t* cur, const uint8_t* nxt, int ks, int ra, int rb, int h, int sa,
                                        int sb, I8Ops<Q, FM, FN>& o) {
#pragma unroll
  for (int q = 0; q < Q; ++q) {
    if constexpr (!SHIFT) {
      i8_read<FM, FN>(cur, ks + q, ra, rb, h, o.a[q], o.b[q]);
    } else {
      const int pa = 2 * (ks + q) + h + sa, pb = 2 * (ks + q) + h + sb;
      const uint8_t* wa = (pa & 8 ? nxt : cur) + 16 * ((pa & 7) ^ i8_swizzle(ra));
      const uint8_t* wb = (pb & 8 ? nxt : cur) + 16 * ((pb & 7) ^ i8_swizzle(rb));
#pragma unroll
      for (int j = 0; j < FN; ++j) o.b[q][j] = *reinterpret_cast<const i32x4_t*>(wb + (rb + j * 32) * 128);
#pragma unroll
      for (int i = 0; i < FM; ++i) o.a[q][i] = *reinterpret_cast<const i32x4_t*>(wa + (ra + i * 32) * 128);
    }
  }
}

// Order of a quarter K-step: its matrix instructions with the next quarter's LDS reads between them, and
// the quarter's LOADS direct loads between its last ones (a wave that waits to issue a load issues no
// matrix instruction either: a quarter of a K-step's loads right after the barrier and the rest in
// the next quarter measured 118 us at 2560 x 2560 x 12288, all of them after the barrier 136, all in
// the next quarter 125; 4096 x 13824 x 5120: 301, 311 and 312).
template <int FM, int FN, int LOADS>
__device__ __forceinline__ void i8_interleave() {
#pragma unroll
  for (int g = 0; g < FM * FN; ++g) {
    __builtin_amdgcn_sched_group_barrier(0x100, 1, 0);  // LDS read
    __builtin_amdgcn_sched_group_barrier(0x008, 1, 0);  // MFMA
    if (g >= FM * FN - LOADS) __builtin_amdgcn_sched_group_barrier(0x020, 1, 0);  // direct load
  }
  __builtin_amdgcn_sched_barrier(0);
}

// The same for Q quarters without loads.
template <int Q, int FM, int FN>
__device__ __forceinline__ void i8_interleave_q() {
  constexpr int MF = Q * FM * FN;
#pragma unroll
  for (int g = 0; g < MF; ++g) {
    __builtin_amdgcn_sched_group_barrier(0x100, (Q * (FM + FN) + MF - 1) / MF, 0);  // LDS reads
    __builtin_amdgcn_sched_group_barrier(0x008, 1, 0);                              // MFMA
  }
  __builtin_amdgcn_sched_barrier(0);
}

// 16 bytes at the alignment of an element.
typedef u32x4_t u32x4_a2 __attribute__((aligned(2)));
typedef u32x4_t u32x4_a4 __attribute__((aligned(4)));

// A wave's epilogue region (32 rows of FN * 32 elements of ES bytes; 16-byte chunk ch of row r at
// (ch + r / 2) % CPR) to y rows m0 .., columns n0 ..: 16 bytes per lane, at any element (the hardware takes them;
// the aligned dwords of each row, with single elements at its ends, took 2893 x 8595 x 272 51 us, this way 27, and
// 2893 x 8600 x 272 26; 301 x 4099 x 1552 10.9 and 9.5; eight single elements per lane are slower still).
template <int FN, int ES>
__device__ __forceinline__ void store_region(const uint8_t* reg, int lane, uint8_t* y, int64_t ldy, int m0, int n0,
                                             int M, int N) {
  constexpr int RSB = FN * 32 * ES, CPR = RSB / 16;
  auto at = [&](int r, int byte) { return reg + r * RSB + 16 * ((byte / 16 + (r >> 1)) % CPR) + byte % 16; };
#pragma unroll
  for (int it = 0; it < CPR / 2; ++it) {
    const int c = it * 64 + lane, r = c / CPR, b = 16 * (c % CPR);
    const int m = m0 + r, n = n0 + b / ES;
    if (m >= M || n >= N) continue;
    const u32x4_t v = *reinterpret_cast<const u32x4_t*>(at(r, b));
    uint8_t* dst = y + ((size_t)m * ldy + n) * ES;
    if (n + 16 / ES <= N) {
      if constexpr (ES == 4) *reinterpret_cast<u32x4_a4*>(dst) = v;
      else *reinterpret_cast<u32x4_a2*>(dst) = v;
    } else {
#pragma unroll
      for (int e = 0; e < 16 / ES; ++e)
        if (n + e < N) {
          if constexpr (ES == 4) reinterpret_cast<uint32_t*>(dst)[e] = v[e];
          else reinterpret_cast<uint16_t*>(dst)[e] = (uint16_t)(v[e >> 1] >> (16 * (e & 1)));
        }
    }
  }
}

template <int WAVES_M, int WAVES_N, int FM, int FN, int S, int KG, int NL, bool SHIFT, int YT>
__global__ __launch_bounds__(64 * (WAVES_M * WAVES_N * KG + NL)) void gemm_i8_kernel(
    const uint8_t* __restrict__ qa, const float* __restrict__ sa, const uint8_t* __restrict__ qw,
    const float* __restrict__ sw, const uint16_t* __restrict__ bias, int M, int N, int K, void* __restrict__ y,
    int64_t ldy) {
  using T = TileI8<WAVES_M, WAVES_N, FM, FN, S, KG, NL, SHIFT>;
  __shared__ __attribute__((aligned(16))) uint8_t lds[T::LDS];
  const int t = threadIdx.x, lane = t & 63;
  const int w = __builtin_amdgcn_readfirstlane(t >> 6);
  const bool loader = NL > 0 && w >= T::WAVES * KG;
  const int wl = loader ? w - T::WAVES * KG : w, per = loader ? T::LW : T::WAVES;  // waves of a group
  const int kg = KG > 1 ? wl / per : 0, wave = KG > 1 ? wl % per : wl;
  const int wm = wave / WAVES_N, wn = wave % WAVES_N;
  const int l32 = lane & 31, h = lane >> 5;
  int tm, tn;
  tile_of((int)blockIdx.x, (int)gridDim.x, (M + T::BM - 1) / T::BM, (N + T::BN - 1) / T::BN, tm, tn);
  const int m0 = tm * T::BM, n0 = tn * T::BN;
  const int nkt = (K + T::STEP - 1) / T::STEP;
  const uint8_t* abase = qa + (size_t)m0 * K;
  const uint8_t* bbase = qw + (size_t)n0 * K;
  const int rows_a = min(T::BM, M - m0), rows_b = min(T::BN, N - n0);

  // how far into a 128-byte line a row starts, in 16-byte chunks
  auto shift_of = [&](const uint8_t* base, int row) {
    return SHIFT ? (int)((reinterpret_cast<uintptr_t>(base) >> 4) + (uint32_t)row * ((uint32_t)K >> 4)) & 7 : 0;
  };
  // byte offset in the operand and K-column of this lane's chunk in every round
  uint32_t off[T::ROUNDS], col[T::ROUNDS];
#pragma unroll
  for (int r = 0; r < T::ROUNDS; ++r) {
    const int row = (r * T::LW + wave) * 8 + (lane >> 3);
    const int src = row < T::BM ? min(row, rows_a - 1) : min(row - T::BM, rows_b - 1);
    col[r] = 16u * (uint32_t)(((lane & 7) ^ i8_swizzle(row)) - shift_of(row < T::BM ? abase : bbase, src));
    off[r] = (uint32_t)src * (uint32_t)K + col[r] + (SHIFT ? 112u : 0u);
  }
  const int ra = wm * FM * 32 + l32, rb = T::BM + wn * FN * 32 + l32;
  const int sha = shift_of(abase, ra), shb = shift_of(bbase, rb - T::BM);
  // Scales and bias, ahead of the K loop.  With loader waves they are on their way while the first K-steps land
  // (1024 x 4096 x 1024: 12.7 to 12.3 us, 1024 x 2048 x 4096: 16.1 to 15.6); in the tiles without, every wave waits for
  // its bias (widened at once) and then for its row scales before it issues its first direct load.
  static_assert(T::THREADS >= T::BN, "a channel for every thread at most");
  const int mb = m0 + wm * FM * 32, nb = n0 + wn * FN * 32;
  const bool has_bias = bias != nullptr;
  float chan_s = 0.0f, chan_b = 0.0f, row_s[FM];
  if (t < T::BN && n0 + t < N) {
    chan_s = sw[n0 + t];
    if (has_bias) chan_b = bf16_bits_to_f32(bias[n0 + t]);
  }
#pragma unroll
  for (int i = 0; i < FM; ++i) row_s[i] = sa[min(mb + i * 32 + l32, M - 1)];
  i32x16_t acc[FM][FN];
#pragma unroll
  for (int i = 0; i < FM; ++i)
#pragma unroll
    for (int j = 0; j < FN; ++j)
#pragma unroll
      for (int r = 0; r < 16; ++r) acc[i][j][r] = 0;

  // K-steps in the order kt0, kt0 + 1, ..., nkt - 1, 0, ..., kt0 - 1 (integer sums do not depend on it):
  // each XCD starts an eighth of K further on, so the eight of them fetch different columns of the
  // panels that they share from HBM and find the others' in the Infinity Cache.  Past the last K-step
  // the last is loaded again, so that every step waits on the same count.
  // A group whose last K-step does not exist takes columns past K, which are zeros.  With SHIFT the groups
  // take runs of K-steps (each needs its successor's window too), and the cycle is padded with K-steps of
  // zeros, one at least: its windows are the last lines of the rows and then the first.
  const int ni = (nkt + (SHIFT ? 1 : 0) + KG - 1) / KG, cycle = SHIFT ? ni * KG : nkt;
  const int kt0 = (int)(blockIdx.x & 7) * cycle / 8;
  auto k_of = [&](int i) {
    const int p = SHIFT ? kg * ni + min(i, ni) : KG * min(i, ni - 1) + kg;
    const int q = p + kt0 >= cycle ? p + kt0 - cycle : p + kt0;
    return (uint32_t)(SHIFT || KG == 1 || p < nkt ? q : nkt) * T::STEP;
  };
  uint8_t* ring = lds + kg * S * T::STAGE;
  constexpr int R = T::ROUNDS, RA = T::ROUNDS / 4;
  if constexpr (NL > 0) {
    if (loader) {
      __builtin_amdgcn_s_setprio(3);  // (1024 x 8192 x 8192 in 128 x 256 tiles: 67.0 us, 68.7 without)
      constexpr int AHEAD = (SHIFT ? S - 3 : S - 2) * R;  // loads of stages that are not needed yet
#pragma unroll
      for (int j = 0; j < S - 1; ++j)
        i8_issue<T, SHIFT, 0, R>(ring + j * T::STAGE, wave, k_of(j), (uint32_t)K, abase, bbase, off, col);
      vm_wait_barrier<AHEAD>();
      int slot = 0;
      for (int kt = 0; kt < ni; ++kt) {
        // stage kt + S - 1 into the slot of kt - 1, whose operands every wave had read at the last barrier
        i8_issue<T, SHIFT, 0, R>(ring + (slot == 0 ? S - 1 : slot - 1) * T::STAGE, wave, k_of(kt + S - 1), (uint32_t)K,
                                 abase, bbase, off, col);
        vm_wait_barrier<AHEAD>();  // stage kt + 1 (SHIFT: kt + 2) has landed
        slot = slot == S - 1 ? 0 : slot + 1;
      }
    } else {
      // operands are read a quarter of a K-step ahead, or half of one where a quarter is a single matrix
      // instruction (64 x 64 tiles, 128 x 8192 x 4096: 12.3 to 11.0 us; more waves or products per wave do not gain)
      constexpr int Q = FM * FN == 1 ? 2 : 1, P = 4 / Q;
      vm_wait_barrier<0>();
      I8Ops<Q, FM, FN> o[2];
      auto after = [](int slot) { return slot == S - 1 ? 0 : slot + 1; };
      int slot = 0;
      i8_read<SHIFT>(ring, ring + T::STAGE, 0, ra, rb, h, sha, shb, o[0]);
      for (int kt = 0; kt < ni; ++kt) {
#pragma unroll
        for (int p = 0; p < P; ++p) {
          if (p == P - 1) {
            vm_wait_barrier<0>();  // the operands of kt are in registers; the loaders saw the next ones land
            slot = after(slot);
          }
          i8_read<SHIFT>(ring + slot * T::STAGE, ring + after(slot) * T::STAGE, (p + 1) * Q % 4, ra, rb, h, sha, shb,
                         o[(p + 1) & 1]);
#pragma unroll
          for (int q = 0; q < Q; ++q) i8_mma<FM, FN>(acc, o[p & 1].a[q], o[p & 1].b[q]);
          i8_interleave_q<Q, FM, FN>();
        }
      }
    }
  } else {
#pragma unroll
    for (int j = 0; j < S - 1; ++j)
      i8_issue<T, false, 0, R>(ring + j * T::STAGE, wave, k_of(j), (uint32_t)K, abase, bbase, off, col);
    vm_wait_barrier<(S - 2) * R>();
    i32x4_t a0[FM], b0[FN], a1[FM], b1[FN];
    int slot = 0;
    i8_read<FM, FN>(ring, 0, ra, rb, h, a0, b0);
    i8_issue<T, false, 0, RA>(ring + (S - 1) * T::STAGE, wave, k_of(S - 1), (uint32_t)K, abase, bbase, off, col);
    for (int kt = 0; kt < ni; ++kt) {
      uint8_t* cur = ring + slot * T::STAGE;
      // the rest of the loads of K-step kt + S - 1, into the slot of kt - 1
      i8_issue<T, false, RA, R>(ring + (slot == 0 ? S - 1 : slot - 1) * T::STAGE, wave, k_of(kt + S - 1), (uint32_t)K, abase,
                         bbase, off, col);
      i8_read<FM, FN>(cur, 1, ra, rb, h, a1, b1);
      i8_mma<FM, FN>(acc, a0, b0);
      i8_interleave<FM, FN, R - RA>();
      i8_read<FM, FN>(cur, 2, ra, rb, h, a0, b0);
      i8_mma<FM, FN>(acc, a1, b1);
      i8_interleave<FM, FN, 0>();
      i8_read<FM, FN>(cur, 3, ra, rb, h, a1, b1);
      i8_mma<FM, FN>(acc, a0, b0);
      i8_interleave<FM, FN, 0>();
      // K-step kt + 1 has landed and every wave has read the operands of kt: its slot is free
      vm_wait_barrier<(S - 2) * R>();
      i8_issue<T, false, 0, RA>(cur, wave, k_of(kt + S), (uint32_t)K, abase, bbase, off, col);
      slot = slot == S - 1 ? 0 : slot + 1;
      i8_read<FM, FN>(ring + slot * T::STAGE, 0, ra, rb, h, a0, b0);
      i8_mma<FM, FN>(acc, a1, b1);
      i8_interleave<FM, FN, RA>();
    }
  }
  vm_wait_barrier<0>();
  if constexpr (KG > 1) {
    int* part = reinterpret_cast<int*>(lds);
    constexpr int N16 = FM * FN * 16;
#pragma unroll
    for (int i = 0; i < FM; ++i)
#pragma unroll
      for (int j = 0; j < FN; ++j)
#pragma unroll
        for (int r = 0; r < 16; ++r)
          if (kg > 0 && !loader) part[(((kg - 1) * T::WAVES + wave) * N16 + (i * FN + j) * 16 + r) * 64 + lane] = acc[i][j][r];
    __syncthreads();
    if (kg == 0 && !loader)
#pragma unroll
      for (int i = 0; i < FM; ++i)
#pragma unroll
        for (int j = 0; j < FN; ++j)
#pragma unroll
          for (int r = 0; r < 16; ++r)
#pragma unroll
            for (int p = 0; p < KG - 1; ++p)
              acc[i][j][r] += part[((p * T::WAVES + wave) * N16 + (i * FN + j) * 16 + r) * 64 + lane];
    __syncthreads();
  }

  // Epilogue: the channel scales and biases of the tile once in LDS; each wave passes one 32-row
  // fragment row at a time through its own region and stores whole 16-byte runs of y rows.
  float* s_lds = reinterpret_cast<float*>(lds + T::WAVES * T::REGION);
  float* b_lds = s_lds + T::BN;
  if (t < T::BN) {
    s_lds[t] = chan_s;
    b_lds[t] = chan_b;
  }
  __syncthreads();
  if (loader || kg > 0) return;
  constexpr int ES = YType<YT>::ES;
  constexpr int RSB = FN * 32 * ES;   // bytes per region row
  constexpr int CPR = RSB / 16;       // 16-byte chunks per region row
  uint8_t* reg = lds + wave * T::REGION;
#pragma unroll
  for (int i = 0; i < FM; ++i) {
    const float as = row_s[i];
#pragma unroll
    for (int j = 0; j < FN; ++j)
#pragma unroll
      for (int q = 0; q < 4; ++q) {
        const int col = wn * FN * 32 + j * 32 + 8 * q + 4 * h;
        const float4_t s = *reinterpret_cast<const float4_t*>(s_lds + col);
        const float4_t b = *reinterpret_cast<const float4_t*>(b_lds + col);
        float v[4];
#pragma unroll
        for (int e = 0; e < 4; ++e) {
          v[e] = ((float)acc[i][j][4 * q + e] * as) * s[e];
          if (has_bias) v[e] += b[e];
        }
        // chunk ch of row r sits at (ch + r / 2) % CPR
        if constexpr (YT == 2) {
          const int ch = 8 * j + 2 * q + h;
          *reinterpret_cast<float4_t*>(reg + l32 * RSB + 16 * ((ch + (l32 >> 1)) % CPR)) = float4_t{v[0], v[1], v[2], v[3]};
        } else {
          const int ch = 4 * j + q;
          const u32x2_t p = YT == 1 ? u32x2_t{pack_f16x2(v[0], v[1]), pack_f16x2(v[2], v[3])}
                                    : u32x2_t{pack_bf16x2(v[0], v[1]), pack_bf16x2(v[2], v[3])};
          *reinterpret_cast<u32x2_t*>(reg + l32 * RSB + 16 * ((ch + (l32 >> 1)) % CPR) + 8 * h) = p;
        }
      }
    wave_lds_sync();
    store_region<FN, ES>(reg, lane, static_cast<uint8_t*>(y), ldy, mb + i * 32, nb, M, N);
    wave_lds_sync();  // the region is rewritten by the next fragment row
  }
}

// ---- small batches: weight streaming ---------------------------------------------------------------
// A workgroup owns 16 NB weight rows and up to 16 MB activation rows; its KW waves split K: wave w takes
// the 128-column K-steps w, w + KW, ..., each through an LDS ring of its own, S - 1 K-steps ahead by
// direct loads of whole 128-byte lines.  Nothing in the loop is shared, so it has no barrier: a wave
// waits for its own loads only.  v_mfma_i32_16x16x64_i8 (row l % 16, columns 16 (l / 16) ..) keeps the
// activation side at 16 rows; the int32 partial sums of the waves meet in LDS.
template <int MB, int NB, int KW, int S>
struct SkinnyI8 {
  static constexpr int ROWS = 16 * (MB + NB);  // activation rows, then weight rows
  static constexpr int STAGE = ROWS * 128;
  static constexpr int LOADS = ROWS / 8;
  static constexpr int RING = KW * S * STAGE;
  static constexpr int PART = KW * MB * NB * 256 * 4;
  static constexpr int LDS = RING > PART ? RING : PART;
  static_assert(LDS <= 160 * 1024 && LOADS * (S - 1) < 64, "LDS of one CU, vmcnt range");
};

template <class T, int MB>
__device__ __forceinline__ void skinny_issue(uint8_t* stage, uint32_t k0, uint32_t K, const uint8_t* qa,
                                             const uint8_t* wbase, const uint32_t* off, const uint32_t* col) {
  const bool whole = k0 + 128 <= K;
#pragma unroll
  for (int r = 0; r < T::LOADS; ++r) {
    const uint8_t* p = (r < 2 * MB ? qa : wbase) + (k0 + off[r]);
    if (!whole && k0 + col[r] >= K) p = reinterpret_cast<const uint8_t*>(zero_chunk);
    load_lds16(p, stage + r * 1024);
  }
}

template <int MB, int NB>
__device__ __forceinline__ void skinny_mma(i32x4_t (&acc)[MB][NB], const i32x4_t (&a)[2][MB], const i32x4_t (&w)[2][NB]) {
#pragma unroll
  for (int s = 0; s < 2; ++s)
#pragma unroll
    for (int i = 0; i < MB; ++i)
#pragma unroll
      for (int j = 0; j < NB; ++j) acc[i][j] = __builtin_amdgcn_mfma_i32_16x16x64_i8(w[s][j], a[s][i], acc[i][j], 0, 0, 0);
}

template <int MB, int NB, int KW, int S, int YT>
__global__ __launch_bounds__(64 * KW) void gemm_i8_skinny_kernel(
    const uint8_t* __restrict__ qa, const float* __restrict__ sa, const uint8_t* __restrict__ qw,
    const float* __restrict__ sw, const uint16_t* __restrict__ bias, int M, int N, int K, void* __restrict__ y,
    int64_t ldy) {
  using T = SkinnyI8<MB, NB, KW, S>;
  __shared__ __attribute__((aligned(16))) uint8_t lds[T::LDS];
  const int t = threadIdx.x, lane = t & 63;
  const int wave = __builtin_amdgcn_readfirstlane(t >> 6);
  const int l16 = lane & 15, g = lane >> 4;
  const int n0 = blockIdx.x * (16 * NB);
  const uint8_t* wbase = qw + (size_t)n0 * K;
  uint8_t* ring = lds + wave * S * T::STAGE;
  uint32_t off[T::LOADS], col[T::LOADS];
#pragma unroll
  for (int r = 0; r < T::LOADS; ++r) {
    const int row = 8 * r + (lane >> 3);
    col[r] = 16u * (uint32_t)((lane & 7) ^ i8_swizzle(row));
    const int src = row < 16 * MB ? min(row, M - 1) : min(row - 16 * MB, N - 1 - n0);
    off[r] = (uint32_t)src * (uint32_t)K + col[r];
  }
  const int nkt = (K + 127) / 128;
  const int steps = (nkt - wave + KW - 1) / KW;  // of this wave
  i32x4_t acc[MB][NB];
#pragma unroll
  for (int i = 0; i < MB; ++i)
#pragma unroll
    for (int j = 0; j < NB; ++j) acc[i][j] = i32x4_t{0, 0, 0, 0};
  if (steps > 0) {
    auto k_of = [&](int i) { return 128u * (uint32_t)(wave + KW * min(i, steps - 1)); };
#pragma unroll
    for (int i = 0; i < S - 1; ++i)
      skinny_issue<T, MB>(ring + i * T::STAGE, k_of(i), (uint32_t)K, qa, wbase, off, col);
    int slot = 0;
    for (int i = 0; i < steps; ++i) {
      // K-step i has landed; the operands of K-step i - 1 are in registers, so its slot is free
      asm volatile("s_waitcnt vmcnt(%0) lgkmcnt(0)" ::"n"((S - 2) * T::LOADS) : "memory");
      skinny_issue<T, MB>(ring + (slot == 0 ? S - 1 : slot - 1) * T::STAGE, k_of(i + S - 1), (uint32_t)K, qa, wbase, off,
                          col);
      const uint8_t* cur = ring + slot * T::STAGE;
      i32x4_t a[2][MB], w[2][NB];
#pragma unroll
      for (int s = 0; s < 2; ++s) {
        const int c = 16 * ((4 * s + g) ^ i8_swizzle(l16));
#pragma unroll
        for (int j = 0; j < NB; ++j) w[s][j] = *reinterpret_cast<const i32x4_t*>(cur + (16 * MB + 16 * j + l16) * 128 + c);
#pragma unroll
        for (int m = 0; m < MB; ++m) a[s][m] = *reinterpret_cast<const i32x4_t*>(cur + (16 * m + l16) * 128 + c);
      }
      skinny_mma<MB, NB>(acc, a, w);
      slot = slot == S - 1 ? 0 : slot + 1;
    }
  }
  asm volatile("s_waitcnt vmcnt(0) lgkmcnt(0)" ::: "memory");
  __syncthreads();  // every wave has left its ring
  // acc[i][j][r] is the partial sum of m = 16 i + l16, n = n0 + 16 j + 4 g + r
  int* part = reinterpret_cast<int*>(lds);
#pragma unroll
  for (int i = 0; i < MB; ++i)
#pragma unroll
    for (int j = 0; j < NB; ++j)
      *reinterpret_cast<i32x4_t*>(part + ((wave * MB * 16 + 16 * i + l16) * 16 * NB + 16 * j + 4 * g)) = acc[i][j];
  __syncthreads();
  for (int o = t; o < MB * NB * 256; o += 64 * KW) {
    const int m = o / (16 * NB), n = n0 + o % (16 * NB);
    if (m >= M || n >= N) continue;
    int sum = 0;
#pragma unroll
    for (int w = 0; w < KW; ++w) sum += part[w * MB * NB * 256 + o];
    float v = ((float)sum * sa[m]) * sw[n];
    if (bias != nullptr) v += bf16_bits_to_f32(bias[n]);
    store_one<YT>(y, (size_t)m * ldy + n, v);
  }
}

// ---- up to four tokens: quantizer and weight streaming in one launch ---------------------------------
// Each workgroup (KW waves, 16 NB channels) starts its weight rings, quantizes the tokens itself (they are in L2)
// into codes in LDS, and goes on as the streaming kernel above with the activation operand read from there.  Every
// workgroup repeats the quantizer's work; what is saved is a launch and the wait between the two (1 x 6144 x 2048:
// 7.3 to 5.3 us, 4 x 4096 x 4096: 8.4 to 7.5, 4 x 13824 x 5120: 15.9 to 15.3), and 3 us of the host's time.  Loads
// complete in order and x is asked for after the rings' first two K-steps, the smoothing factors after x, so the
// quantizer starts when those K-steps have landed: they cover the way of x, but not the quantizer's arithmetic,
// during which no load is in flight.  The codes are those of the quantizer kernel bit for bit.
constexpr int TK_S = 3;

struct TokenArgs {
  const void* x;
  const uint16_t* lam;
  int block;
  float norm;
  const uint8_t* qw;
  const float* sw;
  const uint16_t* bias;
  int64_t ldx;
  int N, K, ydtype;
  void* y;
  int64_t ldy;
};

template <int NB>
__device__ __forceinline__ void token_issue(uint8_t* stage, uint32_t k0, uint32_t K, const uint8_t* wbase,
                                            const uint32_t* off, const uint32_t* col) {
#pragma unroll
  for (int r = 0; r < 2 * NB; ++r) {
    const uint8_t* p = wbase + (k0 + off[r]);
    if (k0 + col[r] >= K) p = reinterpret_cast<const uint8_t*>(zero_chunk);
    load_lds16(p, stage + r * 1024);
  }
}

template <int NB>
__device__ __forceinline__ void token_mma(i32x4_t (&acc)[NB], const i32x4_t (&a)[2], const i32x4_t (&w)[2][NB]) {
#pragma unroll
  for (int s = 0; s < 2; ++s)
#pragma unroll
    for (int j = 0; j < NB; ++j) acc[j] = __builtin_amdgcn_mfma_i32_16x16x64_i8(w[s][j], a[s], acc[j], 0, 0, 0);
}

// C: chunks of 8 columns per thread, 512 KW C >= K; MT: tokens.
template <int DT, bool ROT, int C, int NB, int KW, int MT>
__global__ __launch_bounds__(64 * KW) void linear_i8_token_kernel(const TokenArgs p) {
  constexpr int STAGE = 2048 * NB, COLS = 512 * KW;  // bytes of a K-step's weight rows; columns of one chunk each
  extern __shared__ __attribute__((aligned(16))) uint8_t dyn[];
  __shared__ uint32_t red[MT][KW];
  const int t = threadIdx.x, lane = t & 63;
  const int wave = __builtin_amdgcn_readfirstlane(t >> 6);
  const int l16 = lane & 15, g = lane >> 4;
  const int n0 = blockIdx.x * (16 * NB), N = p.N, K = p.K;
  const uint8_t* wbase = p.qw + (size_t)n0 * K;
  uint8_t* ring = dyn + wave * TK_S * STAGE;
  uint8_t* codes = dyn + KW * TK_S * STAGE;
  uint32_t off[2 * NB], col[2 * NB];
#pragma unroll
  for (int r = 0; r < 2 * NB; ++r) {
    const int row = 8 * r + (lane >> 3);
    col[r] = 16u * (uint32_t)((lane & 7) ^ i8_swizzle(row));
    off[r] = (uint32_t)min(row, N - 1 - n0) * (uint32_t)K + col[r];
  }
  const int nkt = (K + 127) / 128, steps = (nkt - wave + KW - 1) / KW;
  auto k_of = [&](int i) { return 128u * (uint32_t)(wave + KW * min(i, steps - 1)); };
  if (steps > 0) {
#pragma unroll
    for (int i = 0; i < TK_S - 1; ++i) token_issue<NB>(ring + i * STAGE, k_of(i), (uint32_t)K, wbase, off, col);
  }

  const int tc = 8 * (ROT ? chunk_of(t) : t);
  const size_t es = DT == 2 ? 4 : 2;
  float v[MT][C][8];
#pragma unroll
  for (int r = 0; r < MT; ++r) {
    const uint8_t* xr = static_cast<const uint8_t*>(p.x) + (size_t)r * p.ldx * es;
#pragma unroll
    for (int c = 0; c < C; ++c) {
      const int k = COLS * c + tc;
      widen8<DT>(k < K ? load_raw<DT>(xr, k) : zero_raw<DT>(), v[r][c]);
    }
  }
  if (p.lam != nullptr) {
#pragma unroll
    for (int c = 0; c < C; ++c) {
      const int k = COLS * c + tc;
      float l[8], rh[8], rl[8];
#pragma unroll
      for (int i = 0; i < 8; ++i) l[i] = 1.0f;
      if (k < K) lambda8(p.lam, k, l);
      if (__all(reciprocals8(l, rh, rl))) {
#pragma unroll
        for (int r = 0; r < MT; ++r)
#pragma unroll
          for (int i = 0; i < 8; ++i) v[r][c][i] = fmaf(v[r][c][i], rh[i], v[r][c][i] * rl[i]);
      } else {
#pragma unroll
        for (int r = 0; r < MT; ++r)
#pragma unroll
          for (int i = 0; i < 8; ++i) v[r][c][i] = v[r][c][i] / l[i];
      }
    }
  }
  const int kp = (K + 127) / 128 * 128 + 16;  // bytes of a token's codes
#pragma unroll
  for (int r = 0; r < MT; ++r) {
    if (ROT) rotate<C>(v[r], p.block, lane);
    const uint32_t mx = chunk_max<C>(v[r]), mw = wave_max2(mx, mx);
    if (lane == 0) red[r][wave] = mw;
  }
  // (LDS only: every load so far had landed before the values were there)
  asm volatile("s_waitcnt lgkmcnt(0)\n\ts_barrier" ::: "memory");
  const float sign = ROT ? lane_sign(lane, p.block) : 1.0f;
#pragma unroll
  for (int r = 0; r < MT; ++r) {
    uint32_t bits = 0;
#pragma unroll
    for (int w = 0; w < KW; ++w) bits = max(bits, red[r][w]);
    const float inv = row_inv(bits, p.norm) * sign;
#pragma unroll
    for (int c = 0; c < C; ++c) {
      const int k = COLS * c + tc;
      if (k < K) *reinterpret_cast<u32x2_t*>(codes + r * kp + k) = codes8(v[r][c], inv);
    }
  }
  asm volatile("s_waitcnt lgkmcnt(0)\n\ts_barrier" ::: "memory");

  // the activation rows past the tokens repeat the last one and are not stored; columns past K, up to the
  // K-step's end, meet zero weights
  const uint8_t* arow = codes + min(l16, MT - 1) * kp + 16 * g;
  i32x4_t acc[NB];
#pragma unroll
  for (int j = 0; j < NB; ++j) acc[j] = i32x4_t{0, 0, 0, 0};
  if (steps > 0) {
    int slot = 0;
    for (int i = 0; i < steps; ++i) {
      asm volatile("s_waitcnt vmcnt(%0) lgkmcnt(0)" ::"n"((TK_S - 2) * 2 * NB) : "memory");
      token_issue<NB>(ring + (slot == 0 ? TK_S - 1 : slot - 1) * STAGE, k_of(i + TK_S - 1), (uint32_t)K, wbase, off, col);
      const uint8_t* cur = ring + slot * STAGE;
      const uint8_t* ac = arow + k_of(i);
      i32x4_t a[2], w[2][NB];
#pragma unroll
      for (int s = 0; s < 2; ++s) {
        const int c = 16 * ((4 * s + g) ^ i8_swizzle(l16));
        a[s] = *reinterpret_cast<const i32x4_t*>(ac + 64 * s);
#pragma unroll
        for (int j = 0; j < NB; ++j) w[s][j] = *reinterpret_cast<const i32x4_t*>(cur + (16 * j + l16) * 128 + c);
      }
      token_mma<NB>(acc, a, w);
      slot = slot == TK_S - 1 ? 0 : slot + 1;
    }
  }
  asm volatile("s_waitcnt vmcnt(0) lgkmcnt(0)" ::: "memory");
  __syncthreads();  // every wave has left its ring
  int* part = reinterpret_cast<int*>(dyn);
#pragma unroll
  for (int j = 0; j < NB; ++j)
    if (l16 < MT) *reinterpret_cast<i32x4_t*>(part + (wave * MT + l16) * 16 * NB + 16 * j + 4 * g) = acc[j];
  __syncthreads();
  const int r = t / (16 * NB), n = n0 + t % (16 * NB);
  if (r < MT && n < N) {
    int sum = 0;
    uint32_t bits = 0;
#pragma unroll
    for (int w = 0; w < KW; ++w) {
      sum += part[(w * MT + r) * 16 * NB + t % (16 * NB)];
      bits = max(bits, red[r][w]);
    }
    float f = ((float)sum * row_scale(bits, p.norm)) * p.sw[n];
    if (p.bias != nullptr) f += bf16_bits_to_f32(p.bias[n]);
    const size_t at = (size_t)r * p.ldy + n;
    if (p.ydtype == 2) store_one<2>(p.y, at, f);
    else if (p.ydtype == 1) store_one<1>(p.y, at, f);
    else store_one<0>(p.y, at, f);
  }
}

template <int DT, bool ROT, int C, int NB, int KW, int MT>
hipError_t run_token_c(const TokenArgs& a, hipStream_t stream) {
  static_assert(MT * 16 * NB <= 64 * KW, "a thread for every output");
  const size_t lds = KW * TK_S * 2048 * NB + MT * ((size_t)(a.K + 127) / 128 * 128 + 16);
  linear_i8_token_kernel<DT, ROT, C, NB, KW, MT><<<dim3((unsigned)((a.N + 16 * NB - 1) / (16 * NB))), 64 * KW, lds, stream>>>(a);
  return hipGetLastError();
}

template <int DT, bool ROT, int MT>
hipError_t run_token(const TokenArgs& a, hipStream_t stream) {
  // (the split of the streaming kernel: see run)
  if (a.N <= 4096) return a.K <= 4096 ? run_token_c<DT, ROT, 1, 1, 8, MT>(a, stream) : run_token_c<DT, ROT, 2, 1, 8, MT>(a, stream);
  return a.K <= 4096 ? run_token_c<DT, ROT, 2, 2, 4, MT>(a, stream) : run_token_c<DT, ROT, 3, 2, 4, MT>(a, stream);
}

struct GArgs {
  const uint8_t* qa;
  const float* sa;
  const uint8_t* qw;
  const float* sw;
  const uint16_t* bias;
  int M, N, K;
  void* y;
  int64_t ldy;
  hipStream_t stream;
};

template <int WAVES_M, int WAVES_N, int FM, int FN, int S, int KG, int NL, bool SHIFT, int YT>
hipError_t run_tile(const GArgs& a) {
  using T = TileI8<WAVES_M, WAVES_N, FM, FN, S, KG, NL, SHIFT>;
  const int64_t tiles = (int64_t)((a.M + T::BM - 1) / T::BM) * ((a.N + T::BN - 1) / T::BN);
  if (tiles * T::THREADS >= (int64_t)1 << 32) return hipErrorInvalidConfiguration;
  gemm_i8_kernel<WAVES_M, WAVES_N, FM, FN, S, KG, NL, SHIFT, YT><<<dim3((unsigned)tiles), T::THREADS, 0, a.stream>>>(
      a.qa, a.sa, a.qw, a.sw, a.bias, a.M, a.N, a.K, a.y, a.ldy);
  return hipGetLastError();
}

// S stages where rows are whole 128-byte lines, S2 where they are not.
template <int WAVES_M, int WAVES_N, int FM, int FN, int S, int S2, int KG, int YT>
hipError_t run_lines(const GArgs& a, bool lines) {
  return lines ? run_tile<WAVES_M, WAVES_N, FM, FN, S, KG, 4, false, YT>(a)
               : run_tile<WAVES_M, WAVES_N, FM, FN, S2, KG, 4, true, YT>(a);
}

template <int MB, int NB, int KW, int S, int YT>
hipError_t run_skinny(const GArgs& a) {
  gemm_i8_skinny_kernel<MB, NB, KW, S, YT><<<dim3((unsigned)((a.N + 16 * NB - 1) / (16 * NB))), 64 * KW, 0, a.stream>>>(
      a.qa, a.sa, a.qw, a.sw, a.bias, a.M, a.N, a.K, a.y, a.ldy);
  return hipGetLastError();
}

template <int YT>
hipError_t run(const GArgs& a) {
  const char* forced = test_hook("W8A8_GEMM_TILE");
  auto is = [&](const char* s) { return forced && !strcmp(forced, s); };
  auto tiles = [&](int64_t bm, int64_t bn) { return (a.M + bm - 1) / bm * ((a.N + bn - 1) / bn); };
  // Up to 32 rows and 4096 channels: stream the weights, 16 channels and 8 waves per workgroup (16 x 1024 x 8192:
  // 5.9 us, 32 x 32 tiles 7.4; 2 x 4096 x 12288: 10.0 and 12.1).  Up to 8192 channels, 32 and 4 waves, as long as the
  // weights are short (25 MB: 16 x 6144 x 2048 5.3 and 6.2, 16 x 6144 x 4096 equal, 16 x 6144 x 8192 13.8 and 11.0);
  // past them the tiles below (16 x 28672 x 4096: 28.7 and 24.1; 16 x 13824 x 1040: 6.6 and 7.0).
  const bool stream = a.M <= 32 && (a.N <= 4096 || (a.N <= 8192 && (int64_t)a.N * a.K <= 25000000));
  if (forced ? is("skinny") && a.M <= 32 : stream) {
    if (a.N <= 4096) return a.M <= 16 ? run_skinny<1, 1, 8, 3, YT>(a) : run_skinny<2, 1, 8, 3, YT>(a);
    return a.M <= 16 ? run_skinny<1, 2, 4, 3, YT>(a) : run_skinny<2, 2, 4, 3, YT>(a);
  }
  // At most one tile per CU: the K loop's latency bounds the launch, and the smallest tile that still leaves
  // every CU at most one wins (128 x 2048 x 2048: 32 x 32 tiles 5.3 us, 64 x 32 6.0, 64 x 64 7.4; 128 x 4096 x
  // 4096: 64 x 32 9.1, 32 x 32 12.9; 128 x 8192 x 4096: 64 x 64 12.3, 64 x 128 13.3, 128 x 128 17.1).  The two
  // smallest, whose waves are few, split K over groups of them.
  const bool lines = ((reinterpret_cast<uintptr_t>(a.qa) | reinterpret_cast<uintptr_t>(a.qw) | (uintptr_t)a.K) & 127) == 0;
  if (forced ? is("32") : tiles(32, 32) <= 256) return run_lines<1, 1, 1, 1, 3, 4, 4, YT>(a, lines);
  if (forced ? is("64x32") : tiles(64, 32) <= 256) return run_lines<2, 1, 1, 1, 4, 5, 2, YT>(a, lines);
  if (forced ? is("64") : tiles(64, 64) <= 256) return run_lines<2, 2, 1, 1, 4, 5, 1, YT>(a, lines);
  // (four stages from about K = 2048: 256 x 5120 x 5120 16.9 us, 17.8 with three; 301 x 4099 x 1552 11.6 and 11.2)
  if (forced ? is("64x128s4") : tiles(64, 128) <= 256 && a.K >= 2048) return run_lines<2, 4, 1, 1, 4, 5, 1, YT>(a, lines);
  if (forced ? is("64x128") : tiles(64, 128) <= 256) return run_lines<2, 4, 1, 1, 3, 4, 1, YT>(a, lines);
  // Otherwise, in rounds of 256 tiles, the shape with the least time: rounds by the times (10 ns) of a round's
  // first loads and stores and of its 128-column K-steps, fitted to measured products of whole 128 columns.  A last round
  // that is mostly empty then costs little (4096 x 2560 x 12288: 137 us in 224 tiles of 256 x 192, 144 in 160 of 256 x 256;
  // 300 x 13824 x 5120: 33 in 216 of 128 x 192, 36 in 162 of 128 x 256; 1021 x 2050 x 4096: 19 in 136 of 128 x 128, 29 in 88 of
  // 128 x 192).  Over 300 drawn shapes with such K the rule is 0.1 % behind the best of the five on average and 8 % at
  // most, over 300 with any K 0.35 % and 11 % (297 x 11451 x 192: 9.8 us in 128 x 192 tiles, 8.8 in 128 x 256).
  struct { const char* name; int64_t bm, bn, round, step; } const shapes[] = {{"128", 128, 128, 400, 50},
                                                                              {"128x192", 128, 192, 520, 69},
                                                                              {"128x256", 128, 256, 530, 86},
                                                                              {"256x192", 256, 192, 690, 122},
                                                                              {"256", 256, 256, 790, 133}};
  int best = 0;
  int64_t least = 0;
  for (int i = 0; i < 5; ++i) {
    const int64_t cost = (tiles(shapes[i].bm, shapes[i].bn) + 255) / 256 * (shapes[i].round + (a.K + 127) / 128 * shapes[i].step);
    if (forced ? is(shapes[i].name) : i == 0 || cost < least) {
      best = i;
      least = cost;
    }
  }
  switch (best) {
    case 0: return run_lines<2, 4, 2, 1, 3, 4, 1, YT>(a, lines);  // (a fourth stage for whole lines: 0 to 4 % slower)
    case 1: return run_lines<2, 3, 2, 2, 3, 4, 1, YT>(a, lines);
    case 2: return run_tile<2, 4, 2, 2, 3, 1, 4, false, YT>(a);
    case 3: return run_tile<4, 2, 2, 3, 2, 1, 0, false, YT>(a);
    default: return run_tile<2, 4, 4, 2, 2, 1, 0, false, YT>(a);
  }
}

}  // namespace

hipError_t launch_gemm_i8(const void* qact, const float* ascales, const void* qweight, const float* wscales,
                          const void* bias, int64_t M, int64_t N, int64_t K, void* y, int64_t ldy, int ydtype,
                          hipStream_t stream) {
  const GArgs a{static_cast<const uint8_t*>(qact), ascales, static_cast<const uint8_t*>(qweight), wscales,
                static_cast<const uint16_t*>(bias), (int)M, (int)N, (int)K, y, ldy, stream};
  switch (ydtype) {
    case 0: return run<0>(a);
    case 1: return run<1>(a);
    default: return run<2>(a);
  }
}

bool linear_i8_one_launch(int64_t M, int64_t N, int64_t K) {
  const char* forced = test_hook("W8A8_ONE_LAUNCH");  // "0" keeps the two launches
  // (with 32 channels per workgroup long rows cost more than the launch: 4 x 6144 x 5120 10.1 us in one launch and 11.3 in
  // two, x 8192 15.8 and 13.7; the number of channels does not matter: 1 x 128256 x 2048 46.7 and 55.9)
  const bool small = K <= (N <= 4096 ? 8192 : 6144);
  return M <= 4 && small && !(forced && forced[0] == '0');
}

template <int MT>
hipError_t run_token_m(const TokenArgs& a, int xdtype, hipStream_t stream) {
  switch (xdtype) {
    case 0: return a.block ? run_token<0, true, MT>(a, stream) : run_token<0, false, MT>(a, stream);
    case 1: return a.block ? run_token<1, true, MT>(a, stream) : run_token<1, false, MT>(a, stream);
    default: return a.block ? run_token<2, true, MT>(a, stream) : run_token<2, false, MT>(a, stream);
  }
}

hipError_t launch_linear_i8_token(const void* x, int64_t ldx, int xdtype, const void* lam, int block, float norm,
                                  const void* qweight, const float* wscales, const void* bias, int64_t M, int64_t N,
                                  int64_t K, void* y, int64_t ldy, int ydtype, hipStream_t stream) {
  const TokenArgs a{x, static_cast<const uint16_t*>(lam), block, norm, static_cast<const uint8_t*>(qweight), wscales,
                    static_cast<const uint16_t*>(bias), ldx, (int)N, (int)K, ydtype, y, ldy};
  switch (M) {
    case 1: return run_token_m<1>(a, xdtype, stream);
    case 2: return run_token_m<2>(a, xdtype, stream);
    case 3: return run_token_m<3>(a, xdtype, stream);
    default: return run_token_m<4>(a, xdtype, stream);
  }
}

}  // namespace w4a4
