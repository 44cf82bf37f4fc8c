// Attention of many query rows per sequence over a paged cache (gfx950): prompts, pieces of prompts, large trees.
//
// Bound: the matrix cores.  A workgroup of WAVES waves owns a tile of WAVES NQ 32 rows of one (sequence, key / value
// head) pair and walks its keys in blocks of 64, which all waves share in LDS (direct loads, S stages, one barrier
// per block).  Each wave keeps its rows' queries, maxima, sums and outputs in registers.  With few tiles, each tile's
// blocks are cut into `pieces` equal runs, one per workgroup, whose results a second kernel joins.
//
// v_mfma_f32_32x32x16: lane l holds row l % 32 of 32, keys 8 (i / 4) + 4 (l / 32) + i % 4 of 32.
#include "attention.h"

namespace w4a4 {

namespace {

constexpr int BN = 64;  // keys of a block

template <int DP, int NQ, int WAVES, int S>
struct Tile {
  static constexpr int BM = 32 * NQ * WAVES;
  static constexpr int ROW = 2 * DP, CPR = DP / 8;  // bytes and 16-byte chunks of an LDS row
  static constexpr int RPI = 64 / CPR;              // rows of a direct load
  static constexpr int RW = BN / WAVES;             // rows of a block that one wave loads
  static constexpr int NI = RW / RPI;               // its direct loads of K, or of V
  static constexpr int HALF = BN * ROW, STAGE = 2 * HALF;
  // stages; per wave the places of its rows and four blocks' pages
  static constexpr int OWN = RW * (int)sizeof(AttnPlace) + 4 * 256;
  static constexpr int LDS = S * STAGE + WAVES * OWN;
  static_assert(LDS <= 160 * 1024, "LDS of one CU");
  static_assert(S <= 3, "four blocks' pages");
};

// V's chunks are placed for the transposing reads, which take 64 bytes of 8 rows at once: 4 rows in a row
// lie in 4 different quarters of the banks.
template <int DP>
__device__ __forceinline__ int swizzle_v(int row) {
  return DP == 64 ? (row & 2) << 1 : (row & 3) << 2;
}

// Tile slots.  Sequence s's tiles are slots first(s), first(s) + 1, ..., with first(s) = token0(s) group / BM + s:
// they are at least as many as its tiles (a slot of no tile has a number below 0 or past its sequence's rows).
struct TileOf {
  int seq, tile;
};
template <int BM>
__device__ __forceinline__ TileOf tile_at(const AttnArgs& a, int slot) {
  if (a.starts == nullptr) {  // (fewer slots than that; the last ones are past the batch)
    const int per = (int)(((int64_t)a.each * a.group + BM - 1) / BM);
    const int s = slot / per;
    return {min(s, a.batch - 1), s < a.batch ? slot - s * per : -1};
  }
  auto first = [&](int s) { return min(max(a.starts[s], 0), a.tokens) * a.group / BM + s; };
  int lo = 0, hi = a.batch;  // first(lo) <= slot < first(hi)
  while (hi - lo > 1) {
    const int mid = (lo + hi) >> 1;
    if (first(mid) <= slot) lo = mid;
    else hi = mid;
  }
  return {lo, slot - first(lo)};
}

template <int DP, bool EXACT, int NQ, int WAVES, int S, class T>
__global__ __launch_bounds__(64 * WAVES) void attn_tile_kernel(const AttnArgs a, const int slots) {
  using L = Tile<DP, NQ, WAVES, S>;
  constexpr int BM = L::BM, KS = DP / 16, ND = DP / 32;
  extern __shared__ __attribute__((aligned(16))) uint8_t lds[];
  const int lane = threadIdx.x & 63, l32 = lane & 31, h = lane >> 5;
  const int wave = uniform((int)threadIdx.x >> 6);
  // heads in turn (workgroups go round the XCDs, whose L2 keeps a head's keys), the last tiles of a sequence,
  // which have the most keys, first
  const int id = blockIdx.x;
  const int head = id % a.kv_heads, rest = id / a.kv_heads, piece = rest % a.pieces, slot = slots - 1 - rest / a.pieces;
  const TileOf at = tile_at<BM>(a, slot);
  const AttnSeq sq = attn_seq(a, at.seq);
  const int rows = sq.nq * a.group, row0 = at.tile * BM;
  if (at.tile < 0 || row0 >= rows || rows <= a.rows_from || rows > a.rows_to) return;
  const int i0 = attn_query(a, row0), i1 = attn_query(a, min(row0 + BM, rows) - 1);
  const AttnSpan sp = attn_span<BN>(a, sq, i0, a.mask != nullptr ? sq.len : min(sq.len, sq.ctx + i1 + 1));
  const int b0 = (int)((int64_t)sp.blocks * piece / a.pieces), b1 = (int)((int64_t)sp.blocks * (piece + 1) / a.pieces);
  const int32_t* table = a.table + (int64_t)at.seq * a.table_stride;
  const uint8_t* kh = a.k + 2 * (head * a.k_head);
  const uint8_t* vh = a.v + 2 * (head * a.v_head);
  const int my0 = row0 + wave * 32 * NQ;  // this wave's first row

  AttnRow row[NQ];
  typename T::x8 qf[NQ][KS];
  int low_hi = 0x7FFFFFFF, top_hi = 0, top_lo = 0, low_lo = 0x7FFFFFFF;
#pragma unroll
  for (int n = 0; n < NQ; ++n) {
    const int rr = my0 + n * 32 + l32;
    const bool valid = rr < rows;
    const int i = valid ? attn_query(a, rr) : 0, g = valid ? rr - i * a.group : 0;
    row[n] = attn_row(a, sq, i, valid);
    if (valid) {
      low_hi = min(low_hi, row[n].hi);
      top_hi = max(top_hi, row[n].hi);
      top_lo = max(top_lo, row[n].lo);
      low_lo = min(low_lo, row[n].lo);
    }
    const uint8_t* src = a.q + 2 * ((int64_t)(sq.token0 + i) * a.q_ts + (int64_t)(head * a.group + g) * a.q_hs);
#pragma unroll
    for (int k = 0; k < KS; ++k) {
      const int d = 16 * k + 8 * h;
      u32x4_t x = {0, 0, 0, 0};
      if (valid && d < a.D) x = *reinterpret_cast<const u32x4_t*>(src + 2 * d);
      qf[n][k] = __builtin_bit_cast(typename T::x8, x);
    }
  }
#pragma unroll
  for (int d = 1; d < 32; d <<= 1) {
    low_hi = min(low_hi, __shfl_xor(low_hi, d));
    top_hi = max(top_hi, __shfl_xor(top_hi, d));
    top_lo = max(top_lo, __shfl_xor(top_lo, d));
    low_lo = min(low_lo, __shfl_xor(low_lo, d));
  }
  low_hi = uniform(low_hi);
  top_hi = a.mask != nullptr ? sp.hi : uniform(top_hi);
  top_lo = uniform(top_lo);
  low_lo = uniform(low_lo);
  if (my0 >= rows) top_hi = 0;

  uint8_t* const places = lds + S * L::STAGE + wave * L::OWN;
  uint8_t* const pages = places + L::RW * sizeof(AttnPlace);
  auto key0 = [&](int b) { return (b < sp.sink_blocks ? b : b + sp.skip) * BN; };
  auto seen_by_any = [&](int key) { return key < sp.hi && (key >= sp.lo || key < sp.sinks); };
  // starts the load of the pages of block b's 64 keys (of zeros where there is no such key)
  auto load_pages = [&](int b) {
    const int key = key0(b) + lane;
    const void* src = b < b1 && seen_by_any(key) ? (const void*)(table + attn_page(a, key)) : attn_zeros;
    __builtin_amdgcn_global_load_lds(src, (attn_lds_void*)(pages + (b & 3) * 256), 4, 0, 0);
  };
  // starts this wave's share of block b's loads (of zeros past the run); returns which of the block's keys are there
  auto load_block = [&](int b, int stage) {
    const int key = key0(b) + lane;
    const uint32_t page = *reinterpret_cast<const uint32_t*>(pages + (b & 3) * 256 + 4 * lane);
    const bool ok = b < b1 && seen_by_any(key) && page < a.pages;
    const AttnPlace p = attn_place(a, kh, vh, key, page, ok);
    if (lane / L::RW == wave) *reinterpret_cast<AttnPlace*>(places + (lane % L::RW) * sizeof(AttnPlace)) = p;
    wave_lds_sync();
    uint8_t* to = lds + stage * L::STAGE + wave * L::RW * L::ROW;
#pragma unroll
    for (int n = 0; n < L::NI; ++n) {
      const int r = n * L::RPI + lane / L::CPR, lr = wave * L::RW + r;
      const AttnPlace pl = *reinterpret_cast<const AttnPlace*>(places + r * sizeof(AttnPlace));
      attn_load16(attn_chunk<EXACT>(pl.k, (lane % L::CPR) ^ attn_swizzle<DP>(lr), a.D), to + n * 1024);
      attn_load16(attn_chunk<EXACT>(pl.v, (lane % L::CPR) ^ swizzle_v<DP>(lr), a.D), to + L::HALF + n * 1024);
    }
    return (uint64_t)__ballot(ok);
  };

  float m[NQ], l[NQ];
  float16_t o[NQ][ND];
#pragma unroll
  for (int n = 0; n < NQ; ++n) {
    m[n] = ATTN_NONE;
    l[n] = 0.0f;
#pragma unroll
    for (int d = 0; d < ND; ++d)
#pragma unroll
      for (int i = 0; i < 16; ++i) o[n][d][i] = 0.0f;
  }

  // In the order of their issue: pages b + S - 1, block b + S - 2, pages b + S, block b + S - 1.  A pass waits for all but
  // the blocks after b, so for the pages of block b + S - 1 too.
  for (int j = 0; j < S; ++j) load_pages(b0 + j);
  attn_vm_drain();
  uint64_t there[S];
#pragma unroll
  for (int j = 0; j < S - 1; ++j) there[j] = load_block(b0 + j, j);
  int stage = 0;
#pragma unroll 1
  for (int b = b0; b < b1; ++b) {
    // block b has landed, here and in the other waves, and block b - 1's stage is read
    asm volatile("s_waitcnt vmcnt(%0) lgkmcnt(0)\n\ts_barrier" ::"n"((S - 2) * 2 * L::NI) : "memory");
    load_pages(b + S);
    there[S - 1] = load_block(b + S - 1, stage == 0 ? S - 1 : stage - 1);
    const uint64_t here = there[0];
#pragma unroll
    for (int j = 0; j < S - 1; ++j) there[j] = there[j + 1];
    const uint8_t* ks = lds + stage * L::STAGE;
    const uint8_t* vs = ks + L::HALF;
    stage = stage == S - 1 ? 0 : stage + 1;
    const int j0 = key0(b);
    if (j0 >= top_hi || (j0 + BN <= low_lo && j0 >= a.sinks)) continue;  // no row of this wave sees the block

    float16_t s[NQ][2];
#pragma unroll
    for (int t = 0; t < 2; ++t) {
#pragma unroll
      for (int n = 0; n < NQ; ++n)
#pragma unroll
        for (int i = 0; i < 16; ++i) s[n][t][i] = 0.0f;
#pragma unroll
      for (int k = 0; k < KS; ++k) {
        const int lr = 32 * t + l32;
        const auto kf = __builtin_bit_cast(typename T::x8, *reinterpret_cast<const u32x4_t*>(
            ks + lr * L::ROW + 16 * ((2 * k + h) ^ attn_swizzle<DP>(lr))));
#pragma unroll
        for (int n = 0; n < NQ; ++n) s[n][t] = T::mma32(kf, qf[n][k], s[n][t]);
      }
    }

    if (here != ~0ull || j0 + BN > low_hi || (j0 < top_lo && j0 + BN > a.sinks)) {
      // element (t, i) is key j0 + 4 h + 32 t + 8 (i / 4) + i % 4
#pragma unroll
      for (int n = 0; n < NQ; ++n)
#pragma unroll
        for (int t = 0; t < 2; ++t) {
          const uint32_t mine = (uint32_t)(here >> (32 * t)) >> (4 * h);
          uint32_t bits = 0;
#pragma unroll
          for (int i = 0; i < 16; ++i) {
            const int in = 8 * (i >> 2) + (i & 3), j = j0 + 32 * t + 4 * h + in;
            bits |= (j < row[n].hi && (j >= row[n].lo || j < a.sinks) ? 1u : 0u) << in;
          }
          if (a.mask != nullptr && j0 + 32 * t + 32 > sq.ctx && a.mask_width > 0) {
            const int rr = my0 + n * 32 + l32;
            const uint8_t* of = a.mask + (int64_t)(sq.token0 + (rr < rows ? attn_query(a, rr) : 0)) * a.mask_stride;
            const int node = j0 + 32 * t + 4 * h - sq.ctx;
            uint32_t set[16];
#pragma unroll
            for (int i = 0; i < 16; ++i) set[i] = of[min(max(node + 8 * (i >> 2) + (i & 3), 0), a.mask_width - 1)];
            attn_vm_drain();
            uint32_t tree = 0, nodes = 0;
#pragma unroll
            for (int i = 0; i < 16; ++i) {
              const int in = 8 * (i >> 2) + (i & 3);
              tree |= (set[i] != 0 && node + in < a.mask_width ? 1u : 0u) << in;
              nodes |= (node + in >= 0 ? 1u : 0u) << in;
            }
            bits = (bits & ~nodes) | (tree & nodes);
          }
          bits &= mine;
#pragma unroll
          for (int i = 0; i < 16; ++i)
            if (!((bits >> (8 * (i >> 2) + (i & 3))) & 1)) s[n][t][i] = ATTN_NONE;
        }
    }

    typename T::x8 p[NQ][4];
#pragma unroll
    for (int n = 0; n < NQ; ++n) {
      float top = fmaxf(s[n][0][0], s[n][1][0]);
#pragma unroll
      for (int i = 1; i < 16; ++i) top = fmaxf(fmaxf(top, s[n][0][i]), s[n][1][i]);
      top = attn_max32(top) * a.scale_log2;
      if (__any(top > m[n] + ATTN_SLACK)) {
        const float to = fmaxf(m[n], top), f = attn_exp2(m[n] - (to == ATTN_NONE ? 0.0f : to));
        l[n] *= f;
#pragma unroll
        for (int d = 0; d < ND; ++d) o[n][d] *= f;
        m[n] = to;
      }
      const float ref = m[n] == ATTN_NONE ? 0.0f : m[n];
      float sum = 0.0f;
#pragma unroll
      for (int t = 0; t < 2; ++t)
#pragma unroll
        for (int u = 0; u < 2; ++u) {
          float e[8];
#pragma unroll
          for (int i = 0; i < 8; ++i) e[i] = attn_exp2(fmaf(s[n][t][8 * u + i], a.scale_log2, -ref));
          sum += ((e[0] + e[1]) + (e[2] + e[3])) + ((e[4] + e[5]) + (e[6] + e[7]));
          p[n][2 * t + u] = __builtin_bit_cast(typename T::x8, u32x4_t{T::pack2(e[0], e[1]), T::pack2(e[2], e[3]),
                                                                      T::pack2(e[4], e[5]), T::pack2(e[6], e[7])});
        }
      l[n] += sum;
    }

#pragma unroll
    for (int u = 0; u < 4; ++u)
#pragma unroll
      for (int d = 0; d < ND; ++d) {
        const int c16 = lane & 15;
        const int r0 = 16 * u + 4 * h + (c16 >> 2), r1 = r0 + 8;
        const int ch = 4 * d + 2 * ((lane >> 4) & 1) + ((c16 & 3) >> 1), half = 8 * (c16 & 1);
        const auto vf = attn_read_vt<T>(vs + r0 * L::ROW + 16 * (ch ^ swizzle_v<DP>(r0)) + half,
                                        vs + r1 * L::ROW + 16 * (ch ^ swizzle_v<DP>(r1)) + half);
#pragma unroll
        for (int n = 0; n < NQ; ++n) o[n][d] = T::mma32(vf, p[n][u], o[n][d]);
      }
  }
  attn_vm_drain();  // (nothing arrives in the LDS of an ended wave)

#pragma unroll
  for (int n = 0; n < NQ; ++n) {
    const float sum = attn_sum32(l[n]);
    const int rr = my0 + n * 32 + l32;
    if (rr >= rows) continue;
    if (a.pieces == 1) {
      const float f = sum == 0.0f ? 0.0f : 1.0f / sum;
      const int i = attn_query(a, rr), g = rr - i * a.group;
      uint8_t* dst = a.out + 2 * ((int64_t)(sq.token0 + i) * a.o_ts + (int64_t)(head * a.group + g) * a.o_hs);
#pragma unroll
      for (int d = 0; d < ND; ++d)
#pragma unroll
        for (int q = 0; q < 4; ++q) {
          const int e = 32 * d + 8 * q + 4 * h;
          if (e < a.D)
            *reinterpret_cast<u32x2_t*>(dst + 2 * e) = u32x2_t{T::pack2(o[n][d][4 * q] * f, o[n][d][4 * q + 1] * f),
                                                              T::pack2(o[n][d][4 * q + 2] * f, o[n][d][4 * q + 3] * f)};
        }
    } else {
      const int64_t to = (((int64_t)slot * a.kv_heads + head) * a.pieces + piece) * BM + (rr - row0);
      if (h == 0) *reinterpret_cast<float2_t*>(a.stats + 2 * to) = float2_t{m[n], sum};
#pragma unroll
      for (int d = 0; d < ND; ++d)
#pragma unroll
        for (int q = 0; q < 4; ++q)
          *reinterpret_cast<float4_t*>(a.part + to * DP + 32 * d + 8 * q + 4 * h) =
              float4_t{o[n][d][4 * q], o[n][d][4 * q + 1], o[n][d][4 * q + 2], o[n][d][4 * q + 3]};
    }
  }
}

// Joins the pieces of a tile: a thread takes 4 columns of a row.
template <int DP, int BM, class T>
__global__ __launch_bounds__(256) void attn_tile_join_kernel(const AttnArgs a, const int slots) {
  constexpr int PER = DP / 4;
  const int head = blockIdx.x % a.kv_heads, slot = blockIdx.x / a.kv_heads;
  const TileOf at = tile_at<BM>(a, slot);
  const AttnSeq sq = attn_seq(a, at.seq);
  const int rows = sq.nq * a.group, row0 = at.tile * BM;
  if (at.tile < 0 || row0 >= rows || rows <= a.rows_from || rows > a.rows_to) return;
  const int e = 4 * (threadIdx.x % PER);
  if (e >= a.D) return;
  for (int r = blockIdx.y * (256 / PER) + threadIdx.x / PER; r < min(BM, rows - row0); r += gridDim.y * (256 / PER)) {
    const int64_t first = ((int64_t)slot * a.kv_heads + head) * a.pieces * BM + r;
    float top = ATTN_NONE, sum = 0.0f;
    float4_t o = {0, 0, 0, 0};
    for (int p = 0; p < a.pieces; ++p) top = fmaxf(top, a.stats[2 * (first + (int64_t)p * BM)]);
    const float ref = top == ATTN_NONE ? 0.0f : top;
#pragma unroll 4
    for (int p = 0; p < a.pieces; ++p) {
      const int64_t x = first + (int64_t)p * BM;
      const float2_t st = *reinterpret_cast<const float2_t*>(a.stats + 2 * x);
      const float4_t v = *reinterpret_cast<const float4_t*>(a.part + x * DP + e);
      const float f = attn_exp2(st[0] - ref);
      sum = fmaf(st[1], f, sum);
#pragma unroll
      for (int c = 0; c < 4; ++c) o[c] = fmaf(v[c], f, o[c]);
    }
    const float f = sum == 0.0f ? 0.0f : 1.0f / sum;
    const int rr = row0 + r, i = attn_query(a, rr), g = rr - i * a.group;
    uint8_t* dst = a.out + 2 * ((int64_t)(sq.token0 + i) * a.o_ts + (int64_t)(head * a.group + g) * a.o_hs + e);
    *reinterpret_cast<u32x2_t*>(dst) = u32x2_t{T::pack2(o[0] * f, o[1] * f), T::pack2(o[2] * f, o[3] * f)};
  }
}

#ifndef VQ
#define VQ 1
#define VS 2
#endif
// The tiles of a call: rows of one, how many slots they take (see tile_at; without `starts`, sequence by sequence,
// they take no more), and into how many pieces each tile's keys are cut.
struct TilePlan {
  int rows;
  int64_t slots;
  int pieces;
};
TilePlan plan(const AttnArgs& a) {
  TilePlan p;
  p.rows = a.D <= 64 ? 128 : a.D <= 128 ? 128 * VQ : 128;
  const int64_t rows = (int64_t)a.tokens * a.group;
  p.slots = rows / p.rows + a.batch;
  const int64_t tiles = std::max<int64_t>(1, rows / p.rows) * a.kv_heads;
  p.pieces = (int)std::min<int64_t>(16, std::max<int64_t>(1, 512 / tiles));
  return p;
}

template <int DP, int NQ, int WAVES, int S, class T>
hipError_t run(AttnArgs a, void* workspace, hipStream_t st) {
  using L = Tile<DP, NQ, WAVES, S>;
  const TilePlan p = plan(a);
  if (p.rows != L::BM) return hipErrorInvalidValue;
  const int64_t wgs = p.slots * a.kv_heads * p.pieces;
  if (wgs > 0x7FFFFFFF) return hipErrorInvalidValue;
  a.pieces = p.pieces;
  a.stats = static_cast<float*>(workspace);
  a.part = a.stats + (size_t)wgs * L::BM * 2;
  if (a.D == DP) attn_tile_kernel<DP, true, NQ, WAVES, S, T><<<(unsigned)wgs, 64 * WAVES, L::LDS, st>>>(a, (int)p.slots);
  else attn_tile_kernel<DP, false, NQ, WAVES, S, T><<<(unsigned)wgs, 64 * WAVES, L::LDS, st>>>(a, (int)p.slots);
  hipError_t e = hipGetLastError();
  if (e != hipSuccess || p.pieces == 1) return e;
  attn_tile_join_kernel<DP, L::BM, T><<<dim3((unsigned)(p.slots * a.kv_heads), 8), 256, 0, st>>>(a, (int)p.slots);
  return hipGetLastError();
}

template <class T>
hipError_t run_dim(const AttnArgs& a, void* workspace, hipStream_t st) {
  if (a.D <= 64) return run<64, 1, 4, 2, T>(a, workspace, st);
  if (a.D <= 128) return run<128, VQ, 4, VS, T>(a, workspace, st);
  return run<256, 1, 4, 2, T>(a, workspace, st);
}

}  // namespace

size_t attention_tile_bytes(const AttnArgs& a) {
  const int DP = a.D <= 64 ? 64 : a.D <= 128 ? 128 : 256;
  const TilePlan p = plan(a);
  return p.pieces == 1 ? 0 : (size_t)p.slots * a.kv_heads * p.pieces * p.rows * (2 + DP) * sizeof(float);
}

hipError_t launch_attention_tile(const AttnArgs& a, int dtype, void* workspace, hipStream_t stream) {
  return dtype == 0 ? run_dim<Bf16>(a, workspace, stream) : run_dim<F16>(a, workspace, stream);
}

}  // namespace w4a4
