// Attention of many query rows per sequence over a paged cache (gfx950): prompts, pieces of prompts, large trees.
//
// A workgroup of four waves owns a tile of 128 rows of one (sequence, key / value head) pair and walks its keys in
// blocks of 64, which all waves share in LDS (direct loads, two stages each of keys and values, one barrier per block).
// Each wave keeps its 32 rows' queries, maxima, sums and outputs in registers; the scores of the next block are formed
// between the exponentials of this one and its product with the values.  With few tiles, each tile's blocks are
// cut into equal pieces, one per workgroup, whose results a second kernel joins.
//
// Bound: the SIMDs' time, of which the matrix instructions take one half and the vector instructions (exponentials, maxima,
// sums, addresses) nearly the other.  One prompt of 8192 tokens, 32 heads of 128 over 8: 544 to 603 us, 0.91 to 1.0 PFLOP/s of the
// 1.93 that matrix instructions on random operands reach; matrix cores busy 0.50 of the cycles, vector instructions 0.51, LDS
// reads 0.26 of the LDS's cycles without bank conflicts, waves waiting 0.24 of their time, at 1.8 GHz.  Left out in copies of an
// earlier state, which also lowers the power and so raises the clock: the loads of keys and values 436 us, the LDS reads too 331,
// all but the matrix instructions 275 to 302.  64 rows per wave (half the LDS reads) need more registers than two workgroups of a
// CU have; tiles of eight waves measured 588 against 594; one after the other instead of stepped, 590 against 562.  Heads of
// 64 have half the products for the same exponentials: four prompts of 1000 to 4001 tokens in a window of 1024 take 72 to 86 us,
// matrix cores busy 0.18, vector 0.44, waves waiting 0.28, 1.4 waves of the 2 that fit on a SIMD (three
// workgroups on a CU, with 21 registers spilled: 101 against 91 then).
//
// v_mfma_f32_32x32x16: lane l holds row l % 32 of 32, keys 8 (i / 4) + 4 (l / 32) + i % 4 of 32.
#include "attention.h"

#include <type_traits>

namespace w4a4 {

namespace {

constexpr int BN = 64;  // keys of a block

template <int DP, int WAVES>
struct Tile {
  static constexpr int BM = 32 * WAVES;
  static constexpr int ROW = 2 * DP, CPR = DP / 8;  // bytes and 16-byte chunks of an LDS row
  static constexpr int RPI = 64 / CPR;              // rows of a direct load
  static constexpr int RW = BN / WAVES;             // rows of a block that one wave loads
  static constexpr int NI = RW / RPI;               // its direct loads of K, or of V
  static constexpr int BLOCK = BN * ROW;            // two of K, then two of V
  // per wave the places of its rows' keys, and values (of two blocks), and four blocks' pages
  static constexpr int OWN = 3 * RW * 8 + 4 * 256;
  static constexpr int LDS = 4 * BLOCK + WAVES * OWN;
  static_assert(LDS <= 160 * 1024, "LDS of one CU");
};

// V's chunks are placed for the transposing reads, which take 64 bytes of 8 rows at once: 4 rows in a row
// lie in 4 different quarters of the banks.
template <int DP>
__device__ __forceinline__ int swizzle_v(int row) {
  return DP == 64 ? (row & 2) << 1 : (row & 3) << 2;
}

// f(0), f(1), ..., f(N - 1), each with its number as a constant.
template <int N, int I = 0, class F>
__device__ __forceinline__ void each(F&& f) {
  if constexpr (I < N) {
    f(std::integral_constant<int, I>{});
    each<N, I + 1>(f);
  }
}

// Tile slots.  Sequence s's tiles are slots first(s), first(s) + 1, ..., of which there are at least as many as it has
// tiles (a slot of no tile has a number below 0 or past its sequence's rows).  With x rows before the sequence, first(s) is
//   x / BM + s           for any sequences: R rows take at least R / BM + 1 slots, the whole batch rows / BM + batch;
//   x slot_rate / BM     where those of up to rows_from rows are not the tiles', slot_rate = 1 + BM / rows_from: R > rows_from
//                        rows take at least R / BM + R / rows_from, cut off, so also R / BM + 1; fewer than the others in a batch of
//                        many short sequences among long ones.
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
  auto first = [&](int s) {
    const int x = min(max(a.starts[s], 0), a.tokens) * a.group;
    return a.slot_rate == 0 ? x / BM + s : (int)((int64_t)x * a.slot_rate / BM);
  };
  int lo = 0, hi = a.batch;  // first(lo) <= slot < first(hi)
  while (hi - lo > 1) {
    const int mid = (lo + hi) >> 1;
    if (first(mid) <= slot) lo = mid;
    else hi = mid;
  }
  return {lo, slot - first(lo)};
}

template <int BM>
__device__ __forceinline__ AttnSpan span_of(const AttnArgs& a, const AttnSeq& sq, int row0, int rows) {
  const int i0 = attn_query(a, row0), i1 = attn_query(a, min(row0 + BM, rows) - 1);
  return attn_span<BN>(a, sq, i0, a.mask != nullptr ? sq.len : min(sq.len, sq.ctx + i1 + 1));
}
// Into how many of the at most a.pieces a tile is cut (a.piece_gain: see the launcher).
__device__ __forceinline__ int pieces_of(const AttnArgs& a, const AttnSpan& sp) {
  return max(min(min(a.pieces, sp.blocks / 2), (int)sqrtf((float)sp.blocks * a.piece_gain)), 1);
}

template <int DP, bool EXACT, int WAVES, class T>
__global__ __launch_bounds__(64 * WAVES, DP <= 128 ? 2 : 1) void attn_tile_kernel(const AttnArgs a, const int slots) {
  using L = Tile<DP, WAVES>;
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
  const AttnSpan sp = span_of<BM>(a, sq, row0, rows);
  const int pieces = pieces_of(a, sp);
  if (piece >= pieces) return;
  const int b0 = (int)((int64_t)sp.blocks * piece / pieces), b1 = (int)((int64_t)sp.blocks * (piece + 1) / pieces);
  const int32_t* table = a.table + (int64_t)at.seq * a.table_stride;
  const uint8_t* kh = a.k + 2 * (head * a.k_head);
  const uint8_t* vh = a.v + 2 * (head * a.v_head);

  // this lane's row, its query and head of the group.  (What is used seldom is formed again or lies in LDS: every
  // register of the passes counts, and a spilled one would be waited for together with all loads.)
  auto row_of = [&]() {
    int l = l32;
    asm volatile("" : "+v"(l));
    return row0 + wave * 32 + l;
  };
  __shared__ AttnRow seen_by[WAVES][32];
  int low_hi = 0x7FFFFFFF, top_lo = 0;
  typename T::x8 qf[KS];
  {
    const int rr = row_of();
    const bool valid = rr < rows;
    const int i = valid ? attn_query(a, rr) : 0, g = valid ? rr - i * a.group : 0;
    const AttnRow row = attn_row(a, sq, i, valid);
    if (h == 0) seen_by[wave][l32] = row;
    if (valid) low_hi = row.hi;
    top_lo = row.lo;
    const uint8_t* src = a.q + 2 * ((int64_t)(sq.token0 + i) * a.q_ts + (int64_t)(head * a.group + g) * a.q_hs);
#pragma unroll
    for (int k = 0; k < KS; ++k) {
      const int d = 16 * k + 8 * h;
      u32x4_t x = {0, 0, 0, 0};
      if (valid && d < a.D) x = *reinterpret_cast<const u32x4_t*>(src + 2 * d);
      qf[k] = __builtin_bit_cast(typename T::x8, x);
    }
  }
#pragma unroll
  for (int d = 1; d < 32; d <<= 1) {
    low_hi = min(low_hi, __shfl_xor(low_hi, d));
    top_lo = max(top_lo, __shfl_xor(top_lo, d));
  }
  // (of the whole tile: its waves take the same blocks as cut)
  __shared__ int ends[2][WAVES];
  if (lane == 0) {
    ends[0][wave] = low_hi;
    ends[1][wave] = top_lo;
  }
  __syncthreads();
#pragma unroll
  for (int i = 0; i < WAVES; ++i) {
    low_hi = min(low_hi, ends[0][i]);
    top_lo = max(top_lo, ends[1][i]);
  }
  low_hi = uniform(low_hi);
  top_lo = uniform(top_lo);

  uint8_t* const places = lds + 4 * L::BLOCK + wave * L::OWN;
  uint8_t* const pages = places + 3 * L::RW * 8;
  auto key0 = [&](int b) { return (b < sp.sink_blocks ? b : b + sp.skip) * BN; };
  auto seen_by_any = [&](int key) { return key < sp.hi && (key >= sp.lo || key < sp.sinks); };
  // starts the load of the pages of block b's 64 keys (of zeros where there is no such key)
  auto load_pages = [&](int b) {
    const int key = key0(b) + lane;
    const void* src = b < b1 && seen_by_any(key) ? (const void*)(table + attn_page(a, key)) : attn_zeros;
    __builtin_amdgcn_global_load_lds(src, (attn_lds_void*)(pages + (b & 3) * 256), 4, 0, 0);
  };
  // Rows of one wave that lie in one page, all of them seen: their addresses are one scalar each and an offset of
  // the lane, which the swizzles change in bits that a load's number sets alone.
  auto load_rows = [&](const uint8_t* from, uint32_t token, uint8_t* to, auto swizzle) {
    int l = lane;
    asm volatile("" : "+v"(l));
    const uint32_t row = l / L::CPR * 2 * token, chunk = 16 * ((l % L::CPR) ^ swizzle(wave * L::RW + l / L::CPR));
#pragma unroll
    for (int n = 0; n < L::NI; ++n)
      attn_load16(from + (uint64_t)n * L::RPI * 2 * token + ((chunk ^ (16 * swizzle(n * L::RPI))) + row), to + n * 1024);
  };
  auto page_of = [&](int b) { return *reinterpret_cast<const uint32_t*>(pages + (b & 3) * 256 + 4 * lane); };
  const uint8_t *v_at[2];  // the first row of the values of the block of each parity, NULL: see their places
  // starts this wave's share of the loads of block b's keys (of zeros past the run), and keeps the places of its values;
  // returns which of the block's keys are there.  `page`: of the lane's key
  auto load_k = [&](int b, int odd, uint32_t page) {
    const int j0 = key0(b);
    const uint32_t of = __builtin_amdgcn_readlane(page, wave * L::RW);
    if (EXACT && a.page_rows && b < b1 && j0 + BN <= sp.hi && (j0 >= sp.lo || j0 + BN <= sp.sinks) && of < a.pages) {
      const AttnPlace p = attn_place(a, kh, vh, j0 + wave * L::RW, of, true);
      v_at[odd] = p.v;
      load_rows(p.k, a.k_token, lds + odd * L::BLOCK + wave * L::RW * L::ROW, attn_swizzle<DP>);
      return (uint64_t)__ballot(page < a.pages);  // (the other waves' rows too)
    }
    v_at[odd] = nullptr;
    const int key = j0 + lane;
    const bool ok = b < b1 && seen_by_any(key) && page < a.pages;
    const AttnPlace p = attn_place(a, kh, vh, key, page, ok);
    if (lane / L::RW == wave) {
      *reinterpret_cast<const uint8_t**>(places + (lane % L::RW) * 8) = p.k;
      *reinterpret_cast<const uint8_t**>(places + ((1 + odd) * L::RW + lane % L::RW) * 8) = p.v;
    }
    wave_lds_sync();
    int l = lane;
    asm volatile("" : "+v"(l));
    uint8_t* to = lds + odd * L::BLOCK + wave * L::RW * L::ROW;
    const uint8_t* from[L::NI];  // (all read before the first load: the compiler keeps their order)
#pragma unroll
    for (int n = 0; n < L::NI; ++n)
      from[n] = *reinterpret_cast<const uint8_t**>(places + (n * L::RPI + l / L::CPR) * 8);
#pragma unroll
    for (int n = 0; n < L::NI; ++n) {
      const int r = n * L::RPI + l / L::CPR;
      attn_load16(attn_chunk<EXACT>(from[n], (l % L::CPR) ^ attn_swizzle<DP>(wave * L::RW + r), a.D), to + n * 1024);
    }
    return (uint64_t)__ballot(ok);
  };
  auto load_v = [&](int odd) {
    int l = lane;
    asm volatile("" : "+v"(l));
    uint8_t* to = lds + (2 + odd) * L::BLOCK + wave * L::RW * L::ROW;
    if (v_at[odd] != nullptr) {
      load_rows(v_at[odd], a.v_token, to, swizzle_v<DP>);
      return;
    }
    const uint8_t* from[L::NI];
#pragma unroll
    for (int n = 0; n < L::NI; ++n)
      from[n] = *reinterpret_cast<const uint8_t**>(places + ((1 + odd) * L::RW + n * L::RPI + l / L::CPR) * 8);
#pragma unroll
    for (int n = 0; n < L::NI; ++n) {
      const int r = n * L::RPI + l / L::CPR;
      attn_load16(attn_chunk<EXACT>(from[n], (l % L::CPR) ^ swizzle_v<DP>(wave * L::RW + r), a.D), to + n * 1024);
    }
  };
  // Operands in LDS, 16 bytes a lane.  Of K: keys 32 t + l32, elements 16 k + 8 h ..; of V: this lane's column of 32 d ..,
  // keys 16 u + 4 h .. + 3 and 8 further.  What the swizzles move depends on the lane and on the low bits of k and d
  // only, the rest is a constant of the instruction.
  constexpr int KO = KS < 8 ? KS : 8, VO = ND < 4 ? ND : 4;
  const uint8_t *kat[KO], *vat[VO];
#pragma unroll
  for (int k = 0; k < KO; ++k) kat[k] = lds + l32 * L::ROW + 16 * ((2 * k + h) ^ attn_swizzle<DP>(l32));
  {
    const int c16 = lane & 15, r = 4 * h + (c16 >> 2), c = 2 * ((lane >> 4) & 1) + ((c16 & 3) >> 1);
#pragma unroll
    for (int d = 0; d < VO; ++d)
      vat[d] = lds + 2 * L::BLOCK + r * L::ROW + 16 * ((4 * d + c) ^ swizzle_v<DP>(r)) + 8 * (c16 & 1);
  }
  auto fetch_k = [&](int odd, int t, int k) {
    return __builtin_bit_cast(typename T::x8, *reinterpret_cast<const u32x4_t*>(
        kat[k % KO] + odd * L::BLOCK + 32 * t * L::ROW + k / KO * 256));
  };
  auto fetch_v = [&](int odd, int u, int d) {
    const uint8_t* p = vat[d % VO] + odd * L::BLOCK + 16 * u * L::ROW + d / VO * 256;
    return attn_read_vt<T>(p, p + 8 * L::ROW);
  };

  float m = ATTN_NONE, l = 0.0f;
  float16_t o[ND];
#pragma unroll
  for (int d = 0; d < ND; ++d)
#pragma unroll
    for (int i = 0; i < 16; ++i) o[d][i] = 0.0f;

  // Pass b: softmax of block b's scores and the product with its values, and, among their instructions, the
  // scores of block b + 1; meanwhile the keys of block b + 2 and the values of block b + 1 are loaded.
  uint64_t here, there;
  load_pages(b0);
  load_pages(b0 + 1);
  load_pages(b0 + 2);
  load_pages(b0 + 3);
  attn_vm_drain();
  here = load_k(b0, 0, page_of(b0));
  load_v(0);
  there = load_k(b0 + 1, 1, page_of(b0 + 1));
  uint32_t page = page_of(b0 + 2);
  asm volatile("s_waitcnt vmcnt(0) lgkmcnt(0)\n\ts_barrier" ::: "memory");
  float16_t sa[2], sb[2], zero;
#pragma unroll
  for (int i = 0; i < 16; ++i) zero[i] = 0.0f;
#pragma unroll
  for (int t = 0; t < 2; ++t)
#pragma unroll
    for (int k = 0; k < KS; ++k) sa[t] = T::mma32(fetch_k(0, t, k), qf[k], k == 0 ? zero : sa[t]);
  auto larger = [](float top, const float16_t& s, int i) { return fmaxf(fmaxf(top, s[2 * i]), s[2 * i + 1]); };
  float top = fmaxf(sa[0][0], sa[0][1]);
#pragma unroll
  for (int i = 1; i < 16; ++i) top = larger(top, sa[i >> 3], i & 7);

  auto raise = [&](float top) {
    const float to = fmaxf(m, top), f = attn_exp2(m - (to == ATTN_NONE ? 0.0f : to));
    l *= f;
#pragma unroll
    for (int d = 0; d < ND; ++d) o[d] *= f;
    m = to;
  };
  auto pass = [&](auto parity, int b, float16_t (&s)[2], float16_t (&next)[2]) {
    constexpr int ODD = decltype(parity)::value;
    // keys b + 1 and values b have landed, here and in the other waves; keys b and values b - 1 are read
    asm volatile("s_waitcnt vmcnt(0) lgkmcnt(0)\n\ts_barrier" ::: "memory");
    const uint64_t later = load_k(b + 2, ODD, page);
    load_v(1 - ODD);
    load_pages(b + 4);
    page = page_of(b + 3);
    const int j0 = key0(b);
    if (here != ~0ull || j0 + BN > low_hi || (j0 < top_lo && j0 + BN > a.sinks)) {
      uint32_t seen[2];
      const AttnRow row = seen_by[wave][l32];
      // element (t, i) is key j0 + 4 h + 32 t + 8 (i / 4) + i % 4
#pragma unroll
      for (int t = 0; t < 2; ++t) {
        const uint32_t mine = (uint32_t)(here >> (32 * t)) >> (4 * h);
        uint32_t bits = attn_seen(a, row, j0 + 32 * t + 4 * h);
        if (a.mask != nullptr && j0 + 32 * t + 32 > sq.ctx && a.mask_width > 0) {
          const int rr = row_of();
          const uint8_t* of = a.mask + (int64_t)(sq.token0 + (rr < rows ? attn_query(a, rr) : 0)) * a.mask_stride;
          const int node = j0 + 32 * t + 4 * h - sq.ctx;
          uint32_t set[16];
#pragma unroll
          for (int i = 0; i < 16; ++i) set[i] = of[min(max(node + 8 * (i >> 2) + (i & 3), 0), a.mask_width - 1)];
          attn_vm_drain();
          uint32_t tree = 0;
#pragma unroll
          for (int i = 0; i < 16; ++i) tree |= (set[i] != 0 ? 1u : 0u) << (8 * (i >> 2) + (i & 3));
          const uint32_t before = attn_below(-node);
          bits = (bits & before) | (tree & attn_below(a.mask_width - node) & ~before);
        }
        bits &= mine;
        seen[t] = bits;
#pragma unroll
        for (int i = 0; i < 16; ++i) s[t][i] = attn_hide(s[t][i], ~bits, 8 * (i >> 2) + (i & 3));
      }
      top = fmaxf(s[0][0], s[0][1]);
#pragma unroll
      for (int i = 1; i < 16; ++i) top = larger(top, s[i >> 3], i & 7);
      uint8_t* const values = lds + (2 + ODD) * L::BLOCK;
      if (attn_any_odd<T, L::BLOCK>(values, lane)) {  // (the same in all waves)
        raise(attn_reference<T>(attn_max32(top), a.scale_log2));        // (nothing is scaled by 0 afterwards)
        uint64_t odd = attn_odd_rows<T, L::CPR, BN>(values, lane);
        while (odd != 0) {
          const int j = __ffsll((unsigned long long)odd) - 1;
          odd &= odd - 1;
          const uint32_t of = __shfl(j >= 32 ? seen[1] : seen[0], l32 + 8 * (j & 4));
          const bool sees = (of >> (8 * (j >> 3 & 3) + (j & 3))) & 1;
#pragma unroll
          for (int d = 0; d < ND; ++d)
#pragma unroll
            for (int q = 0; q < 4; ++q) {
              float x[4] = {o[d][4 * q], o[d][4 * q + 1], o[d][4 * q + 2], o[d][4 * q + 3]};
              attn_add_odd<T>(values + j * L::ROW + 16 * ((4 * d + q) ^ swizzle_v<DP>(j)) + 8 * h, sees, x);
#pragma unroll
              for (int c = 0; c < 4; ++c) o[d][4 * q + c] = x[c];
            }
        }
        __syncthreads();  // every wave has read them
        attn_clear_odd<T, L::CPR, BN / WAVES>(values + wave * L::RW * L::ROW, lane);
        __syncthreads();
      }
    }
    top = attn_reference<T>(attn_max32(top), a.scale_log2);
    if (__any(top > m + ATTN_SLACK)) raise(top);
    const float ref = m == ATTN_NONE ? 0.0f : m, sc = a.scale_log2;

    // Step i: matrix instruction i (2 KS of the next block's scores, then 4 ND products, 16 keys after 16 keys), the
    // LDS reads of the one PRE further, and its share of the vector work: the 16 pairs of exponentials end
    // before the products that need them (a pair's rounding a step after its exponentials), and the next
    // block's maximum follows its scores.  The barriers keep the compiler from gathering each kind again.
    // A block's probabilities are summed before they are rounded, and by themselves: the running sum takes one addition per
    // 64 keys.  (Rounded pairs added to it by dot products, an instruction less each, took the same: prompt of 8192 550 us both,
    // pieces of prompts 135 against 136, four prompts in a window 75 against 76.)
    constexpr int N1 = 2 * KS, N = N1 + 4 * ND, PRE = 3, LAST = N1 + 3 * ND - 1;
    typename T::x8 f[PRE + 1];
    float e[16][2];
    u32x4_t p[4];
    auto fetch = [&](int i) {
      f[i % (PRE + 1)] = i < N1 ? fetch_k(1 - ODD, i / KS, i % KS) : fetch_v(ODD, (i - N1) / ND, (i - N1) % ND);
    };
    float over = ATTN_NONE, own = 0.0f;  // the next block's largest score, and this one's sum
    __builtin_amdgcn_s_setprio(1);
    __builtin_amdgcn_sched_barrier(0);
#pragma unroll
    for (int i = 0; i < PRE; ++i) fetch(i);
    each<N>([&](auto step) __attribute__((always_inline)) {
      constexpr int i = decltype(step)::value;
      if constexpr (i + PRE < N) fetch(i + PRE);
      const auto& op = f[i % (PRE + 1)];
      if constexpr (i < N1) {
        next[i / KS] = T::mma32(op, qf[i % KS], i % KS == 0 ? zero : next[i / KS]);
      } else {
        constexpr int u = (i - N1) / ND, d = (i - N1) % ND;
        o[d] = T::mma32(op, __builtin_bit_cast(typename T::x8, p[u]), o[d]);
      }
      __builtin_amdgcn_sched_barrier(0);
      each<2>([&](auto y) __attribute__((always_inline)) {
        // pair j: exponentials in step j LAST / 16, rounding in the next one
        constexpr int j1 = (16 * (i - 1) + LAST - 1) / LAST + decltype(y)::value;
        constexpr int j0 = (16 * i + LAST - 1) / LAST + decltype(y)::value;
        if constexpr (i > 0 && j1 < 16 && j1 * LAST / 16 == i - 1) {
          p[j1 / 4][j1 % 4] = T::pack2(e[j1][0], e[j1][1]);
          own = j1 == 0 ? e[j1][0] + e[j1][1] : own + (e[j1][0] + e[j1][1]);
        }
        if constexpr (j0 < 16 && j0 * LAST / 16 == i) {
          e[j0][0] = attn_exp2(fmaf(s[j0 >> 3][2 * (j0 & 7)], sc, -ref));
          e[j0][1] = attn_exp2(fmaf(s[j0 >> 3][2 * (j0 & 7) + 1], sc, -ref));
        }
      });
      // (a score's last matrix instruction is two steps ahead)
      if constexpr (i >= KS + 2 && i < KS + 10) over = larger(over, next[0], i - KS - 2);
      if constexpr (i >= N1 + 2 && i < N1 + 6) {
        over = larger(over, next[1], 2 * (i - N1 - 2));
        over = larger(over, next[1], 2 * (i - N1 - 2) + 1);
      }
      __builtin_amdgcn_sched_barrier(0);
    });
    __builtin_amdgcn_s_setprio(0);
    asm volatile("" : "+v"(over), "+v"(own));  // (not moved out of the steps and behind them)
    top = over;
    l += own;
    here = there;
    there = later;
  };
#pragma unroll 1
  for (int b = b0; b < b1; b += 2) {
    pass(std::integral_constant<int, 0>{}, b, sa, sb);
    if (b + 1 < b1) pass(std::integral_constant<int, 1>{}, b + 1, sb, sa);
  }
  asm volatile("s_waitcnt vmcnt(0)" ::: "memory");  // (nothing arrives in the LDS of an ended wave)

  const float sum = attn_sum32(l);
  const int rr = row_of();
  if (rr >= rows) return;
  if (pieces == 1) {
    const float f = sum == 0.0f ? 0.0f : 1.0f / sum;
    const int i = attn_query(a, rr), g = rr - i * a.group;
    uint8_t* dst = a.out + 2 * ((int64_t)(sq.token0 + i) * a.o_ts + (int64_t)(head * a.group + g) * a.o_hs);
#pragma unroll
    for (int d = 0; d < ND; ++d)
#pragma unroll
      for (int q = 0; q < 4; ++q) {
        const int e = 32 * d + 8 * q + 4 * h;
        if (e < a.D)
          *reinterpret_cast<u32x2_t*>(dst + 2 * e) = u32x2_t{T::pack2(o[d][4 * q] * f, o[d][4 * q + 1] * f),
                                                            T::pack2(o[d][4 * q + 2] * f, o[d][4 * q + 3] * f)};
      }
  } else {
    const int64_t to = (((int64_t)slot * a.kv_heads + head) * a.pieces + piece) * BM + (rr - row0);
    if (h == 0) *reinterpret_cast<float2_t*>(a.stats + 2 * to) = float2_t{m, sum};
#pragma unroll
    for (int d = 0; d < ND; ++d)
#pragma unroll
      for (int q = 0; q < 4; ++q)
        *reinterpret_cast<float4_t*>(a.part + to * DP + 32 * d + 8 * q + 4 * h) =
            float4_t{o[d][4 * q], o[d][4 * q + 1], o[d][4 * q + 2], o[d][4 * q + 3]};
  }
}

// Joins the pieces of a tile.
template <int DP, int BM, class T>
__global__ __launch_bounds__(256) void attn_tile_join_kernel(const AttnArgs a, const int slots) {
  const int head = blockIdx.x % a.kv_heads, slot = blockIdx.x / a.kv_heads;
  const TileOf at = tile_at<BM>(a, slot);
  const AttnSeq sq = attn_seq(a, at.seq);
  const int rows = sq.nq * a.group, row0 = at.tile * BM;
  if (at.tile < 0 || row0 >= rows || rows <= a.rows_from || rows > a.rows_to) return;
  const int pieces = pieces_of(a, span_of<BM>(a, sq, row0, rows));
  if (pieces == 1) return;
  const int64_t first = ((int64_t)slot * a.kv_heads + head) * a.pieces;
  attn_join<DP, BM, T>(a, pieces, min(BM, rows - row0), row0, sq.token0, head, [&](int p) { return first + p; });
}

// The tiles of a call: rows of one, how many slots they take (see tile_at; without `starts`, sequence by sequence,
// they take no more), and into how many pieces each tile's keys are cut at most: so many that all tiles' pieces are
// about the workgroups that the GPU holds (sequences' last tiles are half full on average).  512 queries of 32 heads
// over 8 and 16384 keys, us: 160 with 512 workgroups, 195 with 256, 173 with 1024; heads of 256 dimensions, one workgroup per CU:
// 170 with 256, 186 with 512.  At most 32 (16 queries, 32768 keys: 60 with 16, 47 with 32, 51 with 64).
// Slots are at most about six times the tiles that this counts on, so that grid and workspace stay in proportion to
// what the GPU holds: a piece of 256 queries among 255 single tokens, 32 heads over 8, has 79 slots (271 in the
// first way of numbering) and 168 MB of pieces (577).
struct TilePlan {
  int rows;
  int64_t slots;
  int pieces, slot_rate;
};
TilePlan plan(const AttnArgs& a, int64_t max_q) {
  TilePlan p;
  p.rows = 128;
  const int64_t rows = (int64_t)a.tokens * a.group, sequences = (a.tokens + max_q - 1) / max_q;
  p.slots = rows / p.rows + a.batch;
  p.slot_rate = 0;
  if (a.rows_from > 0) {
    const int rate = 1 + (p.rows + a.rows_from - 1) / a.rows_from;
    const int64_t slots = rows * rate / p.rows;
    if (slots < p.slots) {
      p.slots = slots;
      p.slot_rate = rate;
    }
  }
  const int64_t wgs = (rows / p.rows + (sequences + 1) / 2) * a.kv_heads, resident = a.D <= 128 ? 512 : 256;
  p.pieces = (int)std::min<int64_t>(32, std::max<int64_t>(1, (resident + wgs / 2) / wgs));
  return p;
}

template <int DP, int WAVES, class T>
hipError_t run(AttnArgs a, int64_t max_q, void* workspace, hipStream_t st) {
  using L = Tile<DP, WAVES>;
  const TilePlan p = plan(a, max_q);
  if (p.rows != L::BM) return hipErrorInvalidValue;
  const int64_t wgs = p.slots * a.kv_heads * p.pieces;
  if (wgs >= 0x1000000) return hipErrorInvalidConfiguration;  // (a grid's threads are counted in 32 bits, and so are tiles' rows)
  a.pieces = p.pieces;
  a.slot_rate = p.slot_rate;
  // p pieces take blocks / p passes of about 1 us, and write and read p tokens heads DP floats (twice 0.1 us per 1000 rows of
  // 128 and piece): least for p = sqrt(blocks 5000 / (tokens heads)).  (32 heads, us: 64 queries and 8192 keys 36, 49 with all
  // 32 pieces; 16 queries and 8192 keys 22 and 31; 16 and 32768 39 and 47)
  a.piece_gain = 5000.0f / ((float)a.tokens * (float)a.heads);
  a.stats = static_cast<float*>(workspace);
  a.part = a.stats + (size_t)wgs * L::BM * 2;
  if (a.D == DP) attn_tile_kernel<DP, true, WAVES, T><<<(unsigned)wgs, 64 * WAVES, L::LDS, st>>>(a, (int)p.slots);
  else attn_tile_kernel<DP, false, WAVES, T><<<(unsigned)wgs, 64 * WAVES, L::LDS, st>>>(a, (int)p.slots);
  hipError_t e = hipGetLastError();
  if (e != hipSuccess || p.pieces == 1) return e;
  // (16 trees of 33 to 64 tokens: 161 us with 64 shares of 41 x 8 tiles, 142 with 12)
  const int64_t tiles = p.slots * a.kv_heads, shares = std::min<int64_t>(64, std::max<int64_t>(8, 4096 / tiles));
  attn_tile_join_kernel<DP, L::BM, T><<<dim3((unsigned)tiles, (unsigned)shares), 256, 0, st>>>(a, (int)p.slots);
  return hipGetLastError();
}

template <class T>
hipError_t run_dim(const AttnArgs& a, int64_t max_q, void* workspace, hipStream_t st) {
  if (a.D <= 64) return run<64, 4, T>(a, max_q, workspace, st);
  if (a.D <= 128) return run<128, 4, T>(a, max_q, workspace, st);
  return run<256, 4, T>(a, max_q, workspace, st);
}

}  // namespace

size_t attention_tile_bytes(const AttnArgs& a, int64_t max_q) {
  const int DP = a.D <= 64 ? 64 : a.D <= 128 ? 128 : 256;
  const TilePlan p = plan(a, max_q);
  return p.pieces == 1 ? 0 : (size_t)p.slots * a.kv_heads * p.pieces * p.rows * (2 + DP) * sizeof(float);
}

hipError_t launch_attention_tile(const AttnArgs& a, int dtype, int64_t max_q, void* workspace, hipStream_t stream) {
  return dtype == 0 ? run_dim<Bf16>(a, max_q, workspace, stream) : run_dim<F16>(a, max_q, workspace, stream);
}

}  // namespace w4a4
