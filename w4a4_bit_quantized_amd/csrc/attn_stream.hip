// Attention of few query rows per sequence over a paged cache (gfx950): decoded tokens, drafted trees.
//
// Bound: HBM (every key and value of the batch once).  A workgroup is one wave, and the launch about as many as
// the GPU holds; the blocks of KB keys of all (sequence, key / value head, row tile) triples are numbered through in
// that order, and every wave takes an equal run of them, whatever the sequences' lengths.  Each wave finds its run by
// itself (every lane sums a part of the sequences' block counts), streams it through an LDS ring of its own by direct
// loads (one block ahead, no barrier), and keeps the maximum, sum and output of its rows in registers.  A triple that
// lies in one run is finished there; of one that is cut, every piece goes to the workspace in float32, and a second
// kernel joins the pieces in the order of the runs.
//
// Measured, 32 heads of 128 over 8, with the join (4 us): one token of 64 sequences of 37 to 8191 keys 179 to 182 us, 5.9 to
// 6.0 TB/s (of 4096 keys each 171, 6.3); a window of 4096 keys of 16 sequences, 4 heads, 33 us, 4.0 TB/s; one sequence of 4096
// keys 16 us, of which finding the run takes 1.3, its queries and pages 2.3, the first keys 1.8, and the four blocks of a run
// 6.  Runs of four waves that share the rows' pieces in LDS gained nothing over one-wave workgroups.
//
// Registers: 138 to 310, so that LDS alone limits the waves of a CU (8 at 64 dimensions, 4 at 128, 2 at 256).  Heads of
// 256 with 17 to 32 rows need 484 to 512 and spill 6 to 12 more, to accumulation registers or to memory (a spill only makes the
// counted waits longer): 64 sequences of 4 and of 6 queries over 4096 keys, 16 heads over 4, 184 and 225 us for the same 177 us
// of bytes.
//
// v_mfma_f32_16x16x32: lane l holds row l % 16 of the tile's NQ blocks of 16 rows, keys 4 (l / 16) .. + 3 of 16.
#include "attention.h"

namespace w4a4 {

namespace {

constexpr int KB = 32;  // keys of a block
// What a triple costs before its first block (its queries, pages and first keys follow one another), in blocks: runs
// are equal in blocks and starts.
// (64 sequences of 37 to 8191 keys: 190 us with 0, 183, 184, 180 and 184 with 1 to 4)
constexpr int START = 3;

// 16 bytes per lane from `src` to LDS at dst + 16 lane, not kept in the caches: of keys that one sequence has to itself, as in
// most batches, nobody reads them again (64 sequences of 4096 keys, 8 heads of 128: 173 us, 198 with ordinary loads).  Where
// they are read again it costs some: of 4096 keys half shared by all 64 170 against 161, 3968 shared 161 against 154; several tiles
// per sequence, 16 times 24 queries with max_q stated as 1, 285 against 245.
__device__ __forceinline__ void load16(const uint8_t* src, uint8_t* dst) {
  __builtin_amdgcn_global_load_lds(src, (attn_lds_void*)dst, 16, 0, 2);
}

template <int DP>
struct Stream {
  static constexpr int ROW = 2 * DP, CPR = DP / 8;  // bytes and 16-byte chunks of an LDS row
  static constexpr int RPI = 64 / CPR;              // rows of a direct load
  static constexpr int NI = KB / RPI;               // direct loads of K, or of V, per block
  static constexpr int HALF = KB * ROW;             // K of a stage, then V
  static constexpr int STAGE = 2 * HALF;
  static constexpr int LDS = 2 * STAGE + KB * (int)sizeof(AttnPlace) + 4 * 256;
};

template <int DP, bool EXACT, int NQ, class T>
__global__ __launch_bounds__(64) void attn_stream_kernel(const AttnArgs a) {
  using S = Stream<DP>;
  constexpr int BM = 16 * NQ, KS = DP / 32, ND = DP / 16;
  // two stages, the places of a block's keys, and the pages of four blocks' keys (key lane % 32 of 64)
  __shared__ __attribute__((aligned(16))) uint8_t ring[S::LDS];
  AttnPlace* const places = reinterpret_cast<AttnPlace*>(ring + 2 * S::STAGE);
  uint8_t* const pages = ring + 2 * S::STAGE + KB * sizeof(AttnPlace);
  const int lane = threadIdx.x, c16 = lane & 15, qd = lane >> 4;
  const int w = blockIdx.x;

  // this wave's run [u0, u1) of all blocks, and the sequence that u0 is in.  A lane sums the blocks of a strip of
  // sequences; with at most 64 of them, it keeps its one for later.
  auto tiles_of = [&](const AttnSeq& q) {  // (0: not this launch's)
    const int rows = q.nq * a.group;       // (at most tokens x group, which was checked to fit)
    return rows > a.rows_from && rows <= a.rows_to ? (rows + BM - 1) / BM : 0;
  };
  auto units_of = [&](const AttnSeq& q) {
    const int tiles = tiles_of(q);
    return tiles ? (int64_t)tiles * a.kv_heads * (attn_span<KB>(a, q, 0, q.len).blocks + START) : (int64_t)0;
  };
  const int strip = (a.batch + 63) / 64;
  AttnSeq own = {0, 0, 0, 0};
  int64_t mine = 0;
#pragma unroll 1
  for (int s = lane * strip; s < min((lane + 1) * strip, a.batch); ++s) {
    own = attn_seq(a, s);
    mine += units_of(own);
  }
  auto seq_at = [&](int s) {
    int many = strip;
    asm volatile("" : "+s"(many));  // (a condition that the loop around it does not get a second copy for)
    if (many > 1) return attn_seq(a, s);
    return AttnSeq{__builtin_amdgcn_readlane(own.token0, s), __builtin_amdgcn_readlane(own.nq, s),
                   __builtin_amdgcn_readlane(own.len, s), __builtin_amdgcn_readlane(own.ctx, s)};
  };
  const int64_t upto = attn_scan(mine);
  auto lane_of = [](int64_t x, int l) {
    const uint32_t lo = __builtin_amdgcn_readlane((int)x, l), hi = __builtin_amdgcn_readlane((int)(x >> 32), l);
    return (int64_t)(((uint64_t)hi << 32) | lo);
  };
  const int64_t total = lane_of(upto, 63);
  const int64_t run = max((total + gridDim.x - 1) >> a.log2_waves, (int64_t)a.least);
  const int64_t u0 = w * run, u1 = min(u0 + run, total);
  if (lane == 0) a.desc[8 * w] = 0;
  if (u0 >= u1) return;
  const int at = uniform(__ffsll(__ballot(upto > u0)) - 1);
  int64_t u = u0, before = lane_of(upto - mine, at);

#pragma unroll 1
  for (int seq = at * strip; u < u1; ++seq) {
    const AttnSeq sq = seq_at(seq);
    const int tiles = tiles_of(sq);
    if (tiles == 0) continue;
    const AttnSpan sp = attn_span<KB>(a, sq, 0, sq.len);
    const int each = sp.blocks + START;  // units of a triple
    const int64_t units = (int64_t)tiles * a.kv_heads * each;
    if (before + units <= u) {
      before += units;
      continue;
    }
    const int32_t* table = a.table + (int64_t)seq * a.table_stride;
    const int rows = sq.nq * a.group;
    const int pair = uniform(attn_div(u - before, each));  // head * tiles + tile
    int u_in = (int)(u - before - (int64_t)pair * each);   // this run's first unit of the triple
    int head = tiles == 1 ? pair : uniform(attn_div(pair, tiles)), tile = pair - head * tiles;
#pragma unroll 1
    while (u < u1 && head < a.kv_heads) {
      const int u_end = (int)min((int64_t)each, u_in + (u1 - u));
      const int b0 = max(u_in - START, 0), b1 = max(u_end - START, 0);
      const bool first = u_in == 0, whole = first && u_end == each;
      u += u_end - u_in;
      const uint8_t* kh = a.k + 2 * (head * a.k_head);
      const uint8_t* vh = a.v + 2 * (head * a.v_head);

      // the tile's rows: what each lane's sees, and its operands
      AttnRow row[NQ];
      typename T::x8 qf[NQ][KS];
      int low_hi = 0x7FFFFFFF, top_lo = 0;
#pragma unroll
      for (int n = 0; n < NQ; ++n) {
        const int rr = tile * BM + n * 16 + c16;
        const bool valid = rr < rows;
        const int i = valid ? attn_query(a, rr) : 0, g = valid ? rr - i * a.group : 0;
        row[n] = attn_row(a, sq, i, valid);
        if (valid) {
          low_hi = min(low_hi, row[n].hi);
          top_lo = max(top_lo, row[n].lo);
        }
        const uint8_t* src = a.q + 2 * ((int64_t)(sq.token0 + i) * a.q_ts + (int64_t)(head * a.group + g) * a.q_hs);
#pragma unroll
        for (int k = 0; k < KS; ++k) {
          const int d = 32 * k + 8 * qd;
          u32x4_t x = {0, 0, 0, 0};
          if (valid && d < a.D) x = *reinterpret_cast<const u32x4_t*>(src + 2 * d);
          qf[n][k] = __builtin_bit_cast(typename T::x8, x);
        }
      }
#pragma unroll
      for (int d = 1; d < 16; d <<= 1) {
        low_hi = min(low_hi, __shfl_xor(low_hi, d));
        top_lo = max(top_lo, __shfl_xor(top_lo, d));
      }
      low_hi = uniform(low_hi);
      top_lo = uniform(top_lo);

      auto key0 = [&](int b) { return (b < sp.sink_blocks ? b : b + sp.skip) * KB; };
      auto seen_by_any = [&](int key) { return key < sp.hi && (key >= sp.lo || key < sp.sinks); };
      // starts the load of the pages of block b's keys (of zeros where there is no such key)
      auto load_pages = [&](int b) {
        const int key = key0(b) + (lane & 31);
        const void* src = b < b1 && seen_by_any(key) ? (const void*)(table + attn_page(a, key)) : attn_zeros;
        __builtin_amdgcn_global_load_lds(src, (attn_lds_void*)(pages + (b & 3) * 256), 4, 0, 0);
      };

      float m[NQ], l[NQ];
      float4_t o[NQ][ND];
#pragma unroll
      for (int n = 0; n < NQ; ++n) {
        m[n] = ATTN_NONE;
        l[n] = 0.0f;
#pragma unroll
        for (int d = 0; d < ND; ++d) o[n][d] = float4_t{0, 0, 0, 0};
      }
      // 16 keys that lie in one page, all of them seen: their rows' addresses are one scalar and an offset of the lane,
      // which the swizzle changes in bits that a load's number sets alone.
      const uint32_t k_row = lane / S::CPR * 2 * a.k_token, v_row = lane / S::CPR * 2 * a.v_token;
      const uint32_t chunk = 16 * ((lane % S::CPR) ^ attn_swizzle<DP>(lane / S::CPR));
      auto load_row = [&](const uint8_t* from, uint32_t token, uint32_t row, uint8_t* to, int n) {
        from += (uint64_t)(n * S::RPI % 16) * 2 * token;  // (`from`: of the first of the 16)
        load16(from + ((chunk ^ (16 * attn_swizzle<DP>(n * S::RPI))) + row), to + n * 1024);
      };

      // Pass b works on block b and starts the loads of block b + 2: those of K as soon as this block's
      // scores are formed, those of V at its end, so that one and a half blocks are on their way while the wave
      // computes and two while it waits.  The pages are loaded two passes ahead of their use, into LDS too: for a
      // register the compiler would wait by itself, for all loads.  In the order of their issue: pages b + 2, K b,
      // V b, pages b + 3, K b + 1, V b + 1, pages b + 4, K b + 2, with no K and V past the run; the waits count what
      // may be on its way behind.
      constexpr int NI = S::NI;
      uint32_t here = 0, there = 0, later = 0;  // which keys of blocks b, b + 1, b + 2 are there
      load_pages(b0);
      load_pages(b0 + 1);
      attn_vm_drain();
#pragma unroll 1
      for (int b = b0 - 2; b < b1; ++b) {
        here = there;
        there = later;
        load_pages(b + 4);
        const bool work = b >= b0, more = b + 2 < b1;
        uint8_t* stage = ring + (b & 1) * S::STAGE;
        const uint8_t *ks = stage, *vs = stage + S::HALF;
        const int j0 = key0(b);
        if (work) {
          if (b + 1 < b1) attn_vm_wait<3 * NI + 2>();
          else attn_vm_wait<NI + 2>();
        }
        const uint32_t page = *reinterpret_cast<const uint32_t*>(pages + (b + 2 & 3) * 256 + 4 * lane);

        float4_t s[NQ][2];
        if (work) {
#pragma unroll
          for (int t = 0; t < 2; ++t) {
            typename T::x8 kf[KS];
#pragma unroll
            for (int k = 0; k < KS; ++k) {
              const int lr = 16 * t + c16;
              kf[k] = __builtin_bit_cast(typename T::x8, *reinterpret_cast<const u32x4_t*>(
                  ks + lr * S::ROW + 16 * ((4 * k + qd) ^ attn_swizzle<DP>(lr))));
            }
#pragma unroll
            for (int n = 0; n < NQ; ++n) {
              s[n][t] = float4_t{0, 0, 0, 0};
#pragma unroll
              for (int k = 0; k < KS; ++k) s[n][t] = T::mma16(kf[k], qf[n][k], s[n][t]);
            }
          }
        }
        // block b + 2
        const int n0 = key0(b + 2);
        const bool whole_rows = EXACT && a.page_rows && n0 + KB <= sp.hi && (n0 >= sp.lo || n0 + KB <= sp.sinks);
        later = 0;
        const uint8_t *v0 = nullptr, *v1 = nullptr;
        if (more) {
          const bool ok = seen_by_any(n0 + (lane & 31)) && page < a.pages;
          later = (uint32_t)__ballot(ok);
          wave_lds_sync();  // (this block's keys are read)
          if (whole_rows && later == 0xFFFFFFFFu) {
            const AttnPlace p0 = attn_place(a, kh, vh, n0, __builtin_amdgcn_readlane(page, 0), true);
            const AttnPlace p1 = attn_place(a, kh, vh, n0 + 16, __builtin_amdgcn_readlane(page, 16), true);
            v0 = p0.v;
            v1 = p1.v;
#pragma unroll
            for (int n = 0; n < NI; ++n) load_row(n < NI / 2 ? p0.k : p1.k, a.k_token, k_row, stage, n);
          } else {
            if (lane < KB) places[lane] = attn_place(a, kh, vh, n0 + lane, page, ok);
            wave_lds_sync();
            const uint8_t* from[NI];  // (all read before the first load: the compiler keeps their order)
#pragma unroll
            for (int n = 0; n < NI; ++n) from[n] = places[n * S::RPI + lane / S::CPR].k;
#pragma unroll
            for (int n = 0; n < NI; ++n) {
              const int c = (lane % S::CPR) ^ attn_swizzle<DP>(n * S::RPI + lane / S::CPR);
              load16(attn_chunk<EXACT>(from[n], c, a.D), stage + n * 1024);
            }
          }
        }
        uint32_t seen[NQ];  // (of a cut block: bit 16 t + i)
        bool cut = false;
        if (work) {
          if (here != 0xFFFFFFFFu || j0 + KB > low_hi || (j0 < top_lo && j0 + KB > a.sinks)) {
            cut = true;
            // element (t, i) is key j0 + 4 qd + 16 t + i
            const uint32_t mine = here >> (4 * qd);
#pragma unroll
            for (int n = 0; n < NQ; ++n) {
              uint32_t bits = attn_seen(a, row[n], j0 + 4 * qd);  // (bit 16 t + i)
              if (a.mask != nullptr && j0 + KB > sq.ctx && a.mask_width > 0) {
                const int rr = tile * BM + n * 16 + c16;
                const uint8_t* of = a.mask + (int64_t)(sq.token0 + (rr < rows ? attn_query(a, rr) : 0)) * a.mask_stride;
                const int node = j0 + 4 * qd - sq.ctx;
                uint32_t set[8];
#pragma unroll
                for (int e = 0; e < 8; ++e) set[e] = of[min(max(node + 16 * (e >> 2) + (e & 3), 0), a.mask_width - 1)];
                attn_vm_drain();  // (with one for each, the loop's waits would wait for every load)
                uint32_t tree = 0;
#pragma unroll
                for (int e = 0; e < 8; ++e) tree |= (set[e] != 0 ? 1u : 0u) << (16 * (e >> 2) + (e & 3));
                const uint32_t before = attn_below(-node);
                bits = (bits & before) | (tree & attn_below(a.mask_width - node) & ~before);
              }
              bits &= mine;
              seen[n] = bits;
#pragma unroll
              for (int e = 0; e < 8; ++e)
                s[n][e >> 2][e & 3] = attn_hide(s[n][e >> 2][e & 3], ~bits, 16 * (e >> 2) + (e & 3));
            }
          }

          typename T::x8 p[NQ];
#pragma unroll
          for (int n = 0; n < NQ; ++n) {
            float top = fmaxf(fmaxf(fmaxf(s[n][0][0], s[n][0][1]), fmaxf(s[n][0][2], s[n][0][3])),
                              fmaxf(fmaxf(s[n][1][0], s[n][1][1]), fmaxf(s[n][1][2], s[n][1][3])));
            top = attn_reference<T>(attn_max16(attn_max32(top)), a.scale_log2);
            if (__any(top > m[n] + ATTN_SLACK)) {
              const float to = fmaxf(m[n], top), f = attn_exp2(m[n] - (to == ATTN_NONE ? 0.0f : to));
              l[n] *= f;
#pragma unroll
              for (int d = 0; d < ND; ++d) o[n][d] *= f;
              m[n] = to;
            }
            const float ref = m[n] == ATTN_NONE ? 0.0f : m[n];
            float e[8];
#pragma unroll
            for (int t = 0; t < 2; ++t)
#pragma unroll
              for (int i = 0; i < 4; ++i) e[4 * t + i] = attn_exp2(fmaf(s[n][t][i], a.scale_log2, -ref));
            l[n] += ((e[0] + e[1]) + (e[2] + e[3])) + ((e[4] + e[5]) + (e[6] + e[7]));
            p[n] = __builtin_bit_cast(typename T::x8, u32x4_t{T::pack2(e[0], e[1]), T::pack2(e[2], e[3]),
                                                             T::pack2(e[4], e[5]), T::pack2(e[6], e[7])});
          }
          if (more) attn_vm_wait<3 * NI + 2>();
          else if (b + 1 < b1) attn_vm_wait<2 * NI + 2>();
          else attn_vm_wait<2>();
          if (cut) {
            if (attn_any_odd<T, S::HALF>(vs, lane)) {
              uint32_t odd = (uint32_t)attn_odd_rows<T, S::CPR, KB>(vs, lane);
              while (odd != 0) {
                const int j = __ffs(odd) - 1;
                odd &= odd - 1;
#pragma unroll
                for (int n = 0; n < NQ; ++n) {
                  const bool sees = (__shfl(seen[n], c16 + 16 * ((j >> 2) & 3)) >> (16 * (j >> 4) + (j & 3))) & 1;
#pragma unroll
                  for (int d = 0; d < ND; ++d) {
                    const uint8_t* at = vs + j * S::ROW + 16 * ((2 * d + (qd >> 1)) ^ attn_swizzle<DP>(j)) + 8 * (qd & 1);
                    float x[4] = {o[n][d][0], o[n][d][1], o[n][d][2], o[n][d][3]};
                    attn_add_odd<T>(at, sees, x);
                    o[n][d] = float4_t{x[0], x[1], x[2], x[3]};
                  }
                }
              }
              wave_lds_sync();
              attn_clear_odd<T, S::CPR, KB>(stage + S::HALF, lane);
              wave_lds_sync();
            }
          }
#pragma unroll
          for (int d = 0; d < ND; ++d) {
            const int r0 = 4 * qd + (c16 >> 2), r1 = r0 + 16, ch = 2 * d + ((c16 & 3) >> 1), half = 8 * (c16 & 1);
            const auto vf = attn_read_vt<T>(vs + r0 * S::ROW + 16 * (ch ^ attn_swizzle<DP>(r0)) + half,
                                            vs + r1 * S::ROW + 16 * (ch ^ attn_swizzle<DP>(r1)) + half);
#pragma unroll
            for (int n = 0; n < NQ; ++n) o[n][d] = T::mma16(vf, p[n], o[n][d]);
          }
          wave_lds_sync();  // (the stage is read)
        }
        if (more) {
          if (v0 != nullptr) {
#pragma unroll
            for (int n = 0; n < NI; ++n) load_row(n < NI / 2 ? v0 : v1, a.v_token, v_row, stage + S::HALF, n);
          } else {
            const uint8_t* from[NI];
#pragma unroll
            for (int n = 0; n < NI; ++n) from[n] = places[n * S::RPI + lane / S::CPR].v;
#pragma unroll
            for (int n = 0; n < NI; ++n) {
              const int c = (lane % S::CPR) ^ attn_swizzle<DP>(n * S::RPI + lane / S::CPR);
              load16(attn_chunk<EXACT>(from[n], c, a.D), stage + S::HALF + n * 1024);
            }
          }
        }
      }

      float sum[NQ];
#pragma unroll
      for (int n = 0; n < NQ; ++n) sum[n] = attn_sum16(attn_sum32(l[n]));
      // finished, or a piece: the first of a triple in slot 1 of the wave, any other in slot 0
      if (first && !whole && lane == 0) {
        // pieces, the sequence's first row of q, rows of the tile and the first of them, head
        const int pieces = 1 + (run >= each ? 1 : attn_div(each - u_end + run - 1, (int)run));
        *reinterpret_cast<int4*>(a.desc + 8 * w) = int4{pieces, sq.token0, min(BM, rows - tile * BM), tile * BM};
        a.desc[8 * w + 4] = head;
      }
      const int64_t slot = 2 * (int64_t)w + (first ? 1 : 0);
#pragma unroll
      for (int n = 0; n < NQ; ++n) {
        const int rr = tile * BM + n * 16 + c16;
        if (rr >= rows) continue;
        const int i = attn_query(a, rr), g = rr - i * a.group;
        uint8_t* dst = a.out + 2 * ((int64_t)(sq.token0 + i) * a.o_ts + (int64_t)(head * a.group + g) * a.o_hs);
        const int64_t at = slot * BM + n * 16 + c16;
        if (!whole && qd == 0) *reinterpret_cast<float2_t*>(a.stats + 2 * at) = float2_t{m[n], sum[n]};
        const float f = sum[n] == 0.0f ? 0.0f : 1.0f / sum[n];
#pragma unroll
        for (int d = 0; d < ND; ++d) {
          const int e = 16 * d + 4 * qd;
          if (!whole) {
            *reinterpret_cast<float4_t*>(a.part + at * DP + e) = o[n][d];
          } else if (e < a.D) {
            *reinterpret_cast<u32x2_t*>(dst + 2 * e) = u32x2_t{T::pack2(o[n][d][0] * f, o[n][d][1] * f),
                                                              T::pack2(o[n][d][2] * f, o[n][d][3] * f)};
          }
        }
      }
      u_in = 0;
      if (++tile == tiles) {
        tile = 0;
        ++head;
      }
    }
    before += units;
  }
  attn_vm_drain();  // (nothing arrives in the LDS of an ended wave)
}

// Joins the pieces of the triple that starts in run blockIdx.x and is cut.
template <int DP, int BM, class T>
__global__ __launch_bounds__(256) void attn_join_kernel(const AttnArgs a) {
  const int w = blockIdx.x;
  const int4 d = *reinterpret_cast<const int4*>(a.desc + 8 * w);
  const int head = a.desc[8 * w + 4];
  if (d.x == 0) return;
  attn_join<DP, BM, T>(a, d.x, d.z, d.w, d.y, head, [&](int p) { return p == 0 ? 2 * (int64_t)w + 1 : 2 * (int64_t)(w + p); });
}

// Waves of a launch: as many as the GPU's 256 CUs hold by their LDS.
constexpr int log2_waves(int DP) { return DP == 64 ? 11 : DP == 128 ? 10 : 9; }

template <int DP, int NQ, class T>
hipError_t run(AttnArgs a, void* workspace, hipStream_t st) {
  constexpr int W = 1 << log2_waves(DP), BM = 16 * NQ;
  a.desc = static_cast<int32_t*>(workspace);
  a.stats = reinterpret_cast<float*>(a.desc + 8 * W);
  a.part = a.stats + (size_t)2 * W * BM * 2;
  a.log2_waves = log2_waves(DP);
  a.least = 4;  // (one sequence of 4096 keys, 8 heads: 16.0 us with 4, 3: 16.5, 5: 17.0)
  if (a.D == DP) attn_stream_kernel<DP, true, NQ, T><<<W, 64, 0, st>>>(a);
  else attn_stream_kernel<DP, false, NQ, T><<<W, 64, 0, st>>>(a);
  hipError_t e = hipGetLastError();
  if (e != hipSuccess) return e;
  attn_join_kernel<DP, BM, T><<<dim3(W, 8 * NQ), 256, 0, st>>>(a);  // (32 rows: 27 us with 16 shares, 32 with 8)
  return hipGetLastError();
}

template <int DP, class T>
hipError_t run_rows(const AttnArgs& a, int64_t rows, void* workspace, hipStream_t st) {
  if (rows <= 16) return run<DP, 1, T>(a, workspace, st);
  return run<DP, 2, T>(a, workspace, st);
}

template <class T>
hipError_t run_dim(const AttnArgs& a, int64_t rows, void* workspace, hipStream_t st) {
  if (a.D <= 64) return run_rows<64, T>(a, rows, workspace, st);
  if (a.D <= 128) return run_rows<128, T>(a, rows, workspace, st);
  return run_rows<256, T>(a, rows, workspace, st);
}

}  // namespace

// Sequences of at most this many rows are streamed; longer ones go to the tiles.  (One batch of each kind, us:
// 16 sequences of 4096 keys, 8 heads: 32 rows 61 streamed, 77 in tiles; 48 rows 112 and 78.  With few (sequence, head) pairs
// the tiles are faster from 17 rows on, as they cut them into fewer pieces: one sequence, 32 rows: 27 and 19; two: 31 and 25;
// four: 35 and 38.)
constexpr int STREAM_ROWS = 32;
static int stream_rows(const AttnArgs& a) { return (int64_t)a.batch * a.kv_heads <= 16 ? 16 : STREAM_ROWS; }

// The tiles of a call take sequences of more rows than this.  Of a batch whose sequences have half of max_q queries on average
// they take the short ones too; in one of prompts among single tokens, a second launch for those is worth its time (4096 keys
// each, us: 512 queries and 63 sequences of one 241, 265 by the tiles alone; 12 sequences of 64 and 4 of 4 90, 111 by
// both).
static int tiles_from(const AttnArgs& a, int64_t max_q) {
  return (int64_t)a.batch * max_q <= 2 * (int64_t)a.tokens ? 0 : stream_rows(a);
}

// At least the streams' share for 32 rows, also where 16 are used or the tiles take all, so that a workspace sized for prompts whose
// keys are not cut holds single tokens' calls too.  (For one token 34 MB at 128 dimensions, half of which is used.)
size_t attention_workspace_bytes(const AttnArgs& args, int64_t max_q) {
  AttnArgs a = args;
  const int DP = a.D <= 64 ? 64 : a.D <= 128 ? 128 : 256;
  const size_t W = 1 << log2_waves(DP), BM = STREAM_ROWS;
  const size_t stream = W * 32 + 2 * W * BM * 8 + 2 * W * BM * DP * 4;
  if (max_q * a.group <= stream_rows(a)) return stream;
  a.rows_from = tiles_from(a, max_q);
  return std::max(stream, attention_tile_bytes(a, max_q));
}

hipError_t launch_attention(AttnArgs a, int dtype, int64_t max_q, void* workspace, hipStream_t stream) {
  a.rows_from = 0;
  a.rows_to = 0x7FFFFFFF;
  int64_t rows = max_q * a.group;
  if (rows > stream_rows(a)) {
    a.rows_from = tiles_from(a, max_q);
    hipError_t e = launch_attention_tile(a, dtype, max_q, workspace, stream);
    if (e != hipSuccess || a.rows_from == 0) return e;
    a.rows_to = rows = a.rows_from;
    a.rows_from = 0;
  }
  return dtype == 0 ? run_dim<Bf16>(a, rows, workspace, stream) : run_dim<F16>(a, rows, workspace, stream);
}

}  // namespace w4a4
