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
// v_mfma_f32_16x16x32: lane l holds row l % 16 of the tile's NQ blocks of 16 rows, keys 4 (l / 16) .. + 3 of 16.
#include "attention.h"

namespace w4a4 {

namespace {

constexpr int KB = 32;  // keys of a block

template <int DP>
struct Stream {
  static constexpr int ROW = 2 * DP, CPR = DP / 8;  // bytes and 16-byte chunks of an LDS row
  static constexpr int RPI = 64 / CPR;              // rows of a direct load
  static constexpr int NI = KB / RPI;               // direct loads of K, or of V, per block
  static constexpr int HALF = KB * ROW;             // K of a stage, then V
  static constexpr int STAGE = 2 * HALF;
};

// A lane without a key, or past the head's last element, loads this instead: what nobody sees is zero, so
// whatever the cache holds there stays out of the sums.
__device__ const u32x4_t attn_zeros = {0, 0, 0, 0};

struct Desc {  // of a cut triple, where its first piece is
  int pieces, seq, head, tile;
};

template <int DP, int NQ, class T>
__global__ __launch_bounds__(64) void attn_stream_kernel(const AttnArgs a) {
  using S = Stream<DP>;
  constexpr int BM = 16 * NQ, KS = DP / 32, ND = DP / 16;
  __shared__ __attribute__((aligned(16))) uint8_t ring[2 * S::STAGE];
  __shared__ __attribute__((aligned(16))) AttnPlace places[KB];
  const int lane = threadIdx.x, c16 = lane & 15, qd = lane >> 4;
  const int w = blockIdx.x;

  // blocks of a tile of sequence s, and its tiles (0: not this launch's)
  auto tiles_of = [&](const AttnSeq& q) {
    const int64_t rows = (int64_t)q.nq * a.group;
    return rows > a.rows_from && rows <= a.rows_to ? (int)((rows + BM - 1) / BM) : 0;
  };
  auto units_of = [&](int s) {
    const AttnSeq q = attn_seq(a, s);
    const int tiles = tiles_of(q);
    return tiles ? (int64_t)tiles * a.kv_heads * attn_span<KB>(a, q, 0, q.len).blocks : (int64_t)0;
  };
  // this wave's run [u0, u1) of all blocks, and the sequence that u0 is in
  const int strip = (a.batch + 63) / 64;
  int64_t mine = 0;
  for (int s = lane * strip; s < min((lane + 1) * strip, a.batch); ++s) mine += units_of(s);
  int64_t upto = mine;
#pragma unroll
  for (int d = 1; d < 64; d <<= 1) {
    const int64_t x = __shfl_up(upto, d);
    if (lane >= d) upto += x;
  }
  const int64_t total = __shfl(upto, 63);
  const int64_t run = max((total + gridDim.x - 1) / gridDim.x, (int64_t)a.least);
  const int64_t u0 = w * run, u1 = min(u0 + run, total);
  if (lane == 0) a.desc[4 * w] = 0;
  if (u0 >= u1) return;
  const int at = __ffsll(__ballot(upto > u0)) - 1;
  int64_t u = u0, before = __shfl(upto - mine, at);
  int seq = __builtin_amdgcn_readfirstlane(at * strip);

  const float sc = a.scale_log2;
  for (; u < u1; ++seq) {
    const AttnSeq sq = attn_seq(a, seq);
    const int tiles = tiles_of(sq);
    if (tiles == 0) continue;
    const AttnSpan sp = attn_span<KB>(a, sq, 0, sq.len);
    const int64_t units = (int64_t)tiles * a.kv_heads * sp.blocks;
    if (before + units <= u) {
      before += units;
      continue;
    }
    const int32_t* table = a.table + (int64_t)seq * a.table_stride;
    while (u < u1 && u < before + units) {
      const int64_t r = u - before;
      const int pair = (int)(r / sp.blocks), head = pair / tiles, tile = pair % tiles;
      const int b0 = (int)(r - (int64_t)pair * sp.blocks), b1 = (int)min((int64_t)sp.blocks, b0 + (u1 - u));
      u += b1 - b0;
      const uint8_t* kh = a.k + 2 * (head * a.k_head);
      const uint8_t* vh = a.v + 2 * (head * a.v_head);
      const int rows = sq.nq * a.group;  // (at most tokens x group: checked to fit)

      // the tile's rows: what each lane's sees, and its operands
      AttnRow row[NQ];
      int64_t mrow[NQ];
      typename T::x8 qf[NQ][KS];
      int low_hi = 0x7FFFFFFF, top_lo = 0;
#pragma unroll
      for (int n = 0; n < NQ; ++n) {
        const int rr = tile * BM + n * 16 + c16;
        const bool valid = rr < rows;
        const int i = valid ? rr / a.group : 0, g = valid ? rr - i * a.group : 0;
        row[n] = attn_row(a, sq, i, valid);
        mrow[n] = (int64_t)(sq.token0 + i) * a.mask_stride;
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
      low_hi = __builtin_amdgcn_readfirstlane(low_hi);
      top_lo = __builtin_amdgcn_readfirstlane(top_lo);

      auto key0 = [&](int b) { return (b < sp.sink_blocks ? b : b + sp.skip) * KB; };
      auto seen_by_any = [&](int key) { return key < sp.hi && (key >= sp.lo || key < sp.sinks); };
      // page of this lane's key (lane % 32) of block b
      auto page_of = [&](int b) {
        const int key = key0(b) + (lane & 31);
        return b < b1 && seen_by_any(key) ? (uint32_t)table[attn_page(a, key)] : 0xFFFFFFFFu;
      };
      // starts block b's loads into stage b % 2; returns which of its keys are there
      auto issue = [&](int b, uint32_t page) {
        const int key = key0(b) + (lane & 31);
        const AttnPlace p = attn_place(a, key, page, seen_by_any(key));
        wave_lds_sync();
        if (lane < KB) places[lane] = p;
        wave_lds_sync();
        uint8_t* stage = ring + (b & 1) * S::STAGE;
#pragma unroll
        for (int n = 0; n < S::NI; ++n) {
          const int lr = n * S::RPI + lane / S::CPR;
          const int c = (lane % S::CPR) ^ attn_swizzle<DP>(lr);
          const AttnPlace pl = places[lr];
          const bool none = pl.k < 0 || 8 * c >= a.D;
          const uint8_t* z = reinterpret_cast<const uint8_t*>(&attn_zeros);
          attn_load16(none ? z : kh + 2 * pl.k + 16 * c, stage + n * 1024);
          attn_load16(none ? z : vh + 2 * pl.v + 16 * c, stage + S::HALF + n * 1024);
        }
        return (uint32_t)__ballot(p.k >= 0);
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
      wave_lds_sync();
      uint32_t there[2];
      there[0] = issue(b0, page_of(b0));
      there[1] = 0;
      uint32_t next = page_of(b0 + 1);
      for (int b = b0; b < b1; ++b) {
        const uint32_t here = there[0];
        if (b + 1 < b1) {
          there[1] = issue(b + 1, next);
          next = page_of(b + 2);
          attn_vm_wait<2 * S::NI>();  // (the page's load is one more, after them)
        } else {
          attn_vm_wait<0>();
        }
        __builtin_amdgcn_wave_barrier();
        const uint8_t* ks = ring + (b & 1) * S::STAGE;
        const uint8_t* vs = ks + S::HALF;
        const int j0 = key0(b);

        float4_t s[NQ][2];
#pragma unroll
        for (int t = 0; t < 2; ++t) {
#pragma unroll
          for (int n = 0; n < NQ; ++n) s[n][t] = float4_t{0, 0, 0, 0};
#pragma unroll
          for (int k = 0; k < KS; ++k) {
            const int lr = 16 * t + c16;
            const auto kf = __builtin_bit_cast(typename T::x8, *reinterpret_cast<const u32x4_t*>(
                ks + lr * S::ROW + 16 * ((4 * k + qd) ^ attn_swizzle<DP>(lr))));
#pragma unroll
            for (int n = 0; n < NQ; ++n) s[n][t] = T::mma16(kf, qf[n][k], s[n][t]);
          }
        }
        if (here != 0xFFFFFFFFu || j0 + KB > low_hi || (j0 < top_lo && j0 + KB > a.sinks)) {
#pragma unroll
          for (int n = 0; n < NQ; ++n)
#pragma unroll
            for (int t = 0; t < 2; ++t)
#pragma unroll
              for (int i = 0; i < 4; ++i) {
                const int in = 16 * t + 4 * qd + i, j = j0 + in;
                bool seen = j < row[n].hi && (j >= row[n].lo || j < a.sinks);
                if (a.mask != nullptr && j >= sq.ctx) {
                  const int node = j - sq.ctx;
                  if (node < a.mask_width) seen = a.mask[mrow[n] + node] != 0;
                }
                if (!seen || !((here >> in) & 1)) s[n][t][i] = ATTN_NONE;
              }
        }

        typename T::x8 p[NQ];
#pragma unroll
        for (int n = 0; n < NQ; ++n) {
          float top = fmaxf(fmaxf(fmaxf(s[n][0][0], s[n][0][1]), fmaxf(s[n][0][2], s[n][0][3])),
                            fmaxf(fmaxf(s[n][1][0], s[n][1][1]), fmaxf(s[n][1][2], s[n][1][3])));
          top = fmaxf(m[n], attn_max16(attn_max32(top)) * sc);
          const float ref = top == ATTN_NONE ? 0.0f : top;
          if (__any(top > m[n])) {
            const float f = exp2f(m[n] - ref);
            l[n] *= f;
#pragma unroll
            for (int d = 0; d < ND; ++d) o[n][d] *= f;
            m[n] = top;
          }
          float e[8];
#pragma unroll
          for (int t = 0; t < 2; ++t)
#pragma unroll
            for (int i = 0; i < 4; ++i) e[4 * t + i] = exp2f(fmaf(s[n][t][i], sc, -ref));
          l[n] += ((e[0] + e[1]) + (e[2] + e[3])) + ((e[4] + e[5]) + (e[6] + e[7]));
          p[n] = __builtin_bit_cast(typename T::x8, u32x4_t{T::pack2(e[0], e[1]), T::pack2(e[2], e[3]),
                                                           T::pack2(e[4], e[5]), T::pack2(e[6], e[7])});
        }
#pragma unroll
        for (int d = 0; d < ND; ++d) {
          const int r0 = 4 * qd + (c16 >> 2), r1 = r0 + 16, ch = 2 * d + ((c16 & 3) >> 1), half = 8 * (c16 & 1);
          const auto vf = attn_read_vt<T>(vs + r0 * S::ROW + 16 * (ch ^ attn_swizzle<DP>(r0)) + half,
                                          vs + r1 * S::ROW + 16 * (ch ^ attn_swizzle<DP>(r1)) + half);
#pragma unroll
          for (int n = 0; n < NQ; ++n) o[n][d] = T::mma16(vf, p[n], o[n][d]);
        }
        there[0] = there[1];
      }

      // finished, or a piece: the first of a triple in slot 1 of the wave, any other in slot 0
      const bool whole = b0 == 0 && b1 == sp.blocks;
      if (b0 == 0 && !whole && lane == 0) {
        *reinterpret_cast<int4*>(a.desc + 4 * w) =
            int4{1 + (int)((sp.blocks - b1 + run - 1) / run), seq, head, tile};
      }
      const int64_t slot = 2 * (int64_t)w + (b0 == 0 ? 1 : 0);
#pragma unroll
      for (int n = 0; n < NQ; ++n) {
        const float sum = attn_sum16(attn_sum32(l[n]));
        const int rr = tile * BM + n * 16 + c16;
        if (rr >= rows) continue;
        if (whole) {
          const float f = sum == 0.0f ? 0.0f : 1.0f / sum;
          const int i = rr / a.group, g = rr - i * a.group;
          uint8_t* dst = a.out + 2 * ((int64_t)(sq.token0 + i) * a.o_ts + (int64_t)(head * a.group + g) * a.o_hs);
#pragma unroll
          for (int d = 0; d < ND; ++d) {
            const int e = 16 * d + 4 * qd;
            if (e < a.D)
              *reinterpret_cast<u32x2_t*>(dst + 2 * e) = u32x2_t{T::pack2(o[n][d][0] * f, o[n][d][1] * f),
                                                                T::pack2(o[n][d][2] * f, o[n][d][3] * f)};
          }
        } else {
          const int64_t at = slot * BM + n * 16 + c16;
          if (qd == 0) *reinterpret_cast<float2_t*>(a.stats + 2 * at) = float2_t{m[n], sum};
#pragma unroll
          for (int d = 0; d < ND; ++d) *reinterpret_cast<float4_t*>(a.part + at * DP + 16 * d + 4 * qd) = o[n][d];
        }
      }
    }
    before += units;
  }
}

// Joins the pieces of the triple that starts in run blockIdx.x and is cut.  A thread takes 4 columns of a row.
template <int DP, int BM, class T>
__global__ __launch_bounds__(256) void attn_join_kernel(const AttnArgs a) {
  const int w = blockIdx.x;
  const int4 d = *reinterpret_cast<const int4*>(a.desc + 4 * w);
  if (d.x == 0) return;
  const AttnSeq sq = attn_seq(a, d.y);
  const int rows = min(BM, sq.nq * a.group - d.w * BM), per = a.D / 4;
  for (int x = threadIdx.x; x < rows * per; x += 256) {
    const int r = x / per, e = 4 * (x - r * per);
    auto at = [&](int p) { return (p == 0 ? 2 * (int64_t)w + 1 : 2 * (int64_t)(w + p)) * BM + r; };
    float top = ATTN_NONE;
    for (int p = 0; p < d.x; ++p) top = fmaxf(top, a.stats[2 * at(p)]);
    const float ref = top == ATTN_NONE ? 0.0f : top;
    float sum = 0.0f;
    float4_t o = {0, 0, 0, 0};
    for (int p = 0; p < d.x; ++p) {
      const float2_t st = *reinterpret_cast<const float2_t*>(a.stats + 2 * at(p));
      const float f = exp2f(st[0] - ref);
      sum = fmaf(st[1], f, sum);
      const float4_t v = *reinterpret_cast<const float4_t*>(a.part + at(p) * DP + e);
#pragma unroll
      for (int i = 0; i < 4; ++i) o[i] = fmaf(v[i], f, o[i]);
    }
    const float f = sum == 0.0f ? 0.0f : 1.0f / sum;
    const int rr = d.w * BM + r, i = rr / a.group, g = rr - i * a.group;
    uint8_t* dst = a.out + 2 * ((int64_t)(sq.token0 + i) * a.o_ts + (int64_t)(d.z * a.group + g) * a.o_hs + e);
    *reinterpret_cast<u32x2_t*>(dst) = u32x2_t{T::pack2(o[0] * f, o[1] * f), T::pack2(o[2] * f, o[3] * f)};
  }
}

// Waves of a launch: as many as the GPU's 256 CUs hold by their LDS.
constexpr int waves_of(int DP) { return DP == 64 ? 2048 : DP == 128 ? 1024 : 512; }

template <int DP, int NQ, class T>
hipError_t run(AttnArgs a, void* workspace, hipStream_t st) {
  constexpr int W = waves_of(DP), BM = 16 * NQ;
  a.desc = static_cast<int32_t*>(workspace);
  a.stats = reinterpret_cast<float*>(a.desc + 4 * W);
  a.part = a.stats + (size_t)2 * W * BM * 2;
  a.least = 4;
  attn_stream_kernel<DP, NQ, T><<<W, 64, 0, st>>>(a);
  hipError_t e = hipGetLastError();
  if (e != hipSuccess) return e;
  attn_join_kernel<DP, BM, T><<<W, 256, 0, st>>>(a);
  return hipGetLastError();
}

template <int DP, class T>
hipError_t run_rows(const AttnArgs& a, int64_t rows, void* workspace, hipStream_t st) {
  if (rows <= 16) return run<DP, 1, T>(a, workspace, st);
  if (rows <= 32) return run<DP, 2, T>(a, workspace, st);
  if constexpr (DP <= 128) return run<DP, 4, T>(a, workspace, st);
  return run<DP, 2, T>(a, workspace, st);
}

template <class T>
hipError_t run_dim(const AttnArgs& a, int64_t rows, void* workspace, hipStream_t st) {
  if (a.D <= 64) return run_rows<64, T>(a, rows, workspace, st);
  if (a.D <= 128) return run_rows<128, T>(a, rows, workspace, st);
  return run_rows<256, T>(a, rows, workspace, st);
}

}  // namespace

size_t attention_workspace_bytes(const AttnArgs& a, int64_t max_q) {
  const int DP = a.D <= 64 ? 64 : a.D <= 128 ? 128 : 256;
  const size_t W = waves_of(DP), BM = DP <= 128 ? 64 : 32;
  return W * 16 + 2 * W * BM * 8 + 2 * W * BM * DP * 4;
}

hipError_t launch_attention(AttnArgs a, int dtype, int64_t max_q, void* workspace, hipStream_t stream) {
  a.rows_from = 0;
  a.rows_to = 0x7FFFFFFF;
  const int64_t rows = max_q * a.group;
  return dtype == 0 ? run_dim<Bf16>(a, rows, workspace, stream) : run_dim<F16>(a, rows, workspace, stream);
}

}  // namespace w4a4
