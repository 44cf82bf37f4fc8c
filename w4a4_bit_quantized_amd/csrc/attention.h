// What the attention kernels over the paged cache share (gfx950).
//
// Rows.  The query heads of one key / value head (a group) and all queries of a sequence share its keys: row
// r = i group + g of the pair (sequence, key / value head) is query i's head g of the group, and tiles are made of
// consecutive rows.
//
// Scores are formed transposed, S^T = K Q^T, so that a lane holds one row's scores (a column of the matrix
// instruction's result) for 4 keys in 4, 8 or 16: maxima and sums stay in the lane but for one or two exchanges, the
// factor that rescales a row's sums is the lane's own, and the probabilities are already where the second product,
// O^T = V^T P^T, takes them (its keys are summed in whatever order both operands share).  V's operand comes from
// the row-major LDS tile through the transposing LDS read.
//
// Rounding: scores, maxima, sums and outputs are float32.  The probabilities are rounded to the tensors' 16-bit type for
// the matrix instruction, half a step each (2^-8 of the value in bf16, 2^-11 in f16): less than the output's own
// rounding on average, and the sums below the fraction are of the unrounded ones.  They are taken against a
// reference that a row's maximum passes by at most 2^8 (ATTN_SLACK), in f16 times 2^7 (SHIFT): they end at 2^15 of the 2^16
// that f16 holds, and what is below 2^-21 of the reference is off by 2^-32 of it.  (Without the shift it was 2^-25: the
// weight of thousands of keys with scores 15 below a sink's was off by 5 in a hundred, of those 18 below lost.)
#pragma once

#include <algorithm>

#include "device_common.h"
#include "launch.h"
#include "w4a4.h"

namespace w4a4 {

typedef __attribute__((address_space(3))) void attn_lds_void;
typedef short attn_short4_t __attribute__((ext_vector_type(4)));
typedef __attribute__((address_space(3))) attn_short4_t attn_lds_s4;

struct Bf16 {
  typedef bf16x8_t x8;
  static constexpr uint32_t EXP = 0x7F80;  // the exponent of infinities and NaNs
  static constexpr float SHIFT = 0.0f;     // log2 of what probabilities are multiplied by
  static __device__ __forceinline__ float value(uint32_t bits) { return __uint_as_float(bits << 16); }
  static __device__ __forceinline__ float4_t mma16(x8 a, x8 b, float4_t c) {
    return __builtin_amdgcn_mfma_f32_16x16x32_bf16(a, b, c, 0, 0, 0);
  }
  static __device__ __forceinline__ float16_t mma32(x8 a, x8 b, float16_t c) {
    return __builtin_amdgcn_mfma_f32_32x32x16_bf16(a, b, c, 0, 0, 0);
  }
  static __device__ __forceinline__ uint32_t pack2(float a, float b) {  // round to nearest even
    typedef __bf16 bf16x2_t __attribute__((ext_vector_type(2)));
    return __builtin_bit_cast(uint32_t, __builtin_convertvector(float2_t{a, b}, bf16x2_t));
  }
};

struct F16 {
  typedef half8_t x8;
  static constexpr uint32_t EXP = 0x7C00;
  static constexpr float SHIFT = 7.0f;
  static __device__ __forceinline__ float value(uint32_t bits) {
    const uint16_t b = (uint16_t)bits;
    return (float)__builtin_bit_cast(_Float16, b);
  }
  static __device__ __forceinline__ float4_t mma16(x8 a, x8 b, float4_t c) {
    return __builtin_amdgcn_mfma_f32_16x16x32_f16(a, b, c, 0, 0, 0);
  }
  static __device__ __forceinline__ float16_t mma32(x8 a, x8 b, float16_t c) {
    return __builtin_amdgcn_mfma_f32_32x32x16_f16(a, b, c, 0, 0, 0);
  }
  static __device__ __forceinline__ uint32_t pack2(float a, float b) {
    return __builtin_bit_cast(uint32_t, half2_t{(_Float16)a, (_Float16)b});
  }
};

// One sequence, as the device's arrays describe it, with everything clamped to what the arguments hold.
struct AttnSeq {
  int token0, nq;  // its queries
  int len, ctx;    // its keys, and those before its queries (negative: more queries than keys)
};

__device__ __forceinline__ AttnSeq attn_seq(const AttnArgs& a, int s) {
  AttnSeq q;
  if (a.starts != nullptr) {
    q.token0 = min(max(a.starts[s], 0), a.tokens);
    q.nq = min(max(a.starts[s + 1], q.token0), a.tokens) - q.token0;
  } else {
    q.token0 = s * a.each;
    q.nq = a.each;
  }
  q.len = min(max(a.lens[s], 0), a.max_len);
  q.ctx = q.len - q.nq;
  return q;
}

// The keys that the queries from number i0 on may see: [lo, hi), and below lo the sinks, in blocks of BN keys.
// Block b of the list is block b of the cache below `sink_blocks`, and b + skip from there on.
struct AttnSpan {
  int lo, hi, sinks;  // keys below `sinks` are seen too
  int sink_blocks, skip, blocks;
};

template <int BN>
__device__ __forceinline__ AttnSpan attn_span(const AttnArgs& a, const AttnSeq& q, int i0, int hi) {
  AttnSpan s;
  s.hi = max(hi, 0);
  // (a tree's nodes lie at or behind the tree's start)
  const int first = a.mask != nullptr ? q.ctx : q.ctx + i0;
  s.lo = a.window > 0 && first >= a.window ? min(first - a.window + 1, s.hi) : 0;
  s.sinks = a.window > 0 ? min(a.sinks, s.lo) : 0;
  const int b0 = s.lo / BN;
  s.sink_blocks = min((s.sinks + BN - 1) / BN, b0);
  s.skip = b0 - s.sink_blocks;
  s.blocks = max((s.hi + BN - 1) / BN - s.skip, 1);
  return s;
}

// What one row sees: keys below hi from lo on, or below a.sinks.
struct AttnRow {
  int hi, lo;
};

__device__ __forceinline__ AttnRow attn_row(const AttnArgs& a, const AttnSeq& q, int i, bool valid) {
  AttnRow r;
  r.hi = 0;
  r.lo = 0;
  if (valid) {
    int p = q.ctx + i;
    r.hi = min(p + 1, q.len);
    if (a.mask != nullptr) {
      r.hi = q.ctx;
      p = a.pos != nullptr ? max(a.pos[q.token0 + i], q.ctx) : q.ctx;
    }
    if (a.window > 0 && p >= a.window) r.lo = p - a.window + 1;
  }
  return r;
}

// Masks of a cut block, a bit per key: key base + n is bit n.  (From the ends of the row's ranges at once: four
// prompts of 1000 to 4001 tokens in a window of 1024, heads of 64, 78 us; compared key by key 82.)
__device__ __forceinline__ uint32_t attn_below(int n) { return n >= 32 ? ~0u : (1u << max(n, 0)) - 1u; }  // bits < n
__device__ __forceinline__ uint32_t attn_seen(const AttnArgs& a, const AttnRow& row, int base) {
  return attn_below(row.hi - base) & (~attn_below(row.lo - base) | attn_below(a.sinks - base));
}
// s, or -infinity where bit n of `unseen` is set.
__device__ __forceinline__ float attn_hide(float s, uint32_t unseen, int n) {
  const uint32_t all = (uint32_t)((int)(unseen << (31 - n)) >> 31);
  return __uint_as_float((all & 0xFF800000u) | (~all & __float_as_uint(s)));
}

// x / d for 0 <= x < 2^50, d > 0.  (One step from the hardware's reciprocal of at least 20 bits leaves it off by less than
// 2^-40 of itself and the quotient, of less than 2^31, by less than one.)
__device__ __forceinline__ int attn_div(int64_t x, int d) {
  const double dd = (double)d, r0 = __builtin_amdgcn_rcp(dd), r = fma(fma(-dd, r0, 1.0), r0, r0);
  int64_t q = (int64_t)((double)x * r);
  const int64_t rest = x - q * d;
  return (int)(rest < 0 ? q - 1 : rest >= d ? q + 1 : q);
}

__device__ __forceinline__ int attn_query(const AttnArgs& a, int row) {  // row / group
  return (int)(((uint64_t)(uint32_t)row * a.group_mul) >> a.group_shift);
}
__device__ __forceinline__ int attn_page(const AttnArgs& a, int key) {  // key / page_size
  return (int)(((uint64_t)(uint32_t)key * a.page_mul) >> a.page_shift);
}

// Where a key's row and its value's start in the cache; keys that are not there (behind the last one, out of
// everybody's window, on a page that the pool does not have) start at attn_zeros: what nobody sees is zero, whatever
// the cache holds in its place.
struct AttnPlace {
  const uint8_t *k, *v;
};

static __device__ const u32x4_t attn_zeros[2 * W4A4_ATTENTION_MAX_HEAD_DIM / 16] = {};

__device__ __forceinline__ AttnPlace attn_place(const AttnArgs& a, const uint8_t* k, const uint8_t* v, int key,
                                                uint32_t page, bool ok) {
  const uint32_t in = key - attn_page(a, key) * a.page_size;
  AttnPlace p;
  p.k = k + 2 * ((uint64_t)page * a.k_page + (uint64_t)in * a.k_token);
  p.v = v + 2 * ((uint64_t)page * a.v_page + (uint64_t)in * a.v_token);
  const uint8_t* z = reinterpret_cast<const uint8_t*>(attn_zeros);
  if (!ok) p.k = p.v = z;
  return p;
}

// src + 16 c, or zeros for a chunk past the head's last element (none if EXACT).
template <bool EXACT>
__device__ __forceinline__ const uint8_t* attn_chunk(const uint8_t* src, int c, int D) {
  if constexpr (EXACT) return src + 16 * c;
  uint64_t x = reinterpret_cast<uint64_t>(src) + 16 * c, z = reinterpret_cast<uint64_t>(attn_zeros);
  asm("" : "+v"(x), "+v"(z));  // (a select of two addresses: a branch would split the load in two)
  return reinterpret_cast<const uint8_t*>(8 * c < D ? x : z);
}

__device__ __forceinline__ int64_t uniform(int64_t x) {  // one value of the whole wave
  const uint32_t lo = __builtin_amdgcn_readfirstlane((int)x), hi = __builtin_amdgcn_readfirstlane((int)(x >> 32));
  return (int64_t)(((uint64_t)hi << 32) | lo);
}
__device__ __forceinline__ int uniform(int x) { return __builtin_amdgcn_readfirstlane(x); }

// Sums over the lanes up to each (6 steps within the vector registers).
template <int CTRL, int ROWS>
__device__ __forceinline__ int64_t attn_scan_step(int64_t x) {
  const uint32_t lo = __builtin_amdgcn_update_dpp(0, (int)x, CTRL, ROWS, 0xF, false);
  const uint32_t hi = __builtin_amdgcn_update_dpp(0, (int)(x >> 32), CTRL, ROWS, 0xF, false);
  return x + (int64_t)(((uint64_t)hi << 32) | lo);
}
__device__ __forceinline__ int64_t attn_scan(int64_t x) {
  x = attn_scan_step<0x111, 0xF>(x);  // row_shr 1, 2, 4, 8
  x = attn_scan_step<0x112, 0xF>(x);
  x = attn_scan_step<0x114, 0xF>(x);
  x = attn_scan_step<0x118, 0xF>(x);
  x = attn_scan_step<0x142, 0xA>(x);  // row_bcast 15, 31
  return attn_scan_step<0x143, 0xC>(x);
}

__device__ __forceinline__ float attn_exp2(float x) { return __builtin_amdgcn_exp2f(x); }  // (results below 2^-126: 0)

// Chunk (16 bytes) c of row r of an LDS tile with DP / 8 chunks a row lies at c ^ swizzle(r): 16 consecutive
// rows reading one chunk touch all banks.
template <int DP>
__device__ __forceinline__ int attn_swizzle(int row) {
  return DP == 64 ? (row >> 1) & 7 : row & 15;
}

// 16 bytes per lane from `src` to LDS at dst + 16 lane (dst is the wave's).
__device__ __forceinline__ void attn_load16(const uint8_t* src, uint8_t* dst) {
  __builtin_amdgcn_global_load_lds(src, (attn_lds_void*)dst, 16, 0, 0);
}

// All but the last N of the wave's memory operations are done.  (In the loops' assembly: a wait that the compiler
// counts itself it would make one for all direct loads, before the LDS is read.)
template <int N>
__device__ __forceinline__ void attn_vm_wait() {
  static_assert(N >= 0 && N < 64, "vmcnt range");
  asm volatile("s_waitcnt vmcnt(%0)" ::"n"(N) : "memory");
}
// All of them, and the compiler knows.
__device__ __forceinline__ void attn_vm_drain() {
  __builtin_amdgcn_s_waitcnt(0x0F70);
  __builtin_amdgcn_wave_barrier();
}

__device__ __forceinline__ float attn_max32(float v) {  // with the lane 32 further
  const uint32_t u = __float_as_uint(v);
  const auto s = __builtin_amdgcn_permlane32_swap(u, u, false, false);
  return fmaxf(__uint_as_float(s[0]), __uint_as_float(s[1]));
}
__device__ __forceinline__ float attn_max16(float v) {
  const uint32_t u = __float_as_uint(v);
  const auto s = __builtin_amdgcn_permlane16_swap(u, u, false, false);
  return fmaxf(__uint_as_float(s[0]), __uint_as_float(s[1]));
}
__device__ __forceinline__ float attn_sum32(float v) {
  const uint32_t u = __float_as_uint(v);
  const auto s = __builtin_amdgcn_permlane32_swap(u, u, false, false);
  return __uint_as_float(s[0]) + __uint_as_float(s[1]);
}
__device__ __forceinline__ float attn_sum16(float v) {
  const uint32_t u = __float_as_uint(v);
  const auto s = __builtin_amdgcn_permlane16_swap(u, u, false, false);
  return __uint_as_float(s[0]) + __uint_as_float(s[1]);
}

// Two rows' 8 bytes of V at `a` and `b` (this lane's part of 4 keys x 16 columns each), transposed: the lane's
// column of both.  (restrict gives the reads an alias scope; without one the compiler waits for every direct load
// before each of them.)
template <class T>
__device__ __forceinline__ typename T::x8 attn_read_vt(const uint8_t* __restrict__ a, const uint8_t* __restrict__ b) {
  const attn_short4_t t0 = __builtin_amdgcn_ds_read_tr16_b64_v4i16((attn_lds_s4*)a);
  const attn_short4_t t1 = __builtin_amdgcn_ds_read_tr16_b64_v4i16((attn_lds_s4*)b);
  const u32x2_t w0 = __builtin_bit_cast(u32x2_t, t0), w1 = __builtin_bit_cast(u32x2_t, t1);
  return __builtin_bit_cast(typename T::x8, u32x4_t{w0[0], w0[1], w1[0], w1[1]});
}

// Infinities and NaNs among the values of keys that some of a tile's rows see and others do not.  In the product, the
// others' probability 0 times such a value would be a NaN.  So in a block that a mask cuts, the values are looked
// through first; those rows that see such a value get it added, and it is set to 0 for the product.  (Of an infinity that is
// its product with any positive probability.  One that is too small for the types, 0 here, gives a NaN in the product of
// a block that no mask cuts, and a later factor of 0 makes a NaN of the infinity: infinite or NaN in either case.)
// A lane looks at 16 bytes of every 1024 of the tile.
template <class T>
__device__ __forceinline__ uint32_t attn_odd(uint32_t w) {  // the halves of w that are infinite or NaN, as masks
  constexpr uint32_t E = T::EXP;
  return ((w & E) == E ? 0xFFFFu : 0u) | ((w >> 16 & E) == E ? 0xFFFF0000u : 0u);
}
template <class T, int BYTES>
__device__ __forceinline__ bool attn_any_odd(const uint8_t* tile, int lane) {
  typedef unsigned short ushort2_t __attribute__((ext_vector_type(2)));
  constexpr uint32_t E = T::EXP | T::EXP << 16;
  ushort2_t least = {0xFFFF, 0xFFFF};
#pragma unroll 4
  for (int n = 0; n < BYTES / 1024; ++n) {
    const u32x4_t x = *reinterpret_cast<const u32x4_t*>(tile + n * 1024 + lane * 16);
#pragma unroll
    for (int c = 0; c < 4; ++c) least = __builtin_elementwise_min(least, __builtin_bit_cast(ushort2_t, ~x[c] & E));
  }
  return __any(least[0] == 0 || least[1] == 0);
}
// The rows (a bit each) that have such values, looked for in chunks of 16 bytes, CPR of a row.
template <class T, int CPR, int ROWS>
__device__ __forceinline__ uint64_t attn_odd_rows(const uint8_t* tile, int lane) {
  uint64_t odd = 0;
#pragma unroll 1
  for (int n = 0; n < ROWS * CPR / 64; ++n) {
    const u32x4_t x = *reinterpret_cast<const u32x4_t*>(tile + n * 1024 + lane * 16);
    const uint64_t has = __ballot((attn_odd<T>(x[0]) | attn_odd<T>(x[1]) | attn_odd<T>(x[2]) | attn_odd<T>(x[3])) != 0);
    for (int r = 0; r < 64 / CPR; ++r)
      if ((has >> (r * CPR)) & (((uint64_t)1 << CPR) - 1)) odd |= (uint64_t)1 << (n * (64 / CPR) + r);
  }
  return odd;
}
template <class T, int CPR, int ROWS>
__device__ __forceinline__ void attn_clear_odd(uint8_t* tile, int lane) {
#pragma unroll 1
  for (int n = 0; n < ROWS * CPR / 64; ++n) {
    u32x4_t* at = reinterpret_cast<u32x4_t*>(tile + n * 1024 + lane * 16);
    u32x4_t x = *at;
#pragma unroll
    for (int c = 0; c < 4; ++c) x[c] &= ~attn_odd<T>(x[c]);
    *at = x;
  }
}
// What a row that sees a key (or not) gets of 4 of its values in this way.
template <class T>
__device__ __forceinline__ void attn_add_odd(const uint8_t* values, bool seen, float* o) {
  const u32x2_t x = *reinterpret_cast<const u32x2_t*>(values);
#pragma unroll
  for (int c = 0; c < 2; ++c) {
    const uint32_t w = seen ? x[c] & attn_odd<T>(x[c]) : 0u;
    o[2 * c] += T::value(w & 0xFFFFu);
    o[2 * c + 1] += T::value(w >> 16);
  }
}

constexpr float ATTN_NONE = -__builtin_inff();
// The reference that exponents are taken against is raised to a row's maximum only when that has passed it by more
// than this (in powers of two): probabilities up to 2^8 lose nothing, and rescaling becomes rare.
constexpr float ATTN_SLACK = 8.0f;

// The reference that a largest score asks for.
template <class T>
__device__ __forceinline__ float attn_reference(float top, float scale_log2) {
  if constexpr (T::SHIFT == 0.0f) return top * scale_log2;
  else return fmaf(top, scale_log2, -T::SHIFT);
}

// The second kernels' work: joins `pieces` pieces of rows 0 .. rows - 1 of a tile, whose first is row row0 of its sequence
// and head; piece p lies in slot slot(p) of BM rows.  A row is `split` lines of DP / 4 threads, which take its pieces in
// turn, four at a time, and whose sums meet in LDS; more rows at once where there are few pieces.  Workgroups (of 256) with
// other blockIdx.y take other rows.
template <int DP, int BM, class T, class Slot>
__device__ __forceinline__ void attn_join(const AttnArgs& a, int pieces, int rows, int row0, int token0, int head,
                                          Slot slot) {
  constexpr int PER = DP / 4, LINES = 256 / PER;
  __shared__ float4_t sums[256];
  __shared__ float2_t tops[LINES];
  const int t = threadIdx.x, line = t / PER, e = 4 * (t % PER);
  int log2_split = 0;
  while ((1 << log2_split) < LINES && (4 << log2_split) < pieces) ++log2_split;
  const int split = 1 << log2_split, at_once = LINES >> log2_split, part = line & (split - 1);
  for (int r0 = blockIdx.y * at_once; r0 < rows; r0 += gridDim.y * at_once) {
    const int r = r0 + (line >> log2_split), in = min(r, rows - 1);
    float top = ATTN_NONE, sum = 0.0f;
    float4_t o = {0, 0, 0, 0};
    for (int p0 = part; p0 < pieces; p0 += 4 * split) {
      float2_t st[4];
      float4_t v[4];
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        const int64_t x = slot(min(p0 + i * split, pieces - 1)) * BM + in;
        st[i] = *reinterpret_cast<const float2_t*>(a.stats + 2 * x);
        v[i] = *reinterpret_cast<const float4_t*>(a.part + x * DP + e);
        if (p0 + i * split >= pieces) st[i] = float2_t{ATTN_NONE, 0.0f};
      }
      const float to = fmaxf(fmaxf(fmaxf(st[0][0], st[1][0]), fmaxf(st[2][0], st[3][0])), top);
      const float ref = to == ATTN_NONE ? 0.0f : to, keep = attn_exp2(top - ref);
      sum *= keep;
      o *= keep;
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        if (p0 + i * split >= pieces) continue;  // (not even times 0: a NaN would count twice)
        const float f = attn_exp2(st[i][0] - ref);
        sum = fmaf(st[i][1], f, sum);
#pragma unroll
        for (int c = 0; c < 4; ++c) o[c] = fmaf(v[i][c], f, o[c]);
      }
      top = to;
    }
    if (split > 1) {
      __syncthreads();
      sums[t] = o;
      if (e == 0) tops[line] = float2_t{top, sum};
      __syncthreads();
      if (part != 0) continue;
      for (int i = 0; i < split; ++i) top = fmaxf(top, tops[line + i][0]);
      const float ref = top == ATTN_NONE ? 0.0f : top;
      sum = 0.0f;
      o = float4_t{0, 0, 0, 0};
      for (int i = 0; i < split; ++i) {
        const float f = attn_exp2(tops[line + i][0] - ref);
        sum = fmaf(tops[line + i][1], f, sum);
        const float4_t v = sums[i * PER + t];
#pragma unroll
        for (int c = 0; c < 4; ++c) o[c] = fmaf(v[c], f, o[c]);
      }
    }
    if (r >= rows || e >= a.D) continue;
    const float f = sum == 0.0f ? 0.0f : 1.0f / sum;
    const int rr = row0 + r, i = attn_query(a, rr), g = rr - i * a.group;
    uint8_t* dst = a.out + 2 * ((int64_t)(token0 + i) * a.o_ts + (int64_t)(head * a.group + g) * a.o_hs + e);
    *reinterpret_cast<u32x2_t*>(dst) = u32x2_t{T::pack2(o[0] * f, o[1] * f), T::pack2(o[2] * f, o[3] * f)};
  }
}

}  // namespace w4a4
