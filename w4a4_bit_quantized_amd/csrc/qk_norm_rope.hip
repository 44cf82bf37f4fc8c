// RMS norm of query and key heads with the rotary position rotation in the same pass (gfx950).
//
// For every token t and head of D elements:
//   r = 1 / sqrt(mean(x^2) + eps),  u = (x * r) * weight          (optional norm, optional weight)
//   pair p of the rotary span belongs to one position axis a, is number i of its dim_a / 2 pairs, and
//   turns by  pos[t, a] * theta^(-2 i / dim_a)      (each axis its own frequencies)
//         or  pos[t, a] * theta^(-2 p / rot)        (one ladder of frequencies over all pairs)
//   (u0, u1) -> (u0 cos - u1 sin, u0 sin + u1 cos)
// Elements past the rotary span are only normed.  float32 throughout, one rounding at the store.
// The angle is formed in turns in float64 and reduced to half a turn there: what is left, |r| <= 1/2, is
// rounded to float32 and passed to sincospi, and the rest d of the angle that the rounding dropped (at most
// pi 2^-25) turns its result on, to (c - d s, s + d c): without it, a sine or cosine near 0 would be off by d,
// thousands of times its own last place.  The square of d, below 2^-46, is left out.
// (Two fused multiply-adds for a pair and token, which all its heads share: 0.1 us at one token of 40 heads and at 1237
// tokens of 16 heads of 80 in f32, nothing at 32760 tokens of 48 heads of 128.)
//
// The float64 part is off by at most 6 * 2^-53 of the
// largest angle: each frequency is its ladder's highest (the first pair's, or the last's where theta < 1) times 2^-e,
// with 2.5 roundings in e and so 2.5 ln2 e 2^-e <= 2.5 / 2.7 of the highest; the two products, the highest
// and exp2 itself: 4.  (From the first pair up, e ln2 would not be bounded: 17 * 2^-53 at theta = 1e-8.)
//
// Bound: HBM (every element read and written once).  A group of G lanes (a power of two) holds one
// head of one token, 2 V elements per lane: V pairs, so a rotation never leaves its lane and the only
// exchange is the sum of squares (DPP within 16 lanes).  A workgroup takes a few tokens per pass; their
// cosines and sines are made once, in LDS, and shared by all their heads, and each thread forms its pair's
// frequency once per launch.  Measured: 32760 tokens of 24 + 24 heads of 128 in bf16 152 us (5.3 TB/s of
// reads and writes; copies of that size reach 6.1), 4608 tokens 21.5 us (5.3 TB/s; copies 6.8), one token of 32 + 8
// heads 3.8 us.
#include <math.h>

#include "device_common.h"
#include "launch.h"

namespace w4a4 {

namespace {

constexpr int RT = 256;  // threads per workgroup
// Workgroups of a launch with many tokens: six per CU, all resident, which then walk the tokens in
// strides of the whole launch (2048 of them: 180 us at 32760 tokens of 48 heads of 128, 1536: 159;
// a contiguous run of tokens for each: 172; one pass per workgroup: 169).
constexpr int MAX_WGS = 1536;

template <int DT>
__device__ __forceinline__ constexpr int esize() { return DT == 2 ? 4 : 2; }

// Vectors at the alignment of an element, which the hardware takes.
typedef u32x4_t u32x4_a2 __attribute__((aligned(2)));
typedef u32x2_t u32x2_a2 __attribute__((aligned(2)));
typedef float4_t float4_a4 __attribute__((aligned(4)));

// N consecutive elements (N = 1, 4 or 8).
template <int DT, int N>
__device__ __forceinline__ void load_n(const uint8_t* p, float* v) {
  if constexpr (N == 1) {
    if constexpr (DT == 2) v[0] = *reinterpret_cast<const float*>(p);
    else if constexpr (DT == 1) v[0] = (float)*reinterpret_cast<const _Float16*>(p);
    else v[0] = bf16_bits_to_f32(*reinterpret_cast<const uint16_t*>(p));
  } else if constexpr (DT == 2) {
#pragma unroll
    for (int c = 0; c < N; c += 4) {
      const float4_t f = *reinterpret_cast<const float4_a4*>(p + 4 * c);
#pragma unroll
      for (int e = 0; e < 4; ++e) v[c + e] = f[e];
    }
  } else {
    uint32_t w[N / 2];
    if constexpr (N == 8) {
      const u32x4_t f = *reinterpret_cast<const u32x4_a2*>(p);
#pragma unroll
      for (int e = 0; e < 4; ++e) w[e] = f[e];
    } else {
      const u32x2_t f = *reinterpret_cast<const u32x2_a2*>(p);
      w[0] = f[0];
      w[1] = f[1];
    }
#pragma unroll
    for (int e = 0; e < N / 2; ++e) {
      if constexpr (DT == 1) {
        const half2_t h = __builtin_bit_cast(half2_t, w[e]);
        v[2 * e] = (float)h[0];
        v[2 * e + 1] = (float)h[1];
      } else {
        v[2 * e] = __uint_as_float(w[e] << 16);
        v[2 * e + 1] = __uint_as_float(w[e] & 0xFFFF0000u);
      }
    }
  }
}

template <int DT>
__device__ __forceinline__ uint32_t pack2(float a, float b) {  // round to nearest even
  if constexpr (DT == 1) {
    return __builtin_bit_cast(uint32_t, half2_t{(_Float16)a, (_Float16)b});
  } else {
    typedef __bf16 bf16x2_t __attribute__((ext_vector_type(2)));
    return __builtin_bit_cast(uint32_t, __builtin_convertvector(float2_t{a, b}, bf16x2_t));
  }
}

// (16-bit vectors leave by non-temporal stores: 4608 tokens of 48 heads of 128 took 28.4 us with ordinary
// ones, 22.9 with these; an f32 lane's two halves of 32 bytes are better merged in L2, 87 against 91 us
// for 8000 tokens)
template <int DT, int N>
__device__ __forceinline__ void store_n(uint8_t* p, const float* v) {
  if constexpr (N == 1) {
    if constexpr (DT == 2) *reinterpret_cast<float*>(p) = v[0];
    else *reinterpret_cast<uint16_t*>(p) = (uint16_t)pack2<DT>(v[0], v[0]);
  } else if constexpr (DT == 2) {
#pragma unroll
    for (int c = 0; c < N; c += 4)
      *reinterpret_cast<float4_a4*>(p + 4 * c) = float4_t{v[c], v[c + 1], v[c + 2], v[c + 3]};
  } else if constexpr (N == 8) {
    __builtin_nontemporal_store(u32x4_t{pack2<DT>(v[0], v[1]), pack2<DT>(v[2], v[3]), pack2<DT>(v[4], v[5]),
                                        pack2<DT>(v[6], v[7])}, reinterpret_cast<u32x4_a2*>(p));
  } else {
    __builtin_nontemporal_store(u32x2_t{pack2<DT>(v[0], v[1]), pack2<DT>(v[2], v[3])}, reinterpret_cast<u32x2_a2*>(p));
  }
}

template <int CTRL>
__device__ __forceinline__ float dpp(float v) {
  return __int_as_float(__builtin_amdgcn_mov_dpp(__float_as_int(v), CTRL, 0xF, 0xF, true));
}

// Sum over the aligned group of G lanes (the same value in every lane: each step adds two values
// that all lanes of both halves share).
__device__ __forceinline__ float group_sum(float v, int G) {
  if (G >= 2) v += dpp<0xB1>(v);    // quad_perm [1,0,3,2]
  if (G >= 4) v += dpp<0x4E>(v);    // quad_perm [2,3,0,1]
  if (G >= 8) v += dpp<0x141>(v);   // row_half_mirror
  if (G >= 16) v += dpp<0x140>(v);  // row_mirror
  if (G >= 32) v += __int_as_float(__builtin_amdgcn_ds_swizzle(__float_as_int(v), 0x1F | (16 << 10)));
  if (G >= 64) v += __shfl_xor(v, 32);
  return v;
}

// Where the first and second elements of pairs p .. p + V - 1 start.  Layout 0: interleaved; 1: halves
// of the rotary span; 2: halves of each axis's slice.  Past the span (p >= rot2) the chunk's 2 V
// elements are taken as they lie: they are not rotated.
template <int V>
__device__ __forceinline__ void pair_elements(const RopeArgs& a, int p, int& e0, int& e1) {
  e0 = 2 * p;
  e1 = 2 * p + V;
  if (p < a.rot2) {
    if (a.layout == 1) {
      e0 = p;
      e1 = p + a.rot2;
    } else if (a.layout == 2) {
      int x = 0;
      while (x + 1 < a.axes && p >= a.start[x + 1]) ++x;
      e0 = a.start[x] + p;  // 2 start + (p - start)
      e1 = e0 + a.start[x + 1] - a.start[x];
    }
  }
}

// Bytes between the LDS rows of the staged form (below): a head of 16-bit elements, and 16 more so that the
// lane groups of a wave start on different banks.
__host__ __device__ constexpr int row_stride(int D) { return 2 * D + 16; }

// INTER (V = 4): the lane's V pairs are 2 V consecutive elements; otherwise V consecutive elements at
// e0 and V at e1.  IT: chunks of V pairs per lane; UN: items in flight.
//
// STAGED (V = 1, IT = 4, UN = 1, 16-bit types): for heads of whole 16-byte chunks whose pairs are not in whole
// chunks of 4.  A lane group loads its head in 16-byte chunks into a row of its own in LDS, takes its pairs from there, puts the
// results in their places and stores the row in chunks again; no other wave touches the row.
// 32760 tokens of 48 heads of 128, halves of axes of 44, 42 and 42: 178 us, element by element 283 (two items
// in flight: 206, four: 219).  In 4-byte chunks, for heads of 66, it loses: 57 against 52.
template <int DT, int V, bool INTER, int IT, int UN, bool STAGED>
__global__ __launch_bounds__(RT) void qk_norm_rope_kernel(const RopeArgs a) {
  static_assert(!STAGED || (DT != 2 && V == 1 && IT == 4 && UN == 1 && !INTER), "the staged form");
  // two halves of [tb][D / 2] cosines, then sines; then (STAGED) a row for every lane group
  extern __shared__ __attribute__((aligned(16))) float trig[];
  const int t = threadIdx.x;
  const int D2 = a.D / 2, G = 1 << a.log2g;
  const int heads = a.q.heads + a.k.heads;
  const int h0 = blockIdx.y * a.hb, nh = min(a.hb, heads - h0);
  constexpr int ES = esize<DT>();

  // The angle of this thread's pair (of 2^log2p >= D / 2, for tokens t >> log2p, + 256 >> log2p, ...), in turns
  // per position.
  const int ap = t & ((1 << a.log2p) - 1), at0 = t >> a.log2p, atn = RT >> a.log2p;
  double freq = 0.0;
  int axis = 0;
  if (ap < a.rot2) {
    while (axis + 1 < a.axes && ap >= a.start[axis + 1]) ++axis;
    const RopeLadder& l = a.ladder[axis];
    freq = exp2(-(double)abs(ap - l.origin) * l.step) * l.top;
  }

  // this lane's chunks: the same pairs for every item
  const int gl = t & (G - 1), grp = t >> a.log2g, ng = RT >> a.log2g;
  int e0[IT], e1[IT];
  bool in[IT];
  float wq[IT][2 * V], wk[IT][2 * V];
#pragma unroll
  for (int c = 0; c < IT; ++c) {
    const int p = (gl + c * G) * V;
    in[c] = p < D2;
    pair_elements<V>(a, in[c] ? p : 0, e0[c], e1[c]);
#pragma unroll
    for (int i = 0; i < 2 * V; ++i) wq[c][i] = wk[c][i] = 1.0f;
    if (in[c]) {
      auto weights = [&](const void* w, float* to) {
        if (w == nullptr) return;
        const uint8_t* b = static_cast<const uint8_t*>(w);
        if constexpr (INTER) {
          load_n<DT, 2 * V>(b + e0[c] * ES, to);
        } else {
          load_n<DT, V>(b + e0[c] * ES, to);
          load_n<DT, V>(b + e1[c] * ES, to + V);
        }
      };
      weights(a.q.weight, wq[c]);
      weights(a.k.weight, wk[c]);
    }
  }
  uint8_t* row = reinterpret_cast<uint8_t*>(trig + 2 * a.tb * a.D) + grp * row_stride(a.D);
  const bool has_chunk = 8 * gl < a.D;
  int half = 0;
  for (int64_t t0 = (int64_t)blockIdx.x * a.tb; t0 < a.tokens; t0 += (int64_t)gridDim.x * a.tb, half ^= 1) {
    const int nt = (int)min((int64_t)a.tb, a.tokens - t0);
    float* cos_t = trig + half * a.tb * a.D;
    float* sin_t = cos_t + a.tb * D2;
    if (ap < D2)
      for (int tk = at0; tk < nt; tk += atn) {
        float c = 1.0f, s = 0.0f;
        if (ap < a.rot2) {
          const size_t at = (size_t)(t0 + tk) * a.axes + axis;
          const double pos = a.pos64 ? (double)static_cast<const int64_t*>(a.pos)[at]
                                     : (double)static_cast<const int32_t*>(a.pos)[at];
          const double turns = pos * freq, halves = 2.0 * (turns - rint(turns));
          const float near = (float)halves;
          const float d = (float)((halves - (double)near) * 3.141592653589793);
          sincospif(near, &s, &c);
          const float c0 = c;
          c = fmaf(-d, s, c);
          s = fmaf(d, c0, s);
        }
        cos_t[tk * D2 + ap] = c;
        sin_t[tk * D2 + ap] = s;
      }
    __syncthreads();  // (the other half is rewritten only after the next one)

    int tok = 0, head = grp;  // item of this group: token t0 + tok, head h0 + head
    while (head >= nh) { head -= nh; ++tok; }
    while (tok < nt) {
      float v[UN][IT][2 * V];
      int it_tok[UN];
      bool it_q[UN];
      uint8_t* dst[UN];
#pragma unroll
      for (int u = 0; u < UN; ++u) {
        const bool valid = tok < nt;
        const int hd = h0 + head;
        const bool isq = hd < a.q.heads;
        it_tok[u] = valid ? tok : -1;
        it_q[u] = isq;
        const int hh = isq ? hd : hd - a.q.heads;
        const int64_t tt = t0 + tok;
        const uint8_t* src = static_cast<const uint8_t*>(isq ? a.q.x : a.k.x) +
                             (tt * (isq ? a.q.ts : a.k.ts) + hh * (isq ? a.q.hs : a.k.hs)) * ES;
        dst[u] = static_cast<uint8_t*>(isq ? a.q.y : a.k.y) +
                 (tt * (isq ? a.q.yts : a.k.yts) + hh * (isq ? a.q.yhs : a.k.yhs)) * ES;
        if constexpr (STAGED) {
          if (valid && has_chunk) *reinterpret_cast<u32x4_t*>(row + 16 * gl) = *reinterpret_cast<const u32x4_a2*>(src + 16 * gl);
          wave_lds_sync();
          src = row;
        }
#pragma unroll
        for (int c = 0; c < IT; ++c) {
#pragma unroll
          for (int i = 0; i < 2 * V; ++i) v[u][c][i] = 0.0f;
          if (valid && in[c]) {
            if constexpr (INTER) {
              load_n<DT, 2 * V>(src + e0[c] * ES, v[u][c]);
            } else {
              load_n<DT, V>(src + e0[c] * ES, v[u][c]);
              load_n<DT, V>(src + e1[c] * ES, v[u][c] + V);
            }
          }
        }
        head += ng;
        while (head >= nh) { head -= nh; ++tok; }
      }
#pragma unroll
      for (int u = 0; u < UN; ++u) {
        float r = 1.0f;
        if (a.norm) {
          float s = 0.0f;
#pragma unroll
          for (int c = 0; c < IT; ++c)
#pragma unroll
            for (int i = 0; i < 2 * V; ++i) s = fmaf(v[u][c][i], v[u][c][i], s);
          s = group_sum(s, G);
          r = rsqrtf(fmaf(s, a.inv_d, a.eps));
        }
        if (it_tok[u] < 0) continue;
#pragma unroll
        for (int c = 0; c < IT; ++c) {
          if (!in[c]) continue;
          float o[2 * V];
#pragma unroll
          for (int i = 0; i < 2 * V; ++i) o[i] = a.norm ? (v[u][c][i] * r) * (it_q[u] ? wq[c][i] : wk[c][i]) : v[u][c][i];
          const int at = it_tok[u] * D2 + (gl + c * G) * V;
          float cs[V], sn[V];
          if constexpr (V == 4) {
            const float4_t cc = *reinterpret_cast<const float4_t*>(cos_t + at);
            const float4_t ss = *reinterpret_cast<const float4_t*>(sin_t + at);
#pragma unroll
            for (int i = 0; i < 4; ++i) { cs[i] = cc[i]; sn[i] = ss[i]; }
          } else {
            cs[0] = cos_t[at];
            sn[0] = sin_t[at];
          }
          // pairs of this chunk: (o[i0], o[i1]).  Elements past the span are kept, not turned by an angle of 0:
          // an infinity times the sine 0 would be a NaN in its neighbour.
#pragma unroll
          for (int i = 0; i < V; ++i) {
            const int i0 = INTER ? 2 * i : i, i1 = INTER ? 2 * i + 1 : V + i;
            const bool turn = (gl + c * G) * V + i < a.rot2;
            const float x0 = o[i0], x1 = o[i1];
            o[i0] = turn ? fmaf(x0, cs[i], -(x1 * sn[i])) : x0;
            o[i1] = turn ? fmaf(x0, sn[i], x1 * cs[i]) : x1;
          }
          if constexpr (INTER) {
            store_n<DT, 2 * V>(dst[u] + e0[c] * ES, o);
          } else {
            uint8_t* to = STAGED ? row : dst[u];
            store_n<DT, V>(to + e0[c] * ES, o);
            store_n<DT, V>(to + e1[c] * ES, o + V);
          }
        }
        if constexpr (STAGED) {
          wave_lds_sync();
          if (has_chunk)
            __builtin_nontemporal_store(*reinterpret_cast<const u32x4_t*>(row + 16 * gl),
                                        reinterpret_cast<u32x4_a2*>(dst[u] + 16 * gl));
          wave_lds_sync();  // the row is written again
        }
      }
    }
  }
}

template <int DT, int V, bool INTER, int IT, int UN, bool STAGED>
hipError_t run(const RopeArgs& a, hipStream_t st) {
  const int heads = a.q.heads + a.k.heads;
  const int64_t blocks = ((int64_t)a.tokens + a.tb - 1) / a.tb;
  const dim3 grid((unsigned)(blocks < MAX_WGS ? blocks : MAX_WGS), (unsigned)((heads + a.hb - 1) / a.hb));
  const size_t lds = 2 * (size_t)a.tb * a.D * sizeof(float) + (STAGED ? (size_t)(RT >> a.log2g) * row_stride(a.D) : 0);
  qk_norm_rope_kernel<DT, V, INTER, IT, UN, STAGED><<<grid, RT, lds, st>>>(a);
  return hipGetLastError();
}

template <int DT>
hipError_t run_dt(RopeArgs a, bool vec, bool staged, hipStream_t st) {
  // Element-wise heads: 4 pairs per lane, in f32 with 49 to 64 of them 2 of 2 items (8000 tokens of 48 heads of 128,
  // halves of axes of 44, 42 and 42, f32: 94 us with 2, 105 with 4; of 66, f32: 74 and 64; 40 heads of 126, bf16: 68
  // and 67; 48 heads of 34, f16: 29 and 24).
  const bool two = DT == 2 && !vec && a.D > 96 && a.D <= 128;
  const int lanes = vec ? a.D / 8 : two ? (a.D / 2 + 1) / 2 : (a.D / 2 + 3) / 4;
  a.log2g = 0;
  while ((1 << a.log2g) < lanes) ++a.log2g;
  const int ng = RT >> a.log2g, heads = a.q.heads + a.k.heads;
  a.log2p = 0;
  while ((1 << a.log2p) < a.D / 2) ++a.log2p;
  // few tokens: one pass per workgroup, heads split over workgroups; many: several tokens each
  a.hb = a.tokens < 512 && heads > ng ? ng : heads;
  // tokens per pass: about six items for every lane group, so that a pass is worth its angles and its barrier
  const int64_t per = ((int64_t)a.tokens + MAX_WGS - 1) / MAX_WGS;  // (fewer where not every workgroup has a pass)
  const int full = heads > 0 ? 6 * ng / heads : 1;
  a.tb = full < 1 ? 1 : full > 8 ? 8 : full;
  if (per < a.tb) a.tb = (int)per;
  if (vec) return a.layout == 0 ? run<DT, 4, true, 1, 2, false>(a, st) : run<DT, 4, false, 1, 2, false>(a, st);
  if constexpr (DT == 2) {
    if (two) return run<DT, 1, false, 2, 2, false>(a, st);
  } else {
    if (staged) return run<DT, 1, false, 4, 1, true>(a, st);
  }
  return run<DT, 1, false, 4, 1, false>(a, st);
}

}  // namespace

hipError_t launch_qk_norm_rope(RopeArgs a, int dtype, hipStream_t stream) {
  // 4-pair vectors need whole 8-element chunks of the head, and in the split layouts whole chunks of 4 pairs in
  // the span and in every slice
  bool vec = a.D % 8 == 0;
  if (a.layout == 1) vec = vec && a.rot2 % 4 == 0;
  if (a.layout == 2)
    for (int x = 0; x < a.axes; ++x) vec = vec && a.start[x + 1] % 4 == 0;
  // (16-bit types; one token of 40 heads: 5.1 us, element by element 4.6; 300 tokens: 6.6 and 7.2)
  const bool staged = a.D % 8 == 0 && !vec;
  switch (dtype) {
    case 0: return run_dt<0>(a, vec, staged, stream);
    case 1: return run_dt<1>(a, vec, staged, stream);
    default: return run_dt<2>(a, vec, staged, stream);
  }
}

}  // namespace w4a4
