// rope.cuh -- turning heads by their position: pair j of a row at position p,
// with c = cos_sin[p][j] and s = cos_sin[p][R / 2 + j], becomes
//   (a c - b s, b c + a s);
// pairs are (j, j + R/2), or (2j, 2j + 1) when interleaved.
#pragma once

#include "dsa_device.cuh"
#include "rope_kernels.h"

namespace dsa {

__device__ __forceinline__ float bf_lo(uint32_t w) { return __uint_as_float(w << 16); }
__device__ __forceinline__ float bf_hi(uint32_t w) { return __uint_as_float(w & 0xFFFF0000u); }
__device__ __forceinline__ uint4 ld_row(const __nv_bfloat16* p) { return __ldg(reinterpret_cast<const uint4*>(p)); }

// x c + y s, two roundings (of y s, and of the sum).
__device__ __forceinline__ float turn_quick(float x, float c, float y, float s) {
  return __fmaf_rn(x, c, __fmul_rn(y, s));
}
// x c + y s, correctly rounded but for sums within 2^-45 of a border: both
// products with their remainders (Dekker's two-product by FMA), their sum with
// its own (Knuth's two-sum).  A key's 4-bit code then hangs on its value, not on
// the order of the operations.
__device__ __forceinline__ float turn_exact(float x, float c, float y, float s) {
  const float p = __fmul_rn(x, c), q = __fmul_rn(y, s);
  const float e = __fmaf_rn(x, c, -p), f = __fmaf_rn(y, s, -q);
  const float h = __fadd_rn(p, q), t = __fsub_rn(h, p);
  const float g = __fadd_rn(__fsub_rn(p, __fsub_rn(h, t)), __fsub_rn(q, t));
  const float r = __fadd_rn(h, __fadd_rn(g, __fadd_rn(e, f)));
  return fabsf(h) < INFINITY ? r : h;  // an infinity has no remainder
}
template <bool kExact>
__device__ __forceinline__ float turn(float x, float c, float y, float s) {
  return kExact ? turn_exact(x, c, y, s) : turn_quick(x, c, y, s);
}

// Four interleaved pairs of a 16-byte chunk.
template <bool kExact>
__device__ __forceinline__ uint4 turn_pairs(const uint4& x, const float4& c, const float4& s) {
  uint4 y;
#pragma unroll
  for (int e = 0; e < 4; ++e) {
    const uint32_t w = (&x.x)[e];
    const float a = bf_lo(w), b = bf_hi(w), ce = (&c.x)[e], se = (&s.x)[e];
    (&y.x)[e] = pack_bf16(turn<kExact>(a, ce, b, -se), turn<kExact>(b, ce, a, se));
  }
  return y;
}
// Eight elements x of one half, their partners y, and the partners' sign: x c +
// sg y s (sg = -1 in the lower half, +1 in the upper).
template <bool kExact>
__device__ __forceinline__ uint4 turn_half(const uint4& x, const uint4& y, const float4 (&c)[2], const float4 (&s)[2],
                                           float sg) {
  uint4 z;
#pragma unroll
  for (int e = 0; e < 4; ++e) {
    const uint32_t w = (&x.x)[e], v = (&y.x)[e];
    const float c0 = (&c[e >> 1].x)[2 * (e & 1)], c1 = (&c[e >> 1].x)[2 * (e & 1) + 1];
    const float s0 = (&s[e >> 1].x)[2 * (e & 1)], s1 = (&s[e >> 1].x)[2 * (e & 1) + 1];
    (&z.x)[e] = pack_bf16(turn<kExact>(bf_lo(w), c0, bf_lo(v), sg * s0), turn<kExact>(bf_hi(w), c1, bf_hi(v), sg * s1));
  }
  return z;
}

// A head held by neighbouring lanes, chunk g (8 dimensions) in each: the cosines
// and sines that the chunk needs of the table's row `cs`.
struct RopeChunk {
  float4 c[2], s[2];
};
__device__ __forceinline__ RopeChunk rope_chunk(const RopeView& r, const float* cs, int g, bool on) {
  RopeChunk x = {};
  if (!on || 8 * g >= r.dims) return x;  // (also where there is no rotation)
  const int m = r.dims / 16, j = r.inter ? g : 2 * (g < m ? g : g - m);
  const float4* c = reinterpret_cast<const float4*>(cs) + j;
  const float4* s = reinterpret_cast<const float4*>(cs + r.dims / 2) + j;
  x.c[0] = __ldg(c);
  x.s[0] = __ldg(s);
  if (!r.inter) {
    x.c[1] = __ldg(c + 1);
    x.s[1] = __ldg(s + 1);
  }
  return x;
}
// The chunk turned.  Every lane of the warp calls it; `on`: the lane holds
// something.
__device__ __forceinline__ uint4 turn_chunk(const RopeView& r, const uint4& x, const RopeChunk& t, int g, int lane, bool on) {
  if (r.dims == 0) return x;
  if (r.inter) return !on || 8 * g >= r.dims ? x : turn_pairs<true>(x, t.c[0], t.s[0]);
  const int m = r.dims / 16;  // chunks of a half
  const int from = g < m ? lane + m : g < 2 * m ? lane - m : lane;
  uint4 y;
#pragma unroll
  for (int e = 0; e < 4; ++e) (&y.x)[e] = __shfl_sync(0xffffffffu, (&x.x)[e], from);
  if (!on || g >= 2 * m) return x;
  return turn_half<true>(x, y, t.c, t.s, g < m ? -1.f : 1.f);
}

// Lanes that a head's chunks take: a power of two.
__host__ __device__ inline int rope_chunk_lanes(int dims, bool inter) {
  const int chunks = inter ? dims / 8 : dims / 16;
  int n = 1;
  while (n < chunks) n *= 2;
  return n;
}

// `heads` heads of D dimensions turned by one row of the table, by a group of
// lanes: lane `lane` of `lanes` (a power of two, at least n = rope_chunk_lanes).
// `row()` says which row (null: none, and nothing is written); it is asked after
// the first heads have been asked for, so that looking up a position costs no time
// of its own.  `sure()` is asked after the table's row has been asked for: false,
// and nothing is written either.  `in` and `out` may be the same heads.
template <bool kInter, typename Row, typename Sure>
__device__ __forceinline__ void turn_heads(const __nv_bfloat16* in, __nv_bfloat16* out, int heads, int D, int dims, int n,
                                           float dir, int lane, int lanes, Row&& row, Sure&& sure) {
  constexpr int kU = kInter ? 4 : 2;  // heads under way: four 16-byte loads a lane
  const int chunks = kInter ? dims / 8 : dims / 16;  // what a head has for a lane each
  const int j = lane & (n - 1), step = lanes / n;
  uint4 x[kU], y[kU];
  const auto load = [&](int h0) {
#pragma unroll
    for (int u = 0; u < kU; ++u) {
      const int h = h0 + u * step;
      if (h < heads && j < chunks) {
        x[u] = *reinterpret_cast<const uint4*>(in + h * D + 8 * j);
        if (!kInter) y[u] = *reinterpret_cast<const uint4*>(in + h * D + dims / 2 + 8 * j);
      }
    }
  };
  int h0 = lane / n;
  load(h0);
  const float* cs = row();
  if (cs == nullptr) return;
  const float* sn = cs + dims / 2;
  constexpr int kV = kInter ? 1 : 2;
  float4 c[kV], s[kV];
  if (j < chunks) {
#pragma unroll
    for (int e = 0; e < kV; ++e) {
      c[e] = __ldg(reinterpret_cast<const float4*>(cs) + kV * j + e);
      s[e] = __ldg(reinterpret_cast<const float4*>(sn) + kV * j + e);
    }
  }
  if (!sure()) return;
  if (j < chunks) {
    while (h0 < heads) {
#pragma unroll
      for (int u = 0; u < kU; ++u) {
        const int h = h0 + u * step;
        if (h >= heads) continue;
        if constexpr (kInter) {
          const float4 t = make_float4(dir * s[0].x, dir * s[0].y, dir * s[0].z, dir * s[0].w);
          *reinterpret_cast<uint4*>(out + h * D + 8 * j) = turn_pairs<false>(x[u], c[0], t);
        } else {
          *reinterpret_cast<uint4*>(out + h * D + 8 * j) = turn_half<false>(x[u], y[u], c, s, -dir);
          *reinterpret_cast<uint4*>(out + h * D + dims / 2 + 8 * j) = turn_half<false>(y[u], x[u], c, s, dir);
        }
      }
      h0 += kU * step;
      load(h0);
    }
  }
  // the dimensions that are not turned
  const int rest = (D - dims) / 8, all = heads * rest;
  if (all > 0 && in != out)
    for (int e0 = lane; e0 < all; e0 += 4 * lanes) {
      uint4 x[4];
      int at[4];
#pragma unroll
      for (int u = 0; u < 4; ++u) {
        const int e = e0 + u * lanes;
        at[u] = e / rest * D + dims + e % rest * 8;
        if (e < all) x[u] = *reinterpret_cast<const uint4*>(in + at[u]);
      }
#pragma unroll
      for (int u = 0; u < 4; ++u)
        if (e0 + u * lanes < all) *reinterpret_cast<uint4*>(out + at[u]) = x[u];
    }
}

}  // namespace dsa
