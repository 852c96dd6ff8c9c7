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

// A head held by neighbouring lanes, chunk g (8 dimensions) in each: the chunk
// turned by the table's row `cs` (a shared 16-byte aligned row of cosines and
// sines).  Every lane of the warp calls it; `on`: the lane holds something.
__device__ __forceinline__ uint4 turn_chunk(const RopeView& r, const uint4& x, const float* cs, int g, int lane, bool on) {
  if (r.dims == 0) return x;
  const float* sn = cs + r.dims / 2;
  if (r.inter) {
    if (!on || 8 * g >= r.dims) return x;
    return turn_pairs<true>(x, __ldg(reinterpret_cast<const float4*>(cs) + g),
                            __ldg(reinterpret_cast<const float4*>(sn) + g));
  }
  const int m = r.dims / 16;  // chunks of a half
  const int from = g < m ? lane + m : g < 2 * m ? lane - m : lane;
  uint4 y;
#pragma unroll
  for (int e = 0; e < 4; ++e) (&y.x)[e] = __shfl_sync(0xffffffffu, (&x.x)[e], from);
  if (!on || g >= 2 * m) return x;
  const int j = g < m ? g : g - m;
  float4 c[2], s[2];
#pragma unroll
  for (int e = 0; e < 2; ++e) {
    c[e] = __ldg(reinterpret_cast<const float4*>(cs) + 2 * j + e);
    s[e] = __ldg(reinterpret_cast<const float4*>(sn) + 2 * j + e);
  }
  return turn_half<true>(x, y, c, s, g < m ? -1.f : 1.f);
}

__device__ __forceinline__ int pow2_at_least(int x) { return x <= 1 ? 1 : 1 << (32 - __clz(x - 1)); }

// `heads` heads of D dimensions turned by one row of the table, by a group of
// lanes: lane `lane` of `lanes` (a power of two, at least D / 8).  `in` and
// `out` may be the same heads.
template <bool kInter>
__device__ __forceinline__ void turn_heads(const __nv_bfloat16* in, __nv_bfloat16* out, int heads, int D, int dims,
                                           const float* cs, float dir, int lane, int lanes) {
  constexpr int kU = 4;
  const float* sn = cs + dims / 2;
  const int chunks = kInter ? dims / 8 : dims / 16;  // what a head has for a lane each
  const int n = pow2_at_least(chunks);
  const int j = lane & (n - 1), step = lanes / n;
  if (j < chunks) {
    constexpr int kV = kInter ? 1 : 2;
    float4 c[kV], s[kV];
#pragma unroll
    for (int e = 0; e < kV; ++e) {
      c[e] = __ldg(reinterpret_cast<const float4*>(cs) + kV * j + e);
      s[e] = __ldg(reinterpret_cast<const float4*>(sn) + kV * j + e);
      s[e] = make_float4(dir * s[e].x, dir * s[e].y, dir * s[e].z, dir * s[e].w);
    }
    for (int h0 = lane / n; h0 < heads; h0 += kU * step) {
      uint4 x[kU], y[kU];
#pragma unroll
      for (int u = 0; u < kU; ++u) {
        const int h = h0 + u * step;
        if (h < heads) {
          x[u] = *reinterpret_cast<const uint4*>(in + h * D + 8 * j);
          if (!kInter) y[u] = *reinterpret_cast<const uint4*>(in + h * D + dims / 2 + 8 * j);
        }
      }
#pragma unroll
      for (int u = 0; u < kU; ++u) {
        const int h = h0 + u * step;
        if (h >= heads) continue;
        if (kInter) {
          *reinterpret_cast<uint4*>(out + h * D + 8 * j) = turn_pairs<false>(x[u], c[0], s[0]);
        } else if constexpr (!kInter) {
          *reinterpret_cast<uint4*>(out + h * D + 8 * j) = turn_half<false>(x[u], y[u], c, s, -1.f);
          *reinterpret_cast<uint4*>(out + h * D + dims / 2 + 8 * j) = turn_half<false>(y[u], x[u], c, s, 1.f);
        }
      }
    }
  }
  // the dimensions that are not turned
  const int rest = (D - dims) / 8;
  if (rest > 0 && in != out)
    for (int e = lane; e < heads * rest; e += lanes) {
      const int at = e / rest * D + dims + e % rest * 8;
      *reinterpret_cast<uint4*>(out + at) = *reinterpret_cast<const uint4*>(in + at);
    }
}

}  // namespace dsa
