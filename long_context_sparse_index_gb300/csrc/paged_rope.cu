// paged_rope.cu -- new tokens into a paged cache with their keys turned by their
// positions on the way, into bf16 pages or into pages of 4 bits, and the step's
// queries turned with them; and the rows of a 4-bit cache read back.
//
// What the cache holds is what would be appended had the caller turned the keys
// before: k and k_idx turned in fp32 (correctly rounded, rope.cuh) and rounded to
// bf16; the pooled key is the mean of the four turned bf16 keys; the 4-bit codes
// are those of the turned bf16 key (kv4.cuh).
//
// One launch.  Warps of some blocks append kRows rows each, keys and values in
// one block, indexer keys in the next: 16 lanes hold a row's key and 16 its value,
// 16 B a lane; 8 lanes hold an indexer key.  The other blocks' warps turn a row's
// heads each, 4 KB for 16 heads of 128 or 32 of 64 in two passes, each with all its
// loads before its first store.
// Few rows are bound by the chain offsets -> page and the table's row -> store;
// many by memory (9815 rows with 48 query heads: 30.5 us, 5.95 TB/s).  Asking for
// all offsets and for the page before a query is written costs 64 rows 2.7 us
// instead of 2.5, and 9815 rows 0.5 us.  A warp for keys, values and indexer keys
// together needs more registers and twice the chain (measured without that: 64 rows
// 2.8 us instead of 2.5, in 4 bits 3.2 instead of 2.5; 9815 rows 31.8 instead of
// 30.0).
#include "kv4.cuh"
#include "paged.cuh"
#include "paged_rope_kernels.h"
#include "rope.cuh"

namespace dsa {
namespace {

constexpr int kD = 128;
constexpr int kDi = 64;
constexpr int kWarps = 4;

// The pooled key's chunk of eight dimensions from the four tokens' chunks: hi
// and lo of the fp32 mean.
__device__ __forceinline__ void pooled(const uint4 (&four)[4], uint4* hi, uint4* lo) {
#pragma unroll
  for (int e = 0; e < 4; ++e) {
    float kh[2];
#pragma unroll
    for (int z = 0; z < 2; ++z) {
      float y[4];
#pragma unroll
      for (int t = 0; t < 4; ++t) y[t] = z ? bf_hi((&four[t].x)[e]) : bf_lo((&four[t].x)[e]);
      kh[z] = __fmul_rn(__fadd_rn(__fadd_rn(y[0], y[1]), __fadd_rn(y[2], y[3])), 0.25f);
    }
    const uint32_t h = pack_bf16(kh[0], kh[1]);
    (&hi->x)[e] = h;
    (&lo->x)[e] = pack_bf16(__fsub_rn(kh[0], bf_lo(h)), __fsub_rn(kh[1], bf_hi(h)));
  }
}

// A row's key or value, eight dimensions a lane (16 lanes), to the places of
// token t of the pool at `pool`.  Neighbouring lanes hold a group.
__device__ __forceinline__ void store4(uint8_t* pool, int t, const uint4& x, int lane, bool key, bool on) {
  const int ch = lane & 15;
  float f[8];
#pragma unroll
  for (int e = 0; e < 4; ++e) {
    f[2 * e] = bf_lo((&x.x)[e]);
    f[2 * e + 1] = bf_hi((&x.x)[e]);
  }
  float top = 0.f;
  bool odd = false;  // an infinity or a NaN
#pragma unroll
  for (int e = 0; e < 8; ++e) {
    odd |= !(fabsf(f[e]) < INFINITY);
    top = fmaxf(top, fabsf(f[e]));
  }
  top = fmaxf(top, __shfl_xor_sync(0xffffffffu, top, 1));
  const unsigned any = __ballot_sync(0xffffffffu, odd);
  odd = (any >> (lane & 30)) & 3u;
  const uint32_t bits = odd ? kScaleNan : scale4_of(top);
  const uint32_t w = codes4(f, odd ? 0.f : scale4(bits));
  if (!on) return;
  *reinterpret_cast<uint32_t*>(pool + (key ? k4_code_at(t, 8 * ch) : v4_code_at(t, 8 * ch))) = w;
  if ((ch & 1) == 0) pool[key ? k4_scale_at(t, ch / 2) : v4_scale_at(t, ch / 2)] = static_cast<uint8_t>(bits);
}

// A row's key or value into the cache.
template <bool kFour>
__device__ __forceinline__ void store_row(const CacheView& c, int page, int off, const uint4& x, int lane, bool key) {
  if (kFour) {
    uint8_t* const pool =
        reinterpret_cast<uint8_t*>(c.k + static_cast<int64_t>(page < 0 ? 0 : page) * c.k_stride) + (off >> 2) * kPool4Bytes;
    store4(pool, off & 3, x, lane, key, page >= 0);
  } else if (page >= 0) {
    __nv_bfloat16* dst = key ? c.k + page * c.k_stride : c.v + page * c.v_stride;
    reinterpret_cast<uint4*>(dst + off * kD)[lane & 15] = x;
  }
}

// Rows r0 .. r0 + kRows - 1 (of one warp): their keys and values, or their indexer
// keys.  Keys and values take 16 lanes each: a row's key and value side by side, or
// two rows' keys and then two rows' values.
template <int kRows, bool kFour, bool kKv>
__device__ __forceinline__ void append_rows(const CacheView& c, const BatchView& b, const RopeAppendArgs& x, int64_t r0,
                                            int lane, unsigned* status) {
  constexpr bool kIdx = !kKv;
  const AppendArgs& a = x.a;
  // the rows' sequences: one walk over the offsets; lanes 8u .. 8u + 7 work out
  // row r0 + u (of a single row: every lane)
  const int mine = kRows == 4 ? lane >> 3 : 0;
  const int64_t row = r0 + mine;
  // The rows are asked for before their places are known.
  constexpr int kP = kRows == 4 ? 2 : 1;  // passes
  const int half = lane >> 4, ch = lane & 15, g = lane & 7, tok = lane >> 3;
  const __nv_bfloat16* const idx = a.k_idx + 8 * g;
  uint4 kx[kP], vx[kP], own = make_uint4(0u, 0u, 0u, 0u);
#pragma unroll
  for (int p = 0; p < kP; ++p) {
    kx[p] = vx[p] = make_uint4(0u, 0u, 0u, 0u);
    const int64_t r = r0 + (kRows == 4 ? 2 * p + half : 0);
    if (kKv && kRows == 4 && r < b.rows) vx[p] = ld_row(a.v + r * a.v_stride + 8 * ch);
    if (kKv && r < b.rows) kx[p] = ld_row((kRows == 1 && half ? a.v + r * a.v_stride : a.k + r * a.k_stride) + 8 * ch);
  }
  if (kIdx && row < b.rows) own = ld_row(idx + row * a.kidx_stride);
  int page = -1, older = 0;  // older: how many of the pool's tokens come before the call's rows
  int64_t pos = 0;
  bool astray = a.reserved != nullptr && __ldg(a.reserved) < 0;
  for (int j0 = 0; j0 < b.batch; j0 += 32) {
    const int j = j0 + lane;
    int c0 = 0, c1 = 0, len = 0;
    if (j < b.batch) {
      c0 = __ldg(b.cu + j);
      c1 = __ldg(b.cu + j + 1);
      len = __ldg(b.lens + j);
      astray |= c0 < 0 || c1 < c0 || c1 > b.rows;
    }
    int src = -1;
#pragma unroll
    for (int u = 0; u < kRows; ++u) {
      const unsigned hit =
          __ballot_sync(0xffffffffu, j < b.batch && c0 <= r0 + u && r0 + u < c1 && r0 + u < b.rows);
      if (mine == u && hit != 0u) src = __ffs(hit) - 1;
    }
    const int64_t first = __shfl_sync(0xffffffffu, c0, src & 31), last = __shfl_sync(0xffffffffu, c1, src & 31);
    const int64_t n = __shfl_sync(0xffffffffu, len, src & 31);
    if (src >= 0) {
      const int64_t before = row - first;
      pos = n - last + row;
      if (pos < before || n > (static_cast<int64_t>(b.max_pages) << c.shift) ||
          (x.rope.dims != 0 && pos >= x.rope.positions) || (x.rope_idx.dims != 0 && pos >= x.rope_idx.positions)) {
        record_status(status, kStatusInternal);
      } else {
        page = page_of(b, c.num_pages, j0 + src, static_cast<int>(pos >> c.shift), status);
        older = static_cast<int>(before < 3 ? 3 - before : 0);
      }
    }
  }
  // Then no row's position is sure, and what it would overwrite may be a live
  // token: nothing is written.  (Every warp has seen all offsets.)
  if (__any_sync(0xffffffffu, astray)) {
    if (lane == 0) record_status(status, kStatusInternal);
    return;
  }
  const int mask = (1 << c.shift) - 1;
  const int off = static_cast<int>(pos & mask);
  int pg[kP], of[kP];
  RopeChunk kt[kP];
#pragma unroll
  for (int p = 0; kKv && p < kP; ++p) {
    const int from = kRows == 4 ? 8 * (2 * p + half) : 0;
    pg[p] = __shfl_sync(0xffffffffu, page, from);
    const int64_t at = __shfl_sync(0xffffffffu, pos, from);
    of[p] = static_cast<int>(at & mask);
    kt[p] = rope_chunk(x.rope, x.rope.cs + at * x.rope.stride, ch, pg[p] >= 0 && (kRows == 4 || half == 0));
  }
  // Indexer keys: lanes 8u .. 8u + 7 row r0 + u, and then, for each row that
  // completes a pool, lanes 8t .. 8t + 7 the pool's token t.  (A single row's own
  // lanes are those of its token.)
  const float* const ci = x.rope_idx.cs;
  const int64_t si = x.rope_idx.stride;
  const bool ends = page >= 0 && (off & 3) == 3;
  if (kIdx && kRows == 4) {
    own = turn_chunk(x.rope_idx, own, rope_chunk(x.rope_idx, ci + pos * si, g, page >= 0), g, lane, page >= 0);
    if (page >= 0) *reinterpret_cast<uint4*>(c.k_idx + page * c.kidx_stride + off * kDi + 8 * g) = own;
  }
  unsigned todo = !kIdx ? 0u : kRows == 4 ? __ballot_sync(0xffffffffu, ends && g == 0) : 1u;
  while (todo != 0u) {
    const int src = __ffs(todo) - 1;  // a lane of the row
    todo &= todo - 1;
    const int e_page = __shfl_sync(0xffffffffu, page, src), e_off = __shfl_sync(0xffffffffu, off, src);
    const int e_older = __shfl_sync(0xffffffffu, older, src);
    const int64_t e_pos = __shfl_sync(0xffffffffu, pos, src), e_row = r0 + (kRows == 4 ? src >> 3 : 0);
    const bool whole = kRows == 4 || ends;
    const int t0 = e_off & 3;  // the row's place in its pool
    const bool me = e_page >= 0 && tok == t0, call = me || (whole && tok >= e_older);
    uint4 y = make_uint4(0u, 0u, 0u, 0u);
    __nv_bfloat16* const pidx = c.k_idx + static_cast<int64_t>(e_page < 0 ? 0 : e_page) * c.kidx_stride + 8 * g;
    bool here = false;  // the warp's own rows have been turned
    if (kRows == 4) {
      const int in = (src >> 3) - 3 + tok;
      here = call && in >= 0;
#pragma unroll
      for (int e = 0; e < 4; ++e) {
        const uint32_t w = __shfl_sync(0xffffffffu, (&own.x)[e], 8 * (in & 3) + g);
        if (here) (&y.x)[e] = w;
      }
    } else if (me) {
      y = own;
    }
    const bool load = call && !here;
    if (load && (kRows == 4 || !me)) y = ld_row(idx + (e_row - t0 + tok) * a.kidx_stride);
    if (whole && !call) y = *reinterpret_cast<const uint4*>(pidx + (e_off - 3 + tok) * kDi);
    if (__any_sync(0xffffffffu, load)) {
      const uint4 z = turn_chunk(x.rope_idx, y, rope_chunk(x.rope_idx, ci + (e_pos - t0 + tok) * si, g, load), g, lane, load);
      if (load) y = z;
    }
    if (kRows == 1 && me) *reinterpret_cast<uint4*>(pidx + e_off * kDi) = y;
    if (kRows == 1 && !__any_sync(0xffffffffu, whole)) break;
    uint4 four[4], hi, lo;
#pragma unroll
    for (int t = 0; t < 4; ++t)
#pragma unroll
      for (int e = 0; e < 4; ++e) (&four[t].x)[e] = __shfl_sync(0xffffffffu, (&y.x)[e], 8 * t + g);
    pooled(four, &hi, &lo);
    uint4* to =
        reinterpret_cast<uint4*>(c.khat + static_cast<int64_t>(e_page) * c.khat_stride + (e_off >> 2) * (2 * kDi)) + g;
    if (tok == 0) to[0] = hi;
    if (tok == 1) to[8] = lo;
  }
#pragma unroll
  for (int p = 0; kKv && p < kP; ++p) {
    const uint4 y = turn_chunk(x.rope, kx[p], kt[p], ch, lane, pg[p] >= 0 && (kRows == 4 || half == 0));
    if (kRows == 4 || half == 0) kx[p] = y;
    store_row<kFour>(c, pg[p], of[p], kx[p], lane, kRows == 4 || half == 0);
    if (kRows == 4) store_row<kFour>(c, pg[p], of[p], vx[p], lane, false);
  }
}

// A row of the queries (or of the indexer's), a warp's work.  It is turned where
// append_rows appends it, by the same conditions, so that a step that is repeated
// after an error turns no query in place twice; append_rows records what is wrong.
__device__ __forceinline__ void turn_queries(const CacheView& c, const BatchView& b, const RopeAppendArgs& x,
                                             const RopeView& r, const QueryRows& q, int D, int64_t row, int lane) {
  int page = -1;
  const auto find = [&]() -> const float* {
    if (x.a.reserved != nullptr && __ldg(x.a.reserved) < 0) return nullptr;
    bool astray;
    const RowAt at = warp_locate<true>(b, c.shift, row, lane, nullptr, &astray);
    if (astray || at.seq < 0 || at.pos < 0 || (x.rope.dims != 0 && at.pos >= x.rope.positions) ||
        (x.rope_idx.dims != 0 && at.pos >= x.rope_idx.positions))
      return nullptr;
    page = __ldg(b.table + at.seq * b.table_stride + (at.pos >> c.shift));
    return r.cs + at.pos * r.stride;
  };
  const auto sure = [&] { return static_cast<unsigned>(page) < static_cast<unsigned>(c.num_pages); };
  const __nv_bfloat16* in = q.in + row * q.in_stride;
  __nv_bfloat16* out = q.out + row * q.out_stride;
  const int n = rope_chunk_lanes(r.dims, r.inter);
  if (r.inter) turn_heads<true>(in, out, q.heads, D, r.dims, n, 1.f, lane, 32, find, sure);
  else turn_heads<false>(in, out, q.heads, D, r.dims, n, 1.f, lane, 32, find, sure);
}

template <int kRows, bool kFour>
__global__ void __launch_bounds__(32 * kWarps, kRows == 4 ? 8 : 7)
    append_rope_kernel(const CacheView c, const BatchView b, const RopeAppendArgs x, unsigned append_blocks, unsigned apart,
                       unsigned* status) {
  pdl_wait();  // launched early: what stands before in the stream has ended
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  // Blocks that append: the first ones, or of many rows every apart-th as long as
  // there are some, so that their chains run beside the queries' copies (9815 rows
  // 0.5 us less than with the appends first).
  unsigned nth = blockIdx.x;
  bool appends = nth < append_blocks;
  if constexpr (kRows == 4) {
    nth = blockIdx.x / apart;
    appends = blockIdx.x % apart == 0 && nth < append_blocks;
  }
  if (appends) {
    const int64_t r0 = (static_cast<int64_t>(nth >> 1) * kWarps + warp) * kRows;
    if (r0 >= b.rows) return;
    if (nth & 1) append_rows<kRows, kFour, true>(c, b, x, r0, lane, status);
    else append_rows<kRows, kFour, false>(c, b, x, r0, lane, status);
    return;
  }
  const unsigned before = kRows == 4 ? min(append_blocks, nth + 1) : append_blocks;
  int64_t w = static_cast<int64_t>(blockIdx.x - before) * kWarps + warp;
  if (x.q.heads > 0) {
    if (w < b.rows) return turn_queries(c, b, x, x.rope, x.q, kD, w, lane);
    w -= b.rows;
  }
  if (x.qi.heads > 0 && w < b.rows) turn_queries(c, b, x, x.rope_idx, x.qi, kDi, w, lane);
}

// ----------------------------------------------------------------- reading back
// A warp per row: 16 lanes its key and 16 its value, a word of codes each.
__global__ void __launch_bounds__(32 * kWarps)
    cache4_read_kernel(const CacheView c, const BatchView b, __nv_bfloat16* __restrict__ k, __nv_bfloat16* __restrict__ v,
                       int64_t k_stride, int64_t v_stride, unsigned* status) {
  pdl_wait();  // launched early: what stands before in the stream has ended
  const int lane = threadIdx.x & 31;
  const int64_t row = static_cast<int64_t>(blockIdx.x) * kWarps + (threadIdx.x >> 5);
  if (row >= b.rows) return;
  const RowAt at = warp_locate(b, c.shift, row, lane, status);
  if (at.seq < 0 || at.pos < 0) return;
  const int page = page_of(b, c.num_pages, at.seq, static_cast<int>(at.pos >> c.shift), lane == 0 ? status : nullptr);
  if (page < 0) return;
  const int off = static_cast<int>(at.pos & ((1 << c.shift) - 1)), t = off & 3, ch = lane & 15;
  const uint8_t* pool = reinterpret_cast<const uint8_t*>(c.k + page * c.k_stride) + (off >> 2) * kPool4Bytes;
  const bool key = lane < 16;
  const uint32_t w = *reinterpret_cast<const uint32_t*>(pool + (key ? k4_code_at(t, 8 * ch) : v4_code_at(t, 8 * ch)));
  const uint32_t bits = pool[key ? k4_scale_at(t, ch / 2) : v4_scale_at(t, ch / 2)];
  const uint32_t s2 = bits * 0x00800080u;  // the scale twice, as fp16
  const uint32_t y[4] = {mul_f16x2(f16_of_codes<0>(w), s2), mul_f16x2(f16_of_codes<1>(w), s2),
                         mul_f16x2(f16_of_codes<2>(w), s2), mul_f16x2(f16_of_codes<3>(w), s2)};
  uint4 o;
#pragma unroll
  for (int e = 0; e < 4; ++e) {
    const float2 f = __half22float2(*reinterpret_cast<const __half2*>(&y[e]));
    (&o.x)[e] = pack_bf16(f.x * 0.0625f, f.y * 0.0625f);
  }
  __nv_bfloat16* to = key ? k + row * k_stride : v + row * v_stride;
  reinterpret_cast<uint4*>(to)[ch] = o;
}

template <int kRows, bool kFour>
cudaError_t launch_append(const CacheView& c, const BatchView& b, const RopeAppendArgs& x, const LaunchCtx& ctx) {
  const int64_t per = static_cast<int64_t>(kRows) * kWarps;
  const int64_t ab = (b.rows + per - 1) / per * 2;
  const int64_t turns = b.rows * ((x.q.heads > 0) + (x.qi.heads > 0));
  const int64_t blocks = ab + (turns + kWarps - 1) / kWarps;
  LaunchCtx early = ctx;
  early.pdl = 1;
  return launch_ex(early, append_rope_kernel<kRows, kFour>, dim3(static_cast<unsigned>(blocks)), dim3(32 * kWarps), 0, c,
                   b, x, static_cast<unsigned>(ab), static_cast<unsigned>(blocks / ab), ctx.status);
}

}  // namespace

cudaError_t launch_append_rope(const CacheView& c, bool four, const BatchView& b, const RopeAppendArgs& x,
                               const LaunchCtx& ctx) {
  // One row a warp, or four: bf16 64 rows 2.5 / 3.2 us, 1024 rows 4.9 / 5.1, 1536
  // rows 8.5 / 7.0; in 4 bits 2.5 / 4.5, 4.6 / 6.0, 8.2 / 7.2 (with queries, of one
  // sequence).  Every warp looks at all offsets, so rows of as many sequences take
  // longer: 256 rows 4.0 us, 1024 rows 10, 8192 rows 337 (of one sequence 3.1, 4.9
  // and 26).
  if (b.rows <= 1024)
    return four ? launch_append<1, true>(c, b, x, ctx) : launch_append<1, false>(c, b, x, ctx);
  return four ? launch_append<4, true>(c, b, x, ctx) : launch_append<4, false>(c, b, x, ctx);
}

cudaError_t launch_cache4_read(const CacheView& c, const BatchView& b, void* k, int64_t k_stride, void* v,
                               int64_t v_stride, const LaunchCtx& ctx) {
  LaunchCtx early = ctx;
  early.pdl = 1;
  return launch_ex(early, cache4_read_kernel, dim3(static_cast<unsigned>((b.rows + kWarps - 1) / kWarps)),
                   dim3(32 * kWarps), 0, c, b, static_cast<__nv_bfloat16*>(k), static_cast<__nv_bfloat16*>(v), k_stride,
                   v_stride, ctx.status);
}

}  // namespace dsa
