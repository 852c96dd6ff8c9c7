// paged_cache.cu -- writing new tokens into a paged cache, and the operators
// on its pages: copying, reserving, forking, freeing and compacting.
//
// A page holds `page` tokens of one layer: keys and values (256 B each),
// indexer keys (128 B) and, for every complete pool of four tokens, the pooled
// indexer key as a bf16 hi/lo pair (256 B): 704 B a token.  Pools never cross
// a page.  With keys and values in 4 bits (kv4.cuh) it is 336 B a token.
//
// The pooled key is the one of the contiguous indexer:
//   Khat_p = ((k0 + k1) + (k2 + k3)) * 0.25 in fp32, hi = bf16(Khat),
//   lo = bf16(Khat - hi).
// It is kept with the page so that a decoding step reads 256 B a pool; from
// the indexer keys alone it would read 512 B and add them up again each time.
#include "paged.cuh"

namespace dsa {
namespace {

constexpr int kD = 128;
constexpr int kDi = 64;

// ================================================================= append
// One warp takes four consecutive rows: 16 lanes copy a row's key and 16 its
// value (16 B each), for the four rows at once, and 8 lanes each a row's
// indexer key.  The row whose position ends a pool also computes the pooled
// key: its three predecessors come from the call's rows, or from the page
// where they are older than the call.  Each row's bytes are read once (the
// three indexer keys a second time, from L1 or L2); nothing is staged.
// Bound by latency: 3.4 us for 64 rows, 5.4 us for 9816 rows (13 MB, 2.4 TB/s)
// with inputs and pages in turn, 3.9 with the same ones, which L2 then holds
// (launches in a graph; alone and with all caches empty 6.2 and 7.0).
constexpr int kAppendWarps = 4;

__global__ void __launch_bounds__(32 * kAppendWarps)
    cache_append_kernel(const CacheView c, const BatchView b, const AppendArgs a, unsigned* status) {
  const int lane = threadIdx.x & 31;
  const int64_t r0 = (static_cast<int64_t>(blockIdx.x) * kAppendWarps + (threadIdx.x >> 5)) * 4;
  if (r0 >= b.rows) return;
  // the four rows' sequences: one walk over the offsets; lanes 8u .. 8u+7 work out row r0 + u
  const int mine = lane >> 3;
  const int64_t row = r0 + mine;
  int page = -1, off = 0, older = 0;  // older: how many of the pool's tokens come before the call's rows
  // offsets that descend or leave the call's rows, or a reservation that found too few pages
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
    for (int u = 0; u < 4; ++u) {
      const unsigned hit =
          __ballot_sync(0xffffffffu, j < b.batch && c0 <= r0 + u && r0 + u < c1 && r0 + u < b.rows);
      if (mine == u && hit != 0u) src = __ffs(hit) - 1;
    }
    const int64_t first = __shfl_sync(0xffffffffu, c0, src & 31), last = __shfl_sync(0xffffffffu, c1, src & 31);
    const int64_t n = __shfl_sync(0xffffffffu, len, src & 31);
    if (src >= 0) {
      const int64_t before = row - first, i = n - last + row;  // before: the call's rows of the sequence before this one
      if (i < before || n > (static_cast<int64_t>(b.max_pages) << c.shift)) {
        record_status(status, kStatusInternal);
      } else {
        page = page_of(b, c.num_pages, j0 + src, static_cast<int>(i >> c.shift), status);
        off = static_cast<int>(i & ((1 << c.shift) - 1));
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
  // keys and values: lanes 0..15 the key, 16..31 the value
  const int half = lane >> 4, ch = lane & 15;
  uint4 x[4];
  int pg[4], of[4];
#pragma unroll
  for (int u = 0; u < 4; ++u) {
    pg[u] = __shfl_sync(0xffffffffu, page, 8 * u);
    of[u] = __shfl_sync(0xffffffffu, off, 8 * u);
    if (pg[u] >= 0) {
      const __nv_bfloat16* src = half ? a.v + (r0 + u) * a.v_stride : a.k + (r0 + u) * a.k_stride;
      x[u] = __ldg(reinterpret_cast<const uint4*>(src) + ch);
    }
  }
  const int g = lane & 7;
  uint4 xi = make_uint4(0u, 0u, 0u, 0u);
  if (page >= 0) xi = __ldg(reinterpret_cast<const uint4*>(a.k_idx + row * a.kidx_stride) + g);
#pragma unroll
  for (int u = 0; u < 4; ++u) {
    if (pg[u] < 0) continue;
    __nv_bfloat16* dst = half ? c.v + pg[u] * c.v_stride : c.k + pg[u] * c.k_stride;
    reinterpret_cast<uint4*>(dst + of[u] * kD)[ch] = x[u];
  }
  if (page < 0) return;
  __nv_bfloat16* pidx = c.k_idx + page * c.kidx_stride;
  reinterpret_cast<uint4*>(pidx + off * kDi)[g] = xi;
  if ((off & 3) != 3) return;
  // token t of the pool is this row less 3 - t
  uint4 four[4];
  four[3] = xi;
#pragma unroll
  for (int t = 0; t < 3; ++t)
    four[t] = t < older ? *(reinterpret_cast<const uint4*>(pidx + (off - 3 + t) * kDi) + g)
                        : __ldg(reinterpret_cast<const uint4*>(a.k_idx + (row - 3 + t) * a.kidx_stride) + g);
  uint32_t hi[4], lo[4];
#pragma unroll
  for (int e = 0; e < 4; ++e) {
    float y[4][2];
#pragma unroll
    for (int t = 0; t < 4; ++t) {
      const uint32_t word = (&four[t].x)[e];
      y[t][0] = __uint_as_float(word << 16);
      y[t][1] = __uint_as_float(word & 0xFFFF0000u);
    }
    float kh[2];
#pragma unroll
    for (int z = 0; z < 2; ++z)
      kh[z] = __fmul_rn(__fadd_rn(__fadd_rn(y[0][z], y[1][z]), __fadd_rn(y[2][z], y[3][z])), 0.25f);
    const __nv_bfloat162 h2 = __floats2bfloat162_rn(kh[0], kh[1]);
    const float2 hf = __bfloat1622float2(h2);
    const __nv_bfloat162 l2 = __floats2bfloat162_rn(__fsub_rn(kh[0], hf.x), __fsub_rn(kh[1], hf.y));
    hi[e] = *reinterpret_cast<const uint32_t*>(&h2);
    lo[e] = *reinterpret_cast<const uint32_t*>(&l2);
  }
  uint4* dst = reinterpret_cast<uint4*>(c.khat + page * c.khat_stride + (off >> 2) * (2 * kDi));
  dst[g] = make_uint4(hi[0], hi[1], hi[2], hi[3]);
  dst[8 + g] = make_uint4(lo[0], lo[1], lo[2], lo[3]);
}

// ================================================================= page copies
constexpr int kCopyThreads = 256;
// 16-byte vectors a block copies at a time: a page of 64 tokens, or half of one
// of 128, and so on (704 B a token), so that no block has a remainder to copy
// from pages of 64 tokens on.  8 vectors a thread, which leave a third of every
// second block idle there, take as long: 32.6 us against 33.2 for the copies of a
// compaction of 165 MB, with events around the launch, in turn.
constexpr int kCopyUnroll = 11;
constexpr int kCopyVecs = kCopyThreads * kCopyUnroll;

// 16-byte vectors of a token: 704 B, or 336 B with keys and values in 4 bits
__host__ __device__ constexpr int token_vecs(bool four) { return four ? 21 : 44; }
template <bool kFour>
__device__ __forceinline__ int page_vecs(const CacheView& c) { return token_vecs(kFour) << c.shift; }
template <bool kFour>
__device__ __forceinline__ int page_slices(const CacheView& c) { return (page_vecs<kFour>(c) + kCopyVecs - 1) / kCopyVecs; }

// Vector x of a page: keys, values (in 4 bits both at once, 144 B a token), indexer keys, pooled keys.
template <bool kFour>
__device__ __forceinline__ uint4* page_vec(const CacheView& c, int64_t page, int x) {
  const int n = 16 << c.shift;
  if (kFour) {
    const int m = 9 << c.shift;
    if (x < m) return reinterpret_cast<uint4*>(c.k + page * c.k_stride) + x;
    x -= m;
  } else {
    if (x < n) return reinterpret_cast<uint4*>(c.k + page * c.k_stride) + x;
    x -= n;
    if (x < n) return reinterpret_cast<uint4*>(c.v + page * c.v_stride) + x;
    x -= n;
  }
  if (x < n / 2) return reinterpret_cast<uint4*>(c.k_idx + page * c.kidx_stride) + x;
  return reinterpret_cast<uint4*>(c.khat + page * c.khat_stride) + (x - n / 2);
}

// Slice `sl` of page src to page dst, by a whole block; all loads first.
template <bool kFour>
__device__ __forceinline__ void copy_slice(const CacheView& c, int64_t src, int64_t dst, int sl) {
  const int n = page_vecs<kFour>(c), x0 = sl * kCopyVecs + threadIdx.x;
  uint4 t[kCopyUnroll];
#pragma unroll
  for (int u = 0; u < kCopyUnroll; ++u)
    if (x0 + u * kCopyThreads < n) t[u] = *page_vec<kFour>(c, src, x0 + u * kCopyThreads);
#pragma unroll
  for (int u = 0; u < kCopyUnroll; ++u)
    if (x0 + u * kCopyThreads < n) *page_vec<kFour>(c, dst, x0 + u * kCopyThreads) = t[u];
}

template <bool kFour>
__global__ void __launch_bounds__(kCopyThreads)
    copy_pages_kernel(const __grid_constant__ CacheSet set, const int32_t* __restrict__ src,
                      const int32_t* __restrict__ dst, unsigned* status) {
  const CacheView& c = set.v[blockIdx.z];
  const int s = src[blockIdx.x], d = dst[blockIdx.x];
  if (static_cast<unsigned>(s) >= static_cast<unsigned>(c.num_pages) ||
      static_cast<unsigned>(d) >= static_cast<unsigned>(c.num_pages)) {
    if (threadIdx.x == 0) record_status(status, kStatusInternal);
    return;
  }
  copy_slice<kFour>(c, s, d, blockIdx.y);
}

// ================================================================= planning
// Reserving, forking and compacting need prefix sums over the page counts (a
// page is free when its count is 0).  One cluster of 8 CTAs does it in a
// single launch: each of its 256 warps owns a contiguous stretch of pages,
// counts it, the counts are scanned in shared memory and across the cluster,
// and the warps walk their stretches again (from L2) with their offsets.  A
// cache of few pages is planned by one CTA, which needs no cluster barriers
// (5.4 us against 8.7 for a compaction of 16 thousand pages).
constexpr int kPlanCtas = 8;
constexpr int kPlanAlone = 16384;  // pages up to which one CTA plans
constexpr int kPlanThreads = 1024;
constexpr int kPlanWarps = kPlanThreads / 32;

struct PlanSmem {
  int warp[kPlanWarps];  // this CTA's warps' counts, then their exclusive prefix
  int total;             // read by the other CTAs
  int below;             // compaction: used pages below n_used, from the CTA that finds it (-1: not here)
  int64_t scan[kPlanWarps];
  int bad;
  int carry;
};

template <int kC>
__device__ __forceinline__ void plan_sync() {
  if (kC > 1) cluster_sync();
  else __syncthreads();
}
// a word of CTA u's shared memory
template <int kC>
__device__ __forceinline__ uint32_t plan_peer(const int* p, uint32_t u) {
  return kC > 1 ? cluster_ld_u32(cluster_map(smem_u32(p), u)) : static_cast<uint32_t>(*reinterpret_cast<const volatile int*>(p));
}

// Exclusive prefix of v over the block's threads; *total: the sum.  In 64 bits:
// one request may be 2^27 pages, so those of a block pass 32.  sm.scan is free
// again on return.
__device__ __forceinline__ int64_t block_excl(PlanSmem& sm, int v, int64_t* total) {
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  int64_t x = v;
#pragma unroll
  for (int o = 1; o < 32; o <<= 1) {
    const int64_t y = __shfl_up_sync(0xffffffffu, x, o);
    if (lane >= o) x += y;
  }
  if (lane == 31) sm.scan[warp] = x;
  __syncthreads();
  int64_t before = 0, all = 0;
  for (int w = 0; w < kPlanWarps; ++w) {
    const int64_t t = sm.scan[w];
    before += w < warp ? t : 0;
    all += t;
  }
  __syncthreads();
  *total = all;
  return before + x - v;
}

// The stretch [p0, p1) of warp `gw` of the cluster's 256.
template <int kC>
__device__ __forceinline__ void plan_stretch(int num_pages, int gw, int* p0, int* p1) {
  const int per = ((num_pages + kC * kPlanWarps * 32 - 1) / (kC * kPlanWarps * 32)) * 32;
  *p0 = min(static_cast<int64_t>(gw) * per, static_cast<int64_t>(num_pages));
  *p1 = min(*p0 + per, num_pages);
}

// Counts the pages of this warp's stretch that are used, scans the counts over the cluster: used pages before the stretch;
// *all: used pages in the whole cache.
template <int kC>
__device__ __forceinline__ int plan_scan(PlanSmem& sm, const int32_t* count, int num_pages, uint32_t rank, int* all) {
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  int p0, p1;
  plan_stretch<kC>(num_pages, static_cast<int>(rank) * kPlanWarps + warp, &p0, &p1);
  int n = 0;
#pragma unroll 8
  for (int p = p0; p < p1; p += 32) n += p + lane < p1 && count[p + lane] != 0;
#pragma unroll
  for (int o = 16; o > 0; o >>= 1) n += __shfl_xor_sync(0xffffffffu, n, o);
  if (lane == 0) sm.warp[warp] = n;
  __syncthreads();
  if (threadIdx.x < 32) {
    int x = sm.warp[lane];
    const int v = x;
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
      const int y = __shfl_up_sync(0xffffffffu, x, o);
      if (lane >= o) x += y;
    }
    sm.warp[lane] = x - v;
    if (lane == 31) sm.total = x;
  }
  plan_sync<kC>();
  int before = 0, sum = 0;
  for (uint32_t r = 0; r < kC; ++r) {
    const int t = static_cast<int>(plan_peer<kC>(&sm.total, r));
    before += r < rank ? t : 0;
    sum += t;
  }
  *all = sum;
  return before + sm.warp[warp];
}

// Writes the k-th lowest free page to list[k] for k < need.
template <int kC>
__device__ __forceinline__ void plan_free_list(const int32_t* count, int num_pages, uint32_t rank, int used_before,
                                               int need, int32_t* list) {
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  int p0, p1;
  plan_stretch<kC>(num_pages, static_cast<int>(rank) * kPlanWarps + warp, &p0, &p1);
  int at = p0 - used_before;  // free pages before the stretch
  for (int p = p0; p < p1 && at < need; p += 32) {
    const bool free = p + lane < p1 && count[p + lane] == 0;
    const unsigned m = __ballot_sync(0xffffffffu, free);
    const int k = at + __popc(m & ((1u << lane) - 1u));
    if (free && k < need) list[k] = p + lane;
    at += __popc(m);
  }
}

// ----------------------------------------------------------------- reserve
// ws: off [max_seqs], list [num_pages].  One launch: the plan, then a warp per
// sequence takes its pages, or gives them back.  Bound by latency: 5.1 us for
// 64 sequences of which none needs a page, 5.9 when each takes (or returns) one
// (growing and shrinking in turn in a graph; 7.1 with 70000 pages).  A long
// request is walked 32 pages at a time, each round waiting for memory: 23 us to
// take the 8192 pages of a prompt of 131072 tokens in pages of 16, 119 to give
// them back; 4096 sequences share the warps of one CTA (83 and 126 us) or of a
// cluster (29 and 33).
template <int kC>
__global__ void __cluster_dims__(kC, 1, 1) __launch_bounds__(kPlanThreads)
    cache_reserve_kernel(const PageTableView t, int shift, int num_pages, const int32_t* __restrict__ add,
                         int32_t* result, int32_t* ws, unsigned* status) {
  __shared__ PlanSmem sm;
  const uint32_t rank = kC > 1 ? cluster_rank() : 0u;
  int32_t* off = ws;
  int32_t* list = ws + t.max_seqs;
  const int64_t cap = static_cast<int64_t>(t.max_pages) << shift;
  // every CTA sums the requests; CTA 0 keeps their prefix
  if (threadIdx.x == 0) sm.bad = 0;
  __syncthreads();
  int64_t need = 0;
  for (int s0 = 0; s0 < t.max_seqs; s0 += kPlanThreads) {
    const int s = s0 + static_cast<int>(threadIdx.x);
    int v = 0;
    if (s < t.max_seqs) {
      const int64_t len = t.lens[s], more = add[s], to = len + more;
      if (len < 0 || to < 0 || len > cap || to > cap) {
        sm.bad = 1;
      } else {
        v = static_cast<int>(max(((to + (1 << shift) - 1) >> shift) - ((len + (1 << shift) - 1) >> shift), int64_t{0}));
        if (more < 0 && (to & ((1 << shift) - 1)) != 0) {  // the page that becomes the last is written next: it must be its own
          const int p = t.table[s * t.table_stride + (to >> shift)];
          if (static_cast<unsigned>(p) >= static_cast<unsigned>(num_pages) || t.count[p] > 1) sm.bad = 1;
        }
      }
    }
    int64_t tile;
    const int64_t before = block_excl(sm, v, &tile);
    // (a request too large for the cache is refused below; its prefix is not used)
    if (rank == 0 && s < t.max_seqs) off[s] = static_cast<int32_t>(min(need + before, static_cast<int64_t>(num_pages)));
    need += tile;
  }
  __syncthreads();
  const bool bad = sm.bad != 0;
  int used;
  const int before = plan_scan<kC>(sm, t.count, num_pages, rank, &used);
  const int64_t room = num_pages - used;
  const bool go = !bad && need <= room;
  if (rank == 0 && threadIdx.x == 0) {
    *result = bad ? INT32_MIN : go ? static_cast<int32_t>(need)
                                   : static_cast<int32_t>(-min(need - room, static_cast<int64_t>(INT32_MAX)));
    if (bad) record_status(status, kStatusInternal);
  }
  if (go) plan_free_list<kC>(t.count, num_pages, rank, before, static_cast<int>(need), list);
  plan_sync<kC>();  // the list and the prefix are written; every count has been read
  if (!go) return;
  const int lane = threadIdx.x & 31;
  const int gw = static_cast<int>(rank) * kPlanWarps + (threadIdx.x >> 5);
  for (int s = gw; s < t.max_seqs; s += kC * kPlanWarps) {
    const int64_t len = t.lens[s], more = add[s];
    const int have = static_cast<int>((len + (1 << shift) - 1) >> shift);
    const int want = static_cast<int>((len + more + (1 << shift) - 1) >> shift);
    for (int x = have + lane; x < want; x += 32) {
      const int p = list[off[s] + x - have];
      t.table[s * t.table_stride + x] = p;
      t.count[p] = 1;
    }
    for (int x = want + lane; x < have; x += 32) {  // a shorter sequence gives pages back
      const int p = t.table[s * t.table_stride + x];
      t.table[s * t.table_stride + x] = -1;
      if (static_cast<unsigned>(p) >= static_cast<unsigned>(num_pages)) record_status(status, kStatusInternal);
      else if (atomicSub(t.count + p, 1) <= 0) {
        atomicAdd(t.count + p, 1);  // the page was free already
        record_status(status, kStatusInternal);
      }
    }
    __syncwarp();
    if (lane == 0) t.lens[s] = static_cast<int32_t>(len + more);
  }
}

// ----------------------------------------------------------------- fork
// ws: {go}, len [n], off [n], list [n], claim [max_seqs].  The plan checks the
// request, notes every parent's length and numbers the new pages; a second
// launch copies rows, counts and last pages.
struct ForkWs {
  int32_t *go, *len, *off, *list, *claim;
};
__host__ __device__ inline ForkWs fork_ws(int32_t* ws, int64_t n) {
  return ForkWs{ws, ws + 4, ws + 4 + n, ws + 4 + 2 * n, ws + 4 + 3 * n};
}

template <int kC>
__global__ void __cluster_dims__(kC, 1, 1) __launch_bounds__(kPlanThreads)
    fork_plan_kernel(const PageTableView t, int shift, int num_pages, const int32_t* __restrict__ src,
                     const int32_t* __restrict__ dst, int n, int32_t* result, int32_t* ws_, unsigned* status) {
  __shared__ PlanSmem sm;
  const uint32_t rank = kC > 1 ? cluster_rank() : 0u;
  const ForkWs ws = fork_ws(ws_, n);
  const int64_t cap = static_cast<int64_t>(t.max_pages) << shift;
  const unsigned seqs = static_cast<unsigned>(t.max_seqs);
  if (threadIdx.x == 0) sm.bad = 0;
  for (int j = rank * kPlanThreads + threadIdx.x; j < n; j += kC * kPlanThreads)
    if (static_cast<unsigned>(dst[j]) < seqs) ws.claim[dst[j]] = 0;
  plan_sync<kC>();
  // every CTA checks its part of the request; the same child twice shows in its claim
  for (int j = rank * kPlanThreads + threadIdx.x; j < n; j += kC * kPlanThreads) {
    const int s = src[j], d = dst[j];
    bool ok = static_cast<unsigned>(s) < seqs && static_cast<unsigned>(d) < seqs;
    if (ok) {
      const int len = t.lens[s];
      ok = len >= 0 && len <= cap && t.lens[d] == 0 && atomicExch(&ws.claim[d], 1) == 0;
    }
    if (!ok) sm.bad = 1;
  }
  // every CTA counts all last pages that are partly filled; CTA 0 keeps lengths and prefix
  int need = 0;
  for (int j0 = 0; j0 < n; j0 += kPlanThreads) {
    const int j = j0 + static_cast<int>(threadIdx.x);
    int len = 0;
    if (j < n && static_cast<unsigned>(src[j]) < seqs) len = t.lens[src[j]];
    int64_t tile;
    const int64_t before = block_excl(sm, (len & ((1 << shift) - 1)) != 0, &tile);
    if (rank == 0 && j < n) {
      ws.len[j] = len;
      ws.off[j] = need + static_cast<int>(before);
    }
    need += static_cast<int>(tile);
  }
  int used;
  const int before = plan_scan<kC>(sm, t.count, num_pages, rank, &used);
  bool bad = false;
  for (uint32_t r = 0; r < kC; ++r) bad |= plan_peer<kC>(&sm.bad, r) != 0;
  const int room = num_pages - used;
  const bool go = !bad && need <= room;
  if (rank == 0 && threadIdx.x == 0) {
    *result = bad ? INT32_MIN : go ? need : room - need;
    *ws.go = go;
    if (bad) record_status(status, kStatusInternal);
  }
  if (go) plan_free_list<kC>(t.count, num_pages, rank, before, need, ws.list);
  plan_sync<kC>();  // no CTA leaves while another reads its shared memory
}

// Block (j, y, z): child j's part y in layer z.  Parts 0 .. slices-1 copy a
// slice of the last page; all parts of the first layer share the row and the
// counts.  (No layer reads a row that the first one writes: a child's row was
// free, and what has no tokens has no pages.)
template <bool kFour>
__global__ void __launch_bounds__(kCopyThreads)
    fork_apply_kernel(const __grid_constant__ CacheSet set, bool first, const PageTableView t,
                      const int32_t* __restrict__ src, const int32_t* __restrict__ dst, int n, int32_t* ws_,
                      unsigned* status) {
  const CacheView& c = set.v[blockIdx.z];
  first = first && blockIdx.z == 0;
  const ForkWs ws = fork_ws(ws_, n);
  pdl_wait();  // the plan is written
  if (*ws.go == 0) return;
  const int j = blockIdx.x;
  const int s = src[j], d = dst[j], len = ws.len[j];
  const int full = len >> c.shift;
  const bool part = (len & ((1 << c.shift) - 1)) != 0;
  const int32_t* from = t.table + s * t.table_stride;
  int32_t* to = t.table + d * t.table_stride;
  const int fresh = part ? ws.list[ws.off[j]] : -1;
  for (int x = blockIdx.y * kCopyThreads + threadIdx.x; first && x < t.max_pages; x += gridDim.y * kCopyThreads) {
    int p = -1;
    if (x < full) {
      p = from[x];
      if (static_cast<unsigned>(p) < static_cast<unsigned>(c.num_pages)) atomicAdd(t.count + p, 1);
      else record_status(status, kStatusInternal);
    } else if (x == full && part) {
      p = fresh;
      t.count[fresh] = 1;
    }
    to[x] = p;
  }
  if (first && blockIdx.y == 0 && threadIdx.x == 0) t.lens[d] = len;
  if (part && static_cast<int>(blockIdx.y) < page_slices<kFour>(c)) {
    const int old = from[full];
    if (static_cast<unsigned>(old) < static_cast<unsigned>(c.num_pages)) copy_slice<kFour>(c, old, fresh, blockIdx.y);
    else if (threadIdx.x == 0) record_status(status, kStatusInternal);
  }
}

// ----------------------------------------------------------------- free
// One block per sequence; taking the length out first makes a second mention
// of the same sequence free nothing.
__global__ void __launch_bounds__(kCopyThreads)
    cache_free_kernel(const PageTableView t, int shift, int num_pages, const int32_t* __restrict__ seqs,
                      unsigned* status) {
  __shared__ int s_len;
  const int s = seqs[blockIdx.x];
  if (static_cast<unsigned>(s) >= static_cast<unsigned>(t.max_seqs)) {
    if (threadIdx.x == 0) record_status(status, kStatusInternal);
    return;
  }
  if (threadIdx.x == 0) s_len = atomicExch(t.lens + s, 0);
  __syncthreads();
  const int64_t len = s_len;
  if (len < 0 || len > (static_cast<int64_t>(t.max_pages) << shift)) {
    if (threadIdx.x == 0) record_status(status, kStatusInternal);
    return;
  }
  const int n = static_cast<int>((len + (1 << shift) - 1) >> shift);
  int32_t* row = t.table + s * t.table_stride;
  for (int x = threadIdx.x; x < n; x += kCopyThreads) {
    const int p = row[x];
    row[x] = -1;
    if (static_cast<unsigned>(p) >= static_cast<unsigned>(num_pages)) record_status(status, kStatusInternal);
    else if (atomicSub(t.count + p, 1) <= 0) {
      atomicAdd(t.count + p, 1);  // the page was free already
      record_status(status, kStatusInternal);
    }
  }
}

// ----------------------------------------------------------------- compact
// With U used pages, those at or above U move into the free ones below: the
// k-th to the k-th, both ascending, so every page moves at most once and no
// page is both read and written.  The copies run at 5.5 TB/s (165 MB in all,
// read and written, in 30 us by ncu), 0.8 of the copy peak.  ws: {U, moved}, hole [num_pages], high
// [num_pages], rank_of [num_pages] (for pages at or above U: the place in
// `high`, or -1).
struct CompactWs {
  int32_t *head, *hole, *high, *rank_of;
};
__host__ __device__ inline CompactWs compact_ws(int32_t* ws, int64_t num_pages) {
  return CompactWs{ws, ws + 4, ws + 4 + num_pages, ws + 4 + 2 * num_pages};
}

template <int kC>
__global__ void __cluster_dims__(kC, 1, 1) __launch_bounds__(kPlanThreads)
    compact_plan_kernel(const PageTableView t, int num_pages, int32_t* result, int32_t* ws_) {
  __shared__ PlanSmem sm;
  const uint32_t rank = kC > 1 ? cluster_rank() : 0u;
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  const CompactWs ws = compact_ws(ws_, num_pages);
  if (threadIdx.x == 0) sm.below = -1;
  int used;
  const int before = plan_scan<kC>(sm, t.count, num_pages, rank, &used);  // (its barriers order sm.below)
  int p0, p1;
  plan_stretch<kC>(num_pages, static_cast<int>(rank) * kPlanWarps + warp, &p0, &p1);
  // used pages below page number `used`, found by the warp whose stretch holds that page
  if (used >= p0 && used < p1) {
    int n = 0;
    for (int p = p0; p < used; p += 32) n += __popc(__ballot_sync(0xffffffffu, p + lane < used && t.count[p + lane] != 0));
    if (lane == 0) sm.below = before + n;
  }
  plan_sync<kC>();
  int below = used;  // a full cache: no page is at or above `used`
  for (uint32_t r = 0; r < kC; ++r) {
    const int x = static_cast<int>(plan_peer<kC>(&sm.below, r));
    if (x >= 0) below = x;
  }
  if (rank == 0 && threadIdx.x == 0) {
    ws.head[0] = result[0] = used;
    ws.head[1] = result[1] = used - below;
  }
  int at = before;
  for (int p = p0; p < p1; p += 32) {
    const int q = p + lane;
    const bool in = q < p1, busy = in && t.count[q] != 0;
    const unsigned m = __ballot_sync(0xffffffffu, busy);
    const int ub = at + __popc(m & ((1u << lane) - 1u));  // used pages before q
    if (in && q < used) {
      if (!busy) ws.hole[q - ub] = q;
    } else if (in) {
      ws.rank_of[q] = busy ? ub - below : -1;
      if (busy) ws.high[ub - below] = q;
    }
    at += __popc(m);
  }
  plan_sync<kC>();  // no CTA leaves while another reads its shared memory
}

template <bool kFour>
__global__ void __launch_bounds__(kCopyThreads)
    compact_apply_kernel(const __grid_constant__ CacheSet set, bool first, const PageTableView t, int32_t* ws_) {
  const CacheView& c = set.v[blockIdx.z];
  first = first && blockIdx.z == 0;
  const CompactWs ws = compact_ws(ws_, c.num_pages);
  pdl_wait();  // the plan is written
  const int used = ws.head[0], moved = ws.head[1];
  if (moved == 0) return;
  const int slices = page_slices<kFour>(c);
  for (int64_t x = blockIdx.x; x < static_cast<int64_t>(moved) * slices; x += gridDim.x) {
    const int m = static_cast<int>(x / slices), sl = static_cast<int>(x % slices);
    const int from = ws.high[m], to = ws.hole[m];
    copy_slice<kFour>(c, from, to, sl);
    if (first && sl == 0 && threadIdx.x == 0) {
      t.count[to] = t.count[from];
      t.count[from] = 0;
    }
  }
  if (!first) return;
  // table entries that name a moved page
  const int64_t entries = static_cast<int64_t>(t.max_seqs) * t.max_pages;
  for (int64_t e = static_cast<int64_t>(blockIdx.x) * kCopyThreads + threadIdx.x; e < entries;
       e += static_cast<int64_t>(gridDim.x) * kCopyThreads) {
    int32_t* at = t.table + (e / t.max_pages) * t.table_stride + e % t.max_pages;
    const int p = *at;
    if (p >= used && p < c.num_pages) {
      const int r = ws.rank_of[p];
      if (r >= 0) *at = ws.hole[r];
    }
  }
}

int host_slices(bool four, int shift) { return ((token_vecs(four) << shift) + kCopyVecs - 1) / kCopyVecs; }

}  // namespace

cudaError_t launch_cache_append(const CacheView& c, const BatchView& b, const AppendArgs& a, const LaunchCtx& ctx) {
  const int64_t per = 4 * kAppendWarps;
  cache_append_kernel<<<static_cast<unsigned>((b.rows + per - 1) / per), 32 * kAppendWarps, 0, ctx.stream>>>(
      c, b, a, ctx.status);
  return cudaGetLastError();
}

cudaError_t launch_copy_pages(const CacheSet& set, bool four, const int32_t* src, const int32_t* dst, int64_t n,
                              const LaunchCtx& ctx) {
  const dim3 grid(static_cast<unsigned>(n), host_slices(four, set.v[0].shift), set.n);
  if (four) copy_pages_kernel<true><<<grid, kCopyThreads, 0, ctx.stream>>>(set, src, dst, ctx.status);
  else copy_pages_kernel<false><<<grid, kCopyThreads, 0, ctx.stream>>>(set, src, dst, ctx.status);
  return cudaGetLastError();
}

int64_t fork_ws_words(int64_t n, int max_seqs) { return 4 + 3 * n + max_seqs; }
int64_t reserve_ws_words(int max_seqs, int num_pages) { return static_cast<int64_t>(max_seqs) + num_pages; }
int64_t compact_ws_words(int num_pages) { return 4 + 3 * static_cast<int64_t>(num_pages); }

cudaError_t launch_cache_reserve(const PageTableView& t, int shift, int num_pages, const int32_t* add, int32_t* result,
                                 int32_t* ws, const LaunchCtx& ctx) {
  if (num_pages <= kPlanAlone)
    cache_reserve_kernel<1><<<1, kPlanThreads, 0, ctx.stream>>>(t, shift, num_pages, add, result, ws, ctx.status);
  else
    cache_reserve_kernel<kPlanCtas>
        <<<kPlanCtas, kPlanThreads, 0, ctx.stream>>>(t, shift, num_pages, add, result, ws, ctx.status);
  return cudaGetLastError();
}

cudaError_t launch_fork_plan(const PageTableView& t, int shift, int num_pages, const int32_t* src, const int32_t* dst,
                             int n, int32_t* result, int32_t* ws, const LaunchCtx& ctx) {
  if (num_pages <= kPlanAlone)
    fork_plan_kernel<1><<<1, kPlanThreads, 0, ctx.stream>>>(t, shift, num_pages, src, dst, n, result, ws, ctx.status);
  else
    fork_plan_kernel<kPlanCtas>
        <<<kPlanCtas, kPlanThreads, 0, ctx.stream>>>(t, shift, num_pages, src, dst, n, result, ws, ctx.status);
  return cudaGetLastError();
}

cudaError_t launch_fork_apply(const CacheSet& set, bool four, bool first, const PageTableView& t, const int32_t* src,
                              const int32_t* dst, int n, int32_t* ws, const LaunchCtx& ctx) {
  // parts of a child: one per slice of its last page, and enough that a thread
  // copies at most 4 entries of the row (8 parts at the most for long rows)
  const int slices = host_slices(four, set.v[0].shift);
  const int by_row = first ? (t.max_pages + 4 * kCopyThreads - 1) / (4 * kCopyThreads) : 1;
  const int parts = slices > by_row ? slices : by_row < 8 ? by_row : 8;
  LaunchCtx early = ctx;
  early.pdl = first;  // (only the plan stands right before the first)
  return launch_ex(early, four ? fork_apply_kernel<true> : fork_apply_kernel<false>, dim3(n, parts, set.n),
                   dim3(kCopyThreads), 0, set, first, t, src, dst, n, ws, ctx.status);
}

cudaError_t launch_cache_free(const PageTableView& t, int shift, int num_pages, const int32_t* seqs, int n,
                              const LaunchCtx& ctx) {
  cache_free_kernel<<<n, kCopyThreads, 0, ctx.stream>>>(t, shift, num_pages, seqs, ctx.status);
  return cudaGetLastError();
}

cudaError_t launch_compact_plan(const PageTableView& t, int num_pages, int32_t* result, int32_t* ws,
                                const LaunchCtx& ctx) {
  if (num_pages <= kPlanAlone)
    compact_plan_kernel<1><<<1, kPlanThreads, 0, ctx.stream>>>(t, num_pages, result, ws);
  else
    compact_plan_kernel<kPlanCtas><<<kPlanCtas, kPlanThreads, 0, ctx.stream>>>(t, num_pages, result, ws);
  return cudaGetLastError();
}

cudaError_t launch_compact_apply(const CacheSet& set, bool four, bool first, const PageTableView& t, int32_t* ws,
                                 const LaunchCtx& ctx) {
  LaunchCtx early = ctx;
  early.pdl = first;  // (only the plan stands right before the first)
  return launch_ex(early, four ? compact_apply_kernel<true> : compact_apply_kernel<false>,
                   dim3((ctx.num_sms * 16 + set.n - 1) / set.n, 1, set.n), dim3(kCopyThreads), 0, set, first, t, ws);
}

}  // namespace dsa
