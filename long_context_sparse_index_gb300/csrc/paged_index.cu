// paged_index.cu -- the indexer over a paged cache: scores of new tokens
// against the pooled keys of their sequences' pages, and each row's top-k.
//
//   score(i, p) = sum_h w[i,h] * ReLU(q[i,h,:] . Khat_p),   p < floor(i/4)
//   q . Khat = q . hi + q . lo   (the pooled key's bf16 pair, fp32 sums)
//
// The scores of a group of rows go to a scratch matrix [rows][ld] and each
// row's top-k is taken from there: 4 B a pool against the 256 B of the pooled
// key, so for a decoding step (one row a sequence) the scores' traffic is
// about 3 % of the pooled keys'.
#include "paged.cuh"

namespace dsa {
namespace {

constexpr int kDi = 64;

// ================================================================= scores, single tokens
// Memory-bound: each pooled key is read once for up to kRows rows of its
// sequence.  A warp takes 32 pools (four MMA n-tiles of 8).  The k order of a
// dot product is free, so the MMA fragments are read straight from global
// memory: lane (g, t) holds 16-byte pieces t and t + 4 of pool g's hi (and lo)
// half, which are its B fragments of four k-steps, and the same pieces of
// head g's (and g + 8's) query as A fragments.  No shared memory, no
// transposes, 64 bytes of a row per quad of lanes and load.  Loads evict first
// (each key is read once): 55 us against 62 for 64 sequences of 13 to 131
// thousand tokens, now 52 us: 302 MB at 5.8 TB/s, 0.92 of the rate at which a
// plain read streams.  12 warps an SM at 166 registers; 16 at 128 spilled (73).
//
// Work items are (sequence, group of kRows rows, 128 pools); every CTA walks
// an equal, contiguous range of them.
constexpr int kWarps = 4;
constexpr int kThreads = 32 * kWarps;
constexpr int kTile = 32 * kWarps;  // pools of an item
static_assert(kTile == kRunTile, "the walk's tiles");
constexpr int kRows = 8;            // rows of an item

// Exclusive prefix of the sequences' item counts into off[0 .. batch] (shared
// memory), by all kThreads threads.  The sums saturate, so that offsets which
// contradict each other cannot overflow them.
template <typename F>
__device__ __forceinline__ void item_prefix(int* off, int batch, F&& items_of) {
  __shared__ int s_w[kThreads / 32];
  __shared__ int s_base;
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  if (threadIdx.x == 0) s_base = 0;
  __syncthreads();
  for (int s0 = 0; s0 < batch; s0 += kThreads) {
    const int s = s0 + static_cast<int>(threadIdx.x);
    const int v = s < batch ? items_of(s) : 0;
    int x = v;
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
      const int y = __shfl_up_sync(0xffffffffu, x, o);
      if (lane >= o) x += y;
    }
    if (lane == 31) s_w[warp] = x;
    __syncthreads();
    int before = s_base, all = 0;
#pragma unroll
    for (int w = 0; w < kThreads / 32; ++w) {
      before += w < warp ? s_w[w] : 0;
      all += s_w[w];
    }
    if (s < batch) off[s] = before + x - v;
    __syncthreads();
    if (threadIdx.x == 0) s_base = min(s_base + all, kMaxTotal);
    __syncthreads();
  }
  if (threadIdx.x == 0) off[batch] = s_base;
  __syncthreads();
}

template <int kMt>
__global__ void __launch_bounds__(kThreads, kMt <= 2 ? 3 : 2)
    paged_score_kernel(const CacheView c, const BatchView b, const __nv_bfloat16* __restrict__ q,
                       const float* __restrict__ w, int Hi, int64_t row0, int64_t row1, const TcRule tc,
                       float* __restrict__ scores, float* __restrict__ tops, int64_t ld, unsigned* status) {
  extern __shared__ int off[];

  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  const int g = lane >> 2, t = lane & 3;
  item_prefix(off, b.batch, [&](int s) {
    int64_t first;
    const int n = seq_rows(b, s, row0, row1, &first);
    if (n == 0 || tc_takes(b, tc, s)) return 0;
    const int64_t tiles = (seq_pools(b, c.shift, s, first, n) + kTile - 1) / kTile;
    const int64_t items = tiles * ((n + kRows - 1) / kRows);
    return static_cast<int>(items < kMaxItems ? items : kMaxItems);
  });
  pdl_wait();  // launched early behind the chunk scores (what was read above is older than their launch)
  const int total = off[b.batch];
  int it = static_cast<int>(static_cast<int64_t>(total) * blockIdx.x / gridDim.x);
  const int it1 = static_cast<int>(static_cast<int64_t>(total) * (blockIdx.x + 1) / gridDim.x);
  if (it >= it1) return;
  int s = 0;
  {
    int lo = 0, hi = b.batch - 1;  // the last sequence whose first item is at or before `it`
    while (lo < hi) {
      const int mid = (lo + hi + 1) >> 1;
      if (off[mid] <= it) lo = mid;
      else hi = mid - 1;
    }
    s = lo;
  }
  const int pshift = c.shift - 2, pmask = (1 << pshift) - 1;
  // this lane's piece of pool p + 8 * nt + g of a run (p: the warp's first pool of a tile); null past the row's
  // pools or without a page
  auto source = [&](const Run& x, int p, int nt) -> const uint4* {
    p += nt * 8 + g;
    if (p >= x.pools) return nullptr;
    const int page = __ldg(x.table + (p >> pshift));
    if (static_cast<unsigned>(page) >= static_cast<unsigned>(c.num_pages)) {
      record_status(status, kStatusInternal);
      return nullptr;
    }
    return reinterpret_cast<const uint4*>(c.khat + page * c.khat_stride + (p & pmask) * (2 * kDi)) + t;
  };
  uint4 kf[4][4];
  auto fetch = [&](uint4 (&k)[4], const uint4* src) {
#pragma unroll
    for (int e = 0; e < 4; ++e) k[e] = src ? __ldcs(src + 4 * e) : make_uint4(0u, 0u, 0u, 0u);
  };
  uint4 qa[kMt][2][2];  // [m-tile][head g / g + 8][half of the 64 dims]
  float wv[kMt][2];
  int64_t in_regs = -1;  // the row whose query they hold

  // The pooled keys of the next tile are fetched n-tile by n-tile into the
  // registers that the last row of this one has just used, so that the loads
  // of three n-tiles are always in flight behind the products of the fourth.
  Run cur = next_run(b, c.shift, kRows, off, row0, row1, it1, &it, &s);
  if (cur.nr == 0) return;
  int p = cur.p0 + warp * 32;  // the warp's first pool
#pragma unroll
  for (int nt = 0; nt < 4; ++nt) fetch(kf[nt], source(cur, p, nt));
  while (true) {
    Run nxt = cur;
    int pn = p + kTile;
    if (pn >= cur.p1) {
      nxt = next_run(b, c.shift, kRows, off, row0, row1, it1, &it, &s);
      pn = nxt.p0 + warp * 32;
    }
    const uint4* ahead[4];
#pragma unroll
    for (int nt = 0; nt < 4; ++nt) ahead[nt] = nxt.nr > 0 ? source(nxt, pn, nt) : nullptr;
    for (int rr = 0; rr < cur.nr; ++rr) {
      const int64_t row = cur.ra + rr;
      if (in_regs != row) {
        in_regs = row;
#pragma unroll
        for (int m = 0; m < kMt; ++m)
#pragma unroll
          for (int u = 0; u < 2; ++u) {
            const int h = 16 * m + 8 * u + g;
            const uint4* src = reinterpret_cast<const uint4*>(q + (row * Hi + h) * kDi);
#pragma unroll
            for (int e = 0; e < 2; ++e) qa[m][u][e] = h < Hi ? __ldg(src + t + 4 * e) : make_uint4(0u, 0u, 0u, 0u);
            wv[m][u] = h < Hi ? __ldg(w + row * Hi + h) : 0.f;
          }
      }
      const bool last = rr + 1 == cur.nr;
      float v[4][2];
#pragma unroll
      for (int nt = 0; nt < 4; ++nt) {
        v[nt][0] = v[nt][1] = 0.f;
#pragma unroll
        for (int m = 0; m < kMt; ++m) {
          float acc[4] = {0.f, 0.f, 0.f, 0.f};
#pragma unroll
          for (int e = 0; e < 4; ++e) {  // 0, 1: hi; 2, 3: lo
            const uint4 x = qa[m][0][e & 1], y = qa[m][1][e & 1], z = kf[nt][e];
            const uint32_t a0[4] = {x.x, y.x, x.y, y.y}, a1[4] = {x.z, y.z, x.w, y.w};
            mma_bf16_16816(acc, a0, z.x, z.y);
            mma_bf16_16816(acc, a1, z.z, z.w);
          }
          v[nt][0] = fmaf(wv[m][0], fmaxf(acc[0], 0.f), v[nt][0]);
          v[nt][1] = fmaf(wv[m][0], fmaxf(acc[1], 0.f), v[nt][1]);
          v[nt][0] = fmaf(wv[m][1], fmaxf(acc[2], 0.f), v[nt][0]);
          v[nt][1] = fmaf(wv[m][1], fmaxf(acc[3], 0.f), v[nt][1]);
        }
        if (last) fetch(kf[nt], ahead[nt]);
      }
      // sum over the 8 head lanes, scattering the 8 values over them
      const bool b4 = lane & 16, b3 = lane & 8, b2 = lane & 4;
      float x2[2][2];
#pragma unroll
      for (int a = 0; a < 2; ++a)
#pragma unroll
        for (int z = 0; z < 2; ++z) {
          const float keep = b4 ? v[2 + a][z] : v[a][z], give = b4 ? v[a][z] : v[2 + a][z];
          x2[a][z] = keep + __shfl_xor_sync(0xffffffffu, give, 16);
        }
      float x1[2];
#pragma unroll
      for (int z = 0; z < 2; ++z) {
        const float keep = b3 ? x2[1][z] : x2[0][z], give = b3 ? x2[0][z] : x2[1][z];
        x1[z] = keep + __shfl_xor_sync(0xffffffffu, give, 8);
      }
      const float sum = (b2 ? x1[1] : x1[0]) + __shfl_xor_sync(0xffffffffu, b2 ? x1[0] : x1[1], 4);
      const int at = p + (b4 ? 16 : 0) + (b3 ? 8 : 0) + 2 * t + (b2 ? 1 : 0);
      float top = -INFINITY;
      if (at < cur.pools) {
        scores[(row - row0) * ld + at] = sum;
        top = sum;
      }
      // the largest of each eight pools (an n-tile: lanes alike in bits 3 and 4)
#pragma unroll
      for (int o = 1; o < 8; o <<= 1) top = fmaxf(top, __shfl_xor_sync(0xffffffffu, top, o));
      if ((lane & 7) == 0 && at < cur.pools) tops[((row - row0) * ld + at) >> 3] = top;
    }
    if (nxt.nr == 0) return;
    cur = nxt;
    p = pn;
  }
}

// ================================================================= selection
// One CTA per row of n > topk scores in global memory, with the largest score
// of each eight pools beside them (the score kernels write both):
//   1. n > 8 * topk: the topk-th largest of the groups' maxima is a lower bound
//      t of the row's topk-th largest score T, for topk groups hold a score
//      that reaches it.  Only the groups whose maximum reaches t
//      can hold a score that does; theirs are listed.  (t is taken from a
//      histogram, one step low at the most.)  For independent scores that is
//      little more than topk scores from topk groups: of a row of 32768, 16 KB
//      of maxima and 16 KB of scores are read instead of 128 KB.  Shorter rows
//      are not listed: steps 2 and 3 read the row itself, from L1.
//   2. T: a histogram of equal steps between its extrema (monotone
//      in the score, whatever the rounding) finds the bin that holds T; while
//      that bin has more than kFew scores, a histogram of equal steps of their
//      32-bit keys narrows it; the few left are ranked against each other.
//   3. Scores above T set a bit each, those equal to T one in a second map; the
//      set bits in order are the row, ascending, the first ties with them.
// Latency bounds it: 10.6 us for one row or 64 of 32768 (1024 threads each), 65
// us by ncu for 2048 rows (256 threads, five rows an SM at a time; six, at 40
// registers, 80).  A threshold from a sample and one pass over the row took 118
// us for those; a warp per row 270.
// Should the list run over (hundreds of ties or of neighbours alike), or the
// maxima have no finite range, a long row goes the short rows' way: the same
// result, more passes.
constexpr int kBinBits = 10;  // (11 took 80 us for the 2048 rows)
constexpr int kBins = 1 << kBinBits;
constexpr int kFew = 512;
constexpr int kSelMaxWarps = 32;
constexpr int kSegment = 1 << 17;  // pools whose bits are held at once (2 x 16 KB of bits)

// The order-preserving 32-bit image of a score (-0 and +0 are one), and the
// score of a key.
__device__ __forceinline__ uint32_t score_key(float f) {
  uint32_t u = __float_as_uint(f);
  if ((u & 0x7FFFFFFFu) == 0u) u = 0u;
  return (u & 0x80000000u) ? ~u : (u | 0x80000000u);
}
__device__ __forceinline__ float key_score(uint32_t k) {
  return __uint_as_float((k & 0x80000000u) ? (k & 0x7FFFFFFFu) : ~k);
}

struct alignas(16) SelSmem {
  uint32_t hist[kBins];
  uint32_t few[kFew];
  uint32_t wred[2][2][kSelMaxWarps];  // two buffers, used in turn: one barrier a reduction
  uint32_t lo, hi;
  uint32_t nfew;
  uint32_t bin, above, inbin;
  uint32_t T, take;
};
static_assert(sizeof(SelSmem) % 16 == 0, "what lies after it is read 16 bytes at a time");

// extrema over the block; every thread gets them
template <int kThr>
__device__ __forceinline__ void sel_minmax(SelSmem& sm, uint32_t& lo, uint32_t& hi, int& turn) {
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  lo = __reduce_min_sync(0xffffffffu, lo);
  hi = __reduce_max_sync(0xffffffffu, hi);
  if (lane == 0) {
    sm.wred[turn][0][warp] = lo;
    sm.wred[turn][1][warp] = hi;
  }
  __syncthreads();
  lo = __reduce_min_sync(0xffffffffu, lane < kThr / 32 ? sm.wred[turn][0][lane] : 0xFFFFFFFFu);
  hi = __reduce_max_sync(0xffffffffu, lane < kThr / 32 ? sm.wred[turn][1][lane] : 0u);
  turn ^= 1;
}

// Exclusive prefixes of v and u over the block in thread order, and their totals.
template <int kThr>
__device__ __forceinline__ void sel_scan2(SelSmem& sm, uint32_t& v, uint32_t& u, uint32_t* v_all, uint32_t* u_all,
                                          int& turn) {
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  uint32_t x = v, y = u;
#pragma unroll
  for (int o = 1; o < 32; o <<= 1) {
    const uint32_t a = __shfl_up_sync(0xffffffffu, x, o), b = __shfl_up_sync(0xffffffffu, y, o);
    if (lane >= o) {
      x += a;
      y += b;
    }
  }
  if (lane == 31) {
    sm.wred[turn][0][warp] = x;
    sm.wred[turn][1][warp] = y;
  }
  __syncthreads();
  const uint32_t wx = lane < kThr / 32 ? sm.wred[turn][0][lane] : 0u, wy = lane < kThr / 32 ? sm.wred[turn][1][lane] : 0u;
  *v_all = __reduce_add_sync(0xffffffffu, wx);
  *u_all = __reduce_add_sync(0xffffffffu, wy);
  v = __reduce_add_sync(0xffffffffu, lane < warp ? wx : 0u) + x - v;
  u = __reduce_add_sync(0xffffffffu, lane < warp ? wy : 0u) + y - u;
  turn ^= 1;
}

// The bin of the complete histogram (a barrier precedes) that holds the need-th
// largest: sm.bin, sm.above (scores in higher bins), sm.inbin.
template <int kThr>
__device__ __forceinline__ void sel_find(SelSmem& sm, uint32_t need, int& turn) {
  constexpr int kPer = kBins / kThr;
  static_assert(kPer * kThr == kBins, "a thread's bins");
  uint32_t cnt[kPer], sum = 0;  // bins in descending order: thread 0 has the highest
#pragma unroll
  for (int j = 0; j < kPer; ++j) {
    cnt[j] = sm.hist[kBins - 1 - (kPer * threadIdx.x + j)];
    sum += cnt[j];
  }
  uint32_t before = sum, none = 0u, all, zero;
  sel_scan2<kThr>(sm, before, none, &all, &zero, turn);
  if (before < need && need <= before + sum) {
#pragma unroll
    for (int j = 0; j < kPer; ++j) {
      if (before < need && need <= before + cnt[j]) {
        sm.bin = kBins - 1 - (kPer * threadIdx.x + j);
        sm.above = before;
        sm.inbin = cnt[j];
      }
      before += cnt[j];
    }
  }
  __syncthreads();
}

// Equal steps of the score between two keys: bin(f) is monotone in f (scores
// outside fall into the first and the last).  inv = 0 where the range is not
// finite or empty.
struct Steps {
  float lo, inv;
  __device__ __forceinline__ static Steps of(uint32_t klo, uint32_t khi) {
    Steps s;
    s.lo = key_score(klo);
    const float range = key_score(khi) - s.lo;
    s.inv = range > 0.f && range < INFINITY ? fminf(static_cast<float>(kBins) / range, 3.0e38f) : 0.f;
    return s;
  }
  __device__ __forceinline__ int bin(float f) const {
    return static_cast<int>(fminf(fmaxf((f - lo) * inv, 0.f), static_cast<float>(kBins - 1)));
  }
};

// The need-th largest of the cnt > need scores at v (shared or global memory):
// key T, and how many scores equal to it are among the need largest.  sm.hist
// is their complete histogram by st (a barrier has passed since), or st.inv is
// 0; sm.nfew is zero.
template <int kThr>
__device__ __forceinline__ void sel_kth(SelSmem& sm, uint32_t need, int cnt, const float* v, const Steps& st,
                                        uint32_t* T, uint32_t* take, int& turn) {
  const int tid = threadIdx.x;
  uint32_t lo = 0u, hi = 0u, members = static_cast<uint32_t>(cnt);
  int bin0 = -1;  // -1: every score
  if (st.inv > 0.f) {
    sel_find<kThr>(sm, need, turn);
    members = sm.inbin;
    need -= sm.above;
    bin0 = static_cast<int>(sm.bin);
  }
  bool windowed = false;  // the members are the scores with keys in [lo, hi]
  auto inside = [&](float f, uint32_t k) {
    return windowed ? k >= lo && k <= hi : bin0 < 0 || st.bin(f) == bin0;
  };
  while (members > static_cast<uint32_t>(kFew)) {
    uint32_t a = 0xFFFFFFFFu, z = 0u;
    for (int j = tid; j < cnt; j += kThr) {
      const float f = v[j];
      const uint32_t k = score_key(f);
      if (inside(f, k)) {
        a = min(a, k);
        z = max(z, k);
      }
    }
    for (int j = tid; j < kBins; j += kThr) sm.hist[j] = 0u;
    sel_minmax<kThr>(sm, a, z, turn);
    lo = a;
    hi = z;
    windowed = true;
    if (lo == hi) break;
    const int bits = 32 - __clz(hi - lo);
    const int sh = bits > kBinBits ? bits - kBinBits : 0;
    for (int j = tid; j < cnt; j += kThr) {
      const uint32_t k = score_key(v[j]);
      if (k >= lo && k <= hi) atomicAdd(&sm.hist[(k - lo) >> sh], 1u);
    }
    __syncthreads();
    sel_find<kThr>(sm, need, turn);
    members = sm.inbin;
    need -= sm.above;
    const uint32_t nlo = lo + (sm.bin << sh);
    const uint64_t nhi = static_cast<uint64_t>(nlo) + ((1ull << sh) - 1ull);
    lo = nlo;
    hi = nhi < hi ? static_cast<uint32_t>(nhi) : hi;
    if (sh == 0) break;
  }
  if (windowed && lo == hi) {
    *T = lo;
    *take = need;
    return;
  }
  for (int j = tid; j < cnt; j += kThr) {
    const float f = v[j];
    const uint32_t k = score_key(f);
    if (inside(f, k)) {
      const uint32_t at = atomicAdd(&sm.nfew, 1u);
      if (at < static_cast<uint32_t>(kFew)) sm.few[at] = k;
    }
  }
  __syncthreads();
  const uint32_t m = min(sm.nfew, static_cast<uint32_t>(kFew));
  for (uint32_t j = tid; j < m; j += kThr) {
    const uint32_t mine = sm.few[j];
    uint32_t gt = 0u, eq = 0u;
    for (uint32_t e = 0; e < m; ++e) {
      gt += sm.few[e] > mine;
      eq += sm.few[e] == mine;
    }
    if (gt < need && need <= gt + eq) {  // every thread with T writes the same
      sm.T = mine;
      sm.take = need - gt;
    }
  }
  __syncthreads();
  *T = sm.T;
  *take = sm.take;
}

template <int kCap, int kThr>
__global__ void __launch_bounds__(kThr, kThr == 1024 ? 1 : kThr == 256 ? 5 : kThr == 128 ? 10 : 2)
    paged_select_kernel(const BatchView b, int shift, int64_t row0, const float* __restrict__ scores, int64_t ld,
                        const float* __restrict__ tops, int topk, int words_room, int32_t* __restrict__ pool_idx,
                        unsigned* status) {
  extern __shared__ __align__(16) uint8_t smem_raw[];
  SelSmem& sm = *reinterpret_cast<SelSmem*>(smem_raw);
  float* cval = reinterpret_cast<float*>(smem_raw + sizeof(SelSmem));    // [kCap] candidates
  int32_t* cidx = reinterpret_cast<int32_t*>(cval + kCap);                // [kCap] their pools
  int32_t* gidx = cidx + kCap;                                            // [kCap / 2] groups to look into
  uint32_t* above = reinterpret_cast<uint32_t*>(gidx + kCap / 2);         // [words_room] bits: scores above T
  uint32_t* equal = above + words_room;                                   // [words_room] bits: scores equal to T
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
  const int64_t lrow = blockIdx.x, row = row0 + lrow;
  int turn = 0;
  if (tid == 0) sm.nfew = 0u;
  for (int j = tid; j < kBins; j += kThr) sm.hist[j] = 0u;
  const RowAt at = warp_locate(b, shift, row, lane, status);
  pdl_wait();  // the scores are written (what was read above is older than their launch)
  if (at.seq < 0) return;  // padding behind the last sequence
  int32_t* orow = pool_idx + row * topk;
  const int n = at.pos < 0 ? 0 : static_cast<int>(at.pos >> 2);
  if (n <= topk) {  // every pool (or, for a row without a position, nothing)
    for (int j = tid; j < topk; j += kThr) orow[j] = j < n ? j : -1;
    return;
  }
  const float* srow = scores + lrow * ld;
  for (int k = tid; k < min(kSegment, n + 31) >> 5; k += kThr) above[k] = equal[k] = 0u;

  // ---- candidates
  bool listed = false;
  int m = n;  // scores that T is looked for in: the list's, or the row's
  Steps st{0.f, 0.f};
  if (kCap > 0 && n > 8 * topk) {
    const int groups = n >> 3;  // whole groups of eight; what is left of the row is listed in any case
    const float* trow = tops + ((lrow * ld) >> 3);
    uint32_t lo = 0xFFFFFFFFu, hi = 0u;
    for (int j = tid; j < groups; j += kThr) {
      const uint32_t k = score_key(trow[j]);
      lo = min(lo, k);
      hi = max(hi, k);
    }
    sel_minmax<kThr>(sm, lo, hi, turn);
    st = Steps::of(lo, hi);
    if (st.inv > 0.f) {
      for (int j = tid; j < groups; j += kThr) atomicAdd(&sm.hist[st.bin(trow[j])], 1u);  // (from L1)
      __syncthreads();
      sel_find<kThr>(sm, static_cast<uint32_t>(topk), turn);
      const int bin = static_cast<int>(sm.bin);
      const Steps by = st;  // a score reaches t when it lies in this bin or a higher one
      st = Steps::of(score_key(st.lo + static_cast<float>(bin) / st.inv), hi);
      for (int j = tid; j < kBins; j += kThr) sm.hist[j] = 0u;
      // the groups whose maximum does
      // (4096 at a time: one scan for a row of 32768)
      constexpr int kGu = 4096 / kThr;
      uint32_t found = 0u, none = 0u, all, zero;
      for (int j0 = 0; j0 < groups; j0 += kGu * kThr) {
        uint32_t hit = 0u;
#pragma unroll
        for (int u = 0; u < kGu; ++u) {
          const int j = j0 + u * kThr + tid;
          if (j < groups && by.bin(trow[j]) >= bin) hit |= 1u << u;
        }
        uint32_t to = __popc(hit);
        sel_scan2<kThr>(sm, to, none, &all, &zero, turn);
        to += found;
        found += all;
        while (hit) {
          const int u = __ffs(hit) - 1;
          hit &= hit - 1u;
          if (to < static_cast<uint32_t>(kCap / 2)) gidx[to] = j0 + u * kThr + tid;
          ++to;
        }
      }
      __syncthreads();
      listed = found <= static_cast<uint32_t>(kCap / 2);
      if (listed) {
        // their scores: kHu halves of a group a thread, all asked for before the first is looked at
        constexpr int kHu = kThr == 1024 ? 2 : 4;
        uint32_t before = 0u;
        const int halves = 2 * static_cast<int>(found) + 2;  // and the row's last n % 8
        for (int e0 = 0; e0 < halves; e0 += kHu * kThr) {
          float4 x[kHu];
          int at[kHu];
#pragma unroll
          for (int u = 0; u < kHu; ++u) {
            const int e = e0 + u * kThr + tid;
            at[u] = n;
            x[u] = make_float4(0.f, 0.f, 0.f, 0.f);
            if (e < halves) {
              at[u] = 8 * (e < halves - 2 ? gidx[e >> 1] : groups) + 4 * (e & 1);
              if (at[u] < n) x[u] = *reinterpret_cast<const float4*>(srow + at[u]);  // (rows are whole quads)
            }
          }
          uint32_t hit = 0u;
#pragma unroll
          for (int u = 0; u < kHu; ++u) {
            const float f[4] = {x[u].x, x[u].y, x[u].z, x[u].w};
#pragma unroll
            for (int v = 0; v < 4; ++v)
              if (at[u] + v < n && by.bin(f[v]) >= bin) hit |= 1u << (4 * u + v);
          }
          uint32_t to = __popc(hit);
          sel_scan2<kThr>(sm, to, none, &all, &zero, turn);
          to += before;
          before += all;
#pragma unroll
          for (int u = 0; u < kHu; ++u) {
            const float f[4] = {x[u].x, x[u].y, x[u].z, x[u].w};
#pragma unroll
            for (int v = 0; v < 4; ++v)
              if ((hit >> (4 * u + v)) & 1u) {
                if (to < static_cast<uint32_t>(kCap)) {
                  cval[to] = f[v];
                  cidx[to] = at[u] + v;
                  atomicAdd(&sm.hist[st.bin(f[v])], 1u);
                }
                ++to;
              }
          }
        }
        m = static_cast<int>(before);
        listed = m >= topk && m <= kCap;
      }
      if (!listed) m = n;
    }
  }
  if (!listed) {
    __syncthreads();
    for (int j = tid; j < kBins; j += kThr) sm.hist[j] = 0u;
    uint32_t lo = 0xFFFFFFFFu, hi = 0u;
#pragma unroll 4
    for (int j = tid; j < n; j += kThr) {
      const uint32_t k = score_key(srow[j]);
      lo = min(lo, k);
      hi = max(hi, k);
    }
    sel_minmax<kThr>(sm, lo, hi, turn);
    st = Steps::of(lo, hi);
    if (st.inv > 0.f) {
#pragma unroll 4
      for (int j = tid; j < n; j += kThr) atomicAdd(&sm.hist[st.bin(srow[j])], 1u);
    }
  }
  __syncthreads();

  // ---- T: of the list, or of the row itself
  uint32_t T = 0u, take = static_cast<uint32_t>(topk);  // (a list of topk scores is kept whole: no key is below 0)
  if (m > topk) sel_kth<kThr>(sm, static_cast<uint32_t>(topk), m, listed ? cval : srow, st, &T, &take, turn);

  // ---- the row, segment by segment
  uint32_t done = 0u, ties = 0u;  // written so far; ties met so far
  for (int s0 = 0; s0 < n; s0 += kSegment) {
    const int len = min(kSegment, n - s0), words = (len + 31) >> 5;
    if (listed) {
      if (s0 > 0) {
        for (int k = tid; k < words; k += kThr) above[k] = equal[k] = 0u;
        __syncthreads();
      }
      for (int j = tid; j < m; j += kThr) {
        const int p = cidx[j] - s0;
        const uint32_t k = score_key(cval[j]);
        if (p >= 0 && p < len && k >= T) atomicOr((k > T ? above : equal) + (p >> 5), 1u << (p & 31));
      }
    } else {
      for (int k = warp; k < words; k += kThr / 32) {
        const int j = s0 + 32 * k + lane;
        const uint32_t key = j < n ? score_key(srow[j]) : 0u;
        const uint32_t g = __ballot_sync(0xffffffffu, j < n && key > T), e = __ballot_sync(0xffffffffu, j < n && key == T);
        if (lane == 0) {
          above[k] = g;
          equal[k] = e;
        }
      }
    }
    __syncthreads();
    const int wpt = (words + kThr - 1) / kThr;
    const int k0 = min(tid * wpt, words), k1 = min(k0 + wpt, words);
    uint32_t g = 0u, e = 0u, g_all, e_all;
    for (int k = k0; k < k1; ++k) {
      g += __popc(above[k]);
      e += __popc(equal[k]);
    }
    sel_scan2<kThr>(sm, g, e, &g_all, &e_all, turn);
    uint32_t pe = ties + e;
    uint32_t pos = done + g + (min(pe, take) - min(ties, take));
    for (int k = k0; k < k1; ++k) {
      const uint32_t ek = equal[k];
      uint32_t bits = above[k] | ek;
      while (bits) {
        const int z = __ffs(bits) - 1;
        bits &= bits - 1u;
        const bool tie = (ek >> z) & 1u;
        if (tie && pe++ >= take) continue;
        if (pos < static_cast<uint32_t>(topk)) orow[pos] = s0 + 32 * k + z;
        ++pos;
      }
    }
    done += g_all + (min(ties + e_all, take) - min(ties, take));
    ties += e_all;
    if (s0 + kSegment < n) __syncthreads();  // the bits are read: the next segment may set its own
  }
}

template <int kMt>
cudaError_t launch_scores(const CacheView& c, const BatchView& b, const void* q_idx, const float* w, int Hi,
                          int64_t row0, int64_t nrows, TcRule tc, float* scores, float* tops, int64_t ld,
                          const LaunchCtx& ctx) {
  const size_t smem = static_cast<size_t>(b.batch + 1) * sizeof(int);
  const int grid = ctx.num_sms * (kMt <= 2 ? 3 : 2);
  return launch_ex(ctx, paged_score_kernel<kMt>, dim3(grid), dim3(kThreads), smem, c, b,
                   static_cast<const __nv_bfloat16*>(q_idx), w, Hi, row0, row0 + nrows, tc, scores, tops, ld,
                   ctx.status);
}

template <int kCap, int kThr>
cudaError_t launch_select(const BatchView& b, int shift, int64_t row0, int64_t nrows, const float* scores,
                          const float* tops, int64_t ld, int topk, int32_t* pool_idx, const LaunchCtx& ctx) {
  const int64_t pools = static_cast<int64_t>(b.max_pages) << (shift - 2);
  const int words = static_cast<int>((pools < kSegment ? pools : kSegment) + 31) / 32;
  constexpr size_t kFixed = sizeof(SelSmem) + static_cast<size_t>(kCap) * 10;
  constexpr size_t kMost = kFixed + 2 * (kSegment / 32) * 4;
  static_assert(kMost <= 232448 - 1024, "shared memory per CTA");
  static std::atomic<bool> attr_done[kAttrDevices];
  const cudaError_t e = set_smem_limit_once(paged_select_kernel<kCap, kThr>, static_cast<int>(kMost), attr_done);
  if (e != cudaSuccess) return e;
  LaunchCtx early = ctx;
  early.pdl = 1;
  return launch_ex(early, paged_select_kernel<kCap, kThr>, dim3(static_cast<unsigned>(nrows)), dim3(kThr),
                   kFixed + static_cast<size_t>(words) * 8, b, shift, row0, scores, ld, tops, topk, words,
                   pool_idx, ctx.status);
}

}  // namespace

cudaError_t launch_paged_scores(const CacheView& c, const BatchView& b, const void* q_idx, const float* w, int Hi,
                                int64_t row0, int64_t nrows, TcRule tc, float* scores, float* tops, int64_t ld,
                                bool early, const LaunchCtx& call) {
  LaunchCtx ctx = call;
  ctx.pdl = early;
  if (Hi <= 16) return launch_scores<1>(c, b, q_idx, w, Hi, row0, nrows, tc, scores, tops, ld, ctx);
  if (Hi <= 32) return launch_scores<2>(c, b, q_idx, w, Hi, row0, nrows, tc, scores, tops, ld, ctx);
  return launch_scores<4>(c, b, q_idx, w, Hi, row0, nrows, tc, scores, tops, ld, ctx);
}

cudaError_t launch_paged_select(const BatchView& b, int shift, int64_t row0, int64_t nrows, const float* scores,
                                const float* tops, int64_t ld, int topk, int32_t* pool_idx, const LaunchCtx& ctx) {
  // A list of four times the largest topk of its class.  A row per SM or
  // fewer: 1024 threads, for the latency of a row; more: five of 256 threads
  // share an SM.  1024 / 256 threads at 131072 tokens, with 4 us of event
  // overhead: 14.4 / 17.4 us for 128 rows, 22.9 / 19.9 for 192, 31.7 / 22.7 for 384.
  const bool few = nrows <= ctx.num_sms;
  // Short rows by the thousand: no list is ever made, and ten of 128 threads
  // share an SM.  (The host does not know the rows' lengths: the table's width
  // decides, and short rows in a wide table go the longer rows' way.)  256 / 128
  // threads, 2048 pools: 4096 rows 51.5 / 38.2, 1000 rows 20.5 / 16.6, 300 rows (one
  // turn either way) 12.3 / 14.3; 4096 pools, 2000 rows 44.3 / 45.3.
  const int64_t pools = static_cast<int64_t>(b.max_pages) << (shift - 2);
  if (nrows > 5 * static_cast<int64_t>(ctx.num_sms) && pools <= 2048 && pools <= 8 * topk)
    return launch_select<0, 128>(b, shift, row0, nrows, scores, tops, ld, topk, pool_idx, ctx);
  if (topk <= 512)
    return few ? launch_select<2048, 1024>(b, shift, row0, nrows, scores, tops, ld, topk, pool_idx, ctx)
               : launch_select<2048, 256>(b, shift, row0, nrows, scores, tops, ld, topk, pool_idx, ctx);
  return few ? launch_select<8192, 1024>(b, shift, row0, nrows, scores, tops, ld, topk, pool_idx, ctx)
             : launch_select<8192, 512>(b, shift, row0, nrows, scores, tops, ld, topk, pool_idx, ctx);
}

}  // namespace dsa
