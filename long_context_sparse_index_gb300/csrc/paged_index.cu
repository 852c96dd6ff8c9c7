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

// ================================================================= scores, few rows a sequence
// Memory-bound: each pooled key is read once for up to kRows rows of its
// sequence.  A warp takes 32 pools (four MMA n-tiles of 8).  The k order of a
// dot product is free, so the MMA fragments are read straight from global
// memory: lane (g, t) holds 16-byte pieces t and t + 4 of pool g's hi (and lo)
// half, which are its B fragments of four k-steps, and the same pieces of
// head g's (and g + 8's) query as A fragments.  No shared memory, no
// transposes, 64 bytes of a row per quad of lanes and load.
//
// Work items are (sequence, group of kRows rows, 256 pools); every CTA walks
// an equal, contiguous range of them.
constexpr int kWarps = 8;
constexpr int kThreads = 32 * kWarps;
constexpr int kTile = 32 * kWarps;  // pools of an item
constexpr int kRows = 8;            // rows of an item
constexpr int kMaxItems = 1 << 22;  // items of one sequence (a pass scores at most 2^31 pairs: fewer than half of it)

// Rows of sequence s within launch rows [row0, row1): first row and count.
__device__ __forceinline__ int seq_rows(const BatchView& b, int s, int64_t row0, int64_t row1, int64_t* first) {
  const int64_t c0 = __ldg(b.cu + s), c1 = __ldg(b.cu + s + 1);
  const int64_t lo = c0 > row0 ? c0 : row0, hi = c1 < row1 ? c1 : row1;
  *first = lo;
  return hi > lo ? static_cast<int>(hi - lo) : 0;
}

// Pools that the last of rows [first, first + n) of sequence s may see; 0 for
// lengths and offsets that contradict each other (the selection records them).
__device__ __forceinline__ int64_t seq_pools(const BatchView& b, int shift, int s, int64_t first, int64_t n) {
  const int64_t c1 = __ldg(b.cu + s + 1), len = __ldg(b.lens + s);
  if (len > (static_cast<int64_t>(b.max_pages) << shift)) return 0;
  const int64_t i = len - c1 + first + n - 1;
  return i >= 4 ? i >> 2 : 0;
}

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
    if (threadIdx.x == 0) s_base = min(s_base + all, 1 << 30);
    __syncthreads();
  }
  if (threadIdx.x == 0) off[batch] = s_base;
  __syncthreads();
}

template <int kMt>
__global__ void __launch_bounds__(kThreads, kMt <= 2 ? 2 : 1)
    paged_score_kernel(const CacheView c, const BatchView b, const __nv_bfloat16* __restrict__ q,
                       const float* __restrict__ w, int Hi, int64_t row0, int64_t row1, float* __restrict__ scores,
                       int64_t ld, unsigned* status) {
  extern __shared__ int off[];
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  const int g = lane >> 2, t = lane & 3;
  item_prefix(off, b.batch, [&](int s) {
    int64_t first;
    const int n = seq_rows(b, s, row0, row1, &first);
    if (n == 0) return 0;
    const int64_t tiles = (seq_pools(b, c.shift, s, first, n) + kTile - 1) / kTile;
    const int64_t items = tiles * ((n + kRows - 1) / kRows);
    return static_cast<int>(items < kMaxItems ? items : kMaxItems);
  });
  const int total = off[b.batch];
  const int it0 = static_cast<int>(static_cast<int64_t>(total) * blockIdx.x / gridDim.x);
  const int it1 = static_cast<int>(static_cast<int64_t>(total) * (blockIdx.x + 1) / gridDim.x);
  if (it0 >= it1) return;
  int s = 0;
  {
    int lo = 0, hi = b.batch - 1;  // the last sequence whose first item is at or before it0
    while (lo < hi) {
      const int mid = (lo + hi + 1) >> 1;
      if (off[mid] <= it0) lo = mid;
      else hi = mid - 1;
    }
    s = lo;
  }
  uint4 qa[kMt][2][2];  // [m-tile][head g / g + 8][half of the 64 dims]
  float wv[kMt][2];
  int64_t in_regs = -1;  // the row whose query they hold
  const int pshift = c.shift - 2;
  for (int it = it0; it < it1; ++it) {
    while (s + 1 < b.batch && it >= off[s + 1]) ++s;
    int64_t first;
    const int n = seq_rows(b, s, row0, row1, &first);
    const int tiles = static_cast<int>((seq_pools(b, c.shift, s, first, n) + kTile - 1) / kTile);
    if (tiles == 0) continue;
    const int rg = (it - off[s]) / tiles, tile = (it - off[s]) % tiles;
    const int64_t ra = first + rg * kRows;
    const int nr = static_cast<int>(min(static_cast<int64_t>(kRows), first + n - ra));
    if (nr <= 0) continue;
    const int64_t pools = seq_pools(b, c.shift, s, ra, nr);  // of this group's last row
    const int64_t p0 = static_cast<int64_t>(tile) * kTile + warp * 32;
    if (p0 >= pools) continue;
    // pooled keys of the warp's 32 pools
    uint4 kf[4][4];
#pragma unroll
    for (int nt = 0; nt < 4; ++nt) {
      const int64_t p = p0 + nt * 8 + g;
      const uint4* src = nullptr;
      if (p < pools) {
        const int page = page_of(b, c.num_pages, s, static_cast<int>(p >> pshift), status);
        if (page >= 0)
          src = reinterpret_cast<const uint4*>(c.khat + page * c.khat_stride +
                                               (p & ((1 << pshift) - 1)) * (2 * kDi));
      }
#pragma unroll
      for (int e = 0; e < 4; ++e) kf[nt][e] = src ? __ldg(src + t + 4 * e) : make_uint4(0u, 0u, 0u, 0u);
    }
    for (int rr = 0; rr < nr; ++rr) {
      const int64_t row = ra + rr;
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
      const int64_t p = p0 + (b4 ? 16 : 0) + (b3 ? 8 : 0) + 2 * t + (b2 ? 1 : 0);
      if (p < pools) scores[(row - row0) * ld + p] = sum;
    }
  }
}

// ================================================================= selection
// One CTA per row of n > topk scores in global memory (L2 as a rule):
//   1. n > kCap: a strided sample gives a score t that more than topk scores
//      reach and far fewer than kCap (five standard deviations of the sampling
//      to either side), and one pass over the row lists the scores >= t.  The
//      row is read once.  Shorter rows are listed whole.
//   2. The topk-th largest score T of the list: a histogram of equal steps
//      between its extrema (monotone in the score, whatever the rounding) finds
//      the bin that holds T; while that bin has more than kFew scores, a
//      histogram of equal steps of their 32-bit keys narrows it; the few left
//      are ranked against each other.
//   3. Scores above T set a bit each, those equal to T one in a second map; the
//      set bits in order are the row, ascending, the first ties with them.
// Should the list come out too short or too long (correlated or non-finite
// scores), step 2 and 3 run over the row itself: the same result, more passes.
// Lists and not sorted keys: a row of 32768 costs one read of 128 KB and work
// on about 1200 candidates; several rows share an SM and hide each other's
// barriers.
constexpr int kSelThreads = 512;
constexpr int kSelWarps = kSelThreads / 32;
constexpr int kBins = 2048;
constexpr int kFew = kSelThreads;
constexpr int kSegment = 1 << 18;  // pools whose bits are held at once (2 x 32 KB of bits)

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
  uint32_t wred[2][kSelWarps];
  uint32_t lo, hi;
  uint32_t nfew, nlist;
  uint32_t bin, above, inbin;
  uint32_t T, take;
  int seq;
};
static_assert(sizeof(SelSmem) % 16 == 0, "what lies after it is read 16 bytes at a time");

// extrema over the block; every thread gets them
__device__ __forceinline__ void sel_minmax(SelSmem& sm, uint32_t& lo, uint32_t& hi) {
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  lo = __reduce_min_sync(0xffffffffu, lo);
  hi = __reduce_max_sync(0xffffffffu, hi);
  if (lane == 0) {
    sm.wred[0][warp] = lo;
    sm.wred[1][warp] = hi;
  }
  __syncthreads();
  lo = __reduce_min_sync(0xffffffffu, lane < kSelWarps ? sm.wred[0][lane] : 0xFFFFFFFFu);
  hi = __reduce_max_sync(0xffffffffu, lane < kSelWarps ? sm.wred[1][lane] : 0u);
  __syncthreads();  // read: wred may be written again
}

// Exclusive prefix of v over the block in thread order, and the total.
__device__ __forceinline__ uint32_t sel_scan(SelSmem& sm, uint32_t v, uint32_t* total) {
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  uint32_t x = v;
#pragma unroll
  for (int o = 1; o < 32; o <<= 1) {
    const uint32_t y = __shfl_up_sync(0xffffffffu, x, o);
    if (lane >= o) x += y;
  }
  if (lane == 31) sm.wred[0][warp] = x;
  __syncthreads();
  const uint32_t w = lane < kSelWarps ? sm.wred[0][lane] : 0u;
  *total = __reduce_add_sync(0xffffffffu, w);
  const uint32_t before = __reduce_add_sync(0xffffffffu, lane < warp ? w : 0u);
  __syncthreads();
  return before + x - v;
}

// The bin of the complete histogram (a barrier precedes) that holds the need-th
// largest: sm.bin, sm.above (scores in higher bins), sm.inbin.
__device__ __forceinline__ void sel_find(SelSmem& sm, uint32_t need) {
  constexpr int kPer = kBins / kSelThreads;
  uint32_t cnt[kPer], sum = 0;  // bins in descending order: thread 0 has the highest
#pragma unroll
  for (int j = 0; j < kPer; ++j) {
    cnt[j] = sm.hist[kBins - 1 - (kPer * threadIdx.x + j)];
    sum += cnt[j];
  }
  uint32_t all;
  uint32_t before = sel_scan(sm, sum, &all);
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

// Equal steps of the score between two keys: bin(f) is monotone in f.  inv = 0
// where the range is not finite or empty.
struct Steps {
  float lo, inv;
  __device__ __forceinline__ static Steps of(uint32_t klo, uint32_t khi) {
    Steps s;
    s.lo = key_score(klo);
    const float range = key_score(khi) - s.lo;
    s.inv = range > 0.f && range < INFINITY ? fminf(static_cast<float>(kBins) / range, 3.0e38f) : 0.f;
    return s;
  }
  __device__ __forceinline__ float at(float f) const { return (f - lo) * inv; }
  __device__ __forceinline__ int bin(float f) const {
    const float x = at(f);
    return x >= static_cast<float>(kBins - 1) ? kBins - 1 : static_cast<int>(x);
  }
};

// The need-th largest of the cnt > need scores that `each(f)` walks (f(score),
// every thread its share): key T, and how many scores equal to it are among
// the need largest.
template <typename Each>
__device__ __forceinline__ void sel_kth(SelSmem& sm, uint32_t need, uint32_t cnt, Each&& each, uint32_t* T,
                                        uint32_t* take) {
  const int tid = threadIdx.x;
  for (int j = tid; j < kBins; j += kSelThreads) sm.hist[j] = 0u;
  uint32_t lo = 0xFFFFFFFFu, hi = 0u;
  each([&](float f) {
    const uint32_t k = score_key(f);
    lo = min(lo, k);
    hi = max(hi, k);
  });
  sel_minmax(sm, lo, hi);
  if (lo != hi) {
    const Steps st = Steps::of(lo, hi);
    uint32_t members = cnt;
    int bin0 = -1;  // -1: every score
    if (st.inv > 0.f) {
      each([&](float f) { atomicAdd(&sm.hist[st.bin(f)], 1u); });
      __syncthreads();
      sel_find(sm, need);
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
      each([&](float f) {
        const uint32_t k = score_key(f);
        if (inside(f, k)) {
          a = min(a, k);
          z = max(z, k);
        }
      });
      for (int j = tid; j < kBins; j += kSelThreads) sm.hist[j] = 0u;
      sel_minmax(sm, a, z);
      lo = a;
      hi = z;
      windowed = true;
      if (lo == hi) break;
      const int bits = 32 - __clz(hi - lo);
      const int sh = bits > 11 ? bits - 11 : 0;
      each([&](float f) {
        const uint32_t k = score_key(f);
        if (k >= lo && k <= hi) atomicAdd(&sm.hist[(k - lo) >> sh], 1u);
      });
      __syncthreads();
      sel_find(sm, need);
      members = sm.inbin;
      need -= sm.above;
      const uint32_t nlo = lo + (sm.bin << sh);
      const uint64_t nhi = static_cast<uint64_t>(nlo) + ((1ull << sh) - 1ull);
      lo = nlo;
      hi = nhi < hi ? static_cast<uint32_t>(nhi) : hi;
      if (sh == 0) break;
    }
    if (!(windowed && lo == hi)) {
      if (tid == 0) sm.nfew = 0u;
      __syncthreads();
      each([&](float f) {
        const uint32_t k = score_key(f);
        if (inside(f, k)) {
          const uint32_t at = atomicAdd(&sm.nfew, 1u);
          if (at < static_cast<uint32_t>(kFew)) sm.few[at] = k;
        }
      });
      __syncthreads();
      const uint32_t m = min(sm.nfew, static_cast<uint32_t>(kFew));
      if (tid < static_cast<int>(m)) {
        const uint32_t mine = sm.few[tid];
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
      return;
    }
  }
  *T = lo;
  *take = need;
}

template <int kCap>
__global__ void __launch_bounds__(kSelThreads, kCap <= 4096 ? 3 : 2)
    paged_select_kernel(const BatchView b, int shift, int64_t row0, const float* __restrict__ scores, int64_t ld,
                        int topk, int words_room, int32_t* __restrict__ pool_idx, unsigned* status) {
  extern __shared__ __align__(16) uint8_t smem_raw[];
  SelSmem& sm = *reinterpret_cast<SelSmem*>(smem_raw);
  float* cval = reinterpret_cast<float*>(smem_raw + sizeof(SelSmem));    // [kCap] candidates
  int32_t* cidx = reinterpret_cast<int32_t*>(cval + kCap);                // [kCap] their pools
  uint32_t* above = reinterpret_cast<uint32_t*>(cidx + kCap);             // [words_room] bits: scores above T
  uint32_t* equal = above + words_room;                                   // [words_room] bits: scores equal to T
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
  const int64_t lrow = blockIdx.x, row = row0 + lrow;
  if (warp == 0) {
    const int n = warp_locate(b, row, lane);
    if (lane == 0) {
      sm.seq = n;
      sm.nlist = 0u;
    }
  }
  __syncthreads();
  const int seq = sm.seq;
  if (seq >= b.batch) return;  // padding behind the last sequence
  const int64_t i = row_position(b, shift, seq, row, status);
  int32_t* orow = pool_idx + row * topk;
  const int n = i < 0 ? 0 : static_cast<int>(i >> 2);
  if (n <= topk) {  // every pool (or, for a row without a position, nothing)
    for (int j = tid; j < topk; j += kSelThreads) orow[j] = j < n ? j : -1;
    return;
  }
  const float* srow = scores + lrow * ld;

  // ---- candidates
  bool listed = n <= kCap;
  if (listed) {
    for (int j = tid; j < n; j += kSelThreads) {
      cval[j] = srow[j];
      cidx[j] = j;
    }
    if (tid == 0) sm.nlist = static_cast<uint32_t>(n);
  } else {
    // quads (4 consecutive scores) of the sample: 2 a thread, 8 beyond 2^16 pools
    const int nq = n >> 2, per = n > 65536 ? 8 : 2;
    float4 q[8];
    uint32_t lo = 0xFFFFFFFFu, hi = 0u;
#pragma unroll
    for (int u = 0; u < 8; ++u) {
      if (u >= per) break;
      const int64_t k = static_cast<int64_t>(u * kSelThreads + tid) * nq / (per * kSelThreads);
      q[u] = *reinterpret_cast<const float4*>(srow + 4 * k);
    }
    for (int j = tid; j < kBins; j += kSelThreads) sm.hist[j] = 0u;
#pragma unroll
    for (int u = 0; u < 8; ++u) {
      if (u >= per) break;
      const uint32_t k0 = score_key(q[u].x), k1 = score_key(q[u].y), k2 = score_key(q[u].z), k3 = score_key(q[u].w);
      lo = min(min(lo, min(k0, k1)), min(k2, k3));
      hi = max(max(hi, max(k0, k1)), max(k2, k3));
    }
    sel_minmax(sm, lo, hi);
    const Steps st = Steps::of(lo, hi);
    if (st.inv > 0.f) {
#pragma unroll
      for (int u = 0; u < 8; ++u) {
        if (u >= per) break;
        atomicAdd(&sm.hist[st.bin(q[u].x)], 1u);
        atomicAdd(&sm.hist[st.bin(q[u].y)], 1u);
        atomicAdd(&sm.hist[st.bin(q[u].z)], 1u);
        atomicAdd(&sm.hist[st.bin(q[u].w)], 1u);
      }
      __syncthreads();
      // c candidates with c - 5 sqrt(c sigma) = topk, sigma scores a sample
      const float sigma = static_cast<float>(n) / static_cast<float>(4 * per * kSelThreads);
      const float rc = 0.5f * (5.f * sqrtf(sigma) + sqrtf(25.f * sigma + 4.f * static_cast<float>(topk)));
      const int want = min(static_cast<int>(rc * rc / sigma) + 1, 4 * per * kSelThreads);
      sel_find(sm, static_cast<uint32_t>(want));
      const float edge = static_cast<float>(sm.bin);
      // one pass over the row; four 16-byte loads in flight a thread
      constexpr int kU = 4;
      for (int j0 = 0; j0 < n; j0 += 4 * kU * kSelThreads) {
        float4 x[kU];
#pragma unroll
        for (int u = 0; u < kU; ++u) {
          const int j = j0 + 4 * (u * kSelThreads + tid);
          if (j + 3 < n) x[u] = *reinterpret_cast<const float4*>(srow + j);
          else {
            x[u].x = j < n ? srow[j] : -INFINITY;
            x[u].y = j + 1 < n ? srow[j + 1] : -INFINITY;
            x[u].z = j + 2 < n ? srow[j + 2] : -INFINITY;
            x[u].w = -INFINITY;
          }
        }
#pragma unroll
        for (int u = 0; u < kU; ++u) {
          const int j = j0 + 4 * (u * kSelThreads + tid);
          const float f[4] = {x[u].x, x[u].y, x[u].z, x[u].w};
          bool hit[4];
#pragma unroll
          for (int e = 0; e < 4; ++e) hit[e] = st.at(f[e]) >= edge && j + e < n;
          if (!__any_sync(0xffffffffu, hit[0] || hit[1] || hit[2] || hit[3])) continue;
          uint32_t m[4], all = 0u;
#pragma unroll
          for (int e = 0; e < 4; ++e) {
            m[e] = __ballot_sync(0xffffffffu, hit[e]);
            all += __popc(m[e]);
          }
          uint32_t at = 0u;
          if (lane == 0) at = atomicAdd(&sm.nlist, all);
          at = __shfl_sync(0xffffffffu, at, 0);
#pragma unroll
          for (int e = 0; e < 4; ++e) {
            const uint32_t to = at + __popc(m[e] & ((1u << lane) - 1u));
            if (hit[e] && to < static_cast<uint32_t>(kCap)) {
              cval[to] = f[e];
              cidx[to] = j + e;
            }
            at += __popc(m[e]);
          }
        }
      }
      __syncthreads();
      listed = sm.nlist >= static_cast<uint32_t>(topk) && sm.nlist <= static_cast<uint32_t>(kCap);
    }
  }
  __syncthreads();
  const int m = static_cast<int>(sm.nlist);

  // ---- T
  uint32_t T = 0u, take = 0u;
  if (listed && m > topk) {
    sel_kth(sm, static_cast<uint32_t>(topk), static_cast<uint32_t>(m), [&](auto&& f) {
      for (int j = tid; j < m; j += kSelThreads) f(cval[j]);
    }, &T, &take);
  } else if (!listed) {
    sel_kth(sm, static_cast<uint32_t>(topk), static_cast<uint32_t>(n), [&](auto&& f) {
      for (int j = tid; j < n; j += kSelThreads) f(srow[j]);
    }, &T, &take);
  }  // a list of exactly topk scores is kept whole: every key is above T = 0 (no score's), or equal to it

  // ---- the row, segment by segment
  uint32_t done = 0u, ties = 0u;  // written so far; ties met so far
  if (listed && m == topk) take = static_cast<uint32_t>(topk);
  for (int s0 = 0; s0 < n; s0 += kSegment) {
    const int len = min(kSegment, n - s0), words = (len + 31) >> 5;
    if (listed) {
      for (int k = tid; k < words; k += kSelThreads) above[k] = equal[k] = 0u;
      __syncthreads();
      for (int j = tid; j < m; j += kSelThreads) {
        const int p = cidx[j] - s0;
        const uint32_t k = score_key(cval[j]);
        if (p >= 0 && p < len && k >= T) atomicOr((k > T ? above : equal) + (p >> 5), 1u << (p & 31));
      }
    } else {
      for (int k = warp; k < words; k += kSelWarps) {
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
    const int wpt = (words + kSelThreads - 1) / kSelThreads;
    const int k0 = min(tid * wpt, words), k1 = min(k0 + wpt, words);
    uint32_t g = 0u, e = 0u;
    for (int k = k0; k < k1; ++k) {
      g += __popc(above[k]);
      e += __popc(equal[k]);
    }
    uint32_t g_all, e_all;
    uint32_t pe = ties + sel_scan(sm, e, &e_all);
    const uint32_t pg = sel_scan(sm, g, &g_all);
    uint32_t pos = done + pg + (min(pe, take) - min(ties, take));
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
    __syncthreads();  // the bits are read: the next segment may set its own
  }
}

template <int kMt>
cudaError_t launch_scores(const CacheView& c, const BatchView& b, const void* q_idx, const float* w, int Hi,
                          int64_t row0, int64_t nrows, float* scores, int64_t ld, const LaunchCtx& ctx) {
  const size_t smem = static_cast<size_t>(b.batch + 1) * sizeof(int);
  const int grid = ctx.num_sms * (kMt <= 2 ? 2 : 1);
  paged_score_kernel<kMt><<<grid, kThreads, smem, ctx.stream>>>(c, b, static_cast<const __nv_bfloat16*>(q_idx), w, Hi,
                                                                row0, row0 + nrows, scores, ld, ctx.status);
  return cudaGetLastError();
}

template <int kCap>
cudaError_t launch_select(const BatchView& b, int shift, int64_t row0, int64_t nrows, const float* scores, int64_t ld,
                          int topk, int32_t* pool_idx, const LaunchCtx& ctx) {
  const int64_t pools = static_cast<int64_t>(b.max_pages) << (shift - 2);
  const int words = static_cast<int>((pools < kSegment ? pools : kSegment) + 31) / 32;
  constexpr size_t kFixed = sizeof(SelSmem) + static_cast<size_t>(kCap) * 8;
  constexpr size_t kMost = kFixed + 2 * (kSegment / 32) * 4;
  static_assert(kMost <= 232448 - 1024, "shared memory per CTA");
  static std::atomic<bool> attr_done[kAttrDevices];
  const cudaError_t e = set_smem_limit_once(paged_select_kernel<kCap>, static_cast<int>(kMost), attr_done);
  if (e != cudaSuccess) return e;
  paged_select_kernel<kCap><<<static_cast<unsigned>(nrows), kSelThreads, kFixed + static_cast<size_t>(words) * 8,
                              ctx.stream>>>(b, shift, row0, scores, ld, topk, words, pool_idx, ctx.status);
  return cudaGetLastError();
}

}  // namespace

cudaError_t launch_paged_scores(const CacheView& c, const BatchView& b, const void* q_idx, const float* w, int Hi,
                                int64_t row0, int64_t nrows, float* scores, int64_t ld, const LaunchCtx& ctx) {
  if (Hi <= 16) return launch_scores<1>(c, b, q_idx, w, Hi, row0, nrows, scores, ld, ctx);
  if (Hi <= 32) return launch_scores<2>(c, b, q_idx, w, Hi, row0, nrows, scores, ld, ctx);
  return launch_scores<4>(c, b, q_idx, w, Hi, row0, nrows, scores, ld, ctx);
}

cudaError_t launch_paged_select(const BatchView& b, int shift, int64_t row0, int64_t nrows, const float* scores,
                                int64_t ld, int topk, int32_t* pool_idx, const LaunchCtx& ctx) {
  // the list must hold topk and the spread of the sampling
  if (topk <= 512) return launch_select<4096>(b, shift, row0, nrows, scores, ld, topk, pool_idx, ctx);
  return launch_select<8192>(b, shift, row0, nrows, scores, ld, topk, pool_idx, ctx);
}

}  // namespace dsa
