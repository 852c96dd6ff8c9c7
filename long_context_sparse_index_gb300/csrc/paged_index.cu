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
// One row per cluster of kC CTAs (1, 2, 4 or 8).  Each CTA holds its stretch
// of the row's scores in shared memory (the part past its room is read again
// from global memory).  The topk-th largest score T:
//   1. minimum and maximum; histogram of kBins equal steps between them
//      (monotone in the score, whatever the rounding), summed over the
//      cluster: the bin that holds T;
//   2. while that bin holds more than kFew scores: their minimum and maximum,
//      and a histogram of equal steps of their 32-bit keys;
//   3. the few left are ranked against each other.
// Then every score above T is kept and, of those equal to T, the first ones in
// pool order; one pass counts per warp, one writes, so the output ascends.
constexpr int kSelThreads = 512;
constexpr int kSelWarps = kSelThreads / 32;
constexpr int kBins = 2048;
constexpr int kFew = 512;
constexpr int kSelRoom = 49152;  // scores of a CTA that stay in shared memory (192 KB)

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
  uint32_t wscan[kSelWarps];
  uint32_t lo, hi;        // this CTA's extrema
  uint32_t nfew;
  uint32_t gt, eq;        // this CTA's kept counts
  uint32_t bin, above, inbin;
  uint32_t T, take;
  int seq;
};

static_assert(sizeof(SelSmem) % 16 == 0, "the scores after it are read 16 bytes at a time");

template <int kC>
__device__ __forceinline__ void sel_cluster_sync() {
  if (kC > 1) cluster_sync();
  else __syncthreads();
}
// value of a shared word in CTA u of the cluster
template <int kC>
__device__ __forceinline__ uint32_t sel_peer(const uint32_t* p, int u) {
  return kC > 1 ? cluster_ld_u32(cluster_map(smem_u32(p), u)) : *p;
}

// extrema of (lo, hi) over the cluster; every thread gets them
template <int kC>
__device__ __forceinline__ void sel_minmax(SelSmem& sm, uint32_t& lo, uint32_t& hi) {
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  lo = __reduce_min_sync(0xffffffffu, lo);
  hi = __reduce_max_sync(0xffffffffu, hi);
  if (lane == 0) {
    sm.wred[0][warp] = lo;
    sm.wred[1][warp] = hi;
  }
  __syncthreads();
  if (warp == 0) {
    const uint32_t a = __reduce_min_sync(0xffffffffu, lane < kSelWarps ? sm.wred[0][lane] : 0xFFFFFFFFu);
    const uint32_t z = __reduce_max_sync(0xffffffffu, lane < kSelWarps ? sm.wred[1][lane] : 0u);
    if (lane == 0) {
      sm.lo = a;
      sm.hi = z;
    }
  }
  sel_cluster_sync<kC>();
  lo = 0xFFFFFFFFu;
  hi = 0u;
#pragma unroll
  for (int u = 0; u < kC; ++u) {
    lo = min(lo, sel_peer<kC>(&sm.lo, u));
    hi = max(hi, sel_peer<kC>(&sm.hi, u));
  }
}

// Sums the CTAs' histograms and finds the bin holding the need-th largest:
// sm.bin, sm.above (scores in higher bins), sm.inbin, the same in every CTA.
template <int kC>
__device__ __forceinline__ void sel_find(SelSmem& sm, uint32_t need) {
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  constexpr int kPer = kBins / kSelThreads;
  sel_cluster_sync<kC>();  // every CTA's histogram is complete
  uint32_t cnt[kPer], sum = 0;  // bins in descending order: thread 0 has the highest
#pragma unroll
  for (int j = 0; j < kPer; ++j) cnt[j] = 0;
#pragma unroll
  for (int u = 0; u < kC; ++u)
#pragma unroll
    for (int j = 0; j < kPer; ++j) cnt[j] += sel_peer<kC>(&sm.hist[kBins - 1 - (kPer * threadIdx.x + j)], u);
#pragma unroll
  for (int j = 0; j < kPer; ++j) sum += cnt[j];
  uint32_t x = sum;
#pragma unroll
  for (int o = 1; o < 32; o <<= 1) {
    const uint32_t y = __shfl_up_sync(0xffffffffu, x, o);
    if (lane >= o) x += y;
  }
  if (lane == 31) sm.wscan[warp] = x;
  __syncthreads();
  uint32_t before = x - sum;
  for (int k = 0; k < warp; ++k) before += sm.wscan[k];
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
  sel_cluster_sync<kC>();  // found, and no histogram is read any more
}

template <int kC>
__global__ void __launch_bounds__(kSelThreads)
    paged_select_kernel(const BatchView b, int shift, int64_t row0, const float* __restrict__ scores, int64_t ld,
                        int topk, int room, int32_t* __restrict__ pool_idx, unsigned* status) {
  extern __shared__ __align__(16) uint8_t smem_raw[];
  SelSmem& sm = *reinterpret_cast<SelSmem*>(smem_raw);
  float* kept = reinterpret_cast<float*>(smem_raw + sizeof(SelSmem));
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
  const int rank = kC > 1 ? static_cast<int>(cluster_rank()) : 0;
  const int64_t lrow = blockIdx.x / kC, row = row0 + lrow;
  if (warp == 0) {
    const int n = warp_locate(b, row, lane);
    if (lane == 0) sm.seq = n;
  }
  __syncthreads();
  const int seq = sm.seq;
  if (seq >= b.batch) return;  // padding behind the last sequence (the whole cluster)
  const int64_t i = row_position(b, shift, seq, row, status);
  int32_t* orow = pool_idx + row * topk;
  const int64_t n = i < 0 ? 0 : i >> 2;
  if (n <= topk) {  // every pool (or, for a row without a position, nothing)
    for (int j = rank * kSelThreads + tid; j < topk; j += kC * kSelThreads) orow[j] = j < n ? j : -1;
    return;
  }
  // this CTA's stretch, a multiple of 4 long but for the last
  const int per = static_cast<int>(((n + kC - 1) / kC + 3) & ~int64_t{3});
  const int64_t base = static_cast<int64_t>(rank) * per;
  const int cnt = static_cast<int>(base >= n ? 0 : min(static_cast<int64_t>(per), n - base));
  const float* srow = scores + lrow * ld + base;

  // ---- load; extrema
  uint32_t lo = 0xFFFFFFFFu, hi = 0u;
  for (int j = 4 * tid; j < cnt; j += 4 * kSelThreads) {
    float4 f;
    if (j + 3 < cnt) {
      f = *reinterpret_cast<const float4*>(srow + j);
    } else {
      f.x = srow[j];
      f.y = j + 1 < cnt ? srow[j + 1] : f.x;
      f.z = j + 2 < cnt ? srow[j + 2] : f.x;
      f.w = f.x;
    }
    const uint32_t k0 = score_key(f.x), k1 = score_key(f.y), k2 = score_key(f.z),
                   k3 = score_key(f.w);
    lo = min(min(lo, min(k0, k1)), min(k2, k3));
    hi = max(max(hi, max(k0, k1)), max(k2, k3));
    if (j < room) *reinterpret_cast<float4*>(kept + j) = f;  // room is a multiple of 4
  }
  auto get = [&](int j) { return j < room ? kept[j] : srow[j]; };
  for (int j = tid; j < kBins; j += kSelThreads) sm.hist[j] = 0u;
  sel_minmax<kC>(sm, lo, hi);

  // ---- first round: equal steps of the score
  uint32_t need = static_cast<uint32_t>(topk), T = lo, take = need;
  if (lo != hi) {
    const float flo = key_score(lo), fhi = key_score(hi);
    const float step = fhi - flo;
    const float inv = step > 0.f && step < INFINITY ? fminf(static_cast<float>(kBins) / step, 3.0e38f) : 0.f;
    auto bin_of = [&](float f) {
      const float x = (f - flo) * inv;  // non-finite scores make inv 0 or x a NaN: bin 0 or the last
      return x >= static_cast<float>(kBins - 1) ? kBins - 1 : static_cast<int>(x);
    };
    const bool linear = inv > 0.f;  // (the same in every CTA of the cluster)
    if (!linear) sel_cluster_sync<kC>();  // the extrema have been read: the next round may write its own
    if (linear) {
      for (int j = tid; j < cnt; j += kSelThreads) atomicAdd(&sm.hist[bin_of(get(j))], 1u);
      sel_find<kC>(sm, need);
    }
    uint32_t members = linear ? sm.inbin : static_cast<uint32_t>(min(n, int64_t{0xFFFFFFFF}));
    if (linear) need -= sm.above;
    const int bin0 = linear ? static_cast<int>(sm.bin) : -1;
    // ---- the bin's scores by their keys; window [lo, hi] once it is known
    bool windowed = false;
    auto inside = [&](float f, uint32_t k) { return windowed ? k >= lo && k <= hi : bin0 < 0 || bin_of(f) == bin0; };
    while (members > static_cast<uint32_t>(kFew)) {
      uint32_t a = 0xFFFFFFFFu, z = 0u;
      for (int j = tid; j < cnt; j += kSelThreads) {
        const float f = get(j);
        const uint32_t k = score_key(f);
        if (inside(f, k)) {
          a = min(a, k);
          z = max(z, k);
        }
      }
      for (int j = tid; j < kBins; j += kSelThreads) sm.hist[j] = 0u;
      sel_minmax<kC>(sm, a, z);
      lo = a;
      hi = z;
      windowed = true;
      if (lo == hi) break;
      const int bits = 32 - __clz(hi - lo);
      const int sh = bits > 11 ? bits - 11 : 0;
      for (int j = tid; j < cnt; j += kSelThreads) {
        const uint32_t k = score_key(get(j));
        if (k >= lo && k <= hi) atomicAdd(&sm.hist[(k - lo) >> sh], 1u);
      }
      sel_find<kC>(sm, need);
      need -= sm.above;
      members = sm.inbin;
      const uint32_t nlo = lo + (sm.bin << sh);
      const uint64_t nhi = static_cast<uint64_t>(nlo) + ((1ull << sh) - 1ull);
      lo = nlo;
      hi = nhi < hi ? static_cast<uint32_t>(nhi) : hi;
      if (sh == 0) break;
    }
    if (windowed && lo == hi) {
      T = lo;
      take = need;
    } else {
      // ---- at most kFew in the cluster: every CTA lists its own
      if (tid == 0) sm.nfew = 0u;
      __syncthreads();
      for (int j = tid; j < cnt; j += kSelThreads) {
        const float f = get(j);
        const uint32_t k = score_key(f);
        if (inside(f, k)) {
          const uint32_t at = atomicAdd(&sm.nfew, 1u);
          if (at < static_cast<uint32_t>(kFew)) sm.few[at] = k;
        }
      }
      sel_cluster_sync<kC>();
      // every CTA ranks every listed key: one key a thread
      uint32_t mine = 0u, at = static_cast<uint32_t>(tid);
      bool has = false;
#pragma unroll
      for (int u = 0; u < kC; ++u) {
        const uint32_t m = min(sel_peer<kC>(&sm.nfew, u), static_cast<uint32_t>(kFew));
        if (!has && at < m) {
          mine = sel_peer<kC>(&sm.few[at], u);
          has = true;
        } else if (!has) {
          at -= m;
        }
      }
      uint32_t gt = 0u, eq = 0u;
      if (has) {
        for (int u = 0; u < kC; ++u) {
          const uint32_t m = min(sel_peer<kC>(&sm.nfew, u), static_cast<uint32_t>(kFew));
          for (uint32_t e = 0; e < m; ++e) {
            const uint32_t k = sel_peer<kC>(&sm.few[e], u);
            gt += k > mine;
            eq += k == mine;
          }
        }
        if (gt < need && need <= gt + eq) {  // every thread with T writes the same
          sm.T = mine;
          sm.take = need - gt;
        }
      }
      __syncthreads();
      T = sm.T;
      take = sm.take;
    }
  }

  // ---- keep: counts per warp (each warp a contiguous stretch), prefix over the cluster, then the indices
  const int wper = ((cnt + kSelWarps - 1) / kSelWarps + 31) & ~31;
  const int w0 = min(warp * wper, cnt), w1 = min(w0 + wper, cnt);
  uint32_t ngt = 0u, neq = 0u;
  for (int j = w0; j < w1; j += 32) {
    const uint32_t k = j + lane < w1 ? score_key(get(j + lane)) : 0u;
    ngt += j + lane < w1 && k > T;
    neq += j + lane < w1 && k == T;
  }
  ngt = __reduce_add_sync(0xffffffffu, ngt);
  neq = __reduce_add_sync(0xffffffffu, neq);
  if (lane == 0) {
    sm.wred[0][warp] = ngt;
    sm.wred[1][warp] = neq;
  }
  __syncthreads();
  uint32_t gt = 0u, eq = 0u;
  for (int k = 0; k < kSelWarps; ++k) {
    gt += k < warp ? sm.wred[0][k] : 0u;
    eq += k < warp ? sm.wred[1][k] : 0u;
  }
  if (kC > 1) {
    if (tid == kSelThreads - 1) {  // the last warp's prefix and its own
      sm.gt = gt + ngt;
      sm.eq = eq + neq;
    }
    cluster_sync();
#pragma unroll
    for (int u = 0; u < kC; ++u)
      if (u < rank) {
        gt += sel_peer<kC>(&sm.gt, u);
        eq += sel_peer<kC>(&sm.eq, u);
      }
  }
  const unsigned below = (1u << lane) - 1u;
  for (int j = w0; j < w1; j += 32) {
    const bool in = j + lane < w1;
    const uint32_t k = in ? score_key(get(j + lane)) : 0u;
    const unsigned mg = __ballot_sync(0xffffffffu, in && k > T), me = __ballot_sync(0xffffffffu, in && k == T);
    const uint32_t pe = eq + __popc(me & below);
    if (in && (k > T || (k == T && pe < take))) {
      const uint32_t pos = gt + __popc(mg & below) + min(pe, take);
      if (pos < static_cast<uint32_t>(topk)) orow[pos] = static_cast<int32_t>(base + j + lane);
    }
    gt += __popc(mg);
    eq += __popc(me);
  }
  if (kC > 1) cluster_sync();  // no CTA leaves while another reads its shared memory
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

template <int kC>
cudaError_t launch_select(const BatchView& b, int shift, int64_t row0, int64_t nrows, const float* scores, int64_t ld,
                          int64_t pools, int topk, int32_t* pool_idx, const LaunchCtx& ctx) {
  const int64_t per = ((pools + kC - 1) / kC + 3) & ~int64_t{3};
  const int room = static_cast<int>(per < kSelRoom ? per : kSelRoom);
  constexpr int kMost = static_cast<int>(sizeof(SelSmem)) + kSelRoom * 4;
  static_assert(kMost <= 232448 - 1024, "shared memory per CTA");
  static std::atomic<bool> attr_done[kAttrDevices];
  cudaError_t e = set_smem_limit_once(paged_select_kernel<kC>, kMost, attr_done);
  if (e != cudaSuccess) return e;
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3(static_cast<unsigned>(nrows * kC));
  cfg.blockDim = dim3(kSelThreads);
  cfg.dynamicSmemBytes = sizeof(SelSmem) + static_cast<size_t>(room) * 4;
  cfg.stream = ctx.stream;
  cudaLaunchAttribute attr[1];
  attr[0].id = cudaLaunchAttributeClusterDimension;
  attr[0].val.clusterDim.x = kC;
  attr[0].val.clusterDim.y = 1;
  attr[0].val.clusterDim.z = 1;
  cfg.attrs = attr;
  cfg.numAttrs = kC > 1 ? 1 : 0;
  return cudaLaunchKernelEx(&cfg, paged_select_kernel<kC>, b, shift, row0, scores, ld, topk, room, pool_idx,
                            ctx.status);
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
  const int64_t pools = static_cast<int64_t>(b.max_pages) << (shift - 2);
  if (nrows * 8 <= 2 * ctx.num_sms || pools > 4 * kSelRoom)
    return launch_select<8>(b, shift, row0, nrows, scores, ld, pools, topk, pool_idx, ctx);
  if (nrows * 4 <= 4 * ctx.num_sms || pools > 2 * kSelRoom)
    return launch_select<4>(b, shift, row0, nrows, scores, ld, pools, topk, pool_idx, ctx);
  if (pools > kSelRoom) return launch_select<2>(b, shift, row0, nrows, scores, ld, pools, topk, pool_idx, ctx);
  return launch_select<1>(b, shift, row0, nrows, scores, ld, pools, topk, pool_idx, ctx);
}

}  // namespace dsa
