// paged.cuh -- device helpers shared by the paged-cache kernels: which
// sequence a row belongs to, and where a token or pool lies.
//
// Nothing that steers an access is trusted: rows, lengths, page numbers and
// selections come from device memory, so each is checked against its bounds
// where it is read; what is out of range is never followed and is recorded in
// the status word (DSA_ERR_INTERNAL at dsa_sync_status).
#pragma once

#include "dsa_device.cuh"
#include "paged_kernels.h"

namespace dsa {

// Sequence and position of a row; seq < 0: padding behind the last sequence;
// pos < 0: offsets and lengths that contradict each other (recorded).
struct RowAt {
  int seq;
  int64_t pos;
};

// All lanes of a warp call it together with the same row.  Offsets and lengths
// of 128 sequences are looked at at once, so that a call of up to 128
// sequences waits for memory once.
__device__ __forceinline__ RowAt warp_locate(const BatchView& b, int shift, int64_t row, int lane, unsigned* status) {
  constexpr int kU = 4;
  RowAt x{-1, -1};
  for (int j0 = 0; j0 < b.batch && x.seq < 0; j0 += 32 * kU) {
    int c0[kU], c1[kU], len[kU];
#pragma unroll
    for (int u = 0; u < kU; ++u) {
      const int j = j0 + 32 * u + lane;
      c0[u] = c1[u] = len[u] = 0;  // (an empty stretch: no row lies in it)
      if (j < b.batch) {
        c0[u] = __ldg(b.cu + j);
        c1[u] = __ldg(b.cu + j + 1);
        len[u] = __ldg(b.lens + j);
      }
    }
#pragma unroll
    for (int u = 0; u < kU; ++u) {
      const unsigned hit = __ballot_sync(0xffffffffu, c0[u] <= row && row < c1[u]);
      if (hit == 0u || x.seq >= 0) continue;
      const int src = __ffs(hit) - 1;
      const int64_t first = __shfl_sync(0xffffffffu, c0[u], src), last = __shfl_sync(0xffffffffu, c1[u], src);
      const int64_t n = __shfl_sync(0xffffffffu, len[u], src);
      x.seq = j0 + 32 * u + src;
      x.pos = n - last + row;
      // the sequence's rows must be the call's, the sequence as long as its new
      // tokens, and its table as long as it
      if (first < 0 || last > b.rows || x.pos < row - first || n > (static_cast<int64_t>(b.max_pages) << shift)) {
        x.pos = -1;
        if (lane == 0) record_status(status, kStatusInternal);
      }
    }
  }
  return x;
}

// Page x of sequence s (x < max_pages), or -1 (recorded) for a number that is
// no page.
__device__ __forceinline__ int page_of(const BatchView& b, int num_pages, int s, int x, unsigned* status) {
  const int p = __ldg(b.table + s * b.table_stride + x);
  if (static_cast<unsigned>(p) < static_cast<unsigned>(num_pages)) return p;
  record_status(status, kStatusInternal);
  return -1;
}

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

// A stretch of a CTA's walk over the scores: pools [p0, p1) of one sequence, a
// tile of kRunTile at a time, against up to `group` of its rows.
constexpr int kRunTile = 128;
// Items of one sequence in a pass of the scores, and where the sum over the
// sequences saturates.  A pass has up to eight rows of up to 2^29 pools, or more
// rows with 2^31 scores in all; an item is four rows or more by 128 pools or
// more.  So a sequence of eight rows has at most 2 * 2^22 items, one of n > 8
// rows fewer than n / 3 * 2^24 / n, all of a pass together at most 2^25.  Only
// offsets that contradict each other ask for more.  They are cut off, so that a
// scan of 128 sequences on top of the saturated sum stays in 32 bits.
constexpr int kMaxItems = 1 << 23;
constexpr int kMaxTotal = 1 << 29;
struct Run {
  int64_t ra;            // first row
  const int32_t* table;  // the sequence's pages
  int nr;                // rows; 0: the walk has ended
  int pools;             // pools that the last row may see
  int p0, p1;            // multiples of kRunTile (p1 may lie past `pools`)
};

// Items of a walk are (sequence, group of rows, tile); off[s]: items before
// sequence s.  The run that begins at item `*it` (or at the first one behind it
// that has anything to score) and ends with its rows, or with the walk at it1;
// moves *it past it.  *s is a cursor that only moves forward.
static __device__ __noinline__ Run next_run(const BatchView& b, int shift, int group, const int* off, int64_t row0,
                                            int64_t row1, int it1, int* it, int* s) {
  Run x;
  x.nr = 0;
  while (*it < it1) {
    while (*s + 1 < b.batch && *it >= off[*s + 1]) ++*s;
    int64_t first;
    const int n = seq_rows(b, *s, row0, row1, &first);
    const int tiles = static_cast<int>((seq_pools(b, shift, *s, first, n) + kRunTile - 1) / kRunTile);
    if (tiles == 0) {
      ++*it;
      continue;
    }
    const int rg = (*it - off[*s]) / tiles, tile = (*it - off[*s]) % tiles;
    const int many = min(tiles - tile, it1 - *it);
    *it += many;
    x.ra = first + static_cast<int64_t>(rg) * group;
    x.nr = static_cast<int>(min(static_cast<int64_t>(group), first + n - x.ra));
    if (x.nr > 0) {
      x.pools = static_cast<int>(seq_pools(b, shift, *s, x.ra, x.nr));
      x.p0 = tile * kRunTile;
      x.p1 = min((tile + many) * kRunTile, (x.pools + kRunTile - 1) / kRunTile * kRunTile);
      x.table = b.table + *s * b.table_stride;
      if (x.p0 < x.p1) return x;
    }
    x.nr = 0;
  }
  return x;
}

// Whether the 128-row tiles take sequence s: by its rows and pools in the whole
// call, so that every kernel and pass of the call answers alike.
__device__ __forceinline__ bool tc_takes(const BatchView& b, const TcRule& tc, int s) {
  const int64_t rows = static_cast<int64_t>(__ldg(b.cu + s + 1)) - __ldg(b.cu + s), pools = __ldg(b.lens + s) >> 2;
  return rows >= tc.rows && (rows + 127) / 128 * ((pools + 255) / 256) >= tc.tiles;
}

// ----------------------------------------------------------------- thread-block clusters
__device__ __forceinline__ void cluster_sync() {
  asm volatile("barrier.cluster.arrive.release.aligned;\nbarrier.cluster.wait.acquire.aligned;" ::: "memory");
}
__device__ __forceinline__ uint32_t cluster_rank() {
  uint32_t r;
  asm volatile("mov.u32 %0, %%cluster_ctarank;" : "=r"(r));
  return r;
}
// Address, in CTA `rank` of the cluster, of what lies at shared address `a` here.
__device__ __forceinline__ uint32_t cluster_map(uint32_t a, uint32_t rank) {
  uint32_t r;
  asm volatile("mapa.shared::cluster.u32 %0, %1, %2;" : "=r"(r) : "r"(a), "r"(rank));
  return r;
}
__device__ __forceinline__ uint32_t cluster_ld_u32(uint32_t a) {
  uint32_t v;
  asm volatile("ld.shared::cluster.u32 %0, [%1];" : "=r"(v) : "r"(a) : "memory");
  return v;
}
__device__ __forceinline__ float cluster_ld_f32(uint32_t a) { return __uint_as_float(cluster_ld_u32(a)); }
__device__ __forceinline__ float4 cluster_ld_f32x4(uint32_t a) {
  float4 v;
  asm volatile("ld.shared::cluster.v4.f32 {%0,%1,%2,%3}, [%4];"
               : "=f"(v.x), "=f"(v.y), "=f"(v.z), "=f"(v.w)
               : "r"(a)
               : "memory");
  return v;
}

}  // namespace dsa
