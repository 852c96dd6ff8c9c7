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
      // the sequence must be as long as its new tokens, and its table as long as it
      if (x.pos < row - first || n > (static_cast<int64_t>(b.max_pages) << shift)) {
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

// New tokens of sequence s in the whole call.
__device__ __forceinline__ int64_t call_rows(const BatchView& b, int s) {
  return static_cast<int64_t>(__ldg(b.cu + s + 1)) - __ldg(b.cu + s);
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
