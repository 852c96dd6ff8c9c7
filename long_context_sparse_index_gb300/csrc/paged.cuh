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

// Sequence of `row` (all lanes of a warp call it together with the same row):
// the number of sequences that end at or before it.  batch: past the last.
__device__ __forceinline__ int warp_locate(const BatchView& b, int64_t row, int lane) {
  int n = 0;
  for (int j = lane; j < b.batch; j += 32) n += __ldg(b.cu + j + 1) <= row;
#pragma unroll
  for (int o = 16; o > 0; o >>= 1) n += __shfl_xor_sync(0xffffffffu, n, o);
  return n;
}

// Position of `row` in its sequence s (< batch), or -1 (recorded) when the
// offsets and lengths contradict each other or the block table is too short.
__device__ __forceinline__ int64_t row_position(const BatchView& b, int shift, int s, int64_t row, unsigned* status) {
  const int c0 = __ldg(b.cu + s), c1 = __ldg(b.cu + s + 1), len = __ldg(b.lens + s);
  const int64_t i = static_cast<int64_t>(len) - c1 + row;
  if (row < c0 || row >= c1 || i < row - c0 || len > (static_cast<int64_t>(b.max_pages) << shift)) {
    record_status(status, kStatusInternal);
    return -1;
  }
  return i;
}

// Page x of sequence s (x < max_pages), or -1 (recorded) for a number that is
// no page.
__device__ __forceinline__ int page_of(const BatchView& b, int num_pages, int s, int x, unsigned* status) {
  const int p = __ldg(b.table + s * b.table_stride + x);
  if (static_cast<unsigned>(p) < static_cast<unsigned>(num_pages)) return p;
  record_status(status, kStatusInternal);
  return -1;
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
