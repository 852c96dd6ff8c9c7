// paged_rope_kernels.h -- host-side launchers over a paged cache with rotated
// positions, and over one in 4 bits (internal).
#pragma once

#include "paged_kernels.h"
#include "rope_kernels.h"

namespace dsa {

constexpr int kPool4 = 576;  // bytes of a pool (kv4.cuh)
// A cache in 4 bits is a CacheView whose `k` is the 4-bit buffer (k_stride in
// units of two bytes) and whose `v` is null.

// Heads of the call's rows to be turned, bf16 [rows][heads][d]; heads 0: none.
struct QueryRows {
  const __nv_bfloat16* in;
  __nv_bfloat16* out;
  int64_t in_stride, out_stride;  // elements from row to row
  int heads;
};
struct RopeAppendArgs {
  AppendArgs a;
  RopeView rope, rope_idx;  // of keys and queries, and of the indexer's
  QueryRows q, qi;
};
cudaError_t launch_append_rope(const CacheView& c, bool four, const BatchView& b, const RopeAppendArgs& x,
                               const LaunchCtx& ctx);
// Rows of k and v [rows][128] as the cache holds them.
cudaError_t launch_cache4_read(const CacheView& c, const BatchView& b, void* k, int64_t k_stride, void* v,
                               int64_t v_stride, const LaunchCtx& ctx);
cudaError_t launch_paged4_attn(const CacheView& c, const BatchView& b, const void* q, const int32_t* pool_idx, int topk,
                               float scale, void* o, float* lse, const LaunchCtx& ctx);

}  // namespace dsa
