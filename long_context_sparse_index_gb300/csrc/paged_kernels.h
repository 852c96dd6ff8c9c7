// paged_kernels.h -- host-side launchers of the paged-cache kernels and the
// views they take (internal).
#pragma once

#include <cuda_bf16.h>
#include <cuda_runtime.h>
#include <cstdint>

#include "dsa_kernels.h"

namespace dsa {

// One layer's cache in pages of 2^shift tokens.  Strides are in elements from
// one page to the next; within a page everything is contiguous.
struct CacheView {
  __nv_bfloat16* k;      // [num_pages][page][128]
  __nv_bfloat16* v;      // [num_pages][page][128]
  __nv_bfloat16* k_idx;  // [num_pages][page][64]
  __nv_bfloat16* khat;   // [num_pages][page / 4][128]: hi 0..63, lo 64..127
  int64_t k_stride, v_stride, kidx_stride, khat_stride;
  int num_pages;
  int shift;             // log2(page size), 4..10
};

// The sequences of a call and their new tokens (device arrays).
struct BatchView {
  const int32_t* table;  // [batch][max_pages], rows table_stride apart
  int64_t table_stride;
  int max_pages;
  const int32_t* lens;   // [batch] tokens with the new ones
  const int32_t* cu;     // [batch + 1] rows of the new tokens
  int batch;
  int64_t rows;          // rows of the call's tensors (rows past cu[batch] are padding)
};

// The page bookkeeping of a cache (device arrays, written by the page operators).
struct PageTableView {
  int32_t* table;        // [max_seqs][max_pages]
  int64_t table_stride;
  int max_pages;
  int32_t* lens;         // [max_seqs]
  int max_seqs;
  int32_t* count;        // [num_pages] sequences that hold the page
};

struct AppendArgs {
  const __nv_bfloat16 *k, *v, *k_idx;       // rows of the new tokens
  int64_t k_stride, v_stride, kidx_stride;  // elements from row to row
  const int32_t* reserved;                  // a reservation's result, or null
};

// The layers of one launch that moves pages: their caches have the same pages
// of the same size.  Passed by value as a kernel parameter.
constexpr int kLayerBatch = 32;
struct CacheSet {
  int n;
  CacheView v[kLayerBatch];
};

cudaError_t launch_cache_append(const CacheView& c, const BatchView& b, const AppendArgs& a, const LaunchCtx& ctx);
// (four: caches whose keys and values are in 4 bits)
cudaError_t launch_copy_pages(const CacheSet& set, bool four, const int32_t* src, const int32_t* dst, int64_t n,
                              const LaunchCtx& ctx);
// Scratch words (int32) of the page operators below.
int64_t fork_ws_words(int64_t n, int max_seqs);
int64_t reserve_ws_words(int max_seqs, int num_pages);
int64_t compact_ws_words(int num_pages);
cudaError_t launch_cache_reserve(const PageTableView& t, int shift, int num_pages, const int32_t* add, int32_t* result,
                                 int32_t* ws, const LaunchCtx& ctx);
// Forking and compacting: the plan, then apply once per batch of layers; `first`
// also changes the table and the counts.
cudaError_t launch_fork_plan(const PageTableView& t, int shift, int num_pages, const int32_t* src, const int32_t* dst,
                             int n, int32_t* result, int32_t* ws, const LaunchCtx& ctx);
cudaError_t launch_fork_apply(const CacheSet& set, bool four, bool first, const PageTableView& t, const int32_t* src,
                              const int32_t* dst, int n, int32_t* ws, const LaunchCtx& ctx);
cudaError_t launch_cache_free(const PageTableView& t, int shift, int num_pages, const int32_t* seqs, int n,
                              const LaunchCtx& ctx);
cudaError_t launch_compact_plan(const PageTableView& t, int num_pages, int32_t* result, int32_t* ws,
                                const LaunchCtx& ctx);
cudaError_t launch_compact_apply(const CacheSet& set, bool four, bool first, const PageTableView& t, int32_t* ws,
                                 const LaunchCtx& ctx);

// Which sequences' scores the kernel of 128-row tiles makes: those of at least
// so many rows and so many tiles (128 rows x 256 pools) in the call.
struct TcRule {
  int rows, tiles;
};

// Indexer over the pages: scores of launch rows [row0, row0 + nrows) into
// scores [nrows][ld] (pool p of a row's sequence in column p) and the largest
// of each eight pools into tops [nrows][ld / 8], then each row's top-k.  ld is
// a multiple of 32.  Only the sequences that the rule leaves; early: launched
// early behind the tcgen05 scores of the others.
cudaError_t launch_paged_scores(const CacheView& c, const BatchView& b, const void* q_idx, const float* w, int Hi,
                                int64_t row0, int64_t nrows, TcRule tc, float* scores, float* tops, int64_t ld,
                                bool early, const LaunchCtx& ctx);
// The same on tcgen05, 128 rows of a sequence at a time, for the sequences that
// the rule names: chunks.  q_map: [64, Hi, rows], box {64, 1, 128}; k_map:
// [128, pools per page, pages], box {64, pools per page, 1}; both swizzled by
// 128 bytes.
bool paged_scores_tc_fits(const BatchView& b);
cudaError_t launch_paged_scores_tc(const CUtensorMap& q_map, const CUtensorMap& k_map, const CacheView& c,
                                   const BatchView& b, const float* w, int Hi, int64_t row0, int64_t nrows,
                                   TcRule tc, float* scores, float* tops, int64_t ld, const LaunchCtx& ctx);
// The same on tcgen05 with (row, head) pairs as columns, for the sequences that
// the rule leaves.  q_map: [64, Hi, rows], box {64, Hi, group}; k_map as
// above, box {64, min(pools per page, 128), 1}.
bool paged_scores_rows_fits(const BatchView& b);
int paged_scores_rows_group(int Hi);  // rows of an item
cudaError_t launch_paged_scores_rows(const CUtensorMap& q_map, const CUtensorMap& k_map, const CacheView& c,
                                     const BatchView& b, const float* w, int Hi, int64_t row0, int64_t nrows,
                                     TcRule tc, float* scores, float* tops, int64_t ld, bool early,
                                     const LaunchCtx& ctx);
cudaError_t launch_paged_select(const BatchView& b, int shift, int64_t row0, int64_t nrows, const float* scores,
                                const float* tops, int64_t ld, int topk, int32_t* pool_idx, const LaunchCtx& ctx);

cudaError_t launch_paged_attn(const CacheView& c, const BatchView& b, const void* q, const int32_t* pool_idx, int topk,
                              float scale, void* o, float* lse, const LaunchCtx& ctx);

}  // namespace dsa
