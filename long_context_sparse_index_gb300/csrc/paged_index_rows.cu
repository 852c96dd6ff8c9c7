// paged_index_rows.cu -- indexer scores over a paged cache for a few rows a
// sequence (drafted tokens, ends of prompts), on the tcgen05 tensor cores.
//
//   score(i, p) = sum_h w[i,h] * ReLU(q[i,h,:] . (hi_p + lo_p))
//
// The pooled keys are the M side: a tile of 128 pools against the (row, head)
// pairs of up to 256 / Hi rows of one sequence, which lie one after another in
// q, so N is rows * Hi and no product is spent on padding.  TMA brings the
// pairs once per run of tiles and the 32 KB of hi and lo page by page into a
// ring of four tiles; 8 tcgen05.mma (four for hi, four for lo) fill one of two
// accumulators; an epilogue thread owns a pool and sums over a row's heads in
// its registers, so the sum over heads needs no exchange between threads.
//
// Every persistent CTA takes an equal, contiguous stretch of all tiles.
//
// Measured at 32 heads: 64 sequences of 32768 tokens (134 MB) in 35 us with 2
// rows each, 40 with 7; 16 of them in 16 and 18 us.  The mma.sync kernel, which
// goes row by row and leaves the heads' sum to shuffles, takes 45, 120, 20 and 42.
// Bound by latency up to a few tiles a CTA, then by the reads (537 MB in 97 us,
// 5.5 TB/s).  With all 256 columns in use (64 x 7 rows: 3.5 TB/s, tensor pipe 32 %,
// issue slots 44 %) by the chain load, wait, fold, shuffle of the epilogue's 32
// thousand values a tile, no unit being full: 8 epilogue warps took 53 us for 7
// rows, 16 that go row by row 45.  One TMA warp issued a box every 25 ns, so that
// pages of 16 tokens (64 boxes a tile) took
// 77 us; three warps take 45, and leave the epilogue its 94 registers (with four
// it had 80 and took 2 to 4 us more).  Five stages were no faster than four.
#include "paged.cuh"

namespace dsa {
namespace {

constexpr int kBM = kRunTile;                 // pools of a tile
static_assert(kBM == 128, "the MMA's M");
constexpr int kBN = 256;                      // (row, head) pairs of an item
constexpr int kDi = 64;
constexpr int kStages = 4;
constexpr uint32_t kHalf = kBM * kDi * 2;     // 16 KB: hi (or lo) of a tile
constexpr uint32_t kABytes = 2 * kHalf;
constexpr uint32_t kBBytes = kBN * kDi * 2;   // 32 KB: queries of a run; two buffers
constexpr int kEpiSubs = 4;                   // warps that share a lane quarter's rows
constexpr int kEpiWarps = 4 * kEpiSubs;
constexpr int kTmaWarps = 3;                  // the pages of a tile are shared out over them
constexpr int kMmaWarp = kTmaWarps;
constexpr int kEpiWarp0 = kTmaWarps + 1;
constexpr int kThreads = 32 * (kEpiWarp0 + kEpiWarps);
constexpr uint32_t kTmemCols = 512;           // 2 accumulators x 256 columns
constexpr uint32_t kCtlOff = kStages * kABytes + 2 * kBBytes;
constexpr uint32_t kWOff = kCtlOff + 256;     // each epilogue warp's head weights
constexpr uint32_t kOffOff = kWOff + kEpiWarps * kBN * 4;
constexpr size_t smem_bytes(int batch) { return 1024 + kOffOff + static_cast<size_t>(batch + 1) * sizeof(int); }
constexpr int kMaxBatchRows = 4096;
static_assert(smem_bytes(kMaxBatchRows) <= 232448, "shared memory per CTA");
// control block (bytes from kCtlOff)
constexpr uint32_t kBarAFull = 0, kBarAEmpty = 32, kBarBFull = 64, kBarBEmpty = 80, kBarAccFull = 96, kBarAccEmpty = 112,
                   kBarDrain = 128, kTmemSlot = 136, kAbort = 140;
static_assert(kStages * 8 <= 32, "the control block's barriers");

struct RowsArgs {
  CacheView c;
  BatchView b;
  const float* w;
  int Hi;
  int group;  // rows of an item
  int64_t row0, row1;
  TcRule tc;
  float* scores;
  float* tops;
  int64_t ld;
  unsigned* status;
  uint64_t limit_ns;
  int inject;
};

__global__ void __launch_bounds__(kThreads, 1)
    paged_score_rows_kernel(const __grid_constant__ CUtensorMap q_map, const __grid_constant__ CUtensorMap k_map,
                            const __grid_constant__ RowsArgs a) {
  extern __shared__ uint8_t smem_raw[];

  const uint32_t raw = smem_u32(smem_raw);
  const uint32_t base = (raw + 1023u) & ~1023u;  // 128-B swizzle atoms need 1024-B alignment
  uint8_t* gbase = smem_raw + (base - raw);
  const uint32_t sA = base, sB = base + kStages * kABytes, sCtl = base + kCtlOff;
  const uint32_t bar_a_full = sCtl + kBarAFull, bar_a_empty = sCtl + kBarAEmpty;
  const uint32_t bar_b_full = sCtl + kBarBFull, bar_b_empty = sCtl + kBarBEmpty;
  const uint32_t bar_acc_full = sCtl + kBarAccFull, bar_acc_empty = sCtl + kBarAccEmpty;
  const uint32_t bar_drain = sCtl + kBarDrain;
  uint32_t* tmem_slot = reinterpret_cast<uint32_t*>(gbase + kCtlOff + kTmemSlot);
  volatile int* abort_flag = reinterpret_cast<volatile int*>(gbase + kCtlOff + kAbort);
  int* off = reinterpret_cast<int*>(gbase + kOffOff);
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;

  if (threadIdx.x == 0) {
    for (int s = 0; s < kStages; ++s) {
      mbar_init(bar_a_full + 8 * s, kTmaWarps);
      mbar_init(bar_a_empty + 8 * s, 1);
    }
    for (int s = 0; s < 2; ++s) {
      mbar_init(bar_b_full + 8 * s, 1);
      mbar_init(bar_b_empty + 8 * s, 1);
      mbar_init(bar_acc_full + 8 * s, 1);
      mbar_init(bar_acc_empty + 8 * s, kEpiWarps);
    }
    mbar_init(bar_drain, 1);
    *abort_flag = 0;
    mbar_fence_init();
  }
  if (warp == kMmaWarp) tmem_alloc(smem_u32(tmem_slot), kTmemCols);
  // items of each sequence: groups of rows x tiles of its last row; one warp scans them, saturating
  if (warp == kEpiWarp0) {
    int sum = 0;
    for (int s0 = 0; s0 < a.b.batch; s0 += 32) {
      const int s = s0 + lane;
      int v = 0;
      if (s < a.b.batch) {
        int64_t first;
        const int n = seq_rows(a.b, s, a.row0, a.row1, &first);
        if (n > 0 && !tc_takes(a.b, a.tc, s)) {
          const int64_t items = (seq_pools(a.b, a.c.shift, s, first, n) + kBM - 1) / kBM * ((n + a.group - 1) / a.group);
          v = static_cast<int>(min(items, static_cast<int64_t>(kMaxItems)));
        }
      }
      int x = v;
#pragma unroll
      for (int o = 1; o < 32; o <<= 1) {
        const int y = __shfl_up_sync(0xffffffffu, x, o);
        if (lane >= o) x += y;
      }
      if (s < a.b.batch) off[s] = sum + x - v;
      sum = min(sum + __shfl_sync(0xffffffffu, x, 31), kMaxTotal);
    }
    if (lane == 0) off[a.b.batch] = sum;
  }
  pdl_wait();  // launched early behind the chunk scores (what was read above is older than their launch)
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  const uint32_t tmem = *tmem_slot;
  const int total = off[a.b.batch];
  const int it0 = static_cast<int>(static_cast<int64_t>(total) * blockIdx.x / gridDim.x);
  const int it1 = static_cast<int>(static_cast<int64_t>(total) * (blockIdx.x + 1) / gridDim.x);
  int it = it0, s = 0;
  {
    int lo = 0, hi = a.b.batch - 1;  // the last sequence whose first item is at or before it0
    while (lo < hi) {
      const int mid = (lo + hi + 1) >> 1;
      if (off[mid] <= it0) lo = mid;
      else hi = mid - 1;
    }
    s = lo;
  }
  auto raise = [&] {
    *abort_flag = 1;
    record_status(a.status, kStatusTimeout);
  };
  int as = 0, bs = 0, cs = 0;  // stage of keys, of queries, accumulator; and their phases
  uint32_t aph = 0, bph = 0, cph = 0;
  bool ok = true;

  if (warp < kTmaWarps) {
    // ---------------------------------------------------------------- TMA producers (a lane per page; warp 0 the queries too)
    const int pshift = a.c.shift - 2, per_page = 1 << pshift;
    const int box = per_page < kBM ? per_page : kBM;  // pools of a box
    const int boxes = kBM / box;                      // 1 .. 32
    const int mine = lane * kTmaWarps + warp;         // this lane's box of every tile
    if (lane == 0) {
      if (warp == 0) tma_prefetch_map(&q_map);
      tma_prefetch_map(&k_map);
    }
    uint32_t a_armed = 0, a_par = 0, b_armed = 0, b_par = 0;
    // this lane's page of the tile at p (-1: none), asked for a tile ahead
    auto page_at = [&](const Run& x, int p) {
      p += mine * box;
      return mine < boxes && p < x.pools ? __ldg(x.table + (p >> pshift)) : -1;
    };
    Run x = next_run(a.b, a.c.shift, a.group, off, a.row0, a.row1, it1, &it, &s);
    int ahead = x.nr > 0 ? page_at(x, x.p0) : -1;
    while (x.nr > 0 && ok) {
      if (warp == 0) {
        ok = __all_sync(0xffffffffu, mbar_wait(bar_b_empty + 8 * bs, bph ^ 1, a.limit_ns, abort_flag));
        if (!ok) break;
        if (lane == 0 && !a.inject) {
          mbar_arrive_expect_tx(bar_b_full + 8 * bs, static_cast<uint32_t>(a.group * a.Hi) * (kDi * 2));
          tma_load_3d(sB + bs * kBBytes, &q_map, bar_b_full + 8 * bs, 0, 0, static_cast<int>(x.ra));
          b_armed |= 1u << bs;
          b_par = (b_par & ~(1u << bs)) | (bph << bs);
        }
        if (++bs == 2) {
          bs = 0;
          bph ^= 1;
        }
      }
      Run nxt = x;
      for (int p = x.p0; p < x.p1; p += kBM) {
        const int page = ahead;
        const bool in = mine < boxes && p + mine * box < x.pools;
        const bool good = in && static_cast<unsigned>(page) < static_cast<unsigned>(a.c.num_pages);
        if (in && !good) record_status(a.status, kStatusInternal);
        if (p + kBM < x.p1) {
          ahead = page_at(x, p + kBM);
        } else {
          nxt = next_run(a.b, a.c.shift, a.group, off, a.row0, a.row1, it1, &it, &s);
          ahead = nxt.nr > 0 ? page_at(nxt, nxt.p0) : -1;
        }
        const uint32_t n = __popc(__ballot_sync(0xffffffffu, good));
        ok = __all_sync(0xffffffffu, mbar_wait(bar_a_empty + 8 * as, aph ^ 1, a.limit_ns, abort_flag));
        if (!ok) break;
        if (!a.inject) {
          if (lane == 0) {
            mbar_arrive_expect_tx(bar_a_full + 8 * as, n * box * (2 * kDi * 2));
            a_armed |= 1u << as;
            a_par = (a_par & ~(1u << as)) | (aph << as);
          }
          __syncwarp();
          if (good) {
            const uint32_t to = sA + as * kABytes + static_cast<uint32_t>(mine * box) * (kDi * 2);
            const int y = (p + mine * box) & (per_page - 1);
            tma_load_3d(to, &k_map, bar_a_full + 8 * as, 0, y, page);
            tma_load_3d(to + kHalf, &k_map, bar_a_full + 8 * as, kDi, y, page);
          }
        }
        if (++as == kStages) {
          as = 0;
          aph ^= 1;
        }
      }
      x = nxt;
    }
    if (lane == 0) {
      if (!ok) raise();
      // every copy this warp issued lands before the CTA may exit
      for (int st = 0; st < kStages; ++st)
        if (a_armed & (1u << st)) mbar_wait(bar_a_full + 8 * st, (a_par >> st) & 1u, a.limit_ns, nullptr);
      for (int st = 0; st < 2; ++st)
        if (b_armed & (1u << st)) mbar_wait(bar_b_full + 8 * st, (b_par >> st) & 1u, a.limit_ns, nullptr);
    }
  } else if (warp == kMmaWarp) {
    // ---------------------------------------------------------------- MMA issuer
    if (lane == 0) {
      bool issued = false;
      for (Run x = next_run(a.b, a.c.shift, a.group, off, a.row0, a.row1, it1, &it, &s); x.nr > 0 && ok; x = next_run(a.b, a.c.shift, a.group, off, a.row0, a.row1, it1, &it, &s)) {
        ok = mbar_wait(bar_b_full + 8 * bs, bph, a.limit_ns, abort_flag);
        if (!ok) break;
        const uint32_t idesc = umma_idesc_bf16_f32(kBM, (x.nr * a.Hi + 15) & ~15);
        const uint32_t bb = sB + bs * kBBytes;
        for (int p = x.p0; p < x.p1; p += kBM) {
          if (!mbar_wait(bar_a_full + 8 * as, aph, a.limit_ns, abort_flag) ||
              !mbar_wait(bar_acc_empty + 8 * cs, cph ^ 1, a.limit_ns, abort_flag)) {
            ok = false;
            break;
          }
          tc_fence_after();
          const uint32_t aa = sA + as * kABytes;
#pragma unroll
          for (int kk = 0; kk < 8; ++kk)
            umma_bf16(tmem + cs * kBN, umma_desc_sw128(aa + (kk < 4 ? 0u : kHalf) + (kk & 3) * 32),
                      umma_desc_sw128(bb + (kk & 3) * 32), idesc, kk > 0 ? 1u : 0u);
          issued = true;
          umma_commit(bar_a_empty + 8 * as);
          umma_commit(bar_acc_full + 8 * cs);
          if (++as == kStages) {
            as = 0;
            aph ^= 1;
          }
          if (++cs == 2) {
            cs = 0;
            cph ^= 1;
          }
        }
        if (!ok) break;
        umma_commit(bar_b_empty + 8 * bs);
        if (++bs == 2) {
          bs = 0;
          bph ^= 1;
        }
      }
      if (!ok) raise();
      if (issued) {  // all MMAs done before tensor memory and shared memory are released
        umma_commit(bar_drain);
        mbar_wait(bar_drain, 0, a.limit_ns, nullptr);
      }
    }
  } else {
    // ---------------------------------------------------------------- epilogue
    // Warp w reads TMEM lanes 32 * (w % 4) ..: a pool per thread, and every fourth row.
    const int ew = warp - kEpiWarp0, lq = warp & 3, sub = ew >> 2;
    float* wt = reinterpret_cast<float*>(gbase + kWOff) + ew * kBN;
    const uint32_t tlane = tmem + (static_cast<uint32_t>(lq * 32) << 16);
    const int ld = static_cast<int>(a.ld);
    // 16 heads of a row, added to acc
    auto fold = [](float2& acc, const uint32_t (&v)[16], const float* wc) {
#pragma unroll
      for (int j = 0; j < 4; ++j) {
        const float4 w4 = *reinterpret_cast<const float4*>(wc + 4 * j);
        acc = __ffma2_rn(make_float2(w4.x, w4.y), make_float2(fmaxf(__uint_as_float(v[4 * j]), 0.f),
                                                              fmaxf(__uint_as_float(v[4 * j + 1]), 0.f)), acc);
        acc = __ffma2_rn(make_float2(w4.z, w4.w), make_float2(fmaxf(__uint_as_float(v[4 * j + 2]), 0.f),
                                                              fmaxf(__uint_as_float(v[4 * j + 3]), 0.f)), acc);
      }
    };
    for (Run x = next_run(a.b, a.c.shift, a.group, off, a.row0, a.row1, it1, &it, &s); x.nr > 0 && ok; x = next_run(a.b, a.c.shift, a.group, off, a.row0, a.row1, it1, &it, &s)) {
      __syncwarp();
      for (int j = lane; j < kBN; j += 32) wt[j] = j < x.nr * a.Hi ? __ldg(a.w + x.ra * a.Hi + j) : 0.f;
      __syncwarp();
      const int64_t first = (x.ra - a.row0) * a.ld + lq * 32 + lane;  // (a multiple of 8 but for the lane)
      float* out = a.scores + first;
      float* otop = a.tops + (first >> 3);
      for (int p = x.p0; p < x.p1; p += kBM) {
        // (the loads below are the whole warp's: its lanes agree)
        if (!__all_sync(0xffffffffu, mbar_wait(bar_acc_full + 8 * cs, cph, a.limit_ns, abort_flag))) {
          ok = false;
          break;
        }
        tc_fence_after();
        const uint32_t from = tlane + cs * kBN;
        const bool in = p + lq * 32 + lane < x.pools;
        int r = sub;
        // two rows at a time, so that each one's reads and shuffles hide behind the other's
        for (; r + kEpiSubs < x.nr && (a.Hi & 15) == 0; r += 2 * kEpiSubs) {
          float2 acc[2] = {make_float2(0.f, 0.f), make_float2(0.f, 0.f)};
          int col = r * a.Hi;
          const int apart = kEpiSubs * a.Hi;
          for (const int end = col + a.Hi; col < end; col += 16) {
            uint32_t v[2][16];
            tmem_ld16(from + col, v[0]);
            tmem_ld16(from + col + apart, v[1]);
            tmem_ld_wait();
            fold(acc[0], v[0], wt + col);
            fold(acc[1], v[1], wt + col + apart);
          }
          float sum[2], top[2];
#pragma unroll
          for (int e = 0; e < 2; ++e) {
            sum[e] = acc[e].x + acc[e].y;
            top[e] = in ? sum[e] : -INFINITY;
          }
          // the largest of each eight pools
#pragma unroll
          for (int o = 1; o < 8; o <<= 1)
#pragma unroll
            for (int e = 0; e < 2; ++e) top[e] = fmaxf(top[e], __shfl_xor_sync(0xffffffffu, top[e], o));
          if (in) {
#pragma unroll
            for (int e = 0; e < 2; ++e) {
              const int64_t to = static_cast<int64_t>(r + e * kEpiSubs) * ld + p;
              out[to] = sum[e];
              if ((lane & 7) == 0) otop[to >> 3] = top[e];
            }
          }
        }
        for (; r < x.nr; r += kEpiSubs) {
          float2 acc = make_float2(0.f, 0.f);
          int h0 = 0;
          for (; h0 + 16 <= a.Hi && (a.Hi & 3) == 0; h0 += 16) {
            const int col = r * a.Hi + h0;
            uint32_t v[16];
            tmem_ld16(from + col, v);
            tmem_ld_wait();
            fold(acc, v, wt + col);
          }
          for (; h0 < a.Hi; h0 += 16) {
            const int col = r * a.Hi + h0, c0 = min(col, kBN - 16);  // (never past the accumulator)
            uint32_t v[16];
            tmem_ld16(from + c0, v);
            tmem_ld_wait();
#pragma unroll
            for (int j = 0; j < 16; ++j) {
              const int c = c0 + j;  // this row's heads from h0 on lie in columns col ..; the others are another row's
              if (c >= col && c < (r + 1) * a.Hi) acc.x = fmaf(wt[c], fmaxf(__uint_as_float(v[j]), 0.f), acc.x);
            }
          }
          const float sum = acc.x + acc.y;
          float top = in ? sum : -INFINITY;
#pragma unroll
          for (int o = 1; o < 8; o <<= 1) top = fmaxf(top, __shfl_xor_sync(0xffffffffu, top, o));
          if (in) {
            const int64_t to = static_cast<int64_t>(r) * ld + p;
            out[to] = sum;
            if ((lane & 7) == 0) otop[to >> 3] = top;
          }
        }
        tc_fence_before();
        __syncwarp();
        if (lane == 0) mbar_arrive(bar_acc_empty + 8 * cs);
        if (++cs == 2) {
          cs = 0;
          cph ^= 1;
        }
      }
    }
    if (!ok && lane == 0) raise();
  }

  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  if (warp == kMmaWarp) tmem_dealloc(tmem, kTmemCols);
}

}  // namespace

bool paged_scores_rows_fits(const BatchView& b) { return b.batch <= kMaxBatchRows; }
int paged_scores_rows_group(int Hi) { return kBN / Hi < 32 ? kBN / Hi : 32; }

cudaError_t launch_paged_scores_rows(const CUtensorMap& q_map, const CUtensorMap& k_map, const CacheView& c,
                                     const BatchView& b, const float* w, int Hi, int64_t row0, int64_t nrows,
                                     TcRule tc, float* scores, float* tops, int64_t ld, bool early,
                                     const LaunchCtx& call) {
  static std::atomic<bool> attr_done[kAttrDevices];
  const cudaError_t e =
      set_smem_limit_once(paged_score_rows_kernel, static_cast<int>(smem_bytes(kMaxBatchRows)), attr_done);
  if (e != cudaSuccess) return e;
  const RowsArgs a{c, b, w, Hi, paged_scores_rows_group(Hi), row0, row0 + nrows, tc, scores, tops, ld,
                   call.status, call.wait_limit_ns, call.inject_timeout};
  LaunchCtx ctx = call;
  ctx.pdl = early;
  return launch_ex(ctx, paged_score_rows_kernel, dim3(ctx.num_sms), dim3(kThreads), smem_bytes(b.batch), q_map, k_map, a);
}

}  // namespace dsa
