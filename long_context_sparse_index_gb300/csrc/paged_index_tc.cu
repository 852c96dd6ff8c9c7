// paged_index_tc.cu -- indexer scores over a paged cache for chunks of a
// prompt (many rows a sequence), on the tcgen05 tensor cores.
//
//   score(i, p) = sum_h w[i,h] * ReLU(q[i,h,:] . (hi_p + lo_p))
//
// A work item is 128 rows of one sequence against 256 pools.  TMA brings the
// 64 KB of pooled keys page by page (their page numbers come from the block
// table; one box per page and half, into the 128-byte-swizzled K-major tile
// that the MMA reads) and, per head, the rows' 16 KB query tile; a chain of 8
// tcgen05.mma (M 128, N 256, K 16: four for hi, four for lo) accumulates
// q_h . Khat in tensor memory.  16 epilogue warps fold ReLU, the head weight
// and the sum over heads into registers (64 fp32 sums a thread) while the next
// head's products fill the other accumulator; the 128 x 256 scores leave
// through a staging tile, so that every store covers whole 128-byte lines.
//
// One persistent CTA per SM takes items in turn; items of the same pools are
// neighbours, so their pooled keys come from L2.
//
// Measured: 2048 rows of 32 heads against 32768 pools, the last chunk of a
// context of 131072, in 367 us: 760 TFLOP/s, 1520 executed (hi and lo), 0.89 of
// the measured sustained bf16 rate.  The products of a head take 1300 cycles on
// a full chip (1024 nominal; without any epilogue, too), and an item's end
// costs 8 thousand of its 51: the scores' stores and the next item's keys meet
// those of every other SM.  TMA stores from the staging tile, a ring of items
// worked out ahead and a third half-buffer for the next keys moved that time
// into the products (361-368 us) and were not kept; splitting a head's eight
// products around a wait for lo cost 40 us.
#include "paged.cuh"

namespace dsa {
namespace {

constexpr int kBM = 128;
constexpr int kBN = 256;
constexpr int kDi = 64;
constexpr int kAStages = 4;
constexpr uint32_t kABytes = kBM * kDi * 2;   // 16 KB: query tile of one head
constexpr uint32_t kBHalf = kBN * kDi * 2;    // 32 KB: hi (or lo) halves of the pooled keys
constexpr uint32_t kBBytes = 2 * kBHalf;
constexpr int kEpiWarps = 16;                 // 4 TMEM lane quarters x 4 column quarters
constexpr int kEpiCols = kBN / 4;
constexpr int kEpiWarp0 = 2;
constexpr int kThreads = 32 * (kEpiWarp0 + kEpiWarps);
constexpr uint32_t kTmemCols = 512;           // 2 accumulators x 256 columns
constexpr int kStgLd = 36;
constexpr uint32_t kStgBytes = 32 * kStgLd * 4;
constexpr uint32_t kCtlOff = kBBytes + kAStages * kABytes;
constexpr uint32_t kStgOff = kCtlOff + 256;
constexpr uint32_t kOffOff = kStgOff + kEpiWarps * kStgBytes;  // the sequences' item prefix
constexpr size_t smem_bytes(int batch) { return 1024 + kOffOff + static_cast<size_t>(batch + 1) * sizeof(int); }
constexpr int kMaxBatchTc = 4096;
static_assert(smem_bytes(kMaxBatchTc) <= 232448, "shared memory per CTA");
// control block (bytes from kCtlOff)
constexpr uint32_t kBarAFull = 0, kBarAEmpty = 32, kBarBFull = 64, kBarBEmpty = 72, kBarAccFull = 80, kBarAccEmpty = 96,
                   kBarDrain = 112, kTmemSlot = 120, kAbort = 124;

struct TcArgs {
  CacheView c;
  BatchView b;
  const float* w;
  int Hi;
  int64_t row0, row1;
  TcRule tc;
  float* scores;
  float* tops;
  int64_t ld;
  unsigned* status;
  uint64_t limit_ns;
  int inject;
};

struct TcItem {
  int s;
  int nr;          // rows (<= 128)
  int64_t ra;      // first row
  int64_t p0;      // first pool
  int64_t pools;   // pools that the last row may see
};

// Item `it`; *s is a cursor that only moves forward.  False: nothing to score.
__device__ __forceinline__ bool item_at(const TcArgs& a, const int* off, int it, int* s, TcItem* x) {
  while (*s + 1 < a.b.batch && it >= off[*s + 1]) ++*s;
  int64_t first;
  const int n = seq_rows(a.b, *s, a.row0, a.row1, &first);
  if (n == 0) return false;
  const int row_tiles = (n + kBM - 1) / kBM, local = it - off[*s];
  x->s = *s;
  x->ra = first + static_cast<int64_t>(local % row_tiles) * kBM;
  x->nr = static_cast<int>(min(static_cast<int64_t>(kBM), first + n - x->ra));
  x->p0 = static_cast<int64_t>(local / row_tiles) * kBN;
  x->pools = seq_pools(a.b, a.c.shift, *s, x->ra, x->nr);
  return x->nr > 0 && x->p0 < x->pools;
}

__global__ void __launch_bounds__(kThreads, 1)
    paged_score_tc_kernel(const __grid_constant__ CUtensorMap q_map, const __grid_constant__ CUtensorMap k_map,
                          const TcArgs a) {
  extern __shared__ uint8_t smem_raw[];

  const uint32_t raw = smem_u32(smem_raw);
  const uint32_t base = (raw + 1023u) & ~1023u;  // 128-B swizzle atoms need 1024-B alignment
  uint8_t* gbase = smem_raw + (base - raw);
  const uint32_t sB = base, sA = base + kBBytes, sCtl = base + kCtlOff;
  const uint32_t bar_a_full = sCtl + kBarAFull, bar_a_empty = sCtl + kBarAEmpty;
  const uint32_t bar_b_full = sCtl + kBarBFull, bar_b_empty = sCtl + kBarBEmpty;
  const uint32_t bar_acc_full = sCtl + kBarAccFull, bar_acc_empty = sCtl + kBarAccEmpty;
  const uint32_t bar_drain = sCtl + kBarDrain;
  uint32_t* tmem_slot = reinterpret_cast<uint32_t*>(gbase + kCtlOff + kTmemSlot);
  volatile int* abort_flag = reinterpret_cast<volatile int*>(gbase + kCtlOff + kAbort);
  int* off = reinterpret_cast<int*>(gbase + kOffOff);
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;

  if (threadIdx.x == 0) {
    for (int s = 0; s < kAStages; ++s) {
      mbar_init(bar_a_full + 8 * s, 1);
      mbar_init(bar_a_empty + 8 * s, 1);
    }
    mbar_init(bar_b_full, 1);
    mbar_init(bar_b_empty, 1);
    for (int s = 0; s < 2; ++s) {
      mbar_init(bar_acc_full + 8 * s, 1);
      mbar_init(bar_acc_empty + 8 * s, kEpiWarps);
    }
    mbar_init(bar_drain, 1);
    *abort_flag = 0;
    mbar_fence_init();
  }
  if (warp == 1) tmem_alloc(smem_u32(tmem_slot), kTmemCols);
  // items of each sequence: row tiles x pool tiles of its last row (a chunk's
  // earlier row tiles skip the few past their own end); one warp scans them,
  // saturating
  if (warp == 2) {
    int sum = 0;
    for (int s0 = 0; s0 < a.b.batch; s0 += 32) {
      const int s = s0 + lane;
      int v = 0;
      if (s < a.b.batch) {
        int64_t first;
        const int n = seq_rows(a.b, s, a.row0, a.row1, &first);
        if (n > 0 && tc_takes(a.b, a.tc, s)) {
          const int64_t items = (seq_pools(a.b, a.c.shift, s, first, n) + kBN - 1) / kBN * ((n + kBM - 1) / kBM);
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
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  const uint32_t tmem = *tmem_slot;
  const int total = off[a.b.batch];
  auto raise = [&] {
    *abort_flag = 1;
    record_status(a.status, kStatusTimeout);
  };

  if (warp == 0) {
    // ---------------------------------------------------------------- TMA producer (a lane per page; lane 0 the queries)
    const int pshift = a.c.shift - 2, per_page = 1 << pshift;
    const int pages = kBN >> pshift;  // 1 .. 64
    if (lane == 0) {
      tma_prefetch_map(&q_map);
      tma_prefetch_map(&k_map);
    }
    int as = 0, s = 0;
    uint32_t aph = 0, bph = 0, a_armed = 0, a_par = 0, b_par = 0;
    bool b_armed = false, ok = true;
    for (int it = blockIdx.x; it < total && ok; it += gridDim.x) {
      TcItem x;
      if (!item_at(a, off, it, &s, &x)) continue;
      int page[2];
      unsigned n = 0;
#pragma unroll
      for (int u = 0; u < 2; ++u) {
        const int j = u * 32 + lane;
        const int64_t p = x.p0 + (static_cast<int64_t>(j) << pshift);
        page[u] = -1;
        if (j < pages && p < x.pools)
          page[u] = page_of(a.b, a.c.num_pages, x.s, static_cast<int>(p >> pshift), a.status);
        n += __popc(__ballot_sync(0xffffffffu, page[u] >= 0));
      }
      ok = __all_sync(0xffffffffu, mbar_wait(bar_b_empty, bph ^ 1, a.limit_ns, abort_flag));
      if (!ok) break;
      if (!a.inject) {
        if (lane == 0) {
          mbar_arrive_expect_tx(bar_b_full, n * per_page * (2 * kDi * 2));
          b_armed = true;
          b_par = bph;
        }
        __syncwarp();
#pragma unroll
        for (int u = 0; u < 2; ++u)
          if (page[u] >= 0) {
            const uint32_t at = sB + static_cast<uint32_t>((u * 32 + lane) << pshift) * (kDi * 2);
            tma_load_3d(at, &k_map, bar_b_full, 0, 0, page[u]);
            tma_load_3d(at + kBHalf, &k_map, bar_b_full, kDi, 0, page[u]);
          }
      }
      bph ^= 1;
      if (lane == 0) {
        for (int h = 0; h < a.Hi; ++h) {
          if (!mbar_wait(bar_a_empty + 8 * as, aph ^ 1, a.limit_ns, abort_flag)) {
            ok = false;
            break;
          }
          if (!a.inject) {
            mbar_arrive_expect_tx(bar_a_full + 8 * as, kABytes);
            tma_load_3d(sA + as * kABytes, &q_map, bar_a_full + 8 * as, 0, h, static_cast<int>(x.ra));
            a_armed |= 1u << as;
            a_par = (a_par & ~(1u << as)) | (aph << as);
          }
          if (++as == kAStages) {
            as = 0;
            aph ^= 1;
          }
        }
      }
      ok = __shfl_sync(0xffffffffu, static_cast<int>(ok), 0) != 0;
    }
    if (lane == 0) {
      if (!ok) raise();
      // every copy this warp issued lands before the CTA may exit
      for (int st = 0; st < kAStages; ++st)
        if (a_armed & (1u << st)) mbar_wait(bar_a_full + 8 * st, (a_par >> st) & 1u, a.limit_ns, nullptr);
      if (b_armed) mbar_wait(bar_b_full, b_par, a.limit_ns, nullptr);
    }
  } else if (warp == 1) {
    // ---------------------------------------------------------------- MMA issuer
    if (lane == 0) {
      constexpr uint32_t idesc = umma_idesc_bf16_f32(kBM, kBN);
      int as = 0, cs = 0, s = 0;
      uint32_t aph = 0, bph = 0, cph = 0;
      bool ok = true, issued = false;
      for (int it = blockIdx.x; it < total && ok; it += gridDim.x) {
        TcItem x;
        if (!item_at(a, off, it, &s, &x)) continue;
        if (!mbar_wait(bar_b_full, bph, a.limit_ns, abort_flag)) {
          ok = false;
          break;
        }
        tc_fence_after();
        for (int h = 0; h < a.Hi; ++h) {
          if (!mbar_wait(bar_a_full + 8 * as, aph, a.limit_ns, abort_flag) ||
              !mbar_wait(bar_acc_empty + 8 * cs, cph ^ 1, a.limit_ns, abort_flag)) {
            ok = false;
            break;
          }
          tc_fence_after();
          const uint32_t d = tmem + cs * kBN, aa = sA + as * kABytes;
#pragma unroll
          for (int kk = 0; kk < 8; ++kk)
            umma_bf16(d, umma_desc_sw128(aa + (kk & 3) * 32),
                      umma_desc_sw128(sB + (kk < 4 ? 0u : kBHalf) + (kk & 3) * 32), idesc, kk > 0 ? 1u : 0u);
          issued = true;
          umma_commit(bar_a_empty + 8 * as);
          umma_commit(bar_acc_full + 8 * cs);
          if (++as == kAStages) {
            as = 0;
            aph ^= 1;
          }
          if (++cs == 2) {
            cs = 0;
            cph ^= 1;
          }
        }
        if (!ok) break;
        umma_commit(bar_b_empty);
        bph ^= 1;
      }
      if (!ok) raise();
      if (issued) {  // all MMAs done before tensor memory and shared memory are released
        umma_commit(bar_drain);
        mbar_wait(bar_drain, 0, a.limit_ns, nullptr);
      }
    }
  } else {
    // ---------------------------------------------------------------- epilogue
    // Warp w reads TMEM lanes 32 * (w % 4) .. and 64 columns of each
    // accumulator: one row and 64 pools per thread.
    const int ew = warp - kEpiWarp0, lq = warp & 3, cq = ew >> 2;
    float* stg = reinterpret_cast<float*>(gbase + kStgOff + ew * kStgBytes);
    int cs = 0, s = 0;
    uint32_t cph = 0;
    bool ok = true;
    for (int it = blockIdx.x; it < total && ok; it += gridDim.x) {
      TcItem x;
      if (!item_at(a, off, it, &s, &x)) continue;
      const int r = lq * 32 + lane;
      const bool valid = r < x.nr;
      const float* wrow = a.w + (x.ra + (valid ? r : 0)) * a.Hi;
      float2 acc[kEpiCols / 2];
#pragma unroll
      for (int j = 0; j < kEpiCols / 2; ++j) acc[j] = make_float2(0.f, 0.f);
      // the head weight is fetched one head ahead
      float w_next = valid ? __ldg(wrow) : 0.f;
      for (int h = 0; h < a.Hi; ++h) {
        const float wv = w_next;
        if (h + 1 < a.Hi) w_next = valid ? __ldg(wrow + h + 1) : 0.f;
        // (the loads below are the whole warp's: its lanes agree)
        if (!__all_sync(0xffffffffu, mbar_wait(bar_acc_full + 8 * cs, cph, a.limit_ns, abort_flag))) {
          ok = false;
          break;
        }
        tc_fence_after();
        const float2 w2 = make_float2(wv, wv);
        const uint32_t taddr = tmem + (static_cast<uint32_t>(lq * 32) << 16) + cs * kBN + cq * kEpiCols;
#pragma unroll
        for (int cc = 0; cc < kEpiCols / 16; ++cc) {
          uint32_t v[16];
          tmem_ld16(taddr + cc * 16, v);
          tmem_ld_wait();
          if (cc == kEpiCols / 16 - 1) {  // the last load has landed: the accumulator is free
            tc_fence_before();
            __syncwarp();
            if (lane == 0) mbar_arrive(bar_acc_empty + 8 * cs);
          }
#pragma unroll
          for (int j = 0; j < 8; ++j) {
            const float2 y =
                make_float2(fmaxf(__uint_as_float(v[2 * j]), 0.f), fmaxf(__uint_as_float(v[2 * j + 1]), 0.f));
            acc[cc * 8 + j] = __ffma2_rn(w2, y, acc[cc * 8 + j]);
          }
        }
        if (++cs == 2) {
          cs = 0;
          cph ^= 1;
        }
      }
      if (!ok) break;
      float* out = a.scores + (x.ra - a.row0) * a.ld + x.p0;
      const int64_t room = x.pools - x.p0;  // columns of this tile that exist (stores of four may end past it, inside ld)
#pragma unroll
      for (int half = 0; half < 2; ++half) {
        // the largest of each eight pools of this thread's row (a group past
        // the pools that exist holds anything: nobody reads it)
        float top[4];
#pragma unroll
        for (int k = 0; k < 4; ++k) {
          const float2 u = acc[16 * half + 4 * k], v = acc[16 * half + 4 * k + 1], y = acc[16 * half + 4 * k + 2],
                       z = acc[16 * half + 4 * k + 3];
          top[k] = fmaxf(fmaxf(fmaxf(u.x, u.y), fmaxf(v.x, v.y)), fmaxf(fmaxf(y.x, y.y), fmaxf(z.x, z.y)));
        }
        if (valid && cq * kEpiCols + 32 * half < room)
          *reinterpret_cast<float4*>(a.tops +
                                     (((x.ra - a.row0 + r) * a.ld + x.p0 + cq * kEpiCols + 32 * half) >> 3)) =
              make_float4(top[0], top[1], top[2], top[3]);
#pragma unroll
        for (int j = 0; j < 8; ++j) {
          const float2 u = acc[16 * half + 2 * j], v = acc[16 * half + 2 * j + 1];
          *reinterpret_cast<float4*>(stg + lane * kStgLd + 4 * j) = make_float4(u.x, u.y, v.x, v.y);
        }
        __syncwarp();
#pragma unroll
        for (int k = 0; k < 8; ++k) {
          const int rr = 4 * k + (lane >> 3), col = 4 * (lane & 7);
          const float4 y = *reinterpret_cast<const float4*>(stg + rr * kStgLd + col);
          const int pc = cq * kEpiCols + 32 * half + col;
          if (lq * 32 + rr < x.nr && pc < room)
            *reinterpret_cast<float4*>(out + static_cast<int64_t>(lq * 32 + rr) * a.ld + pc) = y;
        }
        __syncwarp();
      }
    }
    if (!ok && lane == 0) raise();
  }

  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  if (warp == 1) tmem_dealloc(tmem, kTmemCols);
}

}  // namespace

bool paged_scores_tc_fits(const BatchView& b) { return b.batch <= kMaxBatchTc; }

cudaError_t launch_paged_scores_tc(const CUtensorMap& q_map, const CUtensorMap& k_map, const CacheView& c,
                                   const BatchView& b, const float* w, int Hi, int64_t row0, int64_t nrows,
                                   TcRule tc, float* scores, float* tops, int64_t ld, const LaunchCtx& ctx) {
  static std::atomic<bool> attr_done[kAttrDevices];
  const cudaError_t e =
      set_smem_limit_once(paged_score_tc_kernel, static_cast<int>(smem_bytes(kMaxBatchTc)), attr_done);
  if (e != cudaSuccess) return e;
  const TcArgs a{c, b, w, Hi, row0, row0 + nrows, tc, scores, tops, ld, ctx.status, ctx.wait_limit_ns, ctx.inject_timeout};
  paged_score_tc_kernel<<<ctx.num_sms, kThreads, smem_bytes(b.batch), ctx.stream>>>(q_map, k_map, a);
  return cudaGetLastError();
}

}  // namespace dsa
