// paged_attn.cu -- attention of new tokens over their selected pools, keys and
// values read through a block table.
//
// Row r (position i of its sequence) attends to the four keys of each selected
// pool and to its own partial pool {4*floor(i/4), ..., i}; its 16 query heads
// share one KV head:
//   o = sum_j exp(s q.k_j - lse) v_j,  lse = log sum_j exp(s q.k_j)
// in fp32, over bf16 products; P is rounded to bf16 for its product with V
// (at most 2^-8 of each weight, either way over the keys; the normaliser sums
// the unrounded weights), and o once more at the end.
//
// Layout of the work: a cluster of C CTAs (1 to 8) of four warps per row.  CTA
// c takes the row's 64-key blocks c, c + C, ...; each warp gathers the K and V
// rows of its own 16 keys of a block with 16-byte cp.async copies into its quarter of a ring of kStages blocks (rows XOR-swizzled in 16-B
// chunks so that ldmatrix reads are conflict-free) and waits only for its own
// copies.  S = Q K^T and O += P V run on mma.sync m16n8k16 (M = the 16 heads).
// The warps' partial softmax states (m, l, O) are merged through shared
// memory, the CTAs' through distributed shared memory, always in the same
// order: no atomics, no workspace, one launch, the same bits on every run.
//
// Measured with 512 pools a row (launches in a graph; keys and values from HBM,
// by selections in turn that L2 cannot hold together, as one layer of many finds
// them; in brackets the same selection again, which L2 holds):
//   1 row          7.2 us, latency: three dependent reads (selection, page,
//                  key), the copies of five blocks at once, the merge.
//   64 rows        18.0 us (12.3): 67 MB at 3.7 TB/s, 0.55 of the copy peak.  The
//                  copies begin when the row's table of keys is complete, and
//                  two stages of a ring keep too few of them under way.
//   256 rows       49 us: 269 MB at 5.5 TB/s.
//   4096 rows      284 us (a chunk: its rows share keys, which come from L2):
//                  15.2 TB/s of keys and values, 0.75 of the 1 KB-gather rate,
//                  and half of the issue slots: the chains of 12 warps an SM
//                  (168 registers) bound it.  Fewer instructions (precomputed
//                  addresses, no predicates: 283 us) changed nothing; S a block
//                  ahead of the softmax took 334 us, for the copies then have
//                  less time.
#include "paged.cuh"

namespace dsa {
namespace {

constexpr int kHq = 16;
constexpr int kD = 128;
constexpr int kWarps = 4;
constexpr int kThreads = 32 * kWarps;
constexpr int kBlkPools = 16;
constexpr int kBlkKeys = 4 * kBlkPools;                // 64
constexpr int kWarpKeys = kBlkKeys / kWarps;           // 16 keys of each block per warp
constexpr uint32_t kWarpTile = kWarpKeys * kD * 2;     // 4 KB: K (or V) rows of a warp's keys
constexpr uint32_t kWarpStage = 2 * kWarpTile;         // K then V
constexpr uint32_t kStageBytes = kWarps * kWarpStage;  // 32 KB: one block
constexpr int kMaxSplit = 8;                           // CTAs of a row's cluster
constexpr int kRedLd = kD + 4;                         // padded rows of the merge slabs
constexpr uint32_t kSlabBytes = kHq * kRedLd * 4;      // one warp's partial O
constexpr float kLog2e = 1.4426950408889634f;
constexpr float kLn2 = 0.6931471805599453f;
// A row's softmax reference moves up only when a score exceeds it by more
// than this (log2 units): P stays below 2^8, and the accumulators are
// rescaled only then, not whenever the maximum rises a little.
constexpr float kLag = 8.f;

// Position in a block's row table of key kr (0..63): warp w's keys 16w..16w+15
// fill slots 16w..16w+15, its even keys first, so that the lane that gathers keys
// p, p + 2, ..., p + 14 of the warp reads their rows with two 16-byte loads.
__device__ __forceinline__ int row_slot(int kr) { return (kr & ~15) + (kr & 1) * 8 + ((kr & 15) >> 1); }

// byte offset of 16-B chunk ch (0..15) of row r in a swizzled [rows][256 B] tile
__device__ __forceinline__ uint32_t swz(int r, int ch) {
  return static_cast<uint32_t>(r * 256 + ((ch ^ (r & 7)) << 4));
}

// Gathers the K and V rows of warp w's 16 keys of a block into `st`.  `rows`
// holds the block's 64 rows as page * page_size + offset (-1: nothing there,
// zero-filled and masked).  kFlat: pages follow one another without a gap in
// both buffers, so the row number is the address.
template <bool kFlat>
__device__ __forceinline__ void gather_warp(uint32_t st, const CacheView& c, const int32_t* rows, int w, int lane) {
  const int p = lane >> 4, ch = lane & 15;
  const int4 ra = *reinterpret_cast<const int4*>(rows + w * kWarpKeys + p * 8);
  const int4 rb = *reinterpret_cast<const int4*>(rows + w * kWarpKeys + p * 8 + 4);
  const int32_t r8[8] = {ra.x, ra.y, ra.z, ra.w, rb.x, rb.y, rb.z, rb.w};
  const int mask = (1 << c.shift) - 1;
#pragma unroll
  for (int u = 0; u < 8; ++u) {
    const int kl = p + 2 * u;
    const bool ok = r8[u] >= 0;
    const int r = ok ? r8[u] : 0;
    if (kFlat) {
      const int64_t src = static_cast<int64_t>(r) * kD + ch * 8;
      cp_async16(st + swz(kl, ch), c.k + src, ok);
      cp_async16(st + kWarpTile + swz(kl, ch), c.v + src, ok);
    } else {
      const int64_t page = r >> c.shift;
      const int off = (r & mask) * kD + ch * 8;
      cp_async16(st + swz(kl, ch), c.k + page * c.k_stride + off, ok);
      cp_async16(st + kWarpTile + swz(kl, ch), c.v + page * c.v_stride + off, ok);
    }
  }
}

template <int kStages, bool kSplit, bool kFlat>
__global__ void __launch_bounds__(kThreads, kStages == 2 ? 3 : 1)
    paged_attn_kernel(const CacheView c, const BatchView b, const __nv_bfloat16* __restrict__ q,
                      const int32_t* __restrict__ pool_idx, int topk, float scale_log2, __nv_bfloat16* __restrict__ o,
                      float* __restrict__ lse, int split, unsigned* status) {
  extern __shared__ uint8_t smem_raw[];
  const uint32_t raw = smem_u32(smem_raw);
  const uint32_t base = (raw + 127u) & ~127u;
  uint8_t* gbase = smem_raw + (base - raw);
  const uint32_t sKV = base;
  // Q is read into registers before the last stage of the ring is first filled
  const uint32_t sQ = base + (kStages - 1) * kStageBytes;
  int32_t* rows = reinterpret_cast<int32_t*>(gbase + kStages * kStageBytes);
  __shared__ int s_nsel;
  __shared__ float s_m[kWarps][kHq], s_l[kWarps][kHq];
  __shared__ float s_cm[kHq], s_cl[kHq];  // this CTA's merged reference and normaliser

  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
  const int g = lane >> 2, t4 = lane & 3;
  const int kC = kSplit ? split : 1;  // CTAs of the row's cluster
  const int rank = kSplit ? static_cast<int>(cluster_rank()) : 0;
  const int64_t r = kSplit ? blockIdx.x / static_cast<unsigned>(split) : blockIdx.x;

  pdl_wait();  // launched early: what stands before in the stream has ended
  // ---- everything that depends on the row's number alone is asked for at
  // once: Q (swizzled), the selection, the offsets and lengths
  {
    const __nv_bfloat16* qrow = q + r * (kHq * kD);
#pragma unroll
    for (int u = 0; u < (kHq * 16) / kThreads; ++u) {
      const int ch = tid + u * kThreads;
      cp_async16(sQ + swz(ch >> 4, ch & 15), qrow + ch * 8, true);
    }
    cp_async_commit();
  }
  const int32_t* prow = pool_idx + r * topk;
  constexpr int kAhead = 4;
  int sel[kAhead];
#pragma unroll
  for (int u = 0; u < kAhead; ++u) sel[u] = tid + u * kThreads < topk ? __ldg(prow + tid + u * kThreads) : 0;
  if (tid == 0) s_nsel = topk;
  // the row's sequence and position, every warp for itself
  const RowAt at = warp_locate(b, c.shift, r, lane, warp == 0 ? status : nullptr);
  if (at.seq < 0 || at.pos < 0) {  // padding behind the last sequence, or a row without a position:
    cp_async_wait<0>();            // every CTA of the cluster leaves here
    return;
  }
  const int64_t i = at.pos;
  const int64_t n_elig = i >> 2;
  // selected pools: the leading non-negative entries
  int first = topk;
#pragma unroll
  for (int u = kAhead - 1; u >= 0; --u)
    if (sel[u] < 0) first = tid + u * kThreads;
  for (int j = tid + kAhead * kThreads; j < topk; j += kThreads)
    if (__ldg(prow + j) < 0) first = min(first, j);
  __syncthreads();
  first = __reduce_min_sync(0xffffffffu, first);
  if (lane == 0 && first < topk) atomicMin(&s_nsel, first);
  __syncthreads();
  const int nsel = s_nsel;
  const int nblk_all = (nsel + 1 + kBlkPools - 1) / kBlkPools;
  const int nblk = nblk_all > rank ? (nblk_all - rank + kC - 1) / kC : 0;

  // Row table of this CTA's blocks, a pool a thread.  Slot s < nsel holds pool
  // prow[s]; slot nsel is the row's own pool; slots beyond are empty.  An entry
  // that is no eligible pool or breaks ascending order, and a page that is
  // none, are recorded; nothing is read for them.
  bool bad = false;
  const int pshift = c.shift - 2;  // log2(pools per page)
  for (int e = tid; e < nblk * kBlkPools; e += kThreads) {
    const int lb = e / kBlkPools, in = e % kBlkPools;
    const int slot = (rank + lb * kC) * kBlkPools + in;
    int64_t pool = -1;
    int have = 4;  // tokens of the pool
    if (slot < nsel) {
      const int p = __ldg(prow + slot);
      if (p < n_elig) pool = p;
      else bad = true;
      if (slot > 0 && p <= __ldg(prow + slot - 1)) bad = true;
    } else if (slot == nsel) {
      pool = n_elig;
      have = static_cast<int>(i & 3) + 1;
    }
    int32_t row = -1;
    if (pool >= 0) {
      const int page = __ldg(b.table + at.seq * b.table_stride + (pool >> pshift));
      if (static_cast<unsigned>(page) < static_cast<unsigned>(c.num_pages))
        row = (page << c.shift) + static_cast<int>((pool & ((1 << pshift) - 1)) << 2);
      else bad = true;
    }
    // keys 0 and 2 of the pool lie side by side, and so do keys 1 and 3
    int32_t* to = rows + lb * kBlkKeys + row_slot(4 * in);
    *reinterpret_cast<int2*>(to) = make_int2(row, row >= 0 && have > 2 ? row + 2 : -1);
    *reinterpret_cast<int2*>(to + 8) =
        make_int2(row >= 0 && have > 1 ? row + 1 : -1, row >= 0 && have > 3 ? row + 3 : -1);
  }
  if (bad) record_status(status, kStatusInternal);

  // ---- the gather pipeline's prologue
  // the row table is visible; without holes only the row's last block (its
  // own pool and the empty slots after it) needs a mask
  const bool any_hole = __syncthreads_or(bad) != 0;
#pragma unroll
  for (int s = 0; s < kStages - 1; ++s) {
    if (s < nblk) gather_warp<kFlat>(sKV + s * kStageBytes + warp * kWarpStage, c, rows + s * kBlkKeys, warp, lane);
    cp_async_commit();
  }

  float o_acc[16][4];
#pragma unroll
  for (int j = 0; j < 16; ++j) o_acc[j][0] = o_acc[j][1] = o_acc[j][2] = o_acc[j][3] = 0.f;
  float m_run[2] = {-INFINITY, -INFINITY}, l_run[2] = {0.f, 0.f};
  uint32_t qa[8][4];
  cp_async_wait<kStages - 1>();  // this thread's part of Q
  __syncthreads();
#pragma unroll
  for (int kk = 0; kk < 8; ++kk) {
    const int mat = lane >> 3;
    ldsm_x4(sQ + swz((lane & 7) + ((mat & 1) << 3), 2 * kk + (mat >> 1)), qa[kk][0], qa[kk][1], qa[kk][2], qa[kk][3]);
  }
  __syncthreads();  // every warp has Q: the last stage may be filled

  int stage = 0;
  for (int lb = 0; lb < nblk; ++lb) {
    cp_async_wait<kStages - 2>();  // this lane's copies of block lb
    __syncwarp();                  // ... and the other lanes'; block lb - 1 has been read
    {
      const int ahead = lb + kStages - 1;
      const int st = stage == 0 ? kStages - 1 : stage - 1;
      if (ahead < nblk) gather_warp<kFlat>(sKV + st * kStageBytes + warp * kWarpStage, c, rows + ahead * kBlkKeys, warp, lane);
      cp_async_commit();
    }
    const uint32_t sK = sKV + stage * kStageBytes + warp * kWarpStage;
    const uint32_t sV = sK + kWarpTile;
    if (++stage == kStages) stage = 0;

    // S = Q K^T for this warp's 16 keys (two n-tiles of 8)
    float s0[4] = {0.f, 0.f, 0.f, 0.f}, s1[4] = {0.f, 0.f, 0.f, 0.f};
#pragma unroll
    for (int kk = 0; kk < 8; ++kk) {
      const int mat = lane >> 3;
      uint32_t b0, b1, b2, b3;
      ldsm_x4(sK + swz(((mat >> 1) << 3) + (lane & 7), 2 * kk + (mat & 1)), b0, b1, b2, b3);
      mma_bf16_16816(s0, qa[kk], b0, b1);
      mma_bf16_16816(s1, qa[kk], b2, b3);
    }
    float x[8] = {s0[0], s0[1], s0[2], s0[3], s1[0], s1[1], s1[2], s1[3]};
    if (rank + lb * kC + 1 == nblk_all || any_hole) {
      const int key0 = warp * kWarpKeys + 2 * t4;
      const int kc[4] = {key0, key0 + 1, key0 + 8, key0 + 9};
      bool valid[4];
#pragma unroll
      for (int e = 0; e < 4; ++e) valid[e] = rows[lb * kBlkKeys + row_slot(kc[e])] >= 0;
      const bool vm[8] = {valid[0], valid[1], valid[0], valid[1], valid[2], valid[3], valid[2], valid[3]};
#pragma unroll
      for (int e = 0; e < 8; ++e) x[e] = vm[e] ? x[e] : -INFINITY;
    }
    // online softmax: head g holds x[0,1,4,5]; head g+8 holds x[2,3,6,7] (the
    // scale is positive: maxima of the raw scores)
    float mx0 = fmaxf(fmaxf(x[0], x[1]), fmaxf(x[4], x[5]));
    float mx1 = fmaxf(fmaxf(x[2], x[3]), fmaxf(x[6], x[7]));
#pragma unroll
    for (int off = 1; off <= 2; off <<= 1) {
      mx0 = fmaxf(mx0, __shfl_xor_sync(0xffffffffu, mx0, off));
      mx1 = fmaxf(mx1, __shfl_xor_sync(0xffffffffu, mx1, off));
    }
    mx0 *= scale_log2;
    mx1 *= scale_log2;
    const float mn0 = mx0 > m_run[0] + kLag ? mx0 : m_run[0];
    const float mn1 = mx1 > m_run[1] + kLag ? mx1 : m_run[1];
    const float mu0 = mn0 == -INFINITY ? 0.f : mn0, mu1 = mn1 == -INFINITY ? 0.f : mn1;
    const float al0 = ex2_ftz(m_run[0] - mu0), al1 = ex2_ftz(m_run[1] - mu1);
    float p[8];
    p[0] = ex2_ftz(fmaf(x[0], scale_log2, -mu0));
    p[1] = ex2_ftz(fmaf(x[1], scale_log2, -mu0));
    p[4] = ex2_ftz(fmaf(x[4], scale_log2, -mu0));
    p[5] = ex2_ftz(fmaf(x[5], scale_log2, -mu0));
    p[2] = ex2_ftz(fmaf(x[2], scale_log2, -mu1));
    p[3] = ex2_ftz(fmaf(x[3], scale_log2, -mu1));
    p[6] = ex2_ftz(fmaf(x[6], scale_log2, -mu1));
    p[7] = ex2_ftz(fmaf(x[7], scale_log2, -mu1));
    l_run[0] = l_run[0] * al0 + (p[0] + p[1] + p[4] + p[5]);
    l_run[1] = l_run[1] * al1 + (p[2] + p[3] + p[6] + p[7]);
    m_run[0] = mn0;
    m_run[1] = mn1;
    if (__any_sync(0xffffffffu, al0 != 1.f || al1 != 1.f)) {
#pragma unroll
      for (int j = 0; j < 16; ++j) {
        o_acc[j][0] *= al0;
        o_acc[j][1] *= al0;
        o_acc[j][2] *= al1;
        o_acc[j][3] *= al1;
      }
    }
    uint32_t pa[4] = {pack_bf16(p[0], p[1]), pack_bf16(p[2], p[3]), pack_bf16(p[4], p[5]), pack_bf16(p[6], p[7])};
    // O += P V: V rows are the k dimension (ldmatrix .trans)
#pragma unroll
    for (int j = 0; j < 8; ++j) {
      const int mat = lane >> 3;
      uint32_t b0, b1, b2, b3;
      ldsm_x4_t(sV + swz(((mat & 1) << 3) + (lane & 7), 2 * j + (mat >> 1)), b0, b1, b2, b3);
      mma_bf16_16816(o_acc[2 * j], pa, b0, b1);
      mma_bf16_16816(o_acc[2 * j + 1], pa, b2, b3);
    }
  }
  cp_async_wait<0>();

  // ---- merge the four warps' partial states into the CTA's (unnormalised,
  // at the CTA's reference M)
#pragma unroll
  for (int off = 1; off <= 2; off <<= 1) {
    l_run[0] += __shfl_xor_sync(0xffffffffu, l_run[0], off);
    l_run[1] += __shfl_xor_sync(0xffffffffu, l_run[1], off);
  }
  if (t4 == 0) {
    s_m[warp][g] = m_run[0];
    s_m[warp][g + 8] = m_run[1];
    s_l[warp][g] = l_run[0];
    s_l[warp][g + 8] = l_run[1];
  }
  __syncthreads();
  float fac[2];
#pragma unroll
  for (int hh = 0; hh < 2; ++hh) {
    const int h = g + 8 * hh;
    float M = s_m[0][h];
#pragma unroll
    for (int w = 1; w < kWarps; ++w) M = fmaxf(M, s_m[w][h]);
    const float Mu = M == -INFINITY ? 0.f : M;  // a CTA without blocks (C > 1 only)
    float L = 0.f;
#pragma unroll
    for (int w = 0; w < kWarps; ++w) L += s_l[w][h] * exp2f(s_m[w][h] - Mu);
    fac[hh] = exp2f(m_run[hh] - Mu);
    if (!kSplit) fac[hh] /= L;
    if (warp == 0 && t4 == 0) {
      if (!kSplit) {
        lse[r * kHq + h] = (M + log2f(L)) * kLn2;
      } else {
        s_cm[h] = M;
        s_cl[h] = L;
      }
    }
  }
  float* red = reinterpret_cast<float*>(gbase);  // four [16][132] fp32 slabs over the ring
#pragma unroll
  for (int j = 0; j < 16; ++j) {
    const int col = 8 * j + 2 * t4;
    *reinterpret_cast<float2*>(red + (warp * kHq + g) * kRedLd + col) =
        make_float2(o_acc[j][0] * fac[0], o_acc[j][1] * fac[0]);
    *reinterpret_cast<float2*>(red + (warp * kHq + g + 8) * kRedLd + col) =
        make_float2(o_acc[j][2] * fac[1], o_acc[j][3] * fac[1]);
  }
  __syncthreads();
  __nv_bfloat16* orow = o + r * (kHq * kD);
  if (!kSplit) {
#pragma unroll
    for (int m = 0; m < 8; ++m) {
      const int e = 2 * (tid + kThreads * m);
      const int h = e / kD, col = e % kD;
      float a0 = 0.f, a1 = 0.f;
#pragma unroll
      for (int w = 0; w < kWarps; ++w) {
        const float2 y = *reinterpret_cast<const float2*>(red + (w * kHq + h) * kRedLd + col);
        a0 += y.x;
        a1 += y.y;
      }
      *reinterpret_cast<uint32_t*>(orow + e) = pack_bf16(a0, a1);
    }
  } else {
    // the CTA's O into slab 0, then every CTA of the cluster finishes its
    // share of the 2048 outputs from the C slabs
#pragma unroll
    for (int m = 0; m < 4; ++m) {
      const int e = 4 * (tid + kThreads * m);
      const int at = (e / kD) * kRedLd + e % kD;
      float4 y = *reinterpret_cast<const float4*>(red + at);
#pragma unroll
      for (int w = 1; w < kWarps; ++w) {
        const float4 z = *reinterpret_cast<const float4*>(red + w * kHq * kRedLd + at);
        y.x += z.x;
        y.y += z.y;
        y.z += z.z;
        y.w += z.w;
      }
      *reinterpret_cast<float4*>(red + at) = y;
    }
    cluster_sync();
    for (int u4 = rank * kThreads + tid; u4 < kHq * kD / 4; u4 += kC * kThreads) {
      const int e = 4 * u4, h = e / kD, col = e % kD;
      float cm[kMaxSplit], cl[kMaxSplit];
      float4 y[kMaxSplit];
#pragma unroll
      for (int u = 0; u < kMaxSplit; ++u) {
        cm[u] = -INFINITY;
        cl[u] = 0.f;
        y[u] = make_float4(0.f, 0.f, 0.f, 0.f);
        if (u < kC) {
          cm[u] = cluster_ld_f32(cluster_map(smem_u32(&s_cm[h]), u));
          cl[u] = cluster_ld_f32(cluster_map(smem_u32(&s_cl[h]), u));
          y[u] = cluster_ld_f32x4(cluster_map(smem_u32(red + h * kRedLd + col), u));
        }
      }
      float M = cm[0];
#pragma unroll
      for (int u = 1; u < kMaxSplit; ++u) M = fmaxf(M, cm[u]);
      float L = 0.f;
      float4 acc = make_float4(0.f, 0.f, 0.f, 0.f);
#pragma unroll
      for (int u = 0; u < kMaxSplit; ++u) {
        const float f = exp2f(cm[u] - M);  // every row has a key of its own: M is finite
        L += cl[u] * f;
        acc.x += y[u].x * f;
        acc.y += y[u].y * f;
        acc.z += y[u].z * f;
        acc.w += y[u].w * f;
      }
      const float inv = 1.f / L;
      *reinterpret_cast<uint2*>(orow + e) =
          make_uint2(pack_bf16(acc.x * inv, acc.y * inv), pack_bf16(acc.z * inv, acc.w * inv));
      if (col == 0) lse[r * kHq + h] = (M + log2f(L)) * kLn2;
    }
    cluster_sync();  // no CTA leaves while another reads its shared memory
  }
}

template <int kStages>
size_t smem_bytes(int blocks, int split) {
  return 128 + static_cast<size_t>(kStages) * kStageBytes +
         static_cast<size_t>((blocks + split - 1) / split) * kBlkKeys * sizeof(int32_t);
}
constexpr int row_blocks(int topk) { return (topk + 1 + kBlkPools - 1) / kBlkPools; }
constexpr int kBlocksOf[2] = {row_blocks(512), row_blocks(2048)};  // the longest rows of two classes

template <int kStages, bool kSplit, bool kFlat>
cudaError_t allow_smem() {
  // (a split of one never has the long ring)
  constexpr size_t kMost = 128 + static_cast<size_t>(kStages) * kStageBytes +
                           static_cast<size_t>(kStages == 2 ? kBlocksOf[1] : (kBlocksOf[1] + 1) / 2) * kBlkKeys *
                               sizeof(int32_t);
  static_assert(kMost <= 232448 - 1024, "shared memory per CTA");
  static_assert(kWarps * kSlabBytes <= kStages * kStageBytes, "the merge slabs fit in the ring");
  static std::atomic<bool> attr_done[kAttrDevices];
  return set_smem_limit_once(paged_attn_kernel<kStages, kSplit, kFlat>, static_cast<int>(kMost), attr_done);
}

// A launch of clusters of `split` CTAs; attr has room for two.
cudaLaunchConfig_t split_config(cudaLaunchAttribute* attr, int64_t rows, int split, size_t smem, cudaStream_t stream) {
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3(static_cast<unsigned>(rows * split));
  cfg.blockDim = dim3(kThreads);
  cfg.dynamicSmemBytes = smem;
  cfg.stream = stream;
  attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[0].val.programmaticStreamSerializationAllowed = 1;
  attr[1].id = cudaLaunchAttributeClusterDimension;
  attr[1].val.clusterDim.x = static_cast<unsigned>(split);
  attr[1].val.clusterDim.y = 1;
  attr[1].val.clusterDim.z = 1;
  cfg.attrs = attr;
  cfg.numAttrs = split > 1 ? 2 : 1;
  return cfg;
}

// How many rows' clusters of `split` CTAs the device holds at once, at the
// longest rows of the class; asked for once per device, class and split.
template <int kStages, bool kFlat>
cudaError_t rows_at_once(int dev, int cls, int split, int* rows) {
  static std::atomic<int> known[kAttrDevices][2][kMaxSplit + 1];  // plus one; 0: not asked for yet
  const bool cached = dev >= 0 && dev < kAttrDevices;
  const int k = cached ? known[dev][cls][split].load(std::memory_order_relaxed) : 0;
  if (k > 0) {
    *rows = k - 1;
    return cudaSuccess;
  }
  cudaError_t e = allow_smem<kStages, true, kFlat>();
  if (e != cudaSuccess) return e;
  cudaLaunchAttribute attr[2];
  cudaLaunchConfig_t cfg = split_config(attr, 1, split, smem_bytes<kStages>(kBlocksOf[cls], split), nullptr);
  e = cudaOccupancyMaxActiveClusters(rows, paged_attn_kernel<kStages, true, kFlat>, &cfg);
  if (e == cudaSuccess && cached) known[dev][cls][split].store(*rows + 1, std::memory_order_relaxed);
  return e;
}

template <int kStages, bool kSplit, bool kFlat>
cudaError_t launch_variant(const CacheView& c, const BatchView& b, const void* q, const int32_t* pool_idx, int topk,
                           float scale, void* o, float* lse, int split, const LaunchCtx& ctx) {
  const cudaError_t e = allow_smem<kStages, kSplit, kFlat>();
  if (e != cudaSuccess) return e;
  cudaLaunchAttribute attr[2];
  const cudaLaunchConfig_t cfg = split_config(attr, b.rows, split, smem_bytes<kStages>(row_blocks(topk), split), ctx.stream);
  return cudaLaunchKernelEx(&cfg, paged_attn_kernel<kStages, kSplit, kFlat>, c, b,
                            static_cast<const __nv_bfloat16*>(q), pool_idx, topk, scale * kLog2e,
                            static_cast<__nv_bfloat16*>(o), lse, split, ctx.status);
}

// The CTAs of a row: as many as let all rows run at once.  A cluster lies
// within a part of the chip, so this is less than the CTAs that fit (16 rows of
// 8 CTAs with the long ring take two turns, 15.0 us; of 6, 9.6), and the
// runtime is asked.  With 5 CTAs or more a row the long ring, one CTA an SM, is
// taken if it fits: it has all of a CTA's blocks under way at once (25 rows of 5:
// 11.0 us, of 8 with two stages 11.5; 30 rows of 4 13.0 against 11.7).  Rows of up
// to 6 blocks are not split: 5 blocks of 64 rows take 7.8 us with one CTA, 8.4 with
// two, 8.5 with five; of 8 rows 6.9, 7.3 and 6.1; of 100 rows 8.1, 9.4 and 13.6.
// Otherwise, at 512 pools: 64 rows 31.1 us with one CTA each, 21.7 / 19.0 / 18.0 /
// 17.7 / 17.5 with 2 to 6 and 24.0 with 8 (two turns); 100 rows 34.1 / 26.5 / 24.7 /
// 24.6 with 1 to 4 and 31.6 with 5; 128 rows 36.4 / 30.3 / 29.4 with 1 to 3 and 37.9
// with 4; 200 rows 42.7 / 40.2; 256 rows 49.3 / 61.3.  All with keys and values
// from HBM; those that L2 holds take 12.3 us for 64 rows of 4 and the same choices.
constexpr int kWhole = 6;
constexpr int kRing = 5;

template <bool kFlat>
cudaError_t launch_rows(const CacheView& c, const BatchView& b, const void* q, const int32_t* pool_idx, int topk,
                        float scale, void* o, float* lse, const LaunchCtx& ctx) {
  const int blocks = row_blocks(topk), cls = blocks <= kBlocksOf[0] ? 0 : 1;
  const int most = blocks <= kWhole ? 1 : blocks / 2 < kMaxSplit ? blocks / 2 : kMaxSplit;
  // (three CTAs an SM at the most, so no more rows than this have two each)
  if (most > 1 && b.rows <= 3 * static_cast<int64_t>(ctx.num_sms) / 2) {
    int fit = 0, dev = 0;
    const cudaError_t got = cudaGetDevice(&dev);
    if (got != cudaSuccess) return got;
    for (int split = most; split >= (most < kRing ? most : kRing); --split) {
      const cudaError_t e = rows_at_once<6, kFlat>(dev, cls, split, &fit);
      if (e != cudaSuccess) return e;
      if (b.rows <= fit) return launch_variant<6, true, kFlat>(c, b, q, pool_idx, topk, scale, o, lse, split, ctx);
    }
    for (int split = most; split > 1; --split) {
      const cudaError_t e = rows_at_once<2, kFlat>(dev, cls, split, &fit);
      if (e != cudaSuccess) return e;
      if (b.rows <= fit) return launch_variant<2, true, kFlat>(c, b, q, pool_idx, topk, scale, o, lse, split, ctx);
    }
  }
  return launch_variant<2, false, kFlat>(c, b, q, pool_idx, topk, scale, o, lse, 1, ctx);
}

}  // namespace

cudaError_t launch_paged_attn(const CacheView& c, const BatchView& b, const void* q, const int32_t* pool_idx, int topk,
                              float scale, void* o, float* lse, const LaunchCtx& ctx) {
  const int64_t page = static_cast<int64_t>(kD) << c.shift;
  if (c.k_stride == page && c.v_stride == page)
    return launch_rows<true>(c, b, q, pool_idx, topk, scale, o, lse, ctx);
  return launch_rows<false>(c, b, q, pool_idx, topk, scale, o, lse, ctx);
}

}  // namespace dsa
