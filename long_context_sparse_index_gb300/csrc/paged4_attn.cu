// paged4_attn.cu -- attention of new tokens over their selected pools, keys and
// values in 4 bits (kv4.cuh) read through a block table.
//
// Row r (position i of its sequence) attends to the four keys of each selected
// pool and to its own partial pool {4*floor(i/4), ..., i}; its 16 query heads
// share one KV head:
//   o = sum_j exp(s q.k_j - lse) v_j,  lse = log sum_j exp(s q.k_j)
// with the k_j and v_j that the codes stand for.
//
// The products run on mma.sync m16n8k16 in fp16 (M = the 16 heads) with fp32
// sums.  Codes times scales are exact in fp16.  A head's query is brought into
// fp16's range by a power of two of its own (its largest element between 2^13 and
// 2^14), which the factor of its logits takes back: elements down to 2^-27 of the
// largest keep all their bits, and smaller ones are off by 2^-38 of the largest.
// P is rounded to fp16 for its product with V (2^-12 of each weight; the
// normaliser sums the unrounded weights), and o once at the end.
//
// Layout of the work: a cluster of C CTAs (1 to 8) of four warps per row.  CTA c
// takes the row's blocks of 16 pools c, c + C, ...; each warp gathers the 576
// bytes of its own 4 pools of a block by 16-byte cp.async copies into its quarter
// of a ring of kStages blocks, and waits only for its own copies.  Nothing is
// unpacked in shared memory: a lane's codes of a fragment are neighbours (32
// dimensions of a key, 16 dimensions of two tokens' values), so it reads 16 bytes
// at a time and converts in registers.  The order of dimensions in a sum is free,
// so Q's fragments take the keys' order; tokens 0, 1 and 2, 3 of the upper two
// pools change places, which keeps the reads of V free of bank conflicts.  The
// warps' partial softmax states (m, l, O) are merged through shared memory, the
// CTAs' through distributed shared memory, always in the same order: no atomics,
// no workspace, one launch, the same bits on every run.
#include "kv4.cuh"
#include "paged.cuh"
#include "paged_rope_kernels.h"

namespace dsa {
namespace {

constexpr int kHq = 16;
constexpr int kD = 128;
constexpr int kWarps = 4;
constexpr int kThreads = 32 * kWarps;
constexpr int kBlkPools = 16;
constexpr int kWarpPools = kBlkPools / kWarps;             // 4 pools of each block per warp
constexpr uint32_t kWarpStage = kWarpPools * kPool4Bytes;  // 2304 B
constexpr uint32_t kStageBytes = kWarps * kWarpStage;      // 9 KB: one block
constexpr int kStages = 6;
constexpr int kMaxSplit = 8;  // CTAs of a row's cluster
// The merge slabs, a row of 16 per head: four runs of 32 columns, 36 floats apart,
// so that a quarter warp's 16-byte stores reach all banks.
constexpr int kRunLd = 36;
constexpr int kRedLd = 4 * kRunLd;
constexpr uint32_t kSlabBytes = kHq * kRedLd * 4;  // one warp's partial O
static_assert(kWarps * kSlabBytes <= kStages * kStageBytes, "the merge slabs fit in the ring");
constexpr float kLog2e = 1.4426950408889634f;
constexpr float kLn2 = 0.6931471805599453f;
constexpr float kUnit = 0.0625f;  // what code * scale is to be multiplied by
// A row's softmax reference moves up only when a score exceeds it by more than
// this (log2 units): P stays below 2^8, within fp16.
constexpr float kLag = 8.f;

__device__ __forceinline__ int slab_col(int col) { return (col >> 5) * kRunLd + (col & 31); }

__device__ __forceinline__ uint4 lds128(uint32_t a) {
  uint4 v;
  asm volatile("ld.shared.v4.b32 {%0,%1,%2,%3}, [%4];" : "=r"(v.x), "=r"(v.y), "=r"(v.z), "=r"(v.w) : "r"(a) : "memory");
  return v;
}
__device__ __forceinline__ uint32_t lds32(uint32_t a) {
  uint32_t v;
  asm volatile("ld.shared.b32 %0, [%1];" : "=r"(v) : "r"(a) : "memory");
  return v;
}
__device__ __forceinline__ uint32_t pack_f16(float lo, float hi) {
  uint32_t d;
  asm("cvt.rn.f16x2.f32 %0, %1, %2;" : "=r"(d) : "f"(hi), "f"(lo));
  return d;
}
// c += a (16x16 f16, row) * b (16x8 f16, col), fp32 accumulate
__device__ __forceinline__ void mma_f16_16816(float (&c)[4], const uint32_t (&a)[4], uint32_t b0, uint32_t b1) {
  asm volatile(
      "mma.sync.aligned.m16n8k16.row.col.f32.f16.f16.f32 {%0,%1,%2,%3}, {%4,%5,%6,%7}, {%8,%9}, {%0,%1,%2,%3};"
      : "+f"(c[0]), "+f"(c[1]), "+f"(c[2]), "+f"(c[3])
      : "r"(a[0]), "r"(a[1]), "r"(a[2]), "r"(a[3]), "r"(b0), "r"(b1));
}
// Scale bits in byte kB of w as two equal fp16 numbers.
template <int kB>
__device__ __forceinline__ uint32_t scale_twice(uint32_t w) {
  return __byte_perm(w, 0u, 0x4040 | kB | kB << 8) << 7;
}
// Codes of key words: the fragments of dimensions 4 kk .. 4 kk + 3.
template <int kHalf>
__device__ __forceinline__ void key_frag(uint32_t w, uint32_t s, uint32_t& b0, uint32_t& b1) {
  b0 = mul_f16x2(f16_of_codes<2 * kHalf>(w), s);
  b1 = mul_f16x2(f16_of_codes<2 * kHalf + 1>(w), s);
}

// Gathers the 4 pools of warp w into `st`.  `at`: the block's pools as byte
// offsets (-1: nothing there, zero-filled).  Eight lanes a pool.
__device__ __forceinline__ void gather_warp(uint32_t st, const uint8_t* kv, const int64_t* at, int w, int lane) {
  const int p = lane >> 3, c8 = lane & 7;
  const int64_t off = at[w * kWarpPools + p];
  const bool ok = off >= 0;
  const uint8_t* src = kv + (ok ? off : 0) + c8 * 16;
  const uint32_t dst = st + p * kPool4Bytes + c8 * 16;
#pragma unroll
  for (int u = 0; u < 4; ++u) cp_async16(dst + 128 * u, src + 128 * u, ok);
  if (c8 < 4) cp_async16(dst + 512, src + 512, ok);
}

// 32 dimensions of a head's query as fp16, times 2^shift; returns the factor that
// takes it back.
__device__ __forceinline__ float query_f16(const uint4 (&raw)[4], uint32_t (&q)[16]) {
  float top = 0.f;
#pragma unroll
  for (int e = 0; e < 16; ++e) {
    const uint32_t w = (&raw[e >> 2].x)[e & 3];
    top = fmaxf(top, fmaxf(fabsf(__uint_as_float(w << 16)), fabsf(__uint_as_float(w & 0xFFFF0000u))));
  }
#pragma unroll
  for (int off = 1; off <= 2; off <<= 1) top = fmaxf(top, __shfl_xor_sync(0xffffffffu, top, off));
  const int shift = min(140 - static_cast<int>(__float_as_uint(top) >> 23), 126);
  const float f = __uint_as_float(static_cast<uint32_t>(127 + shift) << 23);
#pragma unroll
  for (int e = 0; e < 16; ++e) {
    const uint32_t w = (&raw[e >> 2].x)[e & 3];
    q[e] = pack_f16(__uint_as_float(w << 16) * f, __uint_as_float(w & 0xFFFF0000u) * f);
  }
  return __uint_as_float(static_cast<uint32_t>(127 - shift) << 23);
}

template <bool kSplit>
__global__ void __launch_bounds__(kThreads, 3)
    paged4_attn_kernel(const CacheView c, const BatchView b, const __nv_bfloat16* __restrict__ q,
                       const int32_t* __restrict__ pool_idx, int topk, float scale_log2, __nv_bfloat16* __restrict__ o,
                       float* __restrict__ lse, int split, unsigned* status) {
  extern __shared__ uint8_t smem_raw[];
  const uint32_t raw = smem_u32(smem_raw);
  const uint32_t base = (raw + 127u) & ~127u;
  uint8_t* gbase = smem_raw + (base - raw);
  const uint32_t sKV = base;
  int64_t* pools = reinterpret_cast<int64_t*>(gbase + kStages * kStageBytes);
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
  // once: Q, the selection, the offsets and lengths
  uint4 q0[4], q1[4];
  {
    const uint4* src = reinterpret_cast<const uint4*>(q + r * (kHq * kD) + g * kD + 32 * t4);
#pragma unroll
    for (int e = 0; e < 4; ++e) {
      q0[e] = __ldg(src + e);
      q1[e] = __ldg(src + 8 * kD / 8 + e);
    }
  }
  const int32_t* prow = pool_idx + r * topk;
  constexpr int kAhead = 4;
  int sel[kAhead];
#pragma unroll
  for (int u = 0; u < kAhead; ++u) sel[u] = tid + u * kThreads < topk ? __ldg(prow + tid + u * kThreads) : 0;
  if (tid == 0) s_nsel = topk;
  // the row's sequence and position, every warp for itself
  const RowAt at = warp_locate(b, c.shift, r, lane, warp == 0 ? status : nullptr);
  // padding behind the last sequence, or a row without a position: every CTA of
  // the cluster leaves here
  if (at.seq < 0 || at.pos < 0) return;
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

  // The pools of this CTA's blocks as byte offsets, a pool a thread.  Slot s < nsel
  // holds pool prow[s]; slot nsel is the row's own pool; slots beyond are empty.
  // An entry that is no eligible pool or breaks ascending order, and a page that
  // is none, are recorded; nothing is read for them.
  bool bad = false;
  const int pshift = c.shift - 2;  // log2(pools per page)
  for (int e = tid; e < nblk * kBlkPools; e += kThreads) {
    const int slot = (rank + e / kBlkPools * kC) * kBlkPools + e % kBlkPools;
    int64_t pool = -1, off = -1;
    if (slot < nsel) {
      const int p = __ldg(prow + slot);
      if (p < n_elig) pool = p;
      else bad = true;
      if (slot > 0 && p <= __ldg(prow + slot - 1)) bad = true;
    } else if (slot == nsel) {
      pool = n_elig;
    }
    if (pool >= 0) {
      const int page = __ldg(b.table + at.seq * b.table_stride + (pool >> pshift));
      if (static_cast<unsigned>(page) < static_cast<unsigned>(c.num_pages))
        off = page * (2 * c.k_stride) + (pool & ((1 << pshift) - 1)) * kPool4Bytes;
      else bad = true;
    }
    pools[e] = off;
  }
  if (bad) record_status(status, kStatusInternal);

  // ---- the gather pipeline's prologue
  // the pools are visible; without holes only the row's last block (its own pool
  // and the empty slots after it) needs a mask
  const bool any_hole = __syncthreads_or(bad) != 0;
  const uint8_t* kv = reinterpret_cast<const uint8_t*>(c.k);
#pragma unroll
  for (int s = 0; s < kStages - 1; ++s) {
    if (s < nblk) gather_warp(sKV + s * kStageBytes + warp * kWarpStage, kv, pools + s * kBlkPools, warp, lane);
    cp_async_commit();
  }

  // Q's fragments in the keys' order: step kk takes, of each lane's 32 dimensions,
  // 4 kk .. 4 kk + 3
  uint32_t qa[8][4];
  float f0, f1;  // what a head's products are to be multiplied by (log2 units)
  {
    uint32_t x0[16], x1[16];
    f0 = fmaxf(scale_log2 * kUnit * query_f16(q0, x0), 1.17549435e-38f);
    f1 = fmaxf(scale_log2 * kUnit * query_f16(q1, x1), 1.17549435e-38f);
#pragma unroll
    for (int kk = 0; kk < 8; ++kk) {
      qa[kk][0] = x0[2 * kk];
      qa[kk][1] = x1[2 * kk];
      qa[kk][2] = x0[2 * kk + 1];
      qa[kk][3] = x1[2 * kk + 1];
    }
  }

  float o_acc[16][4];
#pragma unroll
  for (int j = 0; j < 16; ++j) o_acc[j][0] = o_acc[j][1] = o_acc[j][2] = o_acc[j][3] = 0.f;
  float m_run[2] = {-INFINITY, -INFINITY}, l_run[2] = {0.f, 0.f};

  // Where this lane reads.  Column g of the first n-tile is token (g & 1) + 2 (g >> 2)
  // of pool g >> 1, of the second the pool's other token of that parity; the
  // columns 2 t4, 2 t4 + 1 that this lane holds P of are pool t4's.
  const int up = g >> 2;  // the first n-tile has tokens 2 and 3 of this pool
  const uint32_t k_at = (g >> 1) * kPool4Bytes + (g & 1) * 64 + 16 * t4;
  const uint32_t ks_at = (g >> 1) * kPool4Bytes + kPool4KScale + 8 * t4 + 4 * (g & 1);
  const uint32_t v_at = t4 * kPool4Bytes + kPool4V + 32 * g;
  const uint32_t vs_at = t4 * kPool4Bytes + kPool4VScale + 4 * g;
  const uint32_t k_up = 128u * up, v_up = 16u * (t4 >> 1);
  const int k_rot = 16 * up, v_rot = 16 * (t4 >> 1);

  int stage = 0;
  for (int lb = 0; lb < nblk; ++lb) {
    cp_async_wait<kStages - 2>();  // this lane's copies of block lb
    __syncwarp();                  // ... and the other lanes'; block lb - 1 has been read
    {
      const int ahead = lb + kStages - 1;
      const int st = stage == 0 ? kStages - 1 : stage - 1;
      if (ahead < nblk) gather_warp(sKV + st * kStageBytes + warp * kWarpStage, kv, pools + ahead * kBlkPools, warp, lane);
      cp_async_commit();
    }
    const uint32_t sW = sKV + stage * kStageBytes + warp * kWarpStage;
    if (++stage == kStages) stage = 0;

    // S = Q K^T for this warp's 16 keys (two n-tiles of 8)
    float s0[4] = {0.f, 0.f, 0.f, 0.f}, s1[4] = {0.f, 0.f, 0.f, 0.f};
    {
      const uint4 ka = lds128(sW + k_at + k_up), kb = lds128(sW + k_at + (128u - k_up));
      uint32_t ks = lds32(sW + ks_at);
      ks = __funnelshift_r(ks, ks, k_rot);
      const uint32_t sa[2] = {scale_twice<0>(ks), scale_twice<1>(ks)};
      const uint32_t sb[2] = {scale_twice<2>(ks), scale_twice<3>(ks)};
#pragma unroll
      for (int h = 0; h < 4; ++h) {  // a word: steps 2 h and 2 h + 1
        const uint32_t wa = (&ka.x)[h], wb = (&kb.x)[h];
        uint32_t b0, b1;
        key_frag<0>(wa, sa[h >> 1], b0, b1);
        mma_f16_16816(s0, qa[2 * h], b0, b1);
        key_frag<0>(wb, sb[h >> 1], b0, b1);
        mma_f16_16816(s1, qa[2 * h], b0, b1);
        key_frag<1>(wa, sa[h >> 1], b0, b1);
        mma_f16_16816(s0, qa[2 * h + 1], b0, b1);
        key_frag<1>(wb, sb[h >> 1], b0, b1);
        mma_f16_16816(s1, qa[2 * h + 1], b0, b1);
      }
    }
    float x[8] = {s0[0], s0[1], s0[2], s0[3], s1[0], s1[1], s1[2], s1[3]};
    uint32_t vs = lds32(sW + vs_at);
    vs = __funnelshift_r(vs, vs, v_rot);  // scales of the first n-tile's two tokens, then the second's
    if (rank + lb * kC + 1 == nblk_all || any_hole) {
      const int in = warp * kWarpPools + t4;
      const int slot = (rank + lb * kC) * kBlkPools + in;
      const int have = pools[lb * kBlkPools + in] < 0 ? 0 : slot == nsel ? static_cast<int>(i & 3) + 1 : 4;
      const int ta = 2 * (t4 >> 1);
      const bool valid[4] = {ta < have, ta + 1 < have, 2 - ta < have, 3 - ta < have};
      const bool vm[8] = {valid[0], valid[1], valid[0], valid[1], valid[2], valid[3], valid[2], valid[3]};
#pragma unroll
      for (int e = 0; e < 8; ++e) x[e] = vm[e] ? x[e] : -INFINITY;
      // what a token that is not there holds may be a NaN: it stands for zeros
#pragma unroll
      for (int e = 0; e < 4; ++e)
        if (!valid[e]) vs &= ~(0xFFu << (8 * e));
    }
    // online softmax: head g holds x[0,1,4,5]; head g+8 holds x[2,3,6,7] (the
    // factors are positive: maxima of the raw scores)
    float mx0 = fmaxf(fmaxf(x[0], x[1]), fmaxf(x[4], x[5]));
    float mx1 = fmaxf(fmaxf(x[2], x[3]), fmaxf(x[6], x[7]));
#pragma unroll
    for (int off = 1; off <= 2; off <<= 1) {
      mx0 = fmaxf(mx0, __shfl_xor_sync(0xffffffffu, mx0, off));
      mx1 = fmaxf(mx1, __shfl_xor_sync(0xffffffffu, mx1, off));
    }
    mx0 *= f0;
    mx1 *= f1;
    const float mn0 = mx0 > m_run[0] + kLag ? mx0 : m_run[0];
    const float mn1 = mx1 > m_run[1] + kLag ? mx1 : m_run[1];
    const float mu0 = mn0 == -INFINITY ? 0.f : mn0, mu1 = mn1 == -INFINITY ? 0.f : mn1;
    const float al0 = ex2_ftz(m_run[0] - mu0), al1 = ex2_ftz(m_run[1] - mu1);
    float p[8];
    p[0] = ex2_ftz(fmaf(x[0], f0, -mu0));
    p[1] = ex2_ftz(fmaf(x[1], f0, -mu0));
    p[4] = ex2_ftz(fmaf(x[4], f0, -mu0));
    p[5] = ex2_ftz(fmaf(x[5], f0, -mu0));
    p[2] = ex2_ftz(fmaf(x[2], f1, -mu1));
    p[3] = ex2_ftz(fmaf(x[3], f1, -mu1));
    p[6] = ex2_ftz(fmaf(x[6], f1, -mu1));
    p[7] = ex2_ftz(fmaf(x[7], f1, -mu1));
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
    const uint32_t pa[4] = {pack_f16(p[0], p[1]), pack_f16(p[2], p[3]), pack_f16(p[4], p[5]), pack_f16(p[6], p[7])};
    // O += P V: n-tile j is dimension 16 g + j of the lane's group g, its two k
    // pairs the pool's tokens.  Two tokens' codes of a dimension become
    // neighbours, four dimensions at a time.
    {
      const uint4 va = lds128(sW + v_at + v_up), vb = lds128(sW + v_at + (16u - v_up));
      const uint32_t sa = __byte_perm(vs, 0u, 0x4140) << 7, sb = __byte_perm(vs, 0u, 0x4342) << 7;
#pragma unroll
      for (int w = 0; w < 2; ++w) {
        const uint32_t a0 = (&va.x)[w], a1 = (&va.x)[w + 2], c0 = (&vb.x)[w], c1 = (&vb.x)[w + 2];
        constexpr uint32_t kLow = 0x0F0F0F0Fu;
        const uint32_t ea = (a0 & kLow) | ((a1 << 4) & ~kLow), oa = ((a0 >> 4) & kLow) | (a1 & ~kLow);
        const uint32_t eb = (c0 & kLow) | ((c1 << 4) & ~kLow), ob = ((c0 >> 4) & kLow) | (c1 & ~kLow);
        mma_f16_16816(o_acc[8 * w + 0], pa, mul_f16x2(f16_of_codes<0>(ea), sa), mul_f16x2(f16_of_codes<0>(eb), sb));
        mma_f16_16816(o_acc[8 * w + 1], pa, mul_f16x2(f16_of_codes<0>(oa), sa), mul_f16x2(f16_of_codes<0>(ob), sb));
        mma_f16_16816(o_acc[8 * w + 2], pa, mul_f16x2(f16_of_codes<1>(ea), sa), mul_f16x2(f16_of_codes<1>(eb), sb));
        mma_f16_16816(o_acc[8 * w + 3], pa, mul_f16x2(f16_of_codes<1>(oa), sa), mul_f16x2(f16_of_codes<1>(ob), sb));
        mma_f16_16816(o_acc[8 * w + 4], pa, mul_f16x2(f16_of_codes<2>(ea), sa), mul_f16x2(f16_of_codes<2>(eb), sb));
        mma_f16_16816(o_acc[8 * w + 5], pa, mul_f16x2(f16_of_codes<2>(oa), sa), mul_f16x2(f16_of_codes<2>(ob), sb));
        mma_f16_16816(o_acc[8 * w + 6], pa, mul_f16x2(f16_of_codes<3>(ea), sa), mul_f16x2(f16_of_codes<3>(eb), sb));
        mma_f16_16816(o_acc[8 * w + 7], pa, mul_f16x2(f16_of_codes<3>(oa), sa), mul_f16x2(f16_of_codes<3>(ob), sb));
      }
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
    if (!kSplit) fac[hh] *= kUnit / L;
    if (warp == 0 && t4 == 0) {
      if (!kSplit) {
        lse[r * kHq + h] = (M + log2f(L)) * kLn2;
      } else {
        s_cm[h] = M;
        s_cl[h] = L;
      }
    }
  }
  float* red = reinterpret_cast<float*>(gbase);  // four slabs over the ring
#pragma unroll
  for (int hh = 0; hh < 2; ++hh)
#pragma unroll
    for (int x = 0; x < 8; ++x) {  // columns 32 t4 + 4 x .. : dimensions of groups 2 t4 and 2 t4 + 1
      const int j = 4 * (x & 3), e = 2 * hh + (x >> 2);
      *reinterpret_cast<float4*>(red + (warp * kHq + g + 8 * hh) * kRedLd + t4 * kRunLd + 4 * x) =
          make_float4(o_acc[j][e] * fac[hh], o_acc[j + 1][e] * fac[hh], o_acc[j + 2][e] * fac[hh],
                      o_acc[j + 3][e] * fac[hh]);
    }
  __syncthreads();
  __nv_bfloat16* orow = o + r * (kHq * kD);
  // the CTA's O, four columns a thread at a time
#pragma unroll
  for (int m = 0; m < 4; ++m) {
    const int e = 4 * (tid + kThreads * m);
    const int from = (e / kD) * kRedLd + slab_col(e % kD);
    float4 y = *reinterpret_cast<const float4*>(red + from);
#pragma unroll
    for (int w = 1; w < kWarps; ++w) {
      const float4 z = *reinterpret_cast<const float4*>(red + w * kHq * kRedLd + from);
      y.x += z.x;
      y.y += z.y;
      y.z += z.z;
      y.w += z.w;
    }
    if (kSplit) *reinterpret_cast<float4*>(red + from) = y;
    else *reinterpret_cast<uint2*>(orow + e) = make_uint2(pack_bf16(y.x, y.y), pack_bf16(y.z, y.w));
  }
  if (kSplit) {
    // then every CTA of the cluster finishes its share of the 2048 outputs from
    // the C slabs
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
          y[u] = cluster_ld_f32x4(cluster_map(smem_u32(red + h * kRedLd + slab_col(col)), u));
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
      const float inv = kUnit / L;
      *reinterpret_cast<uint2*>(orow + e) =
          make_uint2(pack_bf16(acc.x * inv, acc.y * inv), pack_bf16(acc.z * inv, acc.w * inv));
      if (col == 0) lse[r * kHq + h] = (M + log2f(L)) * kLn2;
    }
    cluster_sync();  // no CTA leaves while another reads its shared memory
  }
}

size_t smem_bytes(int blocks, int split) {
  return 128 + static_cast<size_t>(kStages) * kStageBytes +
         static_cast<size_t>((blocks + split - 1) / split) * kBlkPools * sizeof(int64_t);
}
constexpr int row_blocks(int topk) { return (topk + 1 + kBlkPools - 1) / kBlkPools; }
constexpr int kBlocksOf[2] = {row_blocks(512), row_blocks(2048)};  // the longest rows of two classes

template <bool kSplit>
cudaError_t allow_smem() {
  constexpr size_t kMost =
      128 + static_cast<size_t>(kStages) * kStageBytes + static_cast<size_t>(kBlocksOf[1]) * kBlkPools * sizeof(int64_t);
  static_assert(3 * (kMost + 1024 + 512) <= 228 * 1024, "three CTAs an SM");
  static std::atomic<bool> attr_done[kAttrDevices];
  return set_smem_limit_once(paged4_attn_kernel<kSplit>, static_cast<int>(kMost), attr_done);
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
cudaError_t rows_at_once(int dev, int cls, int split, int* rows) {
  static std::atomic<int> known[kAttrDevices][2][kMaxSplit + 1];  // plus one; 0: not asked for yet
  const bool cached = dev >= 0 && dev < kAttrDevices;
  const int k = cached ? known[dev][cls][split].load(std::memory_order_relaxed) : 0;
  if (k > 0) {
    *rows = k - 1;
    return cudaSuccess;
  }
  cudaError_t e = allow_smem<true>();
  if (e != cudaSuccess) return e;
  cudaLaunchAttribute attr[2];
  cudaLaunchConfig_t cfg = split_config(attr, 1, split, smem_bytes(kBlocksOf[cls], split), nullptr);
  e = cudaOccupancyMaxActiveClusters(rows, paged4_attn_kernel<true>, &cfg);
  if (e == cudaSuccess && cached) known[dev][cls][split].store(*rows + 1, std::memory_order_relaxed);
  return e;
}

template <bool kSplit>
cudaError_t launch_variant(const CacheView& c, const BatchView& b, const void* q, const int32_t* pool_idx, int topk,
                           float scale, void* o, float* lse, int split, const LaunchCtx& ctx) {
  const cudaError_t e = allow_smem<kSplit>();
  if (e != cudaSuccess) return e;
  cudaLaunchAttribute attr[2];
  const cudaLaunchConfig_t cfg = split_config(attr, b.rows, split, smem_bytes(row_blocks(topk), split), ctx.stream);
  return cudaLaunchKernelEx(&cfg, paged4_attn_kernel<kSplit>, c, b, static_cast<const __nv_bfloat16*>(q), pool_idx, topk,
                            scale * kLog2e, static_cast<__nv_bfloat16*>(o), lse, split, ctx.status);
}

// The CTAs of a row: as many as let all rows run at once.
constexpr int kWhole = 6;  // rows of up to so many blocks are not split

}  // namespace

cudaError_t launch_paged4_attn(const CacheView& c, const BatchView& b, const void* q, const int32_t* pool_idx, int topk,
                               float scale, void* o, float* lse, const LaunchCtx& ctx) {
  const int blocks = row_blocks(topk), cls = blocks <= kBlocksOf[0] ? 0 : 1;
  const int most = blocks <= kWhole ? 1 : blocks / 2 < kMaxSplit ? blocks / 2 : kMaxSplit;
  // (three CTAs an SM at the most, so no more rows than this have two each)
  if (most > 1 && b.rows <= 3 * static_cast<int64_t>(ctx.num_sms) / 2) {
    int fit = 0, dev = 0;
    const cudaError_t got = cudaGetDevice(&dev);
    if (got != cudaSuccess) return got;
    for (int split = most; split > 1; --split) {
      const cudaError_t e = rows_at_once(dev, cls, split, &fit);
      if (e != cudaSuccess) return e;
      if (b.rows <= fit) return launch_variant<true>(c, b, q, pool_idx, topk, scale, o, lse, split, ctx);
    }
  }
  return launch_variant<false>(c, b, q, pool_idx, topk, scale, o, lse, 1, ctx);
}

}  // namespace dsa
