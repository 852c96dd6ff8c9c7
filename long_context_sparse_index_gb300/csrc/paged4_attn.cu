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
// A head's reference is one of its raw products, and an exponent is a difference of
// raw products times the head's factor: the reference's own weight is 1 however
// large its logit (a product and the reference multiplied each for itself would
// differ by the rounding of either, 16 and more from logits of 2^28 up).
// P is rounded to fp16 for its product with V (2^-11 of each weight, or 2^-25 of the
// reference's where that is more; the normaliser sums the unrounded weights), and o
// once at the end.
//
// Layout of the work: a cluster of C CTAs (1 to 8) of four warps per row.  CTA c
// takes the row's blocks of 16 pools c, c + C, ..., and each warp its own slice of
// four pools of each; it gathers their 576 bytes each by 16-byte cp.async copies
// into its part of a ring of kStages blocks, waits only for its own copies, and
// takes two slices (32 keys) a step.  Nothing is unpacked in shared memory: a lane's
// codes of a fragment are neighbours (32 dimensions of a key, 16 dimensions of two
// tokens' values), so it reads 16 bytes at a time and converts in registers.  The
// order of dimensions in a sum is free, so Q's fragments take the keys' order;
// tokens 0, 1 and 2, 3 of the upper two pools change places, which keeps the reads
// of V free of bank conflicts.  A head's reference is looked at by a vote and moves
// only when a product is above it by 2^8, so most steps rescale nothing.  The warps'
// partial softmax states (m, l, O) are merged through shared memory; the CTAs hand
// theirs to the one that finishes a part of the row, so nothing is read from
// another CTA.  Always in the same order: no atomics, no workspace, one launch, the
// same bits on every run.
//
// Measured with 512 pools a row, launches in a graph, keys and values from HBM:
//   1 row       7.3 us, latency: selection, page, pool (three dependent reads,
//               0.8 us each), 16 keys a warp at about 0.45 us, the merge.
//   64 rows     14.1 us: 19 MB, 1.4 TB/s.
//   512 rows    47 us.
//   4096 rows   265 us: 259 TFLOP/s, and 4.6 TB/s of pools from L2 (262 us with an
//               exponent in one FMA of the product and the scaled reference).  A
//               slice of 16 keys takes 148 clocks of an SM, of which the 32 products
//               have the tensor pipe for 65; the conversions (64), the scales'
//               products (64) and the pairing of tokens (16) go to pipes that take
//               an instruction every two clocks, and the product's issue and theirs
//               overlap by half only (measured: products' clocks + half of the
//               others').
//               More warps an SM (12 or 16), more registers, one or two slices a
//               step or another order of the instructions moved it by 1 % at most.
#include <type_traits>

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
constexpr int kMaxSplit = 8;  // CTAs of a row's cluster
constexpr int kVecs = kHq * kD / 4;  // a row's output in vectors of four
// The merge slabs, a row of 16 per head: four runs of 32 columns, 36 floats apart,
// so that a quarter warp's 16-byte stores reach all banks.
constexpr int kRunLd = 36;
constexpr int kRedLd = 4 * kRunLd;
constexpr uint32_t kSlabBytes = kHq * kRedLd * 4;  // one warp's partial O
static_assert(kWarps * kSlabBytes <= 4 * kStageBytes, "the merge slabs fit in the shorter ring");
constexpr float kLog2e = 1.4426950408889634f;
constexpr float kLn2 = 0.6931471805599453f;
constexpr float kUnit = 0.0625f;  // what code * scale is to be multiplied by
// A row's softmax reference moves up only when a score exceeds it by more than
// this (log2 units): P stays at 2^8 or below, within fp16.
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
__device__ __forceinline__ void cluster_arrive() {
  asm volatile("barrier.cluster.arrive.release.aligned;" ::: "memory");
}
__device__ __forceinline__ void cluster_wait() { asm volatile("barrier.cluster.wait.acquire.aligned;" ::: "memory"); }
__device__ __forceinline__ void cluster_st_f32(uint32_t a, float v) {
  asm volatile("st.shared::cluster.f32 [%0], %1;" ::"r"(a), "f"(v) : "memory");
}
__device__ __forceinline__ void cluster_st_f32x4(uint32_t a, const float4& v) {
  asm volatile("st.shared::cluster.v4.f32 [%0], {%1,%2,%3,%4};" ::"r"(a), "f"(v.x), "f"(v.y), "f"(v.z), "f"(v.w)
               : "memory");
}
__device__ __forceinline__ void cp_async16_all(uint32_t dst, const void* src) {
  asm volatile("cp.async.cg.shared.global [%0], [%1], 16;" ::"r"(dst), "l"(src) : "memory");
}
// (x0 + c, x1 + c) * (f, f), and sums, two at a time
__device__ __forceinline__ float2 addmul2(float x0, float x1, float c, float f) {
  float2 y;
  asm("{\n .reg .b64 x, f, c, y;\n mov.b64 x, {%2, %3};\n mov.b64 f, {%4, %4};\n mov.b64 c, {%5, %5};\n"
      " add.rn.f32x2 y, x, c;\n mul.rn.f32x2 y, y, f;\n mov.b64 {%0, %1}, y;\n}"
      : "=f"(y.x), "=f"(y.y)
      : "f"(x0), "f"(x1), "f"(f), "f"(c));
  return y;
}
__device__ __forceinline__ float2 add2(float2 a, float2 b) {
  float2 y;
  asm("{\n .reg .b64 a, b, y;\n mov.b64 a, {%2, %3};\n mov.b64 b, {%4, %5};\n add.rn.f32x2 y, a, b;\n"
      " mov.b64 {%0, %1}, y;\n}"
      : "=f"(y.x), "=f"(y.y)
      : "f"(a.x), "f"(a.y), "f"(b.x), "f"(b.y));
  return y;
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
// c = a * b
__device__ __forceinline__ void mma_f16_16816_first(float (&c)[4], const uint32_t (&a)[4], uint32_t b0, uint32_t b1) {
  asm volatile(
      "mma.sync.aligned.m16n8k16.row.col.f32.f16.f16.f32 {%0,%1,%2,%3}, {%4,%5,%6,%7}, {%8,%9}, {%10,%10,%10,%10};"
      : "=f"(c[0]), "=f"(c[1]), "=f"(c[2]), "=f"(c[3])
      : "r"(a[0]), "r"(a[1]), "r"(a[2]), "r"(a[3]), "r"(b0), "r"(b1), "f"(0.f));
}
// Scale bits in byte kB of w as two equal fp16 numbers.
template <int kB>
__device__ __forceinline__ uint32_t scale_twice(uint32_t w) {
  return __byte_perm(w, 0u, 0x4440 | kB) * 0x00800080u;
}
// Codes of key words: the fragments of dimensions 4 kk .. 4 kk + 3.
template <int kHalf>
__device__ __forceinline__ void key_frag(uint32_t w, uint32_t s, uint32_t& b0, uint32_t& b1) {
  b0 = mul_f16x2(f16_of_codes<2 * kHalf>(w), s);
  b1 = mul_f16x2(f16_of_codes<2 * kHalf + 1>(w), s);
}

// Gathers the four pools of a slice into `st`.  `at`: the pools as byte offsets
// (-1: nothing there, zero-filled).  Eight lanes a pool.
__device__ __forceinline__ void gather_slice(uint32_t st, const uint8_t* kv, const int64_t* at, int lane, bool any_hole) {
  const int p = lane >> 3, c8 = lane & 7;
  const int64_t off = at[p];
  const uint8_t* src = kv + off + c8 * 16;
  const uint32_t dst = st + p * kPool4Bytes + c8 * 16;
  if (!any_hole) {
#pragma unroll
    for (int u = 0; u < 4; ++u) cp_async16_all(dst + 128 * u, src + 128 * u);
    if (c8 < 4) cp_async16_all(dst + 512, src + 512);
  } else {
    const bool ok = off >= 0;
    if (!ok) src = kv;
#pragma unroll
    for (int u = 0; u < 4; ++u) cp_async16(dst + 128 * u, src + 128 * u, ok);
    if (c8 < 4) cp_async16(dst + 512, src + 512, ok);
  }
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

template <int kStages, bool kSplit>
__global__ void __launch_bounds__(kThreads, kStages == 4 ? 4 : 3)
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
  // what the cluster's CTAs hand to this one: references, normalisers, partial O
  __shared__ float s_pm[kSplit ? kMaxSplit : 1][kHq], s_pl[kSplit ? kMaxSplit : 1][kHq];
  __shared__ float s_f[kHq];  // the heads' factors
  __shared__ float4 s_po[kSplit ? kVecs + kMaxSplit : 1];
  __shared__ uint4 s_q[8 * 32];           // Q's fragments, a step's for each lane

  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
  const int g = lane >> 2, t4 = lane & 3;
  const int kC = kSplit ? split : 1;  // CTAs of the row's cluster
  const int rank = kSplit ? static_cast<int>(cluster_rank()) : 0;
  const int64_t r = kSplit ? blockIdx.x / static_cast<unsigned>(split) : blockIdx.x;

  if (kSplit) cluster_arrive();  // (this CTA runs: the others may write to its shared memory)
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
  if (at.seq < 0 || at.pos < 0) {
    if (kSplit) cluster_wait();
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
  // This warp's slices (its 4 pools of a block each), in the CTA's blocks 0, 1, ...
  const int nsl = nsel / kWarpPools + 1, first_sl = rank * kWarps + warp;
  const int mine = nsl > first_sl ? (nsl - first_sl + kC * kWarps - 1) / (kC * kWarps) : 0;

  // The pools of this CTA's blocks as byte offsets, a pool a thread.  Slot s < nsel
  // holds pool prow[s]; slot nsel is the row's own pool; slots beyond are empty.
  // An entry that is no eligible pool, and a page that is none, are recorded, and
  // nothing is read for them; an entry that breaks ascending order is recorded, too,
  // and attended to as it stands.
  bool bad = false;
  const int pshift = c.shift - 2;  // log2(pools per page)
  const auto pool_of = [&](int e) -> int64_t {  // -1: none
    const int slot = (rank + e / kBlkPools * kC) * kBlkPools + e % kBlkPools;
    if (slot >= nsel) return slot == nsel ? n_elig : -1;
    const int p = __ldg(prow + slot);
    if (slot > 0 && p <= __ldg(prow + slot - 1)) bad = true;
    if (p < n_elig) return p;
    bad = true;
    return -1;
  };
  const auto page_at = [&](int64_t pool) { return pool < 0 ? 0 : __ldg(b.table + at.seq * b.table_stride + (pool >> pshift)); };
  const auto put = [&](int e, int64_t pool, int page) {
    const bool empty = (rank + e / kBlkPools * kC) * kBlkPools + e % kBlkPools > nsel;
    int64_t off = empty ? 0 : -1;  // (what an empty slot reads is masked)
    if (pool >= 0) {
      if (static_cast<unsigned>(page) < static_cast<unsigned>(c.num_pages))
        off = page * (2 * c.k_stride) + (pool & ((1 << pshift) - 1)) * kPool4Bytes;
      else bad = true;
    }
    pools[e] = off;
  };
  // Q's fragments in the keys' order: step kk takes, of each lane's 32 dimensions,
  // 4 kk .. 4 kk + 3.  All warps have the same ones; each stores two steps'.
  float f0 = 0.f, f1 = 0.f;  // what a head's products are to be multiplied by (log2 units)
  const uint32_t sQ = smem_u32(s_q) + 16 * lane;
  const auto ready_q = [&] {
    uint32_t x0[16], x1[16];
    f0 = fmaxf(scale_log2 * kUnit * query_f16(q0, x0), 1.17549435e-38f);
    f1 = fmaxf(scale_log2 * kUnit * query_f16(q1, x1), 1.17549435e-38f);
#pragma unroll
    for (int kk = 0; kk < 8; ++kk)
      if (kk >> 1 == warp) st_shared_v4(sQ + 512 * kk, x0[2 * kk], x1[2 * kk], x0[2 * kk + 1], x1[2 * kk + 1]);
  };
  const int entries = nblk * kBlkPools;
  int e0 = tid;
  if (kSplit) {  // few entries: Q is made ready while a thread's first page number comes
    const int64_t pool = tid < entries ? pool_of(tid) : -1;
    const int page = page_at(pool);
    ready_q();
    if (tid < entries) put(tid, pool, page);
    e0 += kThreads;
  }
#pragma unroll 4
  for (int e = e0; e < entries; e += kThreads) {
    const int64_t pool = pool_of(e);
    put(e, pool, page_at(pool));
  }
  if (bad) record_status(status, kStatusInternal);

  // ---- the gather pipeline's prologue
  // the pools are visible; without holes only the row's last block (its own
  // pool and the empty slots after it) needs a mask
  const bool any_hole = __syncthreads_or(bad) != 0;
  const uint8_t* kv = reinterpret_cast<const uint8_t*>(c.k);
  const int64_t* const my_pools = pools + warp * kWarpPools;
  const uint32_t ring = sKV + warp * kWarpStage;
  // (a split row has few slices, and all of them under way at once; a whole row
  // keeps the pace of its refills: 4096 rows 268 us with a full ring, 265 so)
  constexpr int kFirst = kSplit ? kStages : kStages - 2;
#pragma unroll
  for (int u = 0; u < kFirst; ++u) {
    if (u < mine) gather_slice(ring + u * kStageBytes, kv, my_pools + u * kBlkPools, lane, any_hole);
    cp_async_commit();
  }
  if (!kSplit) {  // many: while the first slices come
    ready_q();
    __syncthreads();
  }

  float o_acc[16][4];
#pragma unroll
  for (int j = 0; j < 16; ++j) o_acc[j][0] = o_acc[j][1] = o_acc[j][2] = o_acc[j][3] = 0.f;
  float2 l_run[2] = {make_float2(0.f, 0.f), make_float2(0.f, 0.f)};  // even and odd columns
  // A head's reference m, a raw product: minus it (0 before the first key), and the
  // product above which it moves up
  float minus_m[2] = {0.f, 0.f}, rise[2] = {-INFINITY, -INFINITY};

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

  // One step: slices l .. l + kN - 1 of this warp, at sW.
  const auto step = [&](auto count, int l, uint32_t sW) {
    constexpr int kN = decltype(count)::value;
    // S = Q K^T for 16 keys of each slice (two n-tiles of 8)
    float s[2 * kN][4];
    {
      uint4 kw[2 * kN];
      uint32_t sc[2 * kN][2];
#pragma unroll
      for (int u = 0; u < kN; ++u) {
        const uint32_t at = sW + u * kStageBytes;
        kw[2 * u] = lds128(at + k_at + k_up);
        kw[2 * u + 1] = lds128(at + k_at + (128u - k_up));
        uint32_t ks = lds32(at + ks_at);
        ks = __funnelshift_r(ks, ks, k_rot);
        sc[2 * u][0] = scale_twice<0>(ks);
        sc[2 * u][1] = scale_twice<1>(ks);
        sc[2 * u + 1][0] = scale_twice<2>(ks);
        sc[2 * u + 1][1] = scale_twice<3>(ks);
      }
#pragma unroll
      for (int h = 0; h < 4; ++h) {  // a word: steps 2 h and 2 h + 1
        const uint4 qv[2] = {lds128(sQ + 1024 * h), lds128(sQ + 1024 * h + 512)};
#pragma unroll
        for (int e = 0; e < 2; ++e) {
          const uint32_t qa[4] = {qv[e].x, qv[e].y, qv[e].z, qv[e].w};
          uint32_t b[2 * kN][2];
#pragma unroll
          for (int n = 0; n < 2 * kN; ++n) {
            if (e == 0) key_frag<0>((&kw[n].x)[h], sc[n][h >> 1], b[n][0], b[n][1]);
            else key_frag<1>((&kw[n].x)[h], sc[n][h >> 1], b[n][0], b[n][1]);
          }
#pragma unroll
          for (int n = 0; n < 2 * kN; ++n) {
            if (h + e == 0) mma_f16_16816_first(s[n], qa, b[n][0], b[n][1]);
            else mma_f16_16816(s[n], qa, b[n][0], b[n][1]);
          }
        }
      }
    }
    uint32_t vs[kN];  // scales of the first n-tile's two tokens, then the second's
#pragma unroll
    for (int u = 0; u < kN; ++u) {
      vs[u] = lds32(sW + u * kStageBytes + vs_at);
      vs[u] = __funnelshift_r(vs[u], vs[u], v_rot);
    }
    if (l + kN >= mine || any_hole) {  // the own pool, or a slice that is not there
#pragma unroll
      for (int u = 0; u < kN; ++u) {
        const int in = warp * kWarpPools + t4;
        const int slot = (rank + (l + u) * kC) * kBlkPools + in;
        const int have = slot > nsel || pools[(l + u) * kBlkPools + in] < 0 ? 0
                         : slot == nsel ? static_cast<int>(i & 3) + 1
                                        : 4;
        const int ta = 2 * (t4 >> 1);
        const bool valid[4] = {ta < have, ta + 1 < have, 2 - ta < have, 3 - ta < have};
#pragma unroll
        for (int e = 0; e < 4; ++e) {
          s[2 * u + (e >> 1)][e & 1] = valid[e] ? s[2 * u + (e >> 1)][e & 1] : -INFINITY;
          s[2 * u + (e >> 1)][2 + (e & 1)] = valid[e] ? s[2 * u + (e >> 1)][2 + (e & 1)] : -INFINITY;
          // what a token that is not there holds may be a NaN: it stands for zeros
          if (!valid[e]) vs[u] &= ~(0xFFu << (8 * e));
        }
      }
    }
    // online softmax: head g holds s[.][0], s[.][1], head g + 8 the others (the
    // factors are positive: maxima of the raw products)
    float mx[2];
#pragma unroll
    for (int hh = 0; hh < 2; ++hh) {
      mx[hh] = fmaxf(s[0][2 * hh], s[0][2 * hh + 1]);
#pragma unroll
      for (int n = 1; n < 2 * kN; ++n) mx[hh] = fmaxf(mx[hh], fmaxf(s[n][2 * hh], s[n][2 * hh + 1]));
    }
    if (__any_sync(0xffffffffu, mx[0] > rise[0] || mx[1] > rise[1])) {
      float al[2];
#pragma unroll
      for (int hh = 0; hh < 2; ++hh) {
        const float f = hh ? f1 : f0;
#pragma unroll
        for (int off = 1; off <= 2; off <<= 1) mx[hh] = fmaxf(mx[hh], __shfl_xor_sync(0xffffffffu, mx[hh], off));
        al[hh] = 1.f;
        if (mx[hh] > rise[hh]) {
          // (before the first key there is nothing to rescale)
          al[hh] = rise[hh] == -INFINITY ? 0.f : ex2_ftz((-minus_m[hh] - mx[hh]) * f);
          minus_m[hh] = -mx[hh];
          rise[hh] = __fadd_rd(mx[hh], kLag / f);  // (rounded up it could lie twice the lag above)
        }
        l_run[hh].x *= al[hh];
        l_run[hh].y *= al[hh];
      }
#pragma unroll
      for (int j = 0; j < 16; ++j) {
        o_acc[j][0] *= al[0];
        o_acc[j][1] *= al[0];
        o_acc[j][2] *= al[1];
        o_acc[j][3] *= al[1];
      }
    }
    uint32_t pa[kN][4];
#pragma unroll
    for (int n = 0; n < 2 * kN; ++n)
#pragma unroll
      for (int hh = 0; hh < 2; ++hh) {
        float2 p = addmul2(s[n][2 * hh], s[n][2 * hh + 1], minus_m[hh], hh ? f1 : f0);
        p.x = ex2_ftz(p.x);
        p.y = ex2_ftz(p.y);
        l_run[hh] = add2(l_run[hh], p);
        pa[n >> 1][2 * (n & 1) + hh] = pack_f16(p.x, p.y);
      }
    // O += P V: n-tile j is dimension 16 g + j of the lane's group g, its two k
    // pairs the pool's tokens.  Two tokens' codes of a dimension become
    // neighbours, four dimensions at a time.
#pragma unroll
    for (int u = 0; u < kN; ++u) {
      const uint32_t at = sW + u * kStageBytes;
      const uint4 va = lds128(at + v_at + v_up), vb = lds128(at + v_at + (16u - v_up));
      const uint32_t sa = __byte_perm(vs[u], 0u, 0x4140) << 7, sb = __byte_perm(vs[u], 0u, 0x4342) << 7;
#pragma unroll
      for (int w = 0; w < 2; ++w) {
        const uint32_t a0 = (&va.x)[w], a1 = (&va.x)[w + 2], c0 = (&vb.x)[w], c1 = (&vb.x)[w + 2];
        constexpr uint32_t kLow = 0x0F0F0F0Fu;
        const uint32_t ea = (a0 & kLow) | ((a1 << 4) & ~kLow), oa = ((a0 >> 4) & kLow) | (a1 & ~kLow);
        const uint32_t eb = (c0 & kLow) | ((c1 << 4) & ~kLow), ob = ((c0 >> 4) & kLow) | (c1 & ~kLow);
        mma_f16_16816(o_acc[8 * w + 0], pa[u], mul_f16x2(f16_of_codes<0>(ea), sa), mul_f16x2(f16_of_codes<0>(eb), sb));
        mma_f16_16816(o_acc[8 * w + 1], pa[u], mul_f16x2(f16_of_codes<0>(oa), sa), mul_f16x2(f16_of_codes<0>(ob), sb));
        mma_f16_16816(o_acc[8 * w + 2], pa[u], mul_f16x2(f16_of_codes<1>(ea), sa), mul_f16x2(f16_of_codes<1>(eb), sb));
        mma_f16_16816(o_acc[8 * w + 3], pa[u], mul_f16x2(f16_of_codes<1>(oa), sa), mul_f16x2(f16_of_codes<1>(ob), sb));
        mma_f16_16816(o_acc[8 * w + 4], pa[u], mul_f16x2(f16_of_codes<2>(ea), sa), mul_f16x2(f16_of_codes<2>(eb), sb));
        mma_f16_16816(o_acc[8 * w + 5], pa[u], mul_f16x2(f16_of_codes<2>(oa), sa), mul_f16x2(f16_of_codes<2>(ob), sb));
        mma_f16_16816(o_acc[8 * w + 6], pa[u], mul_f16x2(f16_of_codes<3>(ea), sa), mul_f16x2(f16_of_codes<3>(eb), sb));
        mma_f16_16816(o_acc[8 * w + 7], pa[u], mul_f16x2(f16_of_codes<3>(oa), sa), mul_f16x2(f16_of_codes<3>(ob), sb));
      }
    }
  };
  int stage = 0;
  for (int l = 0; l < mine; l += 2) {
    if (l == 0) cp_async_wait<kFirst - 2>();  // this lane's copies of slices l and l + 1
    else cp_async_wait<kStages - 4>();
    __syncwarp();  // ... and the other lanes'; slices l - 2 and l - 1 have been read
    if (!kSplit || l != 0) {
#pragma unroll
      for (int u = 0; u < 2; ++u) {
        const int ahead = l + u + kStages - 2;
        const int st = stage + u < 2 ? stage + u + kStages - 2 : stage + u - 2;
        if (ahead < mine) gather_slice(ring + st * kStageBytes, kv, my_pools + ahead * kBlkPools, lane, any_hole);
        cp_async_commit();
      }
    }
    const uint32_t sW = ring + stage * kStageBytes;
    stage = stage + 2 == kStages ? 0 : stage + 2;
    if (!kSplit || l + 1 < mine) step(std::integral_constant<int, 2>{}, l, sW);
    else step(std::integral_constant<int, 1>{}, l, sW);  // (a whole row masks its last odd slice)
  }
  cp_async_wait<0>();
  const float m_run[2] = {rise[0] == -INFINITY ? -INFINITY : -minus_m[0], rise[1] == -INFINITY ? -INFINITY : -minus_m[1]};

  // ---- merge the four warps' partial states into the CTA's (unnormalised, at
  // the CTA's reference M)
  if (kSplit) cluster_wait();  // every CTA of the cluster runs
  float l_sum[2] = {l_run[0].x + l_run[0].y, l_run[1].x + l_run[1].y};
#pragma unroll
  for (int off = 1; off <= 2; off <<= 1) {
    l_sum[0] += __shfl_xor_sync(0xffffffffu, l_sum[0], off);
    l_sum[1] += __shfl_xor_sync(0xffffffffu, l_sum[1], off);
  }
  if (t4 == 0) {
    s_m[warp][g] = m_run[0];
    s_m[warp][g + 8] = m_run[1];
    s_l[warp][g] = l_sum[0];
    s_l[warp][g + 8] = l_sum[1];
  }
  __syncthreads();
  float fac[2];
#pragma unroll
  for (int hh = 0; hh < 2; ++hh) {
    const int h = g + 8 * hh;
    const float f = hh ? f1 : f0;
    float M = s_m[0][h];
#pragma unroll
    for (int w = 1; w < kWarps; ++w) M = fmaxf(M, s_m[w][h]);
    const float Mu = M == -INFINITY ? 0.f : M;  // a CTA without blocks (C > 1 only)
    float L = 0.f;
#pragma unroll
    for (int w = 0; w < kWarps; ++w) L += s_l[w][h] * exp2f((s_m[w][h] - Mu) * f);
    fac[hh] = exp2f((m_run[hh] - Mu) * f);
    if (!kSplit) fac[hh] *= kUnit / L;
    if (!kSplit && warp == 0 && t4 == 0) lse[r * kHq + h] = __fmaf_rn(M, f, log2f(L)) * kLn2;
    if (kSplit && warp == 0 && t4 == 0) s_f[h] = f;
    if (kSplit && warp + kWarps * t4 < kC) {  // a lane tells a CTA
      cluster_st_f32(cluster_map(smem_u32(&s_pm[rank][h]), warp + kWarps * t4), M);
      cluster_st_f32(cluster_map(smem_u32(&s_pl[rank][h]), warp + kWarps * t4), L);
    }
  }
  float* red = reinterpret_cast<float*>(gbase);  // the warps' slabs over the ring
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
  // the CTA's O, four columns a thread at a time: written, or handed to the CTA of
  // the cluster that finishes this part of the row
  const int per = kSplit ? (kVecs + kC - 1) / kC : kVecs;
#pragma unroll
  for (int m = 0; m < kVecs / kThreads; ++m) {
    const int v = tid + kThreads * m, e = 4 * v;
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
    if (kSplit) cluster_st_f32x4(cluster_map(smem_u32(&s_po[rank * per + v % per]), v / per), y);
    else *reinterpret_cast<uint2*>(orow + e) = make_uint2(pack_bf16(y.x, y.y), pack_bf16(y.z, y.w));
  }
  if (kSplit) {
    cluster_sync();  // everything has been handed over; nothing is read from another CTA
    for (int x = tid; x < per && rank * per + x < kVecs; x += kThreads) {
      const int e = 4 * (rank * per + x), h = e / kD, col = e % kD;
      float cm[kMaxSplit], M = -INFINITY, L = 0.f;
      float4 acc = make_float4(0.f, 0.f, 0.f, 0.f);
#pragma unroll
      for (int u = 0; u < kMaxSplit; ++u) {
        cm[u] = u < kC ? s_pm[u][h] : -INFINITY;
        M = fmaxf(M, cm[u]);
      }
#pragma unroll
      for (int u = 0; u < kMaxSplit; ++u) {
        if (u >= kC) continue;
        const float f = exp2f((cm[u] - M) * s_f[h]);  // every row has a key of its own: M is finite
        const float4 y = s_po[u * per + x];
        L += s_pl[u][h] * f;
        acc.x += y.x * f;
        acc.y += y.y * f;
        acc.z += y.z * f;
        acc.w += y.w * f;
      }
      const float inv = kUnit / L;
      *reinterpret_cast<uint2*>(orow + e) =
          make_uint2(pack_bf16(acc.x * inv, acc.y * inv), pack_bf16(acc.z * inv, acc.w * inv));
      if (col == 0) lse[r * kHq + h] = __fmaf_rn(M, s_f[h], log2f(L)) * kLn2;
    }
  }
}

template <int kStages>
size_t smem_bytes(int blocks, int split) {
  return 128 + static_cast<size_t>(kStages) * kStageBytes +
         static_cast<size_t>((blocks + split - 1) / split) * kBlkPools * sizeof(int64_t);
}
constexpr int row_blocks(int topk) { return (topk + 1 + kBlkPools - 1) / kBlkPools; }
constexpr int kBlocksOf[2] = {row_blocks(512), row_blocks(2048)};  // the longest rows of two classes

template <int kStages, bool kSplit>
cudaError_t allow_smem() {
  constexpr size_t kMost =
      128 + static_cast<size_t>(kStages) * kStageBytes + static_cast<size_t>(kBlocksOf[1]) * kBlkPools * sizeof(int64_t);
  static std::atomic<bool> attr_done[kAttrDevices];
  return set_smem_limit_once(paged4_attn_kernel<kStages, kSplit>, static_cast<int>(kMost), attr_done);
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
  cudaError_t e = allow_smem<6, true>();
  if (e != cudaSuccess) return e;
  cudaLaunchAttribute attr[2];
  cudaLaunchConfig_t cfg = split_config(attr, 1, split, smem_bytes<6>(kBlocksOf[cls], split), nullptr);
  e = cudaOccupancyMaxActiveClusters(rows, paged4_attn_kernel<6, true>, &cfg);
  if (e == cudaSuccess && cached) known[dev][cls][split].store(*rows + 1, std::memory_order_relaxed);
  return e;
}

template <int kStages, bool kSplit>
cudaError_t launch_variant(const CacheView& c, const BatchView& b, const void* q, const int32_t* pool_idx, int topk,
                           float scale, void* o, float* lse, int split, const LaunchCtx& ctx) {
  const cudaError_t e = allow_smem<kStages, kSplit>();
  if (e != cudaSuccess) return e;
  call_param("ctas_per_row", split);
  call_param("ring_blocks", kStages);
  call_variant(kSplit ? "a cluster per row: cp.async gather of 4-bit pools through the block table, codes to fp16 in "
                        "registers, mma.sync, online softmax"
                      : "a CTA per row: cp.async gather of 4-bit pools through the block table, codes to fp16 in "
                        "registers, mma.sync, online softmax");
  cudaLaunchAttribute attr[2];
  const cudaLaunchConfig_t cfg = split_config(attr, b.rows, split, smem_bytes<kStages>(row_blocks(topk), split), ctx.stream);
  return cudaLaunchKernelEx(&cfg, paged4_attn_kernel<kStages, kSplit>, c, b, static_cast<const __nv_bfloat16*>(q),
                            pool_idx, topk, scale * kLog2e, static_cast<__nv_bfloat16*>(o), lse, split, ctx.status);
}

// The CTAs of a row.  A split shortens a row's chain of slices (76 ns each, four
// warps side by side) and costs a merge across the cluster; CTAs that share an SM
// slow one another down, and the rows' clusters have to be on the device at once
// (the runtime says how many are: 51 of 8, 74 of 6).  Measured, in us with 1 / 2 / 4 /
// 6 / 8 CTAs a row, keys and values from HBM:
//   512 pools   1 row 17.9 / 12.5 / 9.2 / 7.9 / 7.4    16 rows 18.4 / 13.2 / 9.5 / 8.1 / 8.9
//               32 rows 20.0 / 14.6 / 10.6 / 10.8 / 9.9    40 rows 20.4 / 14.9 / 12.8 / 11.4 / 11.8
//               64 rows 20.7 / 15.6 / 14.2 / 15.2    100 rows 20.6 / 19.2 / 17.5    228 rows 27.3 / 25.3
//   255 pools   1 row 10.3 / 8.6 / 6.9 / 6.6 / 6.5    32 rows 10.8 / 9.5 / 7.6 / 8.1 / 7.6
//               64 rows 11.9 / 10.3 / 9.7 / 10.0    130 rows 11.2 / 11.7
//   128 pools   1 row 7.7 / 7.3 / 6.5 / 6.1 / 6.1    40 rows 8.2 / 8.0 / 7.8 / 7.4 / 7.8    90 rows 8.2 / 9.3 / 8.8
int split_wanted(int64_t rows, int blocks, int num_sms) {
  const int64_t sms = num_sms;
  if (blocks < 6) return 1;
  if (12 * rows <= sms) return 8;
  if (6 * rows <= sms) return 6;
  if (blocks >= 16 && 8 * rows <= 2 * sms) return 8;
  if (blocks > 20 && 6 * rows <= 2 * sms) return 6;
  return blocks >= 16 || 4 * rows <= sms ? 4 : 1;
}

}  // namespace

cudaError_t launch_paged4_attn(const CacheView& c, const BatchView& b, const void* q, const int32_t* pool_idx, int topk,
                               float scale, void* o, float* lse, const LaunchCtx& ctx) {
  const int blocks = row_blocks(topk), cls = blocks <= kBlocksOf[0] ? 0 : 1;
  // (three CTAs an SM at the most, so no more rows than this have two each)
  if (b.rows <= 3 * static_cast<int64_t>(ctx.num_sms) / 2) {
    int fit = 0, dev = 0;
    const cudaError_t got = cudaGetDevice(&dev);
    if (got != cudaSuccess) return got;
    for (int split = split_wanted(b.rows, blocks, ctx.num_sms); split > 1; split -= 2) {
      if (split == 2 && blocks <= 20) break;
      const cudaError_t e = rows_at_once(dev, cls, split, &fit);
      if (e != cudaSuccess) return e;
      if (b.rows <= fit) return launch_variant<6, true>(c, b, q, pool_idx, topk, scale, o, lse, split, ctx);
    }
  }
  // A long ring and three CTAs an SM while all rows run at once, else a short one
  // and four: 300 rows 28.0 us against 30.2, 456 rows 37.3 and 38.2, 512 rows 51.2
  // and 47.0, 4096 rows 267 and 265.
  if (b.rows <= 3 * static_cast<int64_t>(ctx.num_sms))
    return launch_variant<6, false>(c, b, q, pool_idx, topk, scale, o, lse, 1, ctx);
  return launch_variant<4, false>(c, b, q, pool_idx, topk, scale, o, lse, 1, ctx);
}

}  // namespace dsa
