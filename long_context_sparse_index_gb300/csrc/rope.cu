// rope.cu -- heads turned by their position, on contiguous sequences: the
// rotation before the layer's training calls, and its gradient (the rotation
// back, for the matrix of a pair is orthogonal up to the table's scale: the
// gradient multiplies by the transpose, which turns by -s).
//
// The arithmetic is in fp32 (products of a bf16 and an fp32 number, one FMA),
// rounded once more to bf16.  Bound by memory: every element is read and
// written once, and a row of the table serves all heads of its row.
#include "rope.cuh"

namespace dsa {
namespace {

constexpr int kWarps = 8;

// A warp takes `per` rows (one, or as many as have heads enough for its lanes).
template <bool kInter>
__global__ void __launch_bounds__(32 * kWarps, 4)
    rope_kernel(const RopeView r, const RopeArgs a, int n, int per, int lanes, unsigned* status) {
  pdl_wait();  // launched early: what stands before in the stream has ended
  const int lane = threadIdx.x & 31;
  const int64_t w = static_cast<int64_t>(blockIdx.x) * kWarps + (threadIdx.x >> 5);
  const int64_t row = w * per + lane / lanes;
  if (row >= a.rows) return;
  const auto find = [&]() -> const float* {
    const int64_t pos = a.positions ? static_cast<int64_t>(__ldg(a.positions + row)) : a.begin + row;
    if (pos >= 0 && pos < r.positions) return r.cs + pos * r.stride;
    record_status(status, kStatusInternal);  // a position without an angle: the row is not written
    return nullptr;
  };
  turn_heads<kInter>(a.x + row * a.x_stride, a.out + row * a.out_stride, a.heads, a.D, r.dims, n, a.dir,
                     lane & (lanes - 1), lanes, find, [] { return true; });
}

}  // namespace

cudaError_t launch_rope(const RopeView& r, const RopeArgs& a, const LaunchCtx& ctx) {
  // lanes of a row: all of a warp, or fewer if its heads have less for them
  const int n = rope_chunk_lanes(r.dims, r.inter);
  int lanes = n;
  while (lanes < 32 && lanes < a.heads * n) lanes *= 2;
  const int per = 32 / lanes;
  const int64_t blocks = (a.rows + static_cast<int64_t>(per) * kWarps - 1) / (static_cast<int64_t>(per) * kWarps);
  LaunchCtx early = ctx;
  early.pdl = 1;
  return launch_ex(early, r.inter ? rope_kernel<true> : rope_kernel<false>, dim3(static_cast<unsigned>(blocks)),
                   dim3(32 * kWarps), 0, r, a, n, per, lanes, ctx.status);
}

}  // namespace dsa
