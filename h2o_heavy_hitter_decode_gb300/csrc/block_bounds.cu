// block_bounds.cu — least and largest code of each dimension of a block's
// keys, in 8 bits, for the choice of blocks in block_sparse.cu.
//
//   lo_i = floor(min_j c_ji / u), hi_i = ceil(max_j c_ji / u) over the block's
//   entries j; u = 1 for int8 codes, 4 for e4m3 ones (whole numbers of units
//   then reach 112; the rounding is outwards, so the bounds stay bounds).
//
// One warp per (head, block) for many rows (bound_block in block_tile.cuh).
// Few new rows have theirs made by the warp that appends them.  Bound by
// memory: d bytes read an entry and d / 16 written.  A pass of its own: 16 x 32
// heads x 8,192 new rows 105 us more (537 MB read, 5.4 TB/s); an eviction from
// 8,448 to 1,690 entries of 32 x 32 heads 208 -> 265 us (int8 216 -> 301), and one
// that leaves everything as it is 7 -> 68.
#include "block_tile.cuh"

namespace h2o {
namespace blk {
namespace {

constexpr int kWarps = 4;

// Blocks of a call: those that its rows went to, or (whole) all that hold entries; whole = 2
// passes over lengths out of range, which the call before has reported.
template <typename F, int D>
__global__ void __launch_bounds__(kWarps * 32) bound_kernel(const View c, const Lens l, int whole, int blocks) {
  const int lane = threadIdx.x & 31;
  const int64_t item = (int64_t)blockIdx.x * kWarps + (threadIdx.x >> 5);
  const int64_t bh = item / blocks;
  const int j = (int)(item - bh * blocks);
  if (bh >= (int64_t)c.B * c.H) return;
  const int b = (int)bh / c.H, h = (int)bh - b * c.H;
  int first, total;
  if (whole) {
    first = 0, total = l.lengths[b];
    if (total < 0 || total > c.cap) {
      if (whole == 1 && lane == 0 && j == 0 && h == 0) atomicOr(c.err, H2O_BERR_RANGE);
      return;
    }
  } else {
    const Seq s = seq_of(l, b);  // refused sequences are reported by the append
    if (s.cnt == 0) return;
    first = s.len / kBlock, total = s.total;
  }
  const int blk = first + j;
  if (total <= blk * kBlock) return;
  bound_block<F, D>(c, bh, blk, total);
}

template <typename F, int D> cudaError_t bound_t(const View &c, const Lens &l, int whole, cudaStream_t st) {
  const int blocks = whole ? c.cap / kBlock : (l.n + kBlock - 1) / kBlock + 1;  // the rows may start inside a block
  const int64_t warps = (int64_t)c.B * c.H * blocks;
  bound_kernel<F, D><<<(unsigned)((warps + kWarps - 1) / kWarps), kWarps * 32, 0, st>>>(c, l, whole, blocks);
  return cudaGetLastError();
}

}  // namespace

cudaError_t launch_bound(const View &c, const Lens &l, int whole, cudaStream_t st) {
  if (c.kv == H2O_KV_E4M3)
    return c.d == 128 ? bound_t<E4M3, 128>(c, l, whole, st) : bound_t<E4M3, 64>(c, l, whole, st);
  return c.d == 128 ? bound_t<I8, 128>(c, l, whole, st) : bound_t<I8, 64>(c, l, whole, st);
}

}  // namespace blk
}  // namespace h2o
