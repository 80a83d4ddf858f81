// block_bounds.cu — least and largest code of each dimension of a block's
// keys, in 8 bits, for the choice of blocks in block_sparse.cu.
//
//   lo_i = floor(min_j c_ji / u), hi_i = ceil(max_j c_ji / u) over the block's
//   entries j; u = 1 for int8 codes, 4 for e4m3 ones (whole numbers of units
//   then reach 112; the rounding is outwards, so the bounds stay bounds).
//
// One warp per (head, block): the block's rows in 16-byte loads, all on their
// way together, as f16 (exact); least and largest two dimensions at a time.
// Bound by memory: d bytes read an entry and d / 16 written.
#include "block_tile.cuh"

namespace h2o {
namespace blk {
namespace {

constexpr int kWarps = 4;

template <typename F> constexpr float kPerUnit = 1.f;
template <> constexpr float kPerUnit<E4M3> = 0.25f;

// Blocks of a call: those that its rows went to, or (whole) all that hold entries; whole = 2
// passes over lengths out of range, which the call before has reported.
template <typename F, int D>
__global__ void __launch_bounds__(kWarps * 32) bound_kernel(const View c, const Lens l, int whole, int blocks) {
  using T = ToF16<F>;
  constexpr int LPR = D / 16;       // lanes per row, 16 codes each
  constexpr int RPI = 32 / LPR;     // rows per load of the warp
  constexpr int IT = kBlock / RPI;  // loads
  const int lane = threadIdx.x & 31, sub = lane % LPR, row0 = lane / LPR;
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
  const int blk = first + j, rest = total - blk * kBlock;
  if (rest <= 0) return;
  const uint8_t *codes = c.K + ((size_t)bh * c.cap + (size_t)blk * kBlock) * D + sub * 16;
  uint4 w[IT];
#pragma unroll
  for (int i = 0; i < IT; ++i) {
    const int r = i * RPI + row0;
    w[i] = *(const uint4 *)(codes + (size_t)(r < rest ? r : 0) * D);  // row 0 again in the place of none
  }
  __half2 lo[8], hi[8];
#pragma unroll
  for (int i = 0; i < IT; ++i)
#pragma unroll
    for (int e = 0; e < 4; ++e) {
      uint32_t a, z;
      T::run((&w[i].x)[e], a, z);
      const __half2 x = *(const __half2 *)&a, y = *(const __half2 *)&z;
      lo[2 * e] = i == 0 ? x : __hmin2(lo[2 * e], x), hi[2 * e] = i == 0 ? x : __hmax2(hi[2 * e], x);
      lo[2 * e + 1] = i == 0 ? y : __hmin2(lo[2 * e + 1], y), hi[2 * e + 1] = i == 0 ? y : __hmax2(hi[2 * e + 1], y);
    }
#pragma unroll
  for (int o = LPR; o < 32; o <<= 1)
#pragma unroll
    for (int e = 0; e < 8; ++e) {
      lo[e] = __hmin2(lo[e], __shfl_xor_sync(0xffffffffu, lo[e], o));
      hi[e] = __hmax2(hi[e], __shfl_xor_sync(0xffffffffu, hi[e], o));
    }
  if (row0 > 1) return;
  const bool high = row0 == 1;  // the second group of lanes writes the largest
  uint32_t out[4];
#pragma unroll
  for (int e = 0; e < 4; ++e) {
    const __half2 unit = __float2half2_rn(kPerUnit<F>);
    const __half2 x = __hmul2(high ? hi[2 * e] : lo[2 * e], unit), y = __hmul2(high ? hi[2 * e + 1] : lo[2 * e + 1], unit);
    const __half2 p = high ? h2ceil(x) : h2floor(x), q = high ? h2ceil(y) : h2floor(y);
    const uint32_t p0 = __half2int_rn(__low2half(p)) & 0xff, p1 = __half2int_rn(__high2half(p)) & 0xff;
    const uint32_t q0 = __half2int_rn(__low2half(q)) & 0xff, q1 = __half2int_rn(__high2half(q)) & 0xff;
    out[e] = T::kAdjacent ? p0 | p1 << 8 | q0 << 16 | q1 << 24 : p0 | q0 << 8 | p1 << 16 | q1 << 24;
  }
  int8_t *dst = c.bounds + ((size_t)bh * (c.cap / kBlock) + blk) * 2 * D + (high ? D : 0) + sub * 16;
  *(uint4 *)dst = make_uint4(out[0], out[1], out[2], out[3]);
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
