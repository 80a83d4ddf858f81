// block_append.cu — rows quantised into a block-scaled 8-bit cache.
//
// For each block of 32 entries that receives rows: a = max |x| over its new
// rows, scale s' = max(least 2^e with a <= Q 2^e, scale before), code =
// round(x / s').  Division by a power of two is exact, so each code has one
// rounding.  Where the scale grew, the codes already in the block are
// re-scaled by the power of two s / s' and rounded once more.
//
// append_kernel: one warp per (head, block, K or V).  It holds the block's whole row data
// in registers (32 rows x d bf16 = 8 KB at d = 128: sixteen 16-byte loads per
// lane, all in flight together), so the input is read once and the codes are
// written once.  Bound by memory: 16 x 32 heads x 8,192 rows, 3.26 GB, 490 us,
// 98 % of the copy rate, with four CTAs (128 registers) an SM; three (168): 568.
// append_few_kernel: one warp per (head, K or V) for the rows of a decode
// step, taken one at a time; the block's earlier codes are read only where its
// scale grows.
#include "block_cache.cuh"

namespace h2o {
namespace blk {
namespace {

constexpr int kWarps = 4;

template <typename F, int D>
__global__ void __launch_bounds__(kWarps * 32, 4) append_kernel(const View c, const Lens l, const Rows k, const Rows v,
                                                             const int32_t *__restrict__ position,
                                                             const float *__restrict__ score, int blocks) {
  constexpr int LPR = D / 8;        // lanes per row, 8 elements (16 bytes) each
  constexpr int RPI = 32 / LPR;     // rows per load of the warp
  constexpr int IT = kBlock / RPI;  // loads
  const int lane = threadIdx.x & 31;
  grid_launch_dependents();
  const int64_t item = (int64_t)blockIdx.x * kWarps + (threadIdx.x >> 5);
  const bool is_v = item & 1;
  const int64_t bj = item >> 1;  // (b, h, j): j-th block the sequence's rows may touch
  const int j = (int)(bj % blocks);
  const int64_t bh64 = bj / blocks;
  if (bh64 >= (int64_t)c.B * c.H) return;
  const int bh = (int)bh64, b = bh / c.H, h = bh - b * c.H;
  const Seq s = seq_of(l, b);
  if (!s.ok) {
    if (lane == 0 && j == 0 && h == 0 && !is_v) atomicOr(c.err, H2O_BERR_RANGE);
    return;
  }
  const int blk = s.len / kBlock + j, base = blk * kBlock;
  const int lo = max(s.len, base), hi = min(s.len + s.cnt, base + kBlock);  // new entries of this block
  if (lo >= hi) return;

  const Rows &x = is_v ? v : k;
  uint8_t *codes = (is_v ? c.V : c.K) + ((size_t)bh * c.cap + base) * D;
  float *scale = (is_v ? c.Vsc : c.Ksc) + (size_t)bh * (c.cap / kBlock) + blk;
  const int sub = lane % LPR, row0 = lane / LPR;

  uint4 w[IT];
#pragma unroll
  for (int i = 0; i < IT; ++i) {
    const int t = base + i * RPI + row0;
    w[i] = t >= lo && t < hi ? ld_nc16(x.at(b, h, t - s.len) + sub * 8) : make_uint4(0u, 0u, 0u, 0u);
  }
  const float before = base < s.len ? *scale : 0.f;
  auto words = [&](int i) -> uint32_t * { return &w[i].x; };
  // Absolute values of bf16 order like their bits.
  uint32_t top2 = 0;
#pragma unroll
  for (int i = 0; i < IT; ++i)
#pragma unroll
    for (int e = 0; e < 4; ++e) top2 = __vmaxu2(top2, words(i)[e] & 0x7fff7fffu);
  uint32_t top = __reduce_max_sync(0xffffffffu, max(top2 & 0xffffu, top2 >> 16));
  const bool odd = top >= 0x7f80u;  // an infinity or NaN among them
  if (odd) {
    top = 0;
#pragma unroll
    for (int i = 0; i < IT; ++i)
#pragma unroll
      for (int e = 0; e < 4; ++e) {
        const uint32_t u = words(i)[e];
        const uint32_t a = u & 0x7fffu, z = (u >> 16) & 0x7fffu;
        top = max(top, max(a < 0x7f80u ? a : 0u, z < 0x7f80u ? z : 0u));
      }
    top = __reduce_max_sync(0xffffffffu, top);
    if (lane == 0) atomicOr(c.err, H2O_BERR_NONFINITE);
  }
  const float after = fmaxf(before, block_scale<F>(__uint_as_float(top << 16)));
  const float inv = inverse_pow2(after);
#pragma unroll
  for (int i = 0; i < IT; ++i) {
    const int r = i * RPI + row0, t = base + r;
    float f[8];
    Unpack<__nv_bfloat16>::run(w[i], f);
    if (odd) {
#pragma unroll
      for (int e = 0; e < 8; ++e) f[e] = f[e] != f[e] ? 0.f : fminf(fmaxf(f[e] * inv, -F::kMax), F::kMax);
    }
    const float by = odd ? 1.f : inv;
    const uint32_t lo4 = F::codes(f, by), hi4 = F::codes(f + 4, by);
    if (t >= lo && t < hi) *(uint2 *)(codes + (size_t)r * D + sub * 8) = make_uint2(lo4, hi4);
  }
  if (after > before && before > 0.f) {  // earlier entries of the block take the larger scale
    const typename F::Shift shift(exponent(before) - exponent(after));
    for (int i = 0; i < IT; ++i) {
      const int r = i * RPI + row0;
      if (base + r >= s.len) continue;
      uint2 *at = (uint2 *)(codes + (size_t)r * D + sub * 8);
      const uint2 u = *at;
      *at = make_uint2(shift.run(u.x), shift.run(u.y));
    }
  }
  if (lane == 0) *scale = after;
  const int t = base + lane;
  if (!is_v && t >= lo && t < hi) {
    const size_t at = (size_t)bh * c.cap + t;
    c.pos[at] = (position ? position[b] : s.len) + (t - s.len);
    c.score[at] = score ? score[(size_t)bh * l.n + (t - s.len)] : 0.f;
    c.low[at] = 0.f;
  }
}

// Few rows: a warp per (head, K or V).
template <typename F, int D>
__global__ void __launch_bounds__(kWarps * 32) append_few_kernel(const View c, const Lens l, const Rows k, const Rows v,
                                                                 const int32_t *__restrict__ position) {
  const int lane = threadIdx.x & 31;
  grid_launch_dependents();
  const int item = blockIdx.x * kWarps + (threadIdx.x >> 5);
  const bool is_v = item & 1;
  const int bh = item >> 1;
  if (bh >= c.B * c.H) return;
  const int b = bh / c.H, h = bh - b * c.H;
  const Seq s = seq_of(l, b);
  if (!s.ok) {
    if (lane == 0 && h == 0 && !is_v) atomicOr(c.err, H2O_BERR_RANGE);
    return;
  }
  for (int lo = s.len, end = s.len + s.cnt; lo < end;) {
    const int hi = min(end, (lo / kBlock + 1) * kBlock);
    append_rows<F, D>(c, is_v, is_v ? v : k, b, h, s.len, lo, hi);
    lo = hi;
  }
  if (!is_v && lane < s.cnt) {
    const size_t at = (size_t)bh * c.cap + s.len + lane;
    c.pos[at] = (position ? position[b] : s.len) + lane;
    c.score[at] = 0.f;
    c.low[at] = 0.f;
  }
}

template <typename F, int D>
cudaError_t append_t(const View &c, const Lens &l, const Rows &k, const Rows &v, const int32_t *position,
                     const float *score, cudaStream_t st) {
  if (l.n <= kFewRows && !score) {
    const int64_t warps = (int64_t)c.B * c.H * 2;
    append_few_kernel<F, D><<<(unsigned)((warps + kWarps - 1) / kWarps), kWarps * 32, 0, st>>>(c, l, k, v, position);
    return cudaGetLastError();
  }
  const int blocks = (l.n + kBlock - 1) / kBlock + 1;  // the rows may start inside a block
  const int64_t warps = (int64_t)c.B * c.H * blocks * 2;
  append_kernel<F, D><<<(unsigned)((warps + kWarps - 1) / kWarps), kWarps * 32, 0, st>>>(c, l, k, v, position, score,
                                                                                        blocks);
  return cudaGetLastError();
}

}  // namespace

cudaError_t launch_append(const View &c, const Lens &l, const Rows &k, const Rows &v, const int32_t *position,
                          const float *score, cudaStream_t st) {
  if (c.kv == H2O_KV_E4M3)
    return c.d == 128 ? append_t<E4M3, 128>(c, l, k, v, position, score, st)
                      : append_t<E4M3, 64>(c, l, k, v, position, score, st);
  return c.d == 128 ? append_t<I8, 128>(c, l, k, v, position, score, st)
                    : append_t<I8, 64>(c, l, k, v, position, score, st);
}

}  // namespace blk
}  // namespace h2o
