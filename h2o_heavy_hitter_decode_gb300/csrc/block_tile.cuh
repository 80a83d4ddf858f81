// block_tile.cuh — what a warp does with a block of a block-scaled 8-bit cache
// in attention: codes to f16, the two products on mma.sync, the online softmax
// of its rows (the mathematics stands in block_attend.cu).
#pragma once

#include <cuda.h>

#include <cfloat>

#include "block_cache.cuh"
#include "sm100.cuh"

namespace h2o {
namespace blk {

using namespace sm100;

__device__ __forceinline__ int ceil_div(int a, int b) { return (a + b - 1) / b; }

// ------------------------------------------------------------------- formats
// A word's four codes c0..c3 as two f16x2 registers (exact), and the byte
// selections that bring two words' codes x, y to (x0, y0), (x1, y1) and
// (x2, y2), (x3, y3) through the same conversion.
template <typename F> struct ToF16;
template <> struct ToF16<E4M3> {  // (c0, c1), (c2, c3)
  static constexpr bool kAdjacent = true;
  static constexpr uint32_t kLow = 0x5140, kHigh = 0x7362;
  __device__ __forceinline__ static void run(uint32_t w, uint32_t &a, uint32_t &z) {
    asm("{\n\t.reg .b16 lo, hi;\n\tmov.b32 {lo, hi}, %2;\n\tcvt.rn.f16x2.e4m3x2 %0, lo;\n\t"
        "cvt.rn.f16x2.e4m3x2 %1, hi;\n\t}"
        : "=r"(a), "=r"(z)
        : "r"(w));
  }
};
template <> struct ToF16<I8> {  // (c0, c2), (c1, c3): code + 128 in the low bits of the f16 number 1024, less 1152
  static constexpr bool kAdjacent = false;
  static constexpr uint32_t kLow = 0x5410, kHigh = 0x7632;
  __device__ __forceinline__ static void run(uint32_t w, uint32_t &a, uint32_t &z) {
    const __half2 bias = __halves2half2(__ushort_as_half(0x6480), __ushort_as_half(0x6480));
    const uint32_t x = (w & 0x00ff00ffu) ^ 0x64806480u, y = ((w >> 8) & 0x00ff00ffu) ^ 0x64806480u;
    const __half2 p = __hsub2(*(const __half2 *)&x, bias), q = __hsub2(*(const __half2 *)&y, bias);
    a = *(const uint32_t *)&p;
    z = *(const uint32_t *)&q;
  }
};

// c (+)= A B, 16 x 8 x 16.
__device__ __forceinline__ void mma16816(float (&c)[4], const uint32_t (&a)[4], uint32_t b0, uint32_t b1) {
  asm("mma.sync.aligned.m16n8k16.row.col.f32.f16.f16.f32 {%0,%1,%2,%3}, {%4,%5,%6,%7}, {%8,%9}, {%0,%1,%2,%3};"
      : "+f"(c[0]), "+f"(c[1]), "+f"(c[2]), "+f"(c[3])
      : "r"(a[0]), "r"(a[1]), "r"(a[2]), "r"(a[3]), "r"(b0), "r"(b1));
}
__device__ __forceinline__ void mma16816_new(float (&c)[4], const uint32_t (&a)[4], uint32_t b0, uint32_t b1) {
  asm("mma.sync.aligned.m16n8k16.row.col.f32.f16.f16.f32 {%0,%1,%2,%3}, {%4,%5,%6,%7}, {%8,%9}, {%10,%10,%10,%10};"
      : "=f"(c[0]), "=f"(c[1]), "=f"(c[2]), "=f"(c[3])
      : "r"(a[0]), "r"(a[1]), "r"(a[2]), "r"(a[3]), "r"(b0), "r"(b1), "f"(0.f));
}
// Transpose of an 8 x 8 matrix of f16, a lane holding two neighbours of a row.
__device__ __forceinline__ uint32_t transpose8(uint32_t x) {
  uint32_t y;
  asm("movmatrix.sync.aligned.m8n8.trans.b16 %0, %1;" : "=r"(y) : "r"(x));
  return y;
}

// 2-D tiled TMA load with an L2 eviction policy.
__device__ __forceinline__ void tma_load_2d(void *dst, const CUtensorMap *map, uint64_t *bar, int c0, int c1,
                                            uint64_t policy) {
  asm volatile(
      "cp.async.bulk.tensor.2d.shared::cluster.global.mbarrier::complete_tx::bytes.L2::cache_hint [%0], [%1, {%3, %4}], "
      "[%2], %5;" ::"r"(smem_u32(dst)),
      "l"(map), "r"(smem_u32(bar)), "r"(c0), "r"(c1), "l"(policy)
      : "memory");
}
__device__ __forceinline__ uint64_t l2_policy(bool evict_first) {
  uint64_t p;
  if (evict_first)
    asm volatile("createpolicy.fractional.L2::evict_first.b64 %0, 1.0;" : "=l"(p));
  else
    asm volatile("createpolicy.fractional.L2::evict_normal.b64 %0, 1.0;" : "=l"(p));
  return p;
}

// Byte offset of 16-byte chunk `chunk` of row `row` in a swizzled block.
template <int D> __device__ __forceinline__ int chunk_at(int row, int chunk) {
  return row * D + ((D == 128 ? chunk ^ (row & 7) : chunk ^ ((row >> 1) & 3)) << 4);
}

// ------------------------------------------------------------------- bounds
template <typename F> constexpr float kPerUnit = 1.f;
template <> constexpr float kPerUnit<E4M3> = 0.25f;

// Least and largest key code of each dimension of a block of head bh, in units of 1 (int8) or 4 (e4m3) rounded outwards,
// over its entries below `total`.  One warp: the block's rows in 16-byte loads, all on their way together, as f16 (exact);
// two dimensions at a time.
template <typename F, int D> __device__ __forceinline__ void bound_block(const View &c, int64_t bh, int blk, int total) {
  using T = ToF16<F>;
  constexpr int LPR = D / 16;       // lanes per row, 16 codes each
  constexpr int RPI = 32 / LPR;     // rows per load of the warp
  constexpr int IT = kBlock / RPI;  // loads
  const int lane = threadIdx.x & 31, sub = lane % LPR, row0 = lane / LPR, rest = total - blk * kBlock;
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

// Output sums are held in a unit 2^E of the warp's: bf16 values reach 2^128
// and weights before their division by the sum 2^15, so that plain fp32 sums
// would pass its range (|v| from 2^121 on with one entry, 2^103 with 262,144
// of one sign).  A block whose scale is above 2^kUnitMost units sets the unit
// anew, so that its scale is 2^kUnitSet of them: sums stay below 2^15 (weight)
// * 2^9 (code) * 2^70 * 2^30 (entries) = 2^124, and those of blocks whose scale
// is 2^180 times smaller are normal numbers still.
constexpr float kUnitMost = 0x1p70f, kUnitSet = 0x1p60f, kUnitFirst = 0x1p100f;
// Partial outputs are weighted means (their sums of weights go along): four
// times smaller, since a code times its scale may round up to 2^128.
constexpr float kPartDown = 0.25f, kPartUp = 4.f;
// 1 / x of a sum of weights (0, NaN, or 1 and more: a row's largest weight is at least its reference's), 0 of 0.  Off by
// 2^-23 at most, once a partial and once each time partials meet.
__device__ __forceinline__ float inverse_sum(float x) {
  float y;
  asm("rcp.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
  return x == 0.f ? 0.f : y;
}

// What a row's base-2 logits are taken off to give its weights, from its reference and sum of weights.  Nothing seen: every
// weight is 0.  NaN or infinite logits (a NaN or infinite query): the sum is NaN, and the reference in its place gives
// NaN on the entries that the row sees and 0 on those that it does not, whose logit is -infinity.
__device__ __forceinline__ float weight_base(float m, float l) {
  if (l != l) return m == -INFINITY ? 0.f : m;
  return l > 0.f ? m + log2f(l) : INFINITY;
}

// What a warp holds of a head while it attends: Q, and for its NR tiles of 8
// rows the output, the reference and the sum of the weights so far.  Whole: a
// weight meets V as two f16 numbers, its rounding and what that loses, so with
// 22 bits, where one of them has 11.
template <typename F, int D, int NR, bool QSmem, bool Whole> struct Tile {
  using T = ToF16<F>;
  static constexpr int KS = D / 16;  // k steps of S, words of a lane's share of a K entry
  static constexpr int OT = D / 16;  // 16-row tiles of O^T
  // The lane's rows of tile n: 2 t and 2 t + 1 (columns of S^T and O^T).
  float o[NR][OT][4], m[NR][2], lsum[NR][2], crow[NR][2];
  int end[NR][2];
  uint32_t qr[QSmem ? 1 : NR][KS][2];
  int min_end, live;  // live: bit 2 n + u, the row exists
  float vunit;        // 2^-E: units of o in a value of 1

  // Rows row0 .. of head h (of `group` query heads) of sequence b; qs: this warp's share of shared memory for Q.
  __device__ __forceinline__ void begin(const Rows &q, int group, int causal, const Seq &s, int b, int h, int row0,
                                        uint4 *qs) {
    const int lane = threadIdx.x & 31, g = lane >> 2, t = lane & 3;
    min_end = causal ? s.total - s.cnt + 1 : s.total;
    live = 0;
    vunit = kUnitFirst;
#pragma unroll
    for (int n = 0; n < NR; ++n) {
#pragma unroll
      for (int j = 0; j < OT; ++j) o[n][j][0] = o[n][j][1] = o[n][j][2] = o[n][j][3] = 0.f;
#pragma unroll
      for (int u = 0; u < 2; ++u) {
        const int tok = (row0 + 8 * n + 2 * t + u) / group;
        const bool is = tok < s.cnt;
        live |= (int)is << (2 * n + u);
        end[n][u] = is && causal ? s.total - s.cnt + tok + 1 : s.total;
        m[n][u] = -INFINITY;
        lsum[n][u] = 0.f;
      }
      // Q: the lane's D/4 dimensions of row g
      const int r = row0 + 8 * n + g, tok = r / group;
      const bool is = tok < s.cnt;
      const __nv_bfloat16 *p = q.at(b, h * group + r % group, tok) + t * (D / 4);
      float f[D / 4], top = 0.f;
#pragma unroll
      for (int e = 0; e < D / 32; ++e)
        Unpack<__nv_bfloat16>::run(is ? ld_nc16(p + e * 8) : make_uint4(0u, 0u, 0u, 0u), f + e * 8);
#pragma unroll
      for (int e = 0; e < D / 4; ++e) top = fmaxf(top, fabsf(f[e]));
      top = fmaxf(top, __shfl_xor_sync(0xffffffffu, top, 1));
      top = fmaxf(top, __shfl_xor_sync(0xffffffffu, top, 2));
      // q to f16: a power of two brings the row's largest element to 2^13 .. 2^14; bf16's 8 bits then fit, and
      // only elements 2^-27 of the largest and below lose bits
      int ex = 0;
      frexpf(top, &ex);
      const int sh = top > 0.f && top < INFINITY ? min(14 - ex, 100) : 0;
      const float up = ldexpf(1.f, sh), back = ldexpf(rsqrtf((float)D) * kLog2e, -sh);
      crow[n][0] = __shfl_sync(0xffffffffu, back, 8 * t);
      crow[n][1] = __shfl_sync(0xffffffffu, back, 8 * t + 4);
      uint32_t qh[KS][2];
#pragma unroll
      for (int k = 0; k < KS; ++k) {  // in the order of the codes' conversion
        const __half2 x = __floats2half2_rn(f[4 * k] * up, f[4 * k + (T::kAdjacent ? 1 : 2)] * up);
        const __half2 y = __floats2half2_rn(f[4 * k + (T::kAdjacent ? 2 : 1)] * up, f[4 * k + 3] * up);
        qh[k][0] = *(const uint32_t *)&x;
        qh[k][1] = *(const uint32_t *)&y;
      }
      if constexpr (QSmem) {
#pragma unroll
        for (int k = 0; k < KS; k += 2)  // read by this lane only
          qs[(n * (KS / 2) + k / 2) * 32 + lane] = make_uint4(qh[k][0], qh[k][1], qh[k + 1][0], qh[k + 1][1]);
      } else {
#pragma unroll
        for (int k = 0; k < KS; ++k) qr[n][k][0] = qh[k][0], qr[n][k][1] = qh[k][1];
      }
    }
  }

  // The block's K and V codes (swizzled) under their scales; `rest` entries are left of the head; keep(r, j, ...)
  // receives the base-2 logits of row row0 + r and entries j, j + 8, j + 16 and j + 24.
  template <typename Keep>
  __device__ __forceinline__ void block(const uint8_t *kt, uint8_t *vt, float ks, float vs, int blk, int rest,
                                        const uint4 *qs, Keep keep) {
    const int lane = threadIdx.x & 31, g = lane >> 2, t = lane & 3;
    float s[NR][2][4];  // S^T: entries 16 x + g and + 8, rows 2 t and 2 t + 1
#pragma unroll
    for (int part = 0; part < KS / 4; ++part) {  // 16 bytes of each K row at a time
      uint32_t kw[4][4];
#pragma unroll
      for (int n = 0; n < 4; ++n) {
        const uint4 u = *(const uint4 *)(kt + chunk_at<D>(n * 8 + g, t * (KS / 4) + part));
        kw[n][0] = u.x, kw[n][1] = u.y, kw[n][2] = u.z, kw[n][3] = u.w;
      }
#pragma unroll
      for (int k = 0; k < 4; k += 2) {
        uint32_t q[NR][4];
#pragma unroll
        for (int n = 0; n < NR; ++n) {
          if constexpr (QSmem) {
            const uint4 u = qs[(n * (KS / 2) + part * 2 + k / 2) * 32 + lane];
            q[n][0] = u.x, q[n][1] = u.y, q[n][2] = u.z, q[n][3] = u.w;
          } else {
            q[n][0] = qr[n][part * 4 + k][0], q[n][1] = qr[n][part * 4 + k][1];
            q[n][2] = qr[n][part * 4 + k + 1][0], q[n][3] = qr[n][part * 4 + k + 1][1];
          }
        }
#pragma unroll
        for (int e = 0; e < 2; ++e)
#pragma unroll
          for (int x = 0; x < 2; ++x) {
            uint32_t ka[4];
            T::run(kw[2 * x][k + e], ka[0], ka[2]);
            T::run(kw[2 * x + 1][k + e], ka[1], ka[3]);
#pragma unroll
            for (int n = 0; n < NR; ++n) {
              if (part == 0 && k + e == 0)
                mma16816_new(s[n][x], ka, q[n][0], q[n][1]);
              else
                mma16816(s[n][x], ka, q[n][2 * e], q[n][2 * e + 1]);
            }
          }
      }
    }
    const int j0 = blk * kBlock + g;
    const bool edge = blk * kBlock + kBlock > min_end;
    uint32_t p[NR][4];  // P^T as B: entries 8 e + 2 t and + 1 of row g
    uint32_t rest16[Whole ? NR : 1][4];  // what its rounding to 16 bits loses
#pragma unroll
    for (int n = 0; n < NR; ++n) {
      // finite: an infinite factor (a huge query on a huge scale) would turn the products that are 0 into NaN
      const float f0 = fminf(crow[n][0] * ks, FLT_MAX), f1 = fminf(crow[n][1] * ks, FLT_MAX);
#pragma unroll
      for (int x = 0; x < 2; ++x) s[n][x][0] *= f0, s[n][x][1] *= f1, s[n][x][2] *= f0, s[n][x][3] *= f1;
      if (edge) {
#pragma unroll
        for (int x = 0; x < 2; ++x)
#pragma unroll
          for (int e = 0; e < 4; ++e)
            if (j0 + 16 * x + 8 * (e >> 1) >= end[n][e & 1]) s[n][x][e] = -INFINITY;
      }
#pragma unroll
      for (int u = 0; u < 2; ++u)
        if (live >> (2 * n + u) & 1) keep(8 * n + 2 * t + u, j0, s[n][0][u], s[n][0][2 + u], s[n][1][u], s[n][1][2 + u]);
    }
    float top[NR][2];
    bool moves = false;
#pragma unroll
    for (int n = 0; n < NR; ++n)
#pragma unroll
      for (int u = 0; u < 2; ++u) {
        float x = fmaxf(fmaxf(s[n][0][u], s[n][0][2 + u]), fmaxf(s[n][1][u], s[n][1][2 + u]));
        x = fmaxf(x, __shfl_xor_sync(0xffffffffu, x, 4));
        x = fmaxf(x, __shfl_xor_sync(0xffffffffu, x, 8));
        x = fmaxf(x, __shfl_xor_sync(0xffffffffu, x, 16));
        top[n][u] = x;
        moves |= x > m[n][u] + 15.f || m[n][u] == -INFINITY;
      }
    // The weights' reference lies 2^7 below the maximum when it is set, and moves only when it is passed by more than
    // 2^15.  Weights then stay below 2^15, in f16's range, and one 2^21 times smaller than the largest is still a
    // normal number of it: a long tail of small weights next to a large one is not lost.
    if (__any_sync(0xffffffffu, moves)) {
#pragma unroll
      for (int n = 0; n < NR; ++n)
#pragma unroll
        for (int u = 0; u < 2; ++u) {
          const float mn = fmaxf(m[n][u], top[n][u] - 7.f);
          const float f = m[n][u] == -INFINITY ? 0.f : ex2(m[n][u] - mn);
          m[n][u] = mn;
          lsum[n][u] *= f;
#pragma unroll
          for (int j = 0; j < OT; ++j) o[n][j][u] *= f, o[n][j][2 + u] *= f;
        }
    }
#pragma unroll
    for (int n = 0; n < NR; ++n) {
      const float mu0 = m[n][0] == -INFINITY ? 0.f : m[n][0], mu1 = m[n][1] == -INFINITY ? 0.f : m[n][1];
#pragma unroll
      for (int x = 0; x < 2; ++x) {
        const float e0 = ex2(s[n][x][0] - mu0), e1 = ex2(s[n][x][1] - mu1), e2 = ex2(s[n][x][2] - mu0),
                    e3 = ex2(s[n][x][3] - mu1);
        lsum[n][0] += e0 + e2;
        lsum[n][1] += e1 + e3;
        // 16 bits for the product with V: f16's 2^-11 of each weight, so 2^-11 of sum w |v|: an eighth of the output's own
        // rounding where the values do not cancel.  In two parts 2^-22, and 2^-25 below f16's normal numbers, 2^-32 of
        // the largest weight.
        const __half2 a0 = __floats2half2_rn(e0, e1), a1 = __floats2half2_rn(e2, e3);
        p[n][2 * x] = transpose8(*(const uint32_t *)&a0);
        p[n][2 * x + 1] = transpose8(*(const uint32_t *)&a1);
        if constexpr (Whole) {
          const float2 h0 = __half22float2(a0), h1 = __half22float2(a1);
          const __half2 z0 = __floats2half2_rn(e0 - h0.x, e1 - h0.y), z1 = __floats2half2_rn(e2 - h1.x, e3 - h1.y);
          rest16[n][2 * x] = transpose8(*(const uint32_t *)&z0);
          rest16[n][2 * x + 1] = transpose8(*(const uint32_t *)&z1);
        }
      }
    }
    if (rest < kBlock) {  // codes behind the last entry may be anything, also NaN: weight 0 needs a finite code
      for (int z = rest * D + lane * 16; z < kBlock * D; z += 512) *(uint4 *)(vt + z) = make_uint4(0u, 0u, 0u, 0u);
      fence_proxy_async_smem();
      __syncwarp();
    }
    if (vs * vunit > kUnitMost) {  // rare: the first block, and one of a far larger scale than those before
      const float unit = inverse_pow2(vs) * kUnitSet, f = unit * inverse_pow2(vunit);
      vunit = unit;
#pragma unroll
      for (int n = 0; n < NR; ++n)
#pragma unroll
        for (int j = 0; j < OT; ++j) o[n][j][0] *= f, o[n][j][1] *= f, o[n][j][2] *= f, o[n][j][3] *= f;
    }
    vs *= vunit;
    // O += vs (P V): a fresh product per block, added in fp32 under the block's scale
    constexpr int VW = D == 128 && NR == 1 ? 4 : 2;  // words of the lane's D/8 dimensions of an entry at a time
#pragma unroll
    for (int part = 0; part < D / 32 / VW; ++part) {
      uint32_t vw[8][VW];
#pragma unroll
      for (int e = 0; e < 8; ++e) {
        const int r = (e >> 1) * 8 + 2 * t + (e & 1);
        if constexpr (VW == 4) {
          const uint4 u = *(const uint4 *)(vt + chunk_at<D>(r, g));
          vw[e][0] = u.x, vw[e][1] = u.y, vw[e][2 % VW] = u.z, vw[e][3 % VW] = u.w;
        } else {
          const uint8_t *from = D == 128 ? vt + chunk_at<D>(r, g) + part * 8 : vt + chunk_at<D>(r, g >> 1) + (g & 1) * 8;
          const uint2 u = *(const uint2 *)from;
          vw[e][0] = u.x, vw[e][1] = u.y;
        }
      }
#pragma unroll
      for (int w = 0; w < VW; ++w) {
        uint32_t va[2][2][4];  // [dimensions 4w, 4w+1 | 4w+2, 4w+3][k step]
#pragma unroll
        for (int k = 0; k < 2; ++k) {
          const uint32_t x = vw[4 * k][w], y = vw[4 * k + 1][w], z = vw[4 * k + 2][w], v = vw[4 * k + 3][w];
          T::run(__byte_perm(x, y, T::kLow), va[0][k][0], va[0][k][1]);
          T::run(__byte_perm(x, y, T::kHigh), va[1][k][0], va[1][k][1]);
          T::run(__byte_perm(z, v, T::kLow), va[0][k][2], va[0][k][3]);
          T::run(__byte_perm(z, v, T::kHigh), va[1][k][2], va[1][k][3]);
        }
#pragma unroll
        for (int n = 0; n < NR; ++n)
#pragma unroll
          for (int y = 0; y < 2; ++y) {
            const int j = (part * VW + w) * 2 + y;
            float acc[4];
            // the second parts in a sum of their own, two products deep, while registers allow it (long batch 60.1 us
            // for 61.5 in one sum; not with 16 rows a head, 67.5 for 64.7)
            if constexpr (Whole && NR > 1) {
              mma16816_new(acc, va[y][0], rest16[n][0], rest16[n][1]);
              mma16816(acc, va[y][1], rest16[n][2], rest16[n][3]);
              mma16816(acc, va[y][0], p[n][0], p[n][1]);
            } else {
              mma16816_new(acc, va[y][0], p[n][0], p[n][1]);
            }
            mma16816(acc, va[y][1], p[n][2], p[n][3]);
            if constexpr (Whole && NR == 1) {
              float more[4];
              mma16816_new(more, va[y][0], rest16[n][0], rest16[n][1]);
              mma16816(more, va[y][1], rest16[n][2], rest16[n][3]);
#pragma unroll
              for (int e = 0; e < 4; ++e) acc[e] += more[e];
            }
#pragma unroll
            for (int e = 0; e < 4; ++e) o[n][j][e] = fmaf(acc[e], vs, o[n][j][e]);
          }
      }
    }
  }

  // What a sum of o is as a value.
  __device__ __forceinline__ float unit() const { return inverse_pow2(vunit); }
  // Sum of the lane's row over the warp.
  __device__ __forceinline__ float sum(int n, int u) const {
    float l = lsum[n][u];
    l += __shfl_xor_sync(0xffffffffu, l, 4);
    l += __shfl_xor_sync(0xffffffffu, l, 8);
    l += __shfl_xor_sync(0xffffffffu, l, 16);
    return l;
  }
};

}  // namespace blk
}  // namespace h2o
