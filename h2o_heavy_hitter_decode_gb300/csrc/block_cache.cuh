// block_cache.cuh — what the kernels of the block-scaled 8-bit cache share
// (h2o_bcache_* in include/h2o.h): its device view, the checked lengths of a
// sequence, and the code formats with their power-of-two block scales.
#pragma once

#include <cuda.h>

#include "common.cuh"
#include "smem_limit.h"

#include "../../include/h2o.h"

namespace h2o {
namespace blk {

constexpr int kBlock = H2O_BLOCK;  // entries that share a scale
constexpr int kMinExp = -100;      // least scale exponent

struct View {
  int B, H, d, cap, group, max_rows;  // max_rows = group * max_queries
  int kv;                             // h2o_kv8
  uint8_t *K, *V;                     // [B*H][cap][d] codes
  float *Ksc, *Vsc;                   // [B*H][cap / kBlock]
  int32_t *pos;                       // [B*H][cap]
  float *score;                       // [B*H][cap]
  float *low;                         // [B*H][cap] what the scores' fp32 sums have lost (add_score)
  float *logits;                      // [B*H][max_rows][cap] scratch, base-2 logits
  float *part;                        // scratch, split partials
  int32_t *kept;                      // [B*H][cap] scratch of an eviction (shares the logits' memory)
  int *err;                           // [1] sticky H2O_BERR_* bits
  int sms, l2_bytes;
};

// Rows (b, h, t) of bf16 in memory, strides in elements.
struct Rows {
  const __nv_bfloat16 *p;
  int64_t sb, sh, st;
  __device__ __forceinline__ const __nv_bfloat16 *at(int b, int h, int t) const {
    return p + b * sb + h * sh + t * st;
  }
};

// The lengths of a call.  appends: the call's rows are entries len ..
// len + cnt - 1 (before or after they were written).
struct Lens {
  const int32_t *lengths, *counts;
  int n, appends, cap;
};
struct Seq {
  int len, cnt, total;  // entries before the call, real rows, entries to attend over (none without a query)
  bool ok;              // false: out of range, everything else 0
};
__device__ __forceinline__ Seq seq_of(const Lens &l, int b) {
  Seq s;
  s.len = l.lengths[b];
  s.cnt = l.counts ? l.counts[b] : l.n;
  s.ok = s.len >= 0 && s.cnt >= 0 && s.cnt <= l.n && s.len <= l.cap - (l.appends ? s.cnt : 0);
  if (!s.ok) s.len = s.cnt = 0;
  s.total = s.cnt == 0 ? 0 : s.len + (l.appends ? s.cnt : 0);
  return s;
}

// score + w in fp32; low keeps what the sum loses, and is taken into the next
// one: thousands of weights below half a step of a large score (an entry that
// starts with its prompt's column sum) add up all the same, where plain sums
// stay where they are.  The loss of a sum is exact (D. E. Knuth, The Art of
// Computer Programming, vol. 2, 4.2.2, theorem B).  It is at most half a step of the score:
// one that is larger belongs to a score that the caller has replaced.
__device__ __forceinline__ float add_score(float score, float &low, float w) {
  const float half_step = __uint_as_float(__float_as_uint(score) & 0x7f800000u) * 0x1p-24f;
  const float y = __fadd_rn(w, fabsf(low) <= half_step ? low : 0.f);
  const float sum = __fadd_rn(score, y), z = __fsub_rn(sum, score);
  low = __fadd_rn(__fsub_rn(score, __fsub_rn(sum, z)), __fsub_rn(y, z));
  return sum;
}

// ------------------------------------------------------------------ formats
struct E4M3 {
  static constexpr float kMax = 448.f;  // 1.75 * 2^8
  static constexpr int kMaxExp = 8;
  static constexpr uint32_t kMaxMant = 0x600000u;
  // x (finite, at most kMax up to rounding) to the nearest code, ties to even.
  __device__ __forceinline__ static uint32_t code(float x) {
    return (uint32_t)__nv_cvt_float_to_fp8(x, __NV_SATFINITE, __NV_E4M3);
  }
  // Four codes of a word as floats (exact).
  __device__ __forceinline__ static void values(uint32_t w, float *x) { e4m3x4_to_f32(w, x); }
  // Codes of x[0..3] * inv (at most kMax up to rounding).
  __device__ __forceinline__ static uint32_t codes(const float *x, float inv) {
    const uint32_t a = __nv_cvt_float2_to_fp8x2(make_float2(x[0] * inv, x[1] * inv), __NV_SATFINITE, __NV_E4M3);
    const uint32_t z = __nv_cvt_float2_to_fp8x2(make_float2(x[2] * inv, x[3] * inv), __NV_SATFINITE, __NV_E4M3);
    return a | z << 16;
  }
  // A word's codes times 2^e, e <= 15, rounded to codes (at most kMax up to
  // rounding).  In f16: a code has 4 significant bits, so the product is exact
  // wherever it is 2^-20 or more; below 2^-10 it rounds to 0 in any case.
  struct Shift {
    __half2 a;
    __device__ __forceinline__ explicit Shift(int e) {
      a = __half2half2(__ushort_as_half((unsigned short)(e > -15 ? (e + 15) << 10 : e >= -24 ? 1 << (e + 24) : 0)));
    }
    __device__ __forceinline__ uint32_t run(uint32_t w) const {
      uint32_t x, y;
      asm("{\n\t.reg .b16 lo, hi;\n\tmov.b32 {lo, hi}, %2;\n\tcvt.rn.f16x2.e4m3x2 %0, lo;\n\t"
          "cvt.rn.f16x2.e4m3x2 %1, hi;\n\t}"
          : "=r"(x), "=r"(y)
          : "r"(w));
      const __half2 p = __hmul2(*(const __half2 *)&x, a), q = __hmul2(*(const __half2 *)&y, a);
      asm("{\n\t.reg .b16 lo, hi;\n\tcvt.rn.satfinite.e4m3x2.f16x2 lo, %1;\n\tcvt.rn.satfinite.e4m3x2.f16x2 hi, %2;\n\t"
          "mov.b32 %0, {lo, hi};\n\t}"
          : "=r"(w)
          : "r"(*(const uint32_t *)&p), "r"(*(const uint32_t *)&q));
      return w;
    }
  };
};
struct I8 {
  static constexpr float kMax = 127.f;  // 1.984375 * 2^6
  static constexpr int kMaxExp = 6;
  static constexpr uint32_t kMaxMant = 0x7e0000u;
  __device__ __forceinline__ static uint32_t code(float x) { return (uint32_t)__float2int_rn(x) & 0xffu; }
  // Added to 1.5 * 2^23 a number rounds to an integer, whose low byte is the
  // sum's.
  __device__ __forceinline__ static uint32_t codes(const float *x, float inv) {
    const float magic = 12582912.f;
    const uint32_t a = __byte_perm(__float_as_uint(fmaf(x[0], inv, magic)), __float_as_uint(fmaf(x[1], inv, magic)), 0x40);
    const uint32_t z = __byte_perm(__float_as_uint(fmaf(x[2], inv, magic)), __float_as_uint(fmaf(x[3], inv, magic)), 0x40);
    return __byte_perm(a, z, 0x5410);
  }
  // A word's codes times 2^e, e <= 15, rounded: the same in f16, whose numbers from
  // 1024 to 2048 are the integers; the fused product has one rounding.
  struct Shift {
    __half2 a;
    __device__ __forceinline__ explicit Shift(int e) {
      a = __half2half2(__ushort_as_half((unsigned short)(e > -15 ? (e + 15) << 10 : 0)));  // below -8 all is 0
    }
    __device__ __forceinline__ uint32_t run(uint32_t w) const {
      const __half2 bias = __half2half2(__ushort_as_half(0x6480)), magic = __half2half2(__ushort_as_half(0x6600));
      const uint32_t x = (w & 0x00ff00ffu) ^ 0x64806480u, y = ((w >> 8) & 0x00ff00ffu) ^ 0x64806480u;
      const __half2 p = __hfma2(__hsub2(*(const __half2 *)&x, bias), a, magic);
      const __half2 q = __hfma2(__hsub2(*(const __half2 *)&y, bias), a, magic);
      return __byte_perm(*(const uint32_t *)&p, *(const uint32_t *)&q, 0x6240);
    }
  };
  __device__ __forceinline__ static void values(uint32_t w, float *x) {
    x[0] = (float)(int8_t)(w & 0xffu);
    x[1] = (float)(int8_t)((w >> 8) & 0xffu);
    x[2] = (float)(int8_t)((w >> 16) & 0xffu);
    x[3] = (float)(int8_t)(w >> 24);
  }
};

// The least power of two 2^e, e >= kMinExp, with amax <= F::kMax * 2^e (amax
// finite, >= 0).
template <typename F> __device__ __forceinline__ float block_scale(float amax) {
  const uint32_t u = __float_as_uint(amax);
  const int e = (int)(u >> 23) - 127 - F::kMaxExp + ((u & 0x7fffffu) > F::kMaxMant ? 1 : 0);
  return __uint_as_float((uint32_t)((e < kMinExp ? kMinExp : e) + 127) << 23);
}
// The exponent of a power of two.
__device__ __forceinline__ int exponent(float s) { return (int)(__float_as_uint(s) >> 23) - 127; }
// 1 / s of a power of two between 2^kMinExp and 2^126.
__device__ __forceinline__ float inverse_pow2(float s) { return __uint_as_float((254u << 23) - __float_as_uint(s)); }

// ------------------------------------------------------------ few new rows
constexpr int kFewRows = 8;  // rows of a sequence that are appended one at a time

// Rows lo .. hi-1 of head (b, h), all in one block, appended behind `len`
// entries by one warp, a lane taking D/32 neighbours of a row.  The block's
// earlier codes are read only where its scale grows.
template <typename F, int D>
__device__ __forceinline__ void append_rows(const View &c, bool is_v, const Rows &x, int b, int h, int len, int lo,
                                            int hi) {
  constexpr int E = D / 32;
  const int lane = threadIdx.x & 31, bh = b * c.H + h, blk = lo / kBlock, base = blk * kBlock;
  uint8_t *codes = (is_v ? c.V : c.K) + (size_t)bh * c.cap * D + lane * E;
  float *scale = (is_v ? c.Vsc : c.Ksc) + (size_t)bh * (c.cap / kBlock) + blk;
  auto row = [&](int t, uint32_t (&u)[2]) {  // bf16 bits, two to a word
    const __nv_bfloat16 *p = x.at(b, h, t - len) + lane * E;
    if constexpr (E == 4) {
      const uint2 w = *(const uint2 *)p;
      u[0] = w.x, u[1] = w.y;
    } else {
      u[0] = *(const uint32_t *)p, u[1] = 0u;
    }
  };
  const float before = base < len ? *scale : 0.f;
  uint32_t top = 0, odd = 0;
  for (int t = lo; t < hi; ++t) {
    uint32_t u[2];
    row(t, u);
#pragma unroll
    for (int e = 0; e < E; ++e) {
      const uint32_t y = (u[e >> 1] >> (16 * (e & 1))) & 0x7fffu;
      if (y < 0x7f80u)
        top = max(top, y);
      else
        odd = 1;
    }
  }
  top = __reduce_max_sync(0xffffffffu, top);
  if (odd) atomicOr(c.err, H2O_BERR_NONFINITE);
  const float after = fmaxf(before, block_scale<F>(__uint_as_float(top << 16)));
  const float inv = inverse_pow2(after);
  if (after > before && before > 0.f) {  // earlier entries of the block take the larger scale
    const typename F::Shift shift(exponent(before) - exponent(after));
    for (int t = base; t < len; ++t) {
      uint8_t *p = codes + (size_t)t * D;
      store_codes<E>(p, 0, shift.run(E == 4 ? *(const uint32_t *)p : *(const uint16_t *)p));
    }
  }
  for (int t = lo; t < hi; ++t) {
    uint32_t u[2], out = 0;
    row(t, u);
#pragma unroll
    for (int e = 0; e < E; ++e) {
      float y = (e & 1 ? bf16hi(u[e >> 1]) : bf16lo(u[e >> 1])) * inv;
      y = y != y ? 0.f : fminf(fmaxf(y, -F::kMax), F::kMax);
      out |= F::code(y) << (8 * e);
    }
    store_codes<E>(codes + (size_t)t * D, 0, out);
  }
  if (lane == 0) *scale = after;
}

// A kernel launched behind this one with programmatic serialisation may start;
// what it reads of this one's results it reads after its own wait.
__device__ __forceinline__ void grid_launch_dependents() { asm volatile("griddepcontrol.launch_dependents;"); }
__device__ __forceinline__ void grid_dependency_wait() { asm volatile("griddepcontrol.wait;" ::: "memory"); }

// Launchers (each on the device that is current; arguments checked before).
cudaError_t launch_append(const View &c, const Lens &l, const Rows &k, const Rows &v, const int32_t *position,
                          const float *score, cudaStream_t st);
// kmap, vmap: the codes as rows of d bytes, boxes of kBlock rows (code_map).
cudaError_t launch_attend(const View &c, const Lens &l, const Rows &q, int causal, int accumulate, const Rows &out,
                          float *lse, const CUtensorMap &kmap, const CUtensorMap &vmap, cudaStream_t st);
// Append and causal attention (k, v, position as in launch_append, no scores),
// or attention alone (k, v null), in one launch where a CTA can hold a head:
// head_fits says whether.
bool head_fits(const View &c, int n);
cudaError_t launch_head(const View &c, const Lens &l, const Rows &q, const Rows *k, const Rows *v,
                        const int32_t *position, int causal, int accumulate, const Rows &out, float *lse,
                        const CUtensorMap &kmap, const CUtensorMap &vmap, cudaStream_t st);
size_t attend_scratch_bytes(int B, int H, int d, int max_rows, int sms);
cudaError_t launch_evict(const View &c, const int32_t *lengths, int k_heavy, int k_local, int n_sink, int score_mode,
                         const int32_t *position, int32_t *new_lengths, cudaStream_t st);

}  // namespace blk
}  // namespace h2o
