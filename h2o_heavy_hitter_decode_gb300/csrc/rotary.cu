// rotary.cu — norm and rotation of query and key rows (h2o_rotate in
// include/h2o.h): the kernel, its argument checks and its launch.
//
//   y = x / sqrt(mean x^2 + eps) * w;  (y_a, y_b) turned by position * frequency
//
// A warp takes some heads of one token, or of several where a token has few: a
// row is held by d / 16 lanes, 16 elements each, arranged so that both halves of
// a pair are one lane's.  The
// sines and cosines of a lane's 8 pairs depend on the token alone: they are
// computed once and used for all the warp's heads.  Angles: position times the
// 64-bit fraction of a turn wraps at whole turns by itself, and its upper 32
// bits go through sincospif, 24 of them as its argument.
//
// Bound by memory: 16 prompts of 8,192 tokens, 32 query and 32 key heads of 128
// (4.3 GB) 649 us, 98 % of the copy rate, with five CTAs an SM (four 690, six
// 717 with spills); 6,771 patches of 16 and 16 heads of 64 in fp32 23 us, 69 %,
// by the way from positions to sines to stores, 2.2 waves of it (1,693 CTAs).
// One token by latency, 2.7 us.
#include <cstdint>

#include "common.cuh"
#include "rows.h"

namespace h2o {
namespace {

constexpr int kWarps = 4;

struct Args {
  h2o_rotary r;
  int B, n, heads[2];
  const void *in[2];
  void *out[2];
  int64_t sin[2][3], sout[2][3];  // strides b, h, t
  const int32_t *position, *counts;
  int per_token;
  int chunks[2];  // warps that share a token's query heads, and its key heads
  int both;       // or one warp has all of them
  int heads_at_once;
  int per;        // heads of a warp
};

// 8 elements at p.
__device__ __forceinline__ void load8(const __nv_bfloat16 *p, uint4 (&w)[1]) { w[0] = *(const uint4 *)p; }
__device__ __forceinline__ void load8(const float *p, uint4 (&w)[2]) {
  w[0] = *(const uint4 *)p, w[1] = *(const uint4 *)(p + 4);
}
template <typename T, int N> __device__ __forceinline__ void unpack8(const uint4 (&w)[N], float *x) {
#pragma unroll
  for (int i = 0; i < N; ++i) Unpack<T>::run(w[i], x + i * (8 / N));
}
__device__ __forceinline__ void store8(__nv_bfloat16 *p, const float *x) {
  uint32_t w[4];
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    const __nv_bfloat162 b = __floats2bfloat162_rn(x[2 * i], x[2 * i + 1]);
    w[i] = *(const uint32_t *)&b;
  }
  *(uint4 *)p = make_uint4(w[0], w[1], w[2], w[3]);
}
__device__ __forceinline__ void store8(float *p, const float *x) {
  *(float4 *)p = make_float4(x[0], x[1], x[2], x[3]);
  *(float4 *)(p + 4) = make_float4(x[4], x[5], x[6], x[7]);
}

// Rows of L lanes, by whole warps.  One whose mean square plus eps is below kTiny takes the power of two that brings the
// larger of its largest element and sqrt(eps) to 1 .. 2, which its norm takes out again; squares that are lost then are
// 2^-126 of the mean and below.  Returns the mean square plus eps; the other rows stay as they are.  Rare.
constexpr float kTiny = 0x1p-96f;
template <int L> __device__ __forceinline__ float rescale(float (&x)[16], float mean, float eps) {
  float top = sqrtf(eps);
#pragma unroll
  for (int e = 0; e < 16; ++e) top = fmaxf(top, fabsf(x[e]));
#pragma unroll
  for (int o = 1; o < L; o <<= 1) top = fmaxf(top, __shfl_xor_sync(0xffffffffu, top, o));
  const bool tiny = mean < kTiny && top > 0.f;
  // 2^k in two factors: k is up to 149 (the least number of 32 bits is 2^-149)
  const int k = tiny ? -ilogbf(top) : 0;
  const float up = ldexpf(1.f, k / 2), more = ldexpf(1.f, k - k / 2);
  float s = 0.f;
#pragma unroll
  for (int e = 0; e < 16; ++e) x[e] = x[e] * up * more, s = fmaf(x[e], x[e], s);
#pragma unroll
  for (int o = 1; o < L; o <<= 1) s += __shfl_xor_sync(0xffffffffu, s, o);
  return tiny ? s * (1.f / (16 * L)) + eps * up * more * up * more : mean;
}

// Few: a token has fewer heads than a warp takes at a time.
template <typename T, int D, int kAhead, bool Few>
__global__ void __launch_bounds__(kWarps * 32, 5) rotate_kernel(const Args a) {
  constexpr int L = D / 16;       // lanes of a row
  constexpr int kAtOnce = 32 / L;  // heads
  constexpr int N = 8 / VecN<T>::N;
  const int lane = threadIdx.x & 31, sub = lane % L;
  const int64_t item = (int64_t)blockIdx.x * kWarps + (threadIdx.x >> 5);
  const int all = a.both ? 1 : a.chunks[0] + a.chunks[1];
  // kAtOnce rows at a time: heads of a token, or where it has fewer, of several tokens.
  const int slot = lane / L, heads_at_once = Few ? a.heads_at_once : kAtOnce;
  int chunk = (int)(item % all);
  const int64_t token = item / all * (kAtOnce / heads_at_once) + slot / heads_at_once;
  bool is = token < (int64_t)a.B * a.n;
  if (!Few && !is) return;
  const int b = is ? (int)(token / a.n) : 0, t = is ? (int)(token - (int64_t)b * a.n) : 0;
  if (is && a.counts && t >= a.counts[b]) is = false;
  if (!__any_sync(0xffffffffu, is)) return;
  if (!Few) is = true;  // all lanes or none
  int which = chunk >= a.chunks[0];
  if (which) chunk -= a.chunks[0];

  // The lane's two runs of 8 elements: c0 and c1.  Pair e of them: elements e
  // of both, or (interleaved) neighbours in the 16 elements that they make.
  const h2o_rotary &r = a.r;
  const int turning = r.pairs / 8;  // lanes of a row that turn
  const bool turns = sub < turning && is;
  int c0, c1;
  if (r.interleaved || sub >= turning)
    c0 = 2 * sub, c1 = c0 + 1;
  else
    c0 = sub, c1 = sub + turning;
  float cs[8], sn[8], w[16];
  if (turns) {
#pragma unroll
    for (int e = 0; e < 8; ++e) {
      const int i = 8 * sub + e;
      int64_t p;
      if (a.per_token) {
        const int axis = r.axis ? min((int)r.axis[i], r.axes - 1) : 0;
        p = a.position[((int64_t)axis * a.B + b) * a.n + t];
      } else {
        p = (int64_t)a.position[b] + t;
      }
      // the nearest of 2^32 fractions of a turn, -1/2 .. 1/2; what its rounding to 24 bits loses, 2^-26 of a turn at most,
      // turns the sine and cosine on by itself: z of them, and z^2 below 2^-46 is nothing
      const uint64_t turn = (uint64_t)p * r.turns[i] + 0x80000000u;
      const int at = (int)(turn >> 32);
      const float high = (float)at, z = (float)(at - __float2int_rz(high)) * 1.46291808e-9f;  // 2 pi 2^-32
      float s, c;
      sincospif(high * 0x1p-31f, &s, &c);
      sn[e] = fmaf(z, c, s), cs[e] = fmaf(-z, s, c);
    }
  }
  for (;;) {
    const float *weight = which ? r.k_weight : r.q_weight;
#pragma unroll
    for (int e = 0; e < 16; ++e) w[e] = r.norm && weight ? weight[(e < 8 ? c0 : c1) * 8 + (e & 7)] : 1.f;

    const T *in = (const T *)a.in[which] + b * a.sin[which][0] + t * a.sin[which][2];
    T *out = (T *)a.out[which] + b * a.sout[which][0] + t * a.sout[which][2];
    const int end = min(a.heads[which], (chunk + 1) * a.per);
    // kAhead rows of a lane are on their way at once
    for (int first = chunk * a.per; first < end; first += heads_at_once * kAhead) {
      const int h0 = first + slot % heads_at_once;
      uint4 u[kAhead][2][N];
#pragma unroll
      for (int y = 0; y < kAhead; ++y) {
        const int h = h0 + y * heads_at_once;
        const T *src = in + (int64_t)(h < end ? h : 0) * a.sin[which][1];  // behind the last one head 0 again
        if (is) load8(src + c0 * 8, u[y][0]), load8(src + c1 * 8, u[y][1]);
      }
#pragma unroll
      for (int y = 0; y < kAhead; ++y) {
        const int h = h0 + y * heads_at_once;
        float x[16];
        unpack8<T>(u[y][0], x), unpack8<T>(u[y][1], x + 8);
        if (r.norm) {
          float s = 0.f;
#pragma unroll
          for (int e = 0; e < 16; ++e) s = fmaf(x[e], x[e], s);
#pragma unroll
          for (int o = 1; o < L; o <<= 1) s += __shfl_xor_sync(0xffffffffu, s, o);
          float mean = s * (1.f / D) + r.eps;
          // squares of tiny elements leave fp32's range downwards, which shows where eps does not hide it
          if (__any_sync(0xffffffffu, mean < kTiny)) mean = rescale<L>(x, mean, r.eps);
          const float f = rsqrtf(mean);
#pragma unroll
          for (int e = 0; e < 16; ++e) x[e] *= f * w[e];
        }
        if (turns) {
          auto turn = [&](int e, float &p, float &q) {
            const float p0 = p;
            p = p0 * cs[e] - q * sn[e];
            q = q * cs[e] + p0 * sn[e];
          };
          if (r.interleaved) {
#pragma unroll
            for (int e = 0; e < 8; ++e) turn(e, x[2 * e], x[2 * e + 1]);
          } else {
#pragma unroll
            for (int e = 0; e < 8; ++e) turn(e, x[e], x[e + 8]);
          }
        }
        if (h >= end || !is) continue;
        T *dst = out + (int64_t)h * a.sout[which][1];
        store8(dst + c0 * 8, x);
        store8(dst + c1 * 8, x + 8);
      }
    }
    if (!a.both || which) break;
    which = 1;
  }
}

template <typename T, int D> cudaError_t rotate_t(Args &a, int sms, cudaStream_t st) {
  constexpr int kAtOnce = 32 / (D / 16);
  const int64_t tokens = (int64_t)a.B * a.n;
  const int most = a.heads[0] > a.heads[1] ? a.heads[0] : a.heads[1];
  a.heads_at_once = 1;
  while (a.heads_at_once < kAtOnce && a.heads_at_once < most) a.heads_at_once *= 2;
  // Few tokens: their heads go to several warps each.
  int64_t share = (int64_t)sms * 16 / tokens;
  if (share < 1) share = 1;
  a.per = (int)(((most + share - 1) / share + a.heads_at_once - 1) / a.heads_at_once) * a.heads_at_once;
  for (int i = 0; i < 2; ++i) a.chunks[i] = (a.heads[i] + a.per - 1) / a.per;
  // Many tokens: queries and keys by one warp, under the same sines.
  a.both = share == 1 && a.heads[0] > 0 && a.heads[1] > 0;
  const int at_once = kAtOnce / a.heads_at_once;  // tokens of a warp
  const int64_t ctas = ((tokens + at_once - 1) / at_once * (a.both ? 1 : a.chunks[0] + a.chunks[1]) + kWarps - 1) / kWarps;
  if (ctas > 0x7fffffff) return cudaErrorInvalidConfiguration;
  // 64 bytes a lane on their way where a warp has rows enough (8K prompts 803 -> 708 us), else less code (one token 3.1 -> 2.3)
  const dim3 grid((unsigned)ctas);
  if (a.heads_at_once < kAtOnce)
    rotate_kernel<T, D, 1, true><<<grid, kWarps * 32, 0, st>>>(a);
  else if (a.per > kAtOnce)
    rotate_kernel<T, D, 4 * VecN<T>::N / 8, false><<<grid, kWarps * 32, 0, st>>>(a);
  else
    rotate_kernel<T, D, 1, false><<<grid, kWarps * 32, 0, st>>>(a);
  return cudaGetLastError();
}

}  // namespace
}  // namespace h2o

extern "C" h2o_status h2o_rotate(const h2o_rotary *r, h2o_dtype dtype, int B, int n, int q_heads, int k_heads,
                                 const h2o_rows *q, const h2o_rows *k, const int32_t *position, int per_token,
                                 const int32_t *counts, const h2o_rows *q_out, const h2o_rows *k_out,
                                 void *cuda_stream) {
  using namespace h2o;
  if (!r || (dtype != H2O_F32 && dtype != H2O_BF16)) return H2O_EINVAL;
  if (r->d < 1 || r->pairs < 0 || r->axes < 1 || !(r->eps >= 0.f)) return H2O_EINVAL;
  if (r->d != 64 && r->d != 128) return H2O_EUNSUPPORTED;
  if (r->pairs % 8 || 2 * r->pairs > r->d) return H2O_EINVAL;
  if (r->pairs > 0 && (!r->turns || !aligned(r->turns, 8) || !position || !aligned(position, 4))) return H2O_EINVAL;
  if (!aligned(r->q_weight, 16) || !aligned(r->k_weight, 16) || !aligned(counts, 4)) return H2O_EINVAL;
  if (B < 1 || n < 1 || q_heads < 0 || k_heads < 0 || q_heads + (int64_t)k_heads < 1) return H2O_EINVAL;
  if (q_heads > (1 << 24) || k_heads > (1 << 24) || (int64_t)B * n > 0x7fffffffLL) return H2O_EINVAL;
  Args a = {};
  a.r = *r;
  a.B = B, a.n = n, a.position = position, a.counts = counts, a.per_token = per_token != 0;
  const int step = dtype == H2O_F32 ? 4 : 8;
  const h2o_rows *in[2] = {q, k}, *out[2] = {q_out, k_out};
  for (int i = 0; i < 2; ++i) {
    const int heads = a.heads[i] = i ? k_heads : q_heads;
    if (heads == 0) continue;
    if (!rows_fit(in[i], step) || !rows_fit(out[i], step) || !rows_apart(out[i], B, heads, n, r->d)) return H2O_EINVAL;
    a.in[i] = in[i]->data, a.out[i] = const_cast<void *>(out[i]->data);
    const int64_t si[3] = {in[i]->stride_b, in[i]->stride_h, in[i]->stride_t};
    const int64_t so[3] = {out[i]->stride_b, out[i]->stride_h, out[i]->stride_t};
    for (int x = 0; x < 3; ++x) a.sin[i][x] = si[x], a.sout[i][x] = so[x];
  }
  const int sms = num_sms_current_device();
  if (sms <= 0) {
    note_cuda_error(cudaGetLastError());
    return H2O_ECUDA;
  }
  cudaStream_t st = (cudaStream_t)cuda_stream;
  const cudaError_t e = dtype == H2O_F32 ? (r->d == 128 ? rotate_t<float, 128>(a, sms, st) : rotate_t<float, 64>(a, sms, st))
                                         : (r->d == 128 ? rotate_t<__nv_bfloat16, 128>(a, sms, st)
                                                        : rotate_t<__nv_bfloat16, 64>(a, sms, st));
  if (e != cudaSuccess) {
    note_cuda_error(e);
    return H2O_ECUDA;
  }
  return H2O_OK;
}
