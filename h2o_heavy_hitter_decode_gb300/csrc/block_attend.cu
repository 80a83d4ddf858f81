// block_attend.cu — attention of a group's query rows over a block-scaled
// 8-bit cache, each entry's weights added to its score.
//
//   s_rj = (q_r . code_j) ks_j / sqrt(d),  j < end_r
//   LSE_r = ln sum_j exp s_rj;  O_r = sum_j exp(s_rj - LSE_r) vs_j code_j
//   score_j += sum_r exp(s_rj - LSE_r)
//
// Rows r of a cached head: r = t * group + g for query token t and query head
// g of the group.  One CTA per cached head: the logits of every row go to
// scratch memory, then each row's maximum and sum, its output, and at the end
// the scores.
#include "block_cache.cuh"
#include "sm100.cuh"

namespace h2o {
namespace blk {
namespace {

constexpr int kThreads = 256;

__device__ __forceinline__ float block_reduce(float v, float *s, bool is_max) {
  v = is_max ? warp_max(v) : warp_sum(v);
  __syncthreads();
  if ((threadIdx.x & 31) == 0) s[threadIdx.x >> 5] = v;
  __syncthreads();
  v = s[0];
  for (int i = 1; i < kThreads / 32; ++i) v = is_max ? fmaxf(v, s[i]) : v + s[i];
  return v;
}

template <typename F, int D>
__global__ void __launch_bounds__(kThreads) attend_kernel(const View c, const Lens l, const Rows q, int causal,
                                                          int accumulate, const Rows out, float *__restrict__ lse) {
  __shared__ float qs[D];
  __shared__ float red[kThreads / 32];
  __shared__ float acc[kThreads];
  const int bh = blockIdx.x, b = bh / c.H, h = bh - b * c.H, tid = threadIdx.x;
  const Seq s = seq_of(l, b);
  if (!s.ok && tid == 0) atomicOr(c.err, H2O_BERR_RANGE);
  const int rows = s.cnt * c.group;
  const uint8_t *K = c.K + (size_t)bh * c.cap * D, *V = c.V + (size_t)bh * c.cap * D;
  const float *ks = c.Ksc + (size_t)bh * (c.cap / kBlock), *vs = c.Vsc + (size_t)bh * (c.cap / kBlock);
  float *logits = c.logits + (size_t)bh * c.max_rows * c.cap;
  for (int r = 0; r < rows; ++r) {
    const int t = r / c.group, hq = h * c.group + r % c.group;
    const int end = causal ? s.total - s.cnt + t + 1 : s.total;
    float *lg = logits + (size_t)r * c.cap;
    __syncthreads();
    if (tid < D) qs[tid] = __bfloat162float(q.at(b, hq, t)[tid]) * rsqrtf((float)D) * kLog2e;
    __syncthreads();
    float m = -INFINITY;
    for (int j = tid; j < s.total; j += kThreads) {
      float dot = 0.f;
      for (int i = 0; i < D; i += 4) {
        float x[4];
        F::values(*(const uint32_t *)(K + (size_t)j * D + i), x);
        for (int e = 0; e < 4; ++e) dot = fmaf(qs[i + e], x[e], dot);
      }
      dot = j < end ? dot * ks[j / kBlock] : -INFINITY;
      lg[j] = dot;
      m = fmaxf(m, dot);
    }
    m = block_reduce(m, red, true);
    const float mu = m == -INFINITY ? 0.f : m;
    float sum = 0.f;
    for (int j = tid; j < end; j += kThreads) sum += exp2f(lg[j] - mu);
    sum = block_reduce(sum, red, false);
    const float lse2 = mu + log2f(sum);
    const int dim = tid % D;
    float o = 0.f;
    for (int j = tid / D; j < end; j += kThreads / D) {
      float x[4];
      F::values(*(const uint32_t *)(V + (size_t)j * D + (dim & ~3)), x);
      o = fmaf(exp2f(lg[j] - lse2) * vs[j / kBlock], x[dim & 3], o);
    }
    acc[tid] = o;
    __syncthreads();
    if (tid < D) {
      for (int i = tid + D; i < kThreads; i += D) o += acc[i];
      ((__nv_bfloat16 *)out.at(b, hq, t))[tid] = __float2bfloat16_rn(o);
    }
    if (lse && tid == 0) lse[((size_t)b * c.H * c.group + hq) * l.n + t] = lse2 * kLn2;
    for (int j = tid; j < s.total; j += kThreads) lg[j] = j < end ? exp2f(lg[j] - lse2) : 0.f;
  }
  if (!accumulate) return;
  __syncthreads();
  for (int j = tid; j < s.total; j += kThreads) {
    float w = 0.f;
    for (int r = 0; r < rows; ++r) w += logits[(size_t)r * c.cap + j];
    c.score[(size_t)bh * c.cap + j] += w;
  }
}

template <typename F, int D>
cudaError_t attend_t(const View &c, const Lens &l, const Rows &q, int causal, int accumulate, const Rows &out,
                     float *lse, cudaStream_t st) {
  attend_kernel<F, D><<<c.B * c.H, kThreads, 0, st>>>(c, l, q, causal, accumulate, out, lse);
  return cudaGetLastError();
}

}  // namespace

cudaError_t launch_attend(const View &c, const Lens &l, const Rows &q, int causal, int accumulate, const Rows &out,
                          float *lse, cudaStream_t st) {
  if (c.kv == H2O_KV_E4M3)
    return c.d == 128 ? attend_t<E4M3, 128>(c, l, q, causal, accumulate, out, lse, st)
                      : attend_t<E4M3, 64>(c, l, q, causal, accumulate, out, lse, st);
  return c.d == 128 ? attend_t<I8, 128>(c, l, q, causal, accumulate, out, lse, st)
                    : attend_t<I8, 64>(c, l, q, causal, accumulate, out, lse, st);
}

}  // namespace blk
}  // namespace h2o
