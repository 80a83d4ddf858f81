// block_evict.cu — a block-scaled 8-bit cache cut down to its k_heavy
// highest-ranking entries and its k_local last ones.
//
// One CTA per head.  Selection: keys mapped to unsigned integers that order
// like them; a four-pass radix select (8-bit digits) finds the threshold and
// how many of the entries equal to it stay (the ones with the highest
// indices); one scan gives the kept indices in order.  Move: entry i of the
// result comes from index src(i) >= i, so a round of consecutive destination
// blocks, each read into registers by a warp, may be written once every warp
// of the round has read: later rounds read only behind what was written.
// Every destination block gets a fresh scale from the values it receives.
#include "block_cache.cuh"

namespace h2o {
namespace blk {
namespace {

constexpr int kThreads = 512;
constexpr int kWarps = kThreads / 32;

// Keys ordered as unsigned integers; a NaN below everything, -0 as +0.
__device__ __forceinline__ uint32_t order_bits(float x) {
  x = x != x ? -INFINITY : x + 0.f;
  const uint32_t u = __float_as_uint(x);
  return u & 0x80000000u ? ~u : u | 0x80000000u;
}

template <typename F, int D>
__global__ void __launch_bounds__(kThreads, 1) evict_kernel(const View c, const int32_t *__restrict__ lengths, int kh,
                                                         int kl, int n_sink, int mode,
                                                         const int32_t *__restrict__ position,
                                                         int32_t *__restrict__ new_lengths) {
  __shared__ unsigned hist[256];
  __shared__ unsigned s_digit, s_want, s_eq;
  __shared__ int s_weq[kWarps], s_wkeep[kWarps];
  const int bh = blockIdx.x, b = bh / c.H, tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
  const int len = lengths[b], k = kh + kl;
  const bool ok = len >= 0 && len <= c.cap;
  if (bh == b * c.H && tid == 0) {
    new_lengths[b] = ok ? min(len, k) : len;
    if (!ok) atomicOr(c.err, H2O_BERR_RANGE);
  }
  if (!ok || len <= k) return;
  int32_t *pos = c.pos + (size_t)bh * c.cap;
  float *score = c.score + (size_t)bh * c.cap;
  int32_t *kept = c.kept + (size_t)bh * c.cap;
  const int nc = len - kl;  // candidates 0 .. nc-1
  const int p = position ? position[b] : len;
  auto key_of = [&](int j) -> uint32_t {
    const int pj = pos[j];
    if (pj < n_sink) return 0xffffffffu;
    float v = score[j];
    if (mode) {
      const int seen = p - pj;
      v = __fdiv_rn(v, (float)(seen > 1 ? seen : 1));
    }
    return order_bits(v);
  };

  uint32_t prefix = 0, pmask = 0;
  unsigned want = (unsigned)kh, eq_total = 0;
  if (kh > 0) {
    for (int shift = 24; shift >= 0; shift -= 8) {
      for (int i = tid; i < 256; i += kThreads) hist[i] = 0u;
      __syncthreads();
      for (int j = tid; j < nc; j += kThreads) {
        const uint32_t key = key_of(j);
        if ((key & pmask) == prefix) atomicAdd(&hist[(key >> shift) & 255u], 1u);
      }
      __syncthreads();
      if (tid == 0) {
        unsigned cum = 0;
        int d = 255;
        for (; d > 0; --d) {
          if (cum + hist[d] >= want) break;
          cum += hist[d];
        }
        s_digit = (unsigned)d;
        s_want = want - cum;
        s_eq = hist[d];
      }
      __syncthreads();
      prefix |= s_digit << shift;
      pmask |= 255u << shift;
      want = s_want;
      eq_total = s_eq;
      __syncthreads();
    }
  }
  const unsigned lt = (1u << lane) - 1u;
  int run_eq = 0, run_keep = 0;
  for (int j0 = 0; j0 < nc; j0 += kThreads) {
    const int j = j0 + tid;
    const uint32_t key = j < nc && kh > 0 ? key_of(j) : 0u;
    bool keep = j < nc && kh > 0 && key > prefix;
    const bool eq = j < nc && kh > 0 && key == prefix;
    const unsigned beq = __ballot_sync(0xffffffffu, eq);
    if (lane == 0) s_weq[warp] = __popc(beq);
    __syncthreads();
    int rank = run_eq + __popc(beq & lt), tile = 0;  // equals before this one
    for (int w = 0; w < kWarps; ++w) {
      if (w < warp) rank += s_weq[w];
      tile += s_weq[w];
    }
    run_eq += tile;
    if (eq) keep = rank >= (int)(eq_total - want);
    const unsigned bk = __ballot_sync(0xffffffffu, keep);
    if (lane == 0) s_wkeep[warp] = __popc(bk);
    __syncthreads();
    int slot = run_keep + __popc(bk & lt);
    tile = 0;
    for (int w = 0; w < kWarps; ++w) {
      if (w < warp) slot += s_wkeep[w];
      tile += s_wkeep[w];
    }
    run_keep += tile;
    if (keep && slot < kh) kept[slot] = j;
  }
  if (run_keep != kh) {  // cannot happen: the threshold admits exactly k_heavy
    if (tid == 0) atomicOr(c.err, H2O_BERR_INTERNAL);
    return;
  }
  __syncthreads();

  constexpr int LPR = D / 16;       // lanes per row, 16 codes each
  constexpr int RPI = 32 / LPR;     // rows per load of the warp
  constexpr int IT = kBlock / RPI;  // loads
  const int sub = lane % LPR, row0 = lane / LPR;
  const int blocks = (k + kBlock - 1) / kBlock;
  for (int round = 0; round < blocks; round += kWarps) {
    const int blk = round + warp, base = blk * kBlock;
    const bool work = blk < blocks;
    const int i_own = base + lane;
    const bool own = work && i_own < k;
    const int src_own = own ? (i_own < kh ? kept[i_own] : i_own - kh + nc) : 0;
    const int pos_own = own ? pos[src_own] : 0;
    const float score_own = own ? score[src_own] : 0.f;
    uint4 w[2][IT];
    float sc[2][IT], inv[2];
    float out_scale[2];
#pragma unroll
    for (int kv = 0; kv < 2; ++kv) {
      const uint8_t *codes = (kv ? c.V : c.K) + (size_t)bh * c.cap * D;
      const float *scale = (kv ? c.Vsc : c.Ksc) + (size_t)bh * (c.cap / kBlock);
      float amax = 0.f;
#pragma unroll
      for (int i = 0; i < IT; ++i) {
        const int src = __shfl_sync(0xffffffffu, src_own, i * RPI + row0);
        const bool in = work && base + i * RPI + row0 < k;
        w[kv][i] = in ? *(const uint4 *)(codes + (size_t)src * D + sub * 16) : make_uint4(0u, 0u, 0u, 0u);
        sc[kv][i] = in ? scale[src / kBlock] : 0.f;
      }
#pragma unroll
      for (int i = 0; i < IT; ++i) {
        float top = 0.f;
#pragma unroll
        for (int e = 0; e < 4; ++e) {
          float x[4];
          F::values((&w[kv][i].x)[e], x);
          top = fmaxf(top, fmaxf(fmaxf(fabsf(x[0]), fabsf(x[1])), fmaxf(fabsf(x[2]), fabsf(x[3]))));
        }
        amax = fmaxf(amax, top * sc[kv][i]);
      }
      out_scale[kv] = block_scale<F>(warp_max(amax));
      inv[kv] = inverse_pow2(out_scale[kv]);
    }
    __syncthreads();  // every warp has read its sources
#pragma unroll
    for (int kv = 0; kv < 2; ++kv) {
      uint8_t *codes = (kv ? c.V : c.K) + ((size_t)bh * c.cap + base) * D;
#pragma unroll
      for (int i = 0; i < IT; ++i) {
        const int r = i * RPI + row0;
        const float ratio = fminf(sc[kv][i] * inv[kv], 3e38f);  // finite for rows of zeros under a large scale
        uint4 u;
#pragma unroll
        for (int e = 0; e < 4; ++e) {
          float x[4];
          F::values((&w[kv][i].x)[e], x);
          (&u.x)[e] = F::code(x[0] * ratio) | F::code(x[1] * ratio) << 8 | F::code(x[2] * ratio) << 16 |
                      F::code(x[3] * ratio) << 24;
        }
        if (work && base + r < k) *(uint4 *)(codes + (size_t)r * D + sub * 16) = u;
      }
      if (work && lane == 0) ((kv ? c.Vsc : c.Ksc) + (size_t)bh * (c.cap / kBlock))[blk] = out_scale[kv];
    }
    if (own) {
      pos[i_own] = pos_own;
      score[i_own] = score_own;
    }
    __syncthreads();
  }
}

template <typename F, int D>
cudaError_t evict_t(const View &c, const int32_t *lengths, int kh, int kl, int n_sink, int mode,
                    const int32_t *position, int32_t *new_lengths, cudaStream_t st) {
  evict_kernel<F, D><<<c.B * c.H, kThreads, 0, st>>>(c, lengths, kh, kl, n_sink, mode, position, new_lengths);
  return cudaGetLastError();
}

}  // namespace

cudaError_t launch_evict(const View &c, const int32_t *lengths, int kh, int kl, int n_sink, int mode,
                         const int32_t *position, int32_t *new_lengths, cudaStream_t st) {
  if (c.kv == H2O_KV_E4M3)
    return c.d == 128 ? evict_t<E4M3, 128>(c, lengths, kh, kl, n_sink, mode, position, new_lengths, st)
                      : evict_t<E4M3, 64>(c, lengths, kh, kl, n_sink, mode, position, new_lengths, st);
  return c.d == 128 ? evict_t<I8, 128>(c, lengths, kh, kl, n_sink, mode, position, new_lengths, st)
                    : evict_t<I8, 64>(c, lengths, kh, kl, n_sink, mode, position, new_lengths, st);
}

}  // namespace blk
}  // namespace h2o
