// block_evict.cu — a block-scaled 8-bit cache cut down to its k_heavy
// highest-ranking entries and its k_local last ones.
//
// select_kernel: keys mapped to unsigned integers that order like them; a
// four-pass radix select (8-bit digits) finds the threshold and how many of
// the entries equal to it stay (the ones with the highest indices); one scan
// then gives the kept indices in order.  A head's candidates are shared out
// over a cluster of up to 8 CTAs where there are few heads; each CTA reads its
// share once and keeps the keys in shared memory, and the digits' counts meet
// over distributed shared memory.
//
// move_kernel: entry i of the result comes from index src(i) >= i, so a round
// of consecutive destination blocks, each read into registers by a warp, may
// be written once every warp of the round has read: later rounds read only
// behind what was written.  That makes the move in place with one barrier a
// round (the CTA's, or the cluster's where few heads share the device) and no
// copy of the cache.  Every destination block gets a fresh scale from the
// values it receives; where that equals its sources' scale, as mostly, the
// codes go over unchanged.
#include <cooperative_groups.h>

#include "block_cache.cuh"

namespace h2o {
namespace blk {
namespace {

namespace cg = cooperative_groups;

// Keys ordered as unsigned integers; a NaN below everything, -0 as +0.
__device__ __forceinline__ uint32_t order_bits(float x) {
  x = x != x ? -INFINITY : x + 0.f;
  const uint32_t u = __float_as_uint(x);
  return u & 0x80000000u ? ~u : u | 0x80000000u;
}

struct Args {
  View c;
  const int32_t *lengths, *position;
  int32_t *new_lengths;
  int kh, kl, n_sink, mode;
  int held;  // keys a CTA of select_kernel has room for
};

constexpr int kSelThreads = 512;
constexpr int kSelWarps = kSelThreads / 32;
constexpr int kHists = 4;  // histograms of a CTA (each for a quarter of its warps)

template <int P>
__global__ void __launch_bounds__(kSelThreads) select_kernel(const Args a) {
  extern __shared__ uint32_t keys[];
  __shared__ unsigned hist[kHists][256];
  __shared__ unsigned sums[2][256];  // this CTA's counts, by pass parity
  __shared__ unsigned total[256];
  __shared__ unsigned s_digit, s_want, s_eq;
  __shared__ int s_warp[2][kSelWarps];
  __shared__ int s_count[2];  // this CTA's entries above and at the threshold
  cg::cluster_group cluster = cg::this_cluster();
  const View &c = a.c;
  const int rank = P > 1 ? (int)cluster.block_rank() : 0;
  const int bh = blockIdx.x / P, b = bh / c.H, tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
  const int len = a.lengths[b], k = a.kh + a.kl;
  const bool ok = len >= 0 && len <= c.cap;
  if (bh == b * c.H && rank == 0 && tid == 0) {
    a.new_lengths[b] = ok ? min(len, k) : len;
    if (!ok) atomicOr(c.err, H2O_BERR_RANGE);
  }
  if (!ok || len <= k || a.kh == 0) return;  // the whole cluster
  const int nc = len - a.kl;  // candidates 0 .. nc-1, this CTA's lo .. hi-1
  const int share = (nc + P - 1) / P, lo = min(nc, rank * share), hi = min(nc, lo + share), n = hi - lo;
  const int32_t *pos = c.pos + (size_t)bh * c.cap + lo;
  const float *score = c.score + (size_t)bh * c.cap + lo;
  int32_t *kept = c.kept + (size_t)bh * c.cap;
  const int p = a.position ? a.position[b] : len;
  auto read_key = [&](int j) -> uint32_t {
    float v = score[j];
    if (a.n_sink > 0 || a.mode) {
      const int pj = pos[j];
      if (pj < a.n_sink) return 0xffffffffu;
      if (a.mode) {
        const int seen = p - pj;
        v = __fdiv_rn(v, (float)(seen > 1 ? seen : 1));
      }
    }
    return order_bits(v);
  };
  for (int j = tid; j < min(n, a.held); j += kSelThreads) keys[j] = read_key(j);
  auto key_of = [&](int j) -> uint32_t { return j < a.held ? keys[j] : read_key(j); };

  uint32_t prefix = 0, pmask = 0;
  unsigned want = (unsigned)a.kh, eq_total = 0;
#pragma unroll 1
  for (int pass = 0; pass < 4; ++pass) {
    const int shift = 24 - 8 * pass;
    for (int i = tid; i < kHists * 256; i += kSelThreads) (&hist[0][0])[i] = 0u;
    __syncthreads();
    unsigned *mine = hist[warp & (kHists - 1)];
    for (int j = tid; j < n; j += kSelThreads) {
      const uint32_t key = key_of(j);
      if ((key & pmask) == prefix) atomicAdd(&mine[(key >> shift) & 255u], 1u);
    }
    __syncthreads();
    if (tid < 256) {
      unsigned t = 0;
#pragma unroll
      for (int i = 0; i < kHists; ++i) t += hist[i][tid];
      sums[pass & 1][tid] = t;
      if (P == 1) total[tid] = t;
    }
    if (P > 1) {
      cluster.sync();
      if (tid < 256) {
        unsigned t = 0;
#pragma unroll
        for (int i = 0; i < P; ++i) t += *cluster.map_shared_rank(&sums[pass & 1][tid], i);
        total[tid] = t;
      }
    }
    __syncthreads();
    if (warp == 0) {  // the digit d with count(> d) < want <= count(>= d); lane 0 has the highest digits
      unsigned own = 0;
#pragma unroll
      for (int i = 0; i < 8; ++i) own += total[255 - lane * 8 - i];
      unsigned run = own;
#pragma unroll
      for (int o = 1; o < 32; o <<= 1) {
        const unsigned x = __shfl_up_sync(0xffffffffu, run, o);
        if (lane >= o) run += x;
      }
      const unsigned above = run - own;
      if (above < want && want <= run) {
        unsigned cum = above;
        int d = 255 - lane * 8;
        while (cum + total[d] < want) cum += total[d--];
        s_digit = (unsigned)d;
        s_want = want - cum;
        s_eq = total[d];
      }
    }
    __syncthreads();
    prefix |= s_digit << shift;
    pmask |= 255u << shift;
    want = s_want;
    eq_total = s_eq;
    __syncthreads();
  }

  // Each thread scans a run of consecutive candidates (of odd length: no bank conflicts).
  const int run = (n + kSelThreads - 1) / kSelThreads | 1;
  const int j0 = min(n, tid * run), j1 = min(n, j0 + run);
  int above = 0, equal = 0;
  for (int j = j0; j < j1; ++j) {
    const uint32_t key = key_of(j);
    above += key > prefix;
    equal += key == prefix;
  }
  int ia = above, ie = equal;
#pragma unroll
  for (int o = 1; o < 32; o <<= 1) {
    const int x = __shfl_up_sync(0xffffffffu, ia, o), y = __shfl_up_sync(0xffffffffu, ie, o);
    if (lane >= o) ia += x, ie += y;
  }
  if (lane == 31) s_warp[0][warp] = ia, s_warp[1][warp] = ie;
  __syncthreads();
  int before_a = ia - above, before_e = ie - equal;
  for (int w = 0; w < warp; ++w) before_a += s_warp[0][w], before_e += s_warp[1][w];
  if (P > 1) {
    if (tid == kSelThreads - 1) s_count[0] = before_a + above, s_count[1] = before_e + equal;
    cluster.sync();
    for (int i = 0; i < rank; ++i) {
      before_a += *cluster.map_shared_rank(&s_count[0], i);
      before_e += *cluster.map_shared_rank(&s_count[1], i);
    }
  }
  const int drop = (int)(eq_total - want);  // the first of the equal ones go
  for (int j = j0; j < j1; ++j) {
    const uint32_t key = key_of(j);
    bool keep = key > prefix;
    const int slot = before_a + max(0, before_e - drop);
    if (keep) ++before_a;
    if (key == prefix) keep = before_e++ >= drop;
    if (keep && slot < a.kh) kept[slot] = lo + j;
  }
  if (P > 1) cluster.sync();  // no CTA leaves while its counts are read
}

// The largest magnitude among codes, kept as code numbers.
template <typename F> struct TopCode;
template <> struct TopCode<E4M3> {  // a code's low 7 bits order like its magnitude
  uint32_t m = 0;
  __device__ __forceinline__ void add(uint32_t w) {
    m = __vmaxu2(m, w & 0x007f007fu);
    m = __vmaxu2(m, (w >> 8) & 0x007f007fu);
  }
  __device__ __forceinline__ float value() const {
    float x[4];
    E4M3::values(max(m & 0xffffu, m >> 16), x);
    return x[0];
  }
};
template <> struct TopCode<I8> {  // codes + 128, largest and least
  uint32_t hi = 0x00800080u, lo = 0x00800080u;
  __device__ __forceinline__ void add(uint32_t w) {
    w ^= 0x80808080u;
    const uint32_t x = w & 0x00ff00ffu, y = (w >> 8) & 0x00ff00ffu;
    hi = __vmaxu2(hi, __vmaxu2(x, y));
    lo = __vminu2(lo, __vminu2(x, y));
  }
  __device__ __forceinline__ float value() const {
    const int top = max((int)(hi & 0xffffu), (int)(hi >> 16)) - 128, low = 128 - min((int)(lo & 0xffffu), (int)(lo >> 16));
    return (float)max(top, low);
  }
};

template <typename F, int D, int P, int W>
__global__ void __launch_bounds__(W * 32, 16 / W) move_kernel(const Args a) {
  constexpr int LPR = D / 16;       // lanes per row, 16 codes each
  constexpr int RPI = 32 / LPR;     // rows per load of the warp
  constexpr int IT = kBlock / RPI;  // loads
  cg::cluster_group cluster = cg::this_cluster();
  const View &c = a.c;
  const int rank = P > 1 ? (int)cluster.block_rank() : 0;
  const int bh = blockIdx.x / P, b = bh / c.H, lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  const int len = a.lengths[b], kh = a.kh, k = kh + a.kl;
  asm volatile("griddepcontrol.wait;" ::: "memory");  // the kept indices
  if (len < 0 || len > c.cap || len <= k) return;     // the whole cluster
  const int nc = len - a.kl;
  int32_t *pos = c.pos + (size_t)bh * c.cap;
  float *score = c.score + (size_t)bh * c.cap;
  const int32_t *kept = c.kept + (size_t)bh * c.cap;
  const size_t scales = (size_t)bh * (c.cap / kBlock);
  const int sub = lane % LPR, row0 = lane / LPR;
  const int blocks = (k + kBlock - 1) / kBlock;
  // Source of the lane's entry of a block; 0 behind the last one.
  auto source = [&](int i) { return i < kh ? min(max(kept[i], 0), len - 1) : i < k ? i - kh + nc : 0; };
  int blk = rank * W + warp;
  int src_next = source(min(blk * kBlock + lane, k));
  for (int round = 0; round < blocks; round += P * W, blk += P * W) {
    const int base = blk * kBlock;
    const bool work = blk < blocks;
    const int own = base + lane;
    const int src_own = src_next;
    src_next = blk + P * W < blocks ? source(own + P * W * kBlock) : 0;
    uint4 w[2][IT];
    float sc[2][IT], to[2];
    int pos_own = 0;
    float score_own = 0.f;
    bool same = true;
    if (work) {
#pragma unroll
      for (int kv = 0; kv < 2; ++kv) {
        const uint8_t *codes = (kv ? c.V : c.K) + (size_t)bh * c.cap * D + sub * 16;
        const float *scale = (kv ? c.Vsc : c.Ksc) + scales;
#pragma unroll
        for (int i = 0; i < IT; ++i) {
          const int src = __shfl_sync(0xffffffffu, src_own, i * RPI + row0);
          const bool in = base + i * RPI + row0 < k;
          w[kv][i] = in ? *(const uint4 *)(codes + (size_t)src * D) : make_uint4(0u, 0u, 0u, 0u);
          sc[kv][i] = in ? scale[src / kBlock] : 0.f;
        }
      }
      if (own < k) {
        pos_own = pos[src_own];
        score_own = score[src_own];
      }
#pragma unroll
      for (int kv = 0; kv < 2; ++kv) {
        float amax = 0.f;
#pragma unroll
        for (int i = 0; i < IT; ++i) {
          TopCode<F> top;
          top.add(w[kv][i].x), top.add(w[kv][i].y), top.add(w[kv][i].z), top.add(w[kv][i].w);
          amax = fmaxf(amax, top.value() * sc[kv][i]);
        }
        to[kv] = block_scale<F>(warp_max(amax));
#pragma unroll
        for (int i = 0; i < IT; ++i) same = same && (sc[kv][i] == to[kv] || sc[kv][i] == 0.f);
      }
      if (!__all_sync(0xffffffffu, same)) {
#pragma unroll
        for (int kv = 0; kv < 2; ++kv) {
#pragma unroll
          for (int i = 0; i < IT; ++i) {
            if (sc[kv][i] == to[kv]) continue;
            const typename F::Shift shift(exponent(sc[kv][i]) - exponent(to[kv]));
            w[kv][i] = make_uint4(shift.run(w[kv][i].x), shift.run(w[kv][i].y), shift.run(w[kv][i].z), shift.run(w[kv][i].w));
          }
        }
      }
    }
    if (P > 1)
      cluster.sync();
    else
      __syncthreads();  // every warp of the round has read its sources
    if (work) {
#pragma unroll
      for (int kv = 0; kv < 2; ++kv) {
        uint8_t *codes = (kv ? c.V : c.K) + ((size_t)bh * c.cap + base) * D + sub * 16;
#pragma unroll
        for (int i = 0; i < IT; ++i)
          if (base + i * RPI + row0 < k) *(uint4 *)(codes + (size_t)(i * RPI + row0) * D) = w[kv][i];
        if (lane == 0) ((kv ? c.Vsc : c.Ksc) + scales)[blk] = to[kv];
      }
      if (own < k) {
        pos[own] = pos_own;
        score[own] = score_own;
      }
    }
  }
}

template <typename K>
cudaError_t launch_cluster(K *kernel, int ctas, int cluster, int threads, int smem, bool after, cudaStream_t st,
                           const Args &a) {
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3(ctas);
  cfg.blockDim = dim3(threads);
  cfg.dynamicSmemBytes = smem;
  cfg.stream = st;
  cudaLaunchAttribute at[2];
  at[0].id = cudaLaunchAttributeClusterDimension;
  at[0].val.clusterDim = {(unsigned)cluster, 1, 1};
  at[1].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  at[1].val.programmaticStreamSerializationAllowed = 1;
  cfg.attrs = at;
  cfg.numAttrs = after ? 2 : 1;
  return cudaLaunchKernelEx(&cfg, kernel, a);
}

template <int P> cudaError_t select_p(Args a, cudaStream_t st) {
  constexpr int kRoom = 49152;  // keys, 192 KB
  const int share = (a.c.cap + P - 1) / P;
  a.held = share < kRoom ? share : kRoom;
  const int smem = a.held * 4;
  cudaError_t e = cudaFuncSetAttribute(select_kernel<P>, cudaFuncAttributeMaxDynamicSharedMemorySize, smem);
  if (e != cudaSuccess) return e;
  return launch_cluster(select_kernel<P>, a.c.B * a.c.H * P, P, kSelThreads, smem, false, st, a);
}

template <typename F, int D> cudaError_t move_t(const Args &a, cudaStream_t st) {
  // Few heads: a cluster of 8 wide CTAs for each, so that a round covers 128 blocks; many: one CTA of 8 warps, two
  // to an SM, whose barriers then overlap.
  const int heads = a.c.B * a.c.H;
  if (heads * 8 <= a.c.sms) return launch_cluster(move_kernel<F, D, 8, 16>, heads * 8, 8, 512, 0, true, st, a);
  if (heads * 2 <= a.c.sms) return launch_cluster(move_kernel<F, D, 4, 8>, heads * 4, 4, 256, 0, true, st, a);
  return launch_cluster(move_kernel<F, D, 1, 8>, heads, 1, 256, 0, true, st, a);
}

}  // namespace

cudaError_t launch_evict(const View &c, const int32_t *lengths, int kh, int kl, int n_sink, int mode,
                         const int32_t *position, int32_t *new_lengths, cudaStream_t st) {
  const Args a{c, lengths, position, new_lengths, kh, kl, n_sink, mode, 0};
  // Up to 8 CTAs share a head while that fills empty SMs and leaves each some thousand candidates.
  int p = 1;
  while (p < 8 && c.B * c.H * p * 2 <= 2 * c.sms && c.cap / p > 4096) p *= 2;
  cudaError_t e = p == 8 ? select_p<8>(a, st) : p == 4 ? select_p<4>(a, st) : p == 2 ? select_p<2>(a, st) : select_p<1>(a, st);
  if (e != cudaSuccess) return e;
  if (c.kv == H2O_KV_E4M3) return c.d == 128 ? move_t<E4M3, 128>(a, st) : move_t<E4M3, 64>(a, st);
  return c.d == 128 ? move_t<I8, 128>(a, st) : move_t<I8, 64>(a, st);
}

}  // namespace blk
}  // namespace h2o
