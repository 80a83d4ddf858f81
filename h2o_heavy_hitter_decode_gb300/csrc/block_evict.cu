// block_evict.cu — a block-scaled 8-bit cache cut down to its k_heavy
// highest-ranking entries and its k_local last ones.
//
// One launch; a CTA, or a cluster of up to 16 where there are few heads, takes
// a head through both phases, so that on a busy device one head's selection
// (arithmetic) runs under its neighbours' move (memory).
//
// Selection: keys mapped to unsigned integers that order like them; a
// three-pass radix select (digits of 11, 11 and 10 bits: the first one spreads
// scores of a few octaves over four digits an octave, where atomics on 8-bit
// digits queued up) finds the threshold and how many of the entries equal to
// it stay (the ones with the highest indices); one scan then gives the kept
// indices in order.  A CTA reads its share of the candidates once and keeps
// the keys in shared memory; the digits' counts of a cluster meet over
// distributed shared memory.
//
// Move: entry i of the result comes from index src(i) >= i, so a round of
// consecutive destination blocks, each held by a warp, may be written once
// every warp of the round has read: later rounds read only behind what was
// written.  That makes the move in place, with no copy of the cache.  A warp
// arrives at a round's barrier when it has read; it waits for that barrier
// before it writes only where this round's sources begin inside the round's
// own destination, else (once some entries are gone) for the round before.  A
// warp's items of a round are a block's K and V; those of its next block are on
// their way to shared memory (cp.async, each lane its own 16 bytes) meanwhile.
// Every destination block gets a fresh scale from the values it receives; rows
// whose scale it shares go over unchanged.
//
// Bound by memory in the move and by the first digit's atomics in the selection
// (1024 heads, 8,448 -> 1,690 entries: 174 us in all, 80 % of the copy rate; a
// selection alone takes 60 us, and part of it lies under other heads' moves); on
// few heads by latency (8 heads, 131,072 -> 26,214: 57 us, of it about 20 us
// selection).
#include <cooperative_groups.h>

#include "block_cache.cuh"
#include "sm100.cuh"

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

constexpr int kDigits = 2048;  // bins of the first digit
// Shared memory of a CTA where two share an SM (228 KB, 1 KB of it a CTA's own), and the kernel's static part of it.
constexpr int kSmemOfCta = 228 * 1024 / 2 - 1024;
template <int P> constexpr int kStatic = kDigits * 4 * (P > 1 ? 2 : 1) + (P > 1 ? kDigits / P * 8 : 0) + 256;

struct Args {
  View c;
  const int32_t *lengths, *position;
  int32_t *new_lengths;
  int kh, kl, n_sink, mode;
  int held;  // keys a CTA has room for
};

// The largest magnitude among codes, kept as code numbers.
template <typename F> struct TopCode;
template <> struct TopCode<E4M3> {  // a code's low 7 bits order like its magnitude
  uint32_t m = 0;
  __device__ __forceinline__ void add(uint32_t w) {
    m = __vmaxu2(m, __vmaxu2(w & 0x007f007fu, (w >> 8) & 0x007f007fu));
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

template <int P> __device__ __forceinline__ void head_sync(cg::cluster_group &cluster) {
  if constexpr (P > 1)
    cluster.sync();
  else
    __syncthreads();
}
// The barrier between the reads and the writes of rounds.  What was read is in
// registers when a warp arrives, so the warps only have to meet: a releasing
// arrival would make each round wait for the stores of the one before to reach
// L2.  One CTA: an mbarrier with an arrival for each warp.
template <int P> struct Rounds {
  uint64_t *bar;
  uint32_t phase = 0;
  bool pending = false, ok = true;
  __device__ __forceinline__ void arrive(int lane) {
    if constexpr (P > 1) {
      asm volatile("barrier.cluster.arrive.relaxed.aligned;" ::: "memory");
    } else {
      __syncwarp();
      if (lane == 0) sm100::mbar_arrive(bar);
    }
    pending = true;
  }
  __device__ __forceinline__ void wait() {
    if (!pending) return;
    if constexpr (P > 1) {
      asm volatile("barrier.cluster.wait.aligned;" ::: "memory");
    } else {
      ok = sm100::mbar_wait(bar, phase) && ok;
      phase ^= 1;
    }
    pending = false;
  }
};

// 16 bytes global -> shared, zeros where `in` is false.
__device__ __forceinline__ void copy16(uint32_t dst, const void *src, bool in) {
  asm volatile("cp.async.cg.shared.global [%0], [%1], 16, %2;" ::"r"(dst), "l"(src), "r"(in ? 16 : 0) : "memory");
}

template <typename F, int D, int P, int W>
__global__ void __launch_bounds__(W * 32, 2) evict_kernel(const Args a) {
  constexpr int kThreads = W * 32;
  constexpr int kOwn = kDigits / kThreads;
  extern __shared__ __align__(16) uint32_t dyn[];  // the keys, then the warps' row buffers
  __shared__ __align__(16) unsigned hist[P > 1 ? 2 : 1][kDigits];  // this CTA's counts, in a cluster by pass parity
  __shared__ __align__(16) unsigned totals[P > 1 ? 2 : 1][P > 1 ? kDigits / P : 4];  // the cluster's counts of a slice
  __shared__ unsigned s_digit, s_want, s_eq;
  __shared__ int s_warp[2][W];
  __shared__ unsigned s_sum[W];
  __shared__ __align__(8) uint64_t s_bar;
  __shared__ int s_count[2];  // this CTA's entries above and at the threshold
  static_assert(sizeof(hist) + sizeof(totals) + sizeof(s_warp) + sizeof(s_sum) + 64 <= kStatic<P>,
                "the room for keys leaves this out");
  cg::cluster_group cluster = cg::this_cluster();
  const View &c = a.c;
  const int rank = P > 1 ? (int)cluster.block_rank() : 0;
  const int bh = blockIdx.x / P, b = bh / c.H, tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
  const int len = a.lengths[b], kh = a.kh, k = a.kh + a.kl;
  const bool ok = len >= 0 && len <= c.cap;
  if (bh == b * c.H && rank == 0 && tid == 0) {
    a.new_lengths[b] = ok ? min(len, k) : len;
    if (!ok) atomicOr(c.err, H2O_BERR_RANGE);
  }
  if (!ok || len <= k) return;  // the whole cluster
  const int nc = len - a.kl;    // candidates 0 .. nc-1
  int32_t *pos = c.pos + (size_t)bh * c.cap;
  float *score = c.score + (size_t)bh * c.cap, *low = c.low + (size_t)bh * c.cap;
  int32_t *kept = c.kept + (size_t)bh * c.cap;

  if (kh > 0) {
    // this CTA's candidates lo .. lo + n - 1
    const int share = ((nc + P - 1) / P + 3) & ~3, lo = min(nc, rank * share), n = min(nc, lo + share) - lo;
    const int p = a.position ? a.position[b] : len;
    auto to_key = [&](float v, int j) -> uint32_t {
      if (a.n_sink > 0 || a.mode) {
        const int pj = pos[lo + j];
        if (pj < a.n_sink) return 0xffffffffu;
        if (a.mode) {
          const int seen = p - pj;
          v = __fdiv_rn(v, (float)(seen > 1 ? seen : 1));
        }
      }
      return order_bits(v);
    };
    auto key_of = [&](int j) -> uint32_t { return j < a.held ? dyn[j] : to_key(score[lo + j], j); };

    uint32_t prefix = 0, pmask = 0;
    unsigned want = (unsigned)kh, eq_total = 0;
#pragma unroll 1
    for (int pass = 0; pass < 3; ++pass) {
      const int shift = pass == 0 ? 21 : pass == 1 ? 10 : 0;
      const uint32_t dmask = pass == 2 ? 1023u : 2047u;
      unsigned *mine = hist[P > 1 ? pass & 1 : 0];
      for (int i = tid * 4; i < kDigits; i += kThreads * 4) *(uint4 *)(mine + i) = make_uint4(0u, 0u, 0u, 0u);
      __syncthreads();
      auto count = [&](uint32_t key) {
        if ((key & pmask) == prefix) atomicAdd(&mine[(key >> shift) & dmask], 1u);
      };
      const int whole = min(n, a.held) & ~3;
      if (pass == 0) {
        constexpr int kBatch = 8;  // fours of scores on their way at once
        for (int jb = tid * 4; jb < whole; jb += kThreads * 4 * kBatch) {
          float4 v[kBatch];
#pragma unroll
          for (int i = 0; i < kBatch; ++i) v[i] = *(const float4 *)(score + lo + min(jb + i * kThreads * 4, whole - 4));
#pragma unroll
          for (int i = 0; i < kBatch; ++i) {
            const int j = jb + i * kThreads * 4;
            if (j >= whole) break;
            const uint4 u = make_uint4(to_key(v[i].x, j), to_key(v[i].y, j + 1), to_key(v[i].z, j + 2), to_key(v[i].w, j + 3));
            *(uint4 *)(dyn + j) = u;
            count(u.x), count(u.y), count(u.z), count(u.w);
          }
        }
        for (int j = whole + tid; j < n; j += kThreads) {
          const uint32_t u = to_key(score[lo + j], j);
          if (j < a.held) dyn[j] = u;
          count(u);
        }
      } else {
#pragma unroll 4
        for (int j = tid * 4; j < whole; j += kThreads * 4) {
          const uint4 u = *(const uint4 *)(dyn + j);
          count(u.x), count(u.y), count(u.z), count(u.w);
        }
        for (int j = whole + tid; j < n; j += kThreads) count(key_of(j));
      }
      head_sync<P>(cluster);
      if constexpr (P > 1) {
        // Each CTA adds up its slice of the digits over the cluster, and every CTA then
        // reads all the slices.
        constexpr int kSlice = kDigits / P;
        for (int d = tid; d < kSlice; d += kThreads) {
          unsigned t = 0;
#pragma unroll
          for (int i = 0; i < P; ++i) t += *cluster.map_shared_rank(mine + rank * kSlice + d, i);
          totals[pass & 1][d] = t;
        }
        cluster.sync();
      }
      // The digit d with count(> d) < want <= count(>= d): thread i sums its digits, the highest ones first.
      unsigned own[kOwn], sum = 0;
      const int top = kDigits - kOwn * (tid + 1);  // its lowest digit
#pragma unroll
      for (int e = 0; e < kOwn; e += 4) {
        uint4 t;
        if constexpr (P > 1) {
          constexpr int kSlice = kDigits / P;
          t = *(const uint4 *)(cluster.map_shared_rank(totals[pass & 1], (top + e) / kSlice) + (top + e) % kSlice);
        } else {
          t = *(const uint4 *)(mine + top + e);
        }
        own[e] = t.x, own[e + 1] = t.y, own[e + 2] = t.z, own[e + 3] = t.w;
        sum += t.x + t.y + t.z + t.w;
      }
      unsigned run = sum;
#pragma unroll
      for (int o = 1; o < 32; o <<= 1) {
        const unsigned x = __shfl_up_sync(0xffffffffu, run, o);
        if (lane >= o) run += x;
      }
      if (lane == 31) s_sum[warp] = run;
      __syncthreads();
      for (int w = 0; w < warp; ++w) run += s_sum[w];
      unsigned cum = run - sum;
      if (cum < want && want <= run) {
#pragma unroll
        for (int e = kOwn - 1; e >= 0; --e) {
          if (cum < want && want <= cum + own[e]) {
            s_digit = (unsigned)(top + e);
            s_want = want - cum;
            s_eq = own[e];
          }
          cum += own[e];
        }
      }
      __syncthreads();
      prefix |= s_digit << shift;
      pmask |= dmask << shift;
      want = s_want;
      eq_total = s_eq;
    }

    // Each thread scans a run of consecutive candidates, four at a time (an odd number of fours: no bank conflicts).
    const int run = ((n + kThreads * 4 - 1) / (kThreads * 4) | 1) * 4;
    const int j0 = min(n, tid * run), j1 = min(n, j0 + run);
    auto four = [&](int j) -> uint4 {  // 0, below every threshold that is kept, behind the last one
      if (j + 4 <= min(n, a.held)) return *(const uint4 *)(dyn + j);
      return make_uint4(key_of(j), j + 1 < j1 ? key_of(j + 1) : 0u, j + 2 < j1 ? key_of(j + 2) : 0u,
                        j + 3 < j1 ? key_of(j + 3) : 0u);
    };
    int above = 0, equal = 0;
    for (int j = j0; j < j1; j += 4) {
      const uint4 u = four(j);
      above += (u.x > prefix) + (u.y > prefix) + (u.z > prefix) + (u.w > prefix);
      equal += (u.x == prefix) + (u.y == prefix) + (u.z == prefix) + (u.w == prefix);
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
      if (tid == kThreads - 1) s_count[0] = before_a + above, s_count[1] = before_e + equal;
      cluster.sync();
      for (int i = 0; i < rank; ++i) {
        before_a += *cluster.map_shared_rank(&s_count[0], i);
        before_e += *cluster.map_shared_rank(&s_count[1], i);
      }
    }
    const int drop = (int)(eq_total - want);  // the first of the equal ones go
    for (int j = j0; j < j1; j += 4) {
      const uint4 u = four(j);
#pragma unroll
      for (int e = 0; e < 4; ++e) {
        const uint32_t key = (&u.x)[e];
        bool keep = key > prefix;
        const int slot = before_a + max(0, before_e - drop);
        if (keep) ++before_a;
        if (key == prefix) keep = before_e++ >= drop;
        if (keep && slot < kh) kept[slot] = lo + j + e;
      }
    }
    head_sync<P>(cluster);  // every index written, every key and count read
  }

  if constexpr (P == 1) {
    if (tid == 0) {
      sm100::mbar_init(&s_bar, W);
      sm100::fence_mbar_init();
    }
    __syncthreads();
  }
  Rounds<P> rounds{&s_bar};
  constexpr int LPR = D / 16;          // lanes per row, 16 codes each
  constexpr int RPI = 32 / LPR;        // rows per copy of the warp
  constexpr int IT = kBlock / RPI;     // copies
  constexpr int kItem = kBlock * D;    // bytes
  const size_t scales = (size_t)bh * (c.cap / kBlock);
  const int sub = lane % LPR, row0 = lane / LPR;
  const int items = (k + kBlock - 1) / kBlock * 2;  // K and V of every block
  const uint32_t buf = (uint32_t)__cvta_generic_to_shared(dyn) + warp * 2 * kItem + lane * 16;
  const uint4 *held = (const uint4 *)((const uint8_t *)dyn + warp * 2 * kItem) + lane;
  // The lane's entry of an item, and what travels with it.
  struct Entry {
    int pos;
    float scale, score, low;
  };
  auto source = [&](int q) {  // 0 behind the last entry
    const int i = (q >> 1) * kBlock + lane;
    return q >= items || i >= k ? 0 : i < kh ? min(max(kept[i], 0), len - 1) : i - kh + nc;
  };
  auto fetch = [&](int q, int slot, int src) {  // an item's rows into its buffer
    Entry x{0, 0.f, 0.f, 0.f};
    if (q < items) {
      const bool is_v = q & 1;
      const int base = (q >> 1) * kBlock;
      const uint8_t *codes = (is_v ? c.V : c.K) + (size_t)bh * c.cap * D + sub * 16;
#pragma unroll
      for (int i = 0; i < IT; ++i) {
        const int from = __shfl_sync(0xffffffffu, src, i * RPI + row0);
        copy16(buf + slot * kItem + i * 512, codes + (size_t)from * D, base + i * RPI + row0 < k);
      }
      if (base + lane < k) {
        x.scale = ((is_v ? c.Vsc : c.Ksc) + scales)[src / kBlock];
        if (!is_v) {
          x.pos = pos[src];
          x.score = score[src];
          x.low = low[src];
        }
      }
    }
    return x;
  };
  // A round has two items, K and V of a block, for each warp: two independent chains of work, and half the barriers of
  // one (1024 heads 4 us less of 174, 8 long ones 7 us less of 57).  The next round's are on their way meanwhile.
  const int stride = P * W * 2;
  int q = (rank * W + warp) * 2;
  Entry next[2];
  auto fetch_round = [&](int q, int src) {
#pragma unroll
    for (int u = 0; u < 2; ++u) next[u] = fetch(q + u, u, src);
    asm volatile("cp.async.commit_group;" ::: "memory");
  };
  fetch_round(q, source(q));
  int src = source(q + stride);
  // Where the round's first entry comes from; its destination ends 16 * stride entries behind 16 * round.
  auto first_source = [&](int round) {
    const int i = round * (kBlock / 2);
    return i >= k ? len : i < kh ? min(max(kept[i], 0), len - 1) : i - kh + nc;
  };
  int from = first_source(0);
  for (int round = 0; round < items; round += stride, q += stride) {
    const bool inside = from < (round + stride) * (kBlock / 2);
    from = first_source(round + stride);
    asm volatile("cp.async.wait_group 0;" ::: "memory");  // each lane reads back what it copied
    uint4 w[2][IT];
    float scale_own[2], to[2];
#pragma unroll
    for (int u = 0; u < 2; ++u) {
#pragma unroll
      for (int i = 0; i < IT; ++i) w[u][i] = held[u * (kItem / 16) + i * 32];
      scale_own[u] = __shfl_sync(0xffffffffu, next[u].scale, lane);  // the loads have come back
    }
    const int pos_own = __shfl_sync(0xffffffffu, next[0].pos, lane);
    const float score_own = __shfl_sync(0xffffffffu, next[0].score, lane);
    const float low_own = __shfl_sync(0xffffffffu, next[0].low, lane);
    rounds.wait();  // everyone has read the round before
    rounds.arrive(lane);
    fetch_round(q + stride, src);
    src = source(q + 2 * stride);
    const bool work = q < items;
    const int base = (q >> 1) * kBlock;
    if (work) {
#pragma unroll
      for (int u = 0; u < 2; ++u) {
        float amax = 0.f;
#pragma unroll
        for (int i = 0; i < IT; ++i) {
          TopCode<F> top;
          top.add(w[u][i].x), top.add(w[u][i].y), top.add(w[u][i].z), top.add(w[u][i].w);
          amax = fmaxf(amax, top.value() * __shfl_sync(0xffffffffu, scale_own[u], i * RPI + row0));
        }
        to[u] = block_scale<F>(warp_max(amax));
      }
#pragma unroll
      for (int u = 0; u < 2; ++u) {
        // Times 2^(exponent of its scale - the new one's).  More than 15 is rare (small codes of a far larger scale)
        // and takes two steps, the first of them exact; more than 30 is a row of zeros.
        int left = min(exponent(scale_own[u]) - exponent(to[u]), 30);
        while (__any_sync(0xffffffffu, left != 0)) {
          const int step = min(left, 15);
          left = max(left - 15, 0);
#pragma unroll
          for (int i = 0; i < IT; ++i) {
            const int e = __shfl_sync(0xffffffffu, step, i * RPI + row0);
            if (e == 0) continue;
            const typename F::Shift by(e);
            w[u][i] = make_uint4(by.run(w[u][i].x), by.run(w[u][i].y), by.run(w[u][i].z), by.run(w[u][i].w));
          }
        }
      }
    }
    if (inside) rounds.wait();  // this round's sources lie in what it writes: everyone has to have read them
    if (work) {
#pragma unroll
      for (int u = 0; u < 2; ++u) {
        const bool is_v = u;
        uint8_t *codes = (is_v ? c.V : c.K) + ((size_t)bh * c.cap + base) * D + sub * 16;
#pragma unroll
        for (int i = 0; i < IT; ++i)
          if (base + i * RPI + row0 < k) *(uint4 *)(codes + (size_t)(i * RPI + row0) * D) = w[u][i];
        if (lane == 0) ((is_v ? c.Vsc : c.Ksc) + scales)[q >> 1] = to[u];
      }
      if (base + lane < k) {
        pos[base + lane] = pos_own;
        score[base + lane] = score_own;
        low[base + lane] = low_own;
      }
    }
  }
  rounds.wait();
  asm volatile("cp.async.wait_all;" ::: "memory");
  if (!rounds.ok && lane == 0) atomicOr(c.err, H2O_BERR_INTERNAL);
}

template <typename F, int D, int P, int W> cudaError_t evict_p(Args a, cudaStream_t st) {
  constexpr int kRing = W * 2 * kBlock * D;
  // Keys, as many as leave room for two CTAs an SM (the clusters of evict_t count on both).  Against 110 KB of them,
  // where the larger caches had one: 300 heads of 32,768 entries 265 -> 242 us, 64 of 131,072 276 -> 239, 16 of 262,144
  // 207 -> 156; 300 of 65,536, more of whose keys are read again, 730 -> 765.
  constexpr int most = (kSmemOfCta - kStatic<P>) / 4 & ~3;
  const int share = ((a.c.cap + P - 1) / P + 3) & ~3;
  const int keys = share < most ? share : most;
  const int smem = keys * 4 > kRing ? keys * 4 : kRing;
  a.held = smem / 4;
  static SmemLimit limit;
  const void *kernel = (const void *)evict_kernel<F, D, P, W>;
  cudaError_t e = limit.raise(kernel, smem);
  if (e == cudaSuccess && P > 8) e = cudaFuncSetAttribute(kernel, cudaFuncAttributeNonPortableClusterSizeAllowed, 1);
  if (e != cudaSuccess) return e;
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3(a.c.B * a.c.H * P);
  cfg.blockDim = dim3(W * 32);
  cfg.dynamicSmemBytes = smem;
  cfg.stream = st;
  cudaLaunchAttribute at;
  at.id = cudaLaunchAttributeClusterDimension;
  at.val.clusterDim = {(unsigned)P, 1, 1};
  cfg.attrs = &at;
  cfg.numAttrs = P > 1 ? 1 : 0;
  return cudaLaunchKernelEx(&cfg, evict_kernel<F, D, P, W>, a);
}

template <typename F, int D> cudaError_t evict_t(const Args &a, cudaStream_t st) {
  // Up to 16 CTAs share a head while the clusters all fit the device (two CTAs an SM; of 16, whose CTAs have to find
  // room in one GPC, 14 clusters fit) and each has a thousand entries.  8 heads of 131,072 entries: 57 us with 16, 64
  // with 8, 149 with 4.
  const int heads = a.c.B * a.c.H;
  auto shared = [&](int p) { return heads * p <= a.c.sms * 15 / 8 && a.c.cap / p >= 1024; };
  if (heads * 32 <= a.c.sms * 3 && a.c.cap >= 16384) return evict_p<F, D, 16, 8>(a, st);
  if (shared(8)) return evict_p<F, D, 8, 8>(a, st);
  if (shared(4)) return evict_p<F, D, 4, 8>(a, st);
  if (shared(2)) return evict_p<F, D, 2, 8>(a, st);
  return evict_p<F, D, 1, 8>(a, st);
}

}  // namespace

cudaError_t launch_evict(const View &c, const int32_t *lengths, int kh, int kl, int n_sink, int mode,
                         const int32_t *position, int32_t *new_lengths, cudaStream_t st) {
  const Args a{c, lengths, position, new_lengths, kh, kl, n_sink, mode, 0};
  if (c.kv == H2O_KV_E4M3) return c.d == 128 ? evict_t<E4M3, 128>(a, st) : evict_t<E4M3, 64>(a, st);
  return c.d == 128 ? evict_t<I8, 128>(a, st) : evict_t<I8, 64>(a, st);
}

}  // namespace blk
}  // namespace h2o
