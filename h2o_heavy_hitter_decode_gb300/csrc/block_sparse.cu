// block_sparse.cu — attention of a token's query rows over the blocks of a
// block-scaled 8-bit cache that a bound on their logits chooses.
//
//   x_gi = round(q_gi / 2^e), |x| <= 127, one e for the token's group of rows
//   m_j = max_g sum_i (x_gi > 0 ? x_gi hi_ji : x_gi lo_ji)      (block_bounds.cu)
//   key_j = m_j ks_j; the first n_first and the last n_last blocks, and of the
//   rest those with the highest keys, lowest index first among equals; then as
//   in block_attend.cu over the chosen blocks' entries.
//
// The sums are whole numbers below 2^24 and the scales powers of two, so keys
// are exact and the choice does not depend on the order of any sum.
//
// A cluster of P CTAs takes a token's rows of a cached head from the choice to
// the output.  Keys: each CTA a run of the candidates.  Choice: radix select
// over the keys' bits, 8 at a time, the digits' counts of the cluster met over
// distributed shared memory.  Attention: the chosen blocks in turn over the
// cluster's warps, each with its own ring of TMA loads and its own partial
// output; the CTA's and then the cluster's parts meet in shared memory.  With
// one token a sequence the weights go to the scores in the same launch (each
// CTA those of its own blocks); several tokens may choose the same block, so
// theirs are added by scores_kernel, in the tokens' order.
#include <cooperative_groups.h>

#include <climits>

#include "block_tile.cuh"

namespace h2o {
namespace blk {
namespace {

namespace cg = cooperative_groups;

constexpr int kW = 4;         // warps of a CTA
constexpr int kThreads = kW * 32;
constexpr int kStages = 2;    // blocks of a warp on their way
constexpr int kBins = 256;
constexpr int kHeldMost = 4096;  // keys of a CTA that stay in shared memory

struct Args {
  View c;
  Lens l;
  Rows q, out;
  float *lse;
  int32_t *blocks;  // [B*H][n][n_blocks]
  int causal, accumulate, n_blocks, n_first, n_last;
  int held;  // keys a CTA has room for
};

// What token t of a sequence sees: `end` entries in nb blocks, S of them chosen.
struct View1 {
  int end, nb, S;
};
__device__ __forceinline__ View1 view_of(const Args &a, const Seq &s, int t) {
  View1 v;
  v.end = max(0, a.causal ? s.total - s.cnt + t + 1 : s.total);
  v.nb = ceil_div(v.end, kBlock);
  v.S = min(v.nb, a.n_blocks);
  return v;
}
__device__ __forceinline__ int32_t *list_of(const Args &a, int bh, int t) {
  return a.blocks + ((size_t)bh * a.l.n + t) * a.n_blocks;
}
// Base-2 logits of row r of the token's group, in the order of the list.
__device__ __forceinline__ float *logits_of(const Args &a, int bh, int t, int r) {
  return a.c.logits + ((size_t)bh * a.c.max_rows + t * a.c.group + r) * a.c.cap;
}

template <int P> __device__ __forceinline__ void team_sync() {
  if constexpr (P > 1)
    cg::this_cluster().sync();
  else
    __syncthreads();
}
// `p` of this CTA's shared memory in CTA `rank` of the cluster.
template <int P, typename T> __device__ __forceinline__ T *peer(T *p, int rank) {
  if constexpr (P > 1)
    return cg::this_cluster().map_shared_rank(p, rank);
  else
    return p;
}

// Shared memory of a CTA, in order.
template <int D> struct Room {
  static constexpr int kRing = kW * kStages * 2 * kBlock * D;
  static constexpr int kOut = 16 * D * 4;  // the CTA's partial output
  __host__ __device__ static int codes(int group) { return 2 * group * D; }
  __host__ __device__ static int bytes(int group, int held) { return 1024 + kRing + kOut + codes(group) + held * 4; }
};

template <typename F, int D, int NR, int P>
__global__ void __launch_bounds__(kThreads) sparse_kernel(const Args a, const __grid_constant__ CUtensorMap kmap,
                                                          const __grid_constant__ CUtensorMap vmap) {
  constexpr int OT = D / 16, kStage = 2 * kBlock * D, kRows = 8 * NR;
  extern __shared__ uint8_t smem_raw[];
  uint8_t *smem = smem_raw + (-smem_u32(smem_raw) & 1023u);  // swizzled tiles start at multiples of 1024
  float *cta_o = (float *)(smem + Room<D>::kRing);            // [kRows][D]
  int8_t *xs = (int8_t *)(cta_o + 16 * D);                    // [group][2][D] query codes: the positive ones, the negative ones
  __shared__ __align__(8) uint64_t full[kW][kStages];
  __shared__ unsigned hist[2][kBins];
  __shared__ unsigned s_sum[kW], s_digit, s_want, s_top;
  __shared__ int s_scan[2][kW], s_count[2];
  __shared__ float2 part_ml[kW][kRows], cta_ml[kRows];
  __shared__ float row_base[H2O_BLOCK_MAX_ROWS];
  const View &c = a.c;
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5, g = lane >> 2, t4 = lane & 3;
  const int rank = P > 1 ? (int)cg::this_cluster().block_rank() : 0;
  const int64_t item = blockIdx.x / P;
  const int bh = (int)(item / a.l.n), t = (int)(item - (int64_t)bh * a.l.n), b = bh / c.H, h = bh - b * c.H;
  const int group = c.group;
  const Seq s = seq_of(a.l, b);
  if (!s.ok && h == 0 && t == 0 && rank == 0 && tid == 0) atomicOr(c.err, H2O_BERR_RANGE);
  if (t >= s.cnt) return;  // the whole cluster
  const View1 v = view_of(a, s, t);
  const Rows q{a.q.p + t * a.q.st, a.q.sb, a.q.sh, a.q.st};  // the token's rows alone
  const Seq one{s.len, 1, v.end, true};
  int32_t *list = list_of(a, bh, t);
  const size_t scales = (size_t)bh * (c.cap / kBlock);

  if (warp < kW && lane == 0) {
    for (int i = 0; i < kStages; ++i) mbar_init(&full[warp][i], 1);
    fence_mbar_init();
  }
  if (tid == 0) s_top = 0;
  __syncthreads();

  // ------------------------------------------------------------- the choice
  if (rank == 0)
    for (int i = v.S + tid; i < a.n_blocks; i += kThreads) list[i] = -1;
  if (v.nb <= a.n_blocks) {
    for (int i = rank * kThreads + tid; i < v.nb; i += P * kThreads) list[i] = i;
  } else {
    if (rank == 0) {
      for (int i = tid; i < a.n_first; i += kThreads) list[i] = i;
      for (int i = tid; i < a.n_last; i += kThreads) list[a.n_blocks - a.n_last + i] = v.nb - a.n_last + i;
    }
    const int nc = v.nb - a.n_first - a.n_last;
    unsigned want = (unsigned)(a.n_blocks - a.n_first - a.n_last);
    const int share = ceil_div(nc, P), lo = a.n_first + min(nc, rank * share);
    const int n = min(a.n_first + nc, lo + share) - lo;  // this CTA's candidates lo .. lo + n - 1
    uint32_t *keys = share <= a.held ? (uint32_t *)(xs + Room<D>::codes(group))
                                     : (uint32_t *)logits_of(a, bh, t, 0) + rank * share;  // read before any logit is written
    if (want > 0) {
      // query codes
      for (int x = tid; x < group * (D / 8); x += kThreads) {
        const uint4 w = *(const uint4 *)(q.at(b, h * group + x / (D / 8), 0) + x % (D / 8) * 8);
        unsigned top = 0;
#pragma unroll
        for (int e = 0; e < 4; ++e) {
          const uint32_t u = (&w.x)[e], y = u & 0x7fffu, z = (u >> 16) & 0x7fffu;
          top = max(top, max(y < 0x7f80u ? y : 0u, z < 0x7f80u ? z : 0u));
        }
        atomicMax(&s_top, top);
      }
      __syncthreads();
      const float inv = inverse_pow2(block_scale<I8>(__uint_as_float(s_top << 16)));
      for (int x = tid; x < group * (D / 8); x += kThreads) {
        float f[8];
        Unpack<__nv_bfloat16>::run(*(const uint4 *)(q.at(b, h * group + x / (D / 8), 0) + x % (D / 8) * 8), f);
        int8_t *dst = xs + x / (D / 8) * 2 * D + x % (D / 8) * 8;
#pragma unroll
        for (int e = 0; e < 8; ++e) {
          float y = f[e] * inv;
          y = y != y ? 0.f : fminf(fmaxf(y, -127.f), 127.f);
          const int k = __float2int_rn(y);
          dst[e] = (int8_t)max(k, 0);
          dst[D + e] = (int8_t)min(k, 0);
        }
      }
      __syncthreads();
      // keys: D / 16 lanes to a block
      constexpr int L = D / 16;
      for (int x0 = 0; x0 < n; x0 += kThreads / L) {
        const int x = x0 + tid / L, sub = tid % L;
        const int8_t *bd = c.bounds + (scales + lo + min(x, n - 1)) * 2 * D + sub * 16;
        const int4 low = *(const int4 *)bd, high = *(const int4 *)(bd + D);
        int m = INT_MIN;
        for (int r = 0; r < group; ++r) {
          const int4 up = *(const int4 *)(xs + r * 2 * D + sub * 16), dn = *(const int4 *)(xs + r * 2 * D + D + sub * 16);
          int k = 0;
#pragma unroll
          for (int e = 0; e < 4; ++e) k = __dp4a((&dn.x)[e], (&low.x)[e], __dp4a((&up.x)[e], (&high.x)[e], k));
#pragma unroll
          for (int o = 1; o < L; o <<= 1) k += __shfl_xor_sync(0xffffffffu, k, o);
          m = max(m, k);
        }
        // 2^-20: a key of the largest scale stays in fp32's range, one of the least scale a normal number
        const float key = (float)m * 0x1p-20f * c.Ksc[scales + lo + min(x, n - 1)];
        const uint32_t u = __float_as_uint(key);
        if (sub == 0 && x < n) keys[x] = u & 0x80000000u ? ~u : u | 0x80000000u;
      }
      __syncthreads();
    }
    uint32_t prefix = 0, pmask = 0;
    if (want > 0) {
      constexpr int kOwn = kBins / kThreads;
#pragma unroll 1
      for (int pass = 0; pass < 4; ++pass) {
        const int shift = 24 - 8 * pass;
        unsigned *mine = hist[pass & 1];
        for (int i = tid; i < kBins; i += kThreads) mine[i] = 0;
        __syncthreads();
        for (int x = tid; x < n; x += kThreads) {
          const uint32_t u = keys[x];
          if ((u & pmask) == prefix) atomicAdd(&mine[(u >> shift) & 255u], 1u);
        }
        team_sync<P>();
        // thread i sums its digits over the cluster, the highest ones first
        unsigned own[kOwn], sum = 0;
        const int top = kBins - kOwn * (tid + 1);
#pragma unroll
        for (int e = 0; e < kOwn; ++e) {
          own[e] = 0;
#pragma unroll
          for (int i = 0; i < P; ++i) own[e] += *peer<P>(mine + top + e, i);
          sum += own[e];
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
            if (cum < want && want <= cum + own[e]) s_digit = (unsigned)(top + e), s_want = want - cum;
            cum += own[e];
          }
        }
        __syncthreads();
        prefix |= s_digit << shift;
        pmask |= 255u << shift;
        want = s_want;
      }
      // each thread scans a run of consecutive candidates
      const int run = ceil_div(n, kThreads), x0 = min(n, tid * run), x1 = min(n, x0 + run);
      int above = 0, equal = 0;
      for (int x = x0; x < x1; ++x) above += keys[x] > prefix, equal += keys[x] == prefix;
      int ia = above, ie = equal;
#pragma unroll
      for (int o = 1; o < 32; o <<= 1) {
        const int x = __shfl_up_sync(0xffffffffu, ia, o), y = __shfl_up_sync(0xffffffffu, ie, o);
        if (lane >= o) ia += x, ie += y;
      }
      if (lane == 31) s_scan[0][warp] = ia, s_scan[1][warp] = ie;
      __syncthreads();
      int before_a = ia - above, before_e = ie - equal;
      for (int w = 0; w < warp; ++w) before_a += s_scan[0][w], before_e += s_scan[1][w];
      if (P > 1) {
        if (tid == kThreads - 1) s_count[0] = before_a + above, s_count[1] = before_e + equal;
        team_sync<P>();
        for (int i = 0; i < rank; ++i) before_a += *peer<P>(&s_count[0], i), before_e += *peer<P>(&s_count[1], i);
      }
      for (int x = x0; x < x1; ++x) {
        const uint32_t u = keys[x];
        const int slot = before_a + min(before_e, (int)want);  // the first of the equal ones stay
        const bool keep = u > prefix || (u == prefix && before_e < (int)want);
        before_a += u > prefix;
        before_e += u == prefix;
        if (keep) list[a.n_first + slot] = lo + x;
      }
    }
  }
  team_sync<P>();  // the list is whole; every key and count has been read

  // ----------------------------------------------------------- the attention
  // Slot rank + P (warp + kW i) of the list is the i-th block of a warp.
  uint8_t *ring = smem + warp * kStages * kStage;
  const uint64_t policy = l2_policy(false);
  const int first_slot = rank + P * warp;
  bool lost = false;
  uint32_t phases = 0;
  for (int row0 = 0; row0 < group; row0 += kRows) {
    auto fetch = [&](int i) {
      const int slot = first_slot + i * P * kW;
      if (slot >= v.S || lane != 0 || lost) return;
      asm volatile("fence.proxy.async;" ::: "memory");
      uint8_t *dst = ring + i % kStages * kStage;
      uint64_t *bar = &full[warp][i % kStages];
      const int row = bh * c.cap + list[slot] * kBlock;
      mbar_expect_tx(bar, kStage);
      tma_load_2d(dst, &kmap, bar, 0, row, policy);
      tma_load_2d(dst + kBlock * D, &vmap, bar, 0, row, policy);
    };
    for (int i = 0; i < kStages; ++i) fetch(i);
    Tile<F, D, NR, false> tl;
    tl.begin(q, group, 0, one, b, h, row0, nullptr);
    for (int i = 0; first_slot + i * P * kW < v.S; ++i) {
      const int slot = first_slot + i * P * kW, blk = list[slot];
      const float ks = c.Ksc[scales + blk], vs = c.Vsc[scales + blk];
      const int st = i % kStages;
      if (!lost && !mbar_wait(&full[warp][st], phases >> st & 1)) lost = true;
      if (lost) break;
      phases ^= 1u << st;
      uint8_t *kt = ring + st * kStage;
      tl.block(kt, kt + kBlock * D, ks, vs, blk, v.end - blk * kBlock, nullptr,
               [&](int r, int j, float s0, float s1, float s2, float s3) {
                 if (!a.accumulate) return;
                 float *lg = logits_of(a, bh, t, row0 + r) + slot * kBlock + (j - blk * kBlock);
                 lg[0] = s0, lg[8] = s1, lg[16] = s2, lg[24] = s3;
               });
      __syncwarp();  // this warp has read the stage
      fetch(i + kStages);
    }
    if (lost) {  // a copy never arrived: report, and wait for the other one before the memory goes
      if (lane == 0) atomicOr(c.err, H2O_BERR_INTERNAL);
      for (int i = 0; i < kStages; ++i) mbar_wait(&full[warp][i], 0), mbar_wait(&full[warp][i], 1);
    }
    __syncthreads();  // every warp is done with its ring: the partial outputs go there
    float *po = (float *)smem;  // [kW][kRows][D]
    const float part = tl.unit() * kPartDown;
#pragma unroll
    for (int n = 0; n < NR; ++n)
#pragma unroll
      for (int u = 0; u < 2; ++u) {
        const float l = tl.sum(n, u);
        const int r = 8 * n + 2 * t4 + u;
        if (g == 0) part_ml[warp][r] = make_float2(tl.m[n][u], l);
        const float inv = inverse_sum(l);
        float *dst = po + (warp * kRows + r) * D + g * (D / 8);
#pragma unroll
        for (int j = 0; j < OT; j += 2)
          *(float4 *)(dst + 2 * j) = make_float4(tl.o[n][j][u] * inv * part, tl.o[n][j][2 + u] * inv * part,
                                                 tl.o[n][j + 1][u] * inv * part, tl.o[n][j + 1][2 + u] * inv * part);
      }
    __syncthreads();
    // the CTA's warps, then the cluster's CTAs: weighted means of weighted means
    auto meet = [&](int parts, auto ml_of, auto o_of, float &m, float &l, float4 &o) {
      m = -INFINITY, l = 0.f, o = make_float4(0.f, 0.f, 0.f, 0.f);
      for (int i = 0; i < parts; ++i) m = fmaxf(m, ml_of(i).x);
      for (int i = 0; i < parts; ++i) {
        const float2 p = ml_of(i);
        l += p.x == -INFINITY ? p.y : p.y * ex2(p.x - m);
      }
      const bool any = l > 0.f || l != l;
      const float inv = any ? 1.f / l : 0.f;
      for (int i = 0; i < parts; ++i) {
        const float2 p = ml_of(i);
        const float z = (p.x == -INFINITY ? p.y : p.y * ex2(p.x - m)) * inv;
        const float4 e = o_of(i);
        o.x = fmaf(e.x, z, o.x), o.y = fmaf(e.y, z, o.y), o.z = fmaf(e.z, z, o.z), o.w = fmaf(e.w, z, o.w);
      }
    };
    const int rows = min(group - row0, kRows);
    for (int x = tid; x < rows * (D / 4); x += kThreads) {
      const int r = x / (D / 4), d0 = x % (D / 4) * 4;
      float m, l;
      float4 o;
      meet(kW, [&](int i) { return part_ml[i][r]; }, [&](int i) { return *(const float4 *)(po + (i * kRows + r) * D + d0); },
           m, l, o);
      *(float4 *)(cta_o + r * D + d0) = o;
      if (d0 == 0) cta_ml[r] = make_float2(m, l);
    }
    team_sync<P>();
    for (int x = rank * kThreads + tid; x < rows * (D / 4); x += P * kThreads) {
      const int r = x / (D / 4), d0 = x % (D / 4) * 4, hq = h * group + row0 + r;
      float m, l;
      float4 o;
      meet(P, [&](int i) { return *peer<P>(&cta_ml[r], i); },
           [&](int i) { return *(const float4 *)peer<P>(cta_o + r * D + d0, i); }, m, l, o);
      const __nv_bfloat162 p0 = __floats2bfloat162_rn(o.x * kPartUp, o.y * kPartUp),
                           p1 = __floats2bfloat162_rn(o.z * kPartUp, o.w * kPartUp);
      *(uint2 *)(const_cast<__nv_bfloat16 *>(a.out.at(b, hq, t)) + d0) =
          make_uint2(*(const uint32_t *)&p0, *(const uint32_t *)&p1);
      if (d0 == 0) {
        const bool any = l > 0.f || l != l;
        if (a.lse) a.lse[((size_t)b * c.H * group + hq) * a.l.n + t] = any ? (m + log2f(l)) * kLn2 : -INFINITY;
        if (a.l.n > 1) c.part[(size_t)bh * c.max_rows + t * group + row0 + r] = weight_base(m, l);
      }
    }
    if (a.l.n == 1 && a.accumulate && tid < rows) {
      float m = -INFINITY, l = 0.f;
      for (int i = 0; i < P; ++i) m = fmaxf(m, peer<P>(&cta_ml[tid], i)->x);
      for (int i = 0; i < P; ++i) {
        const float2 p = *peer<P>(&cta_ml[tid], i);
        l += p.x == -INFINITY ? p.y : p.y * ex2(p.x - m);
      }
      row_base[row0 + tid] = weight_base(m, l);
    }
    fence_proxy_async_smem();  // the next rows' copies land where the parts were
    team_sync<P>();            // the parts have been read
  }

  // -------------------------------------------------------------- the scores
  if (a.l.n > 1 || !a.accumulate) return;
  float *score = c.score + (size_t)bh * c.cap, *low = c.low + (size_t)bh * c.cap;
  const float *lg = logits_of(a, bh, t, 0);
  for (int x = tid; rank + x / kBlock * P < v.S; x += kThreads) {
    const int slot = rank + x / kBlock * P, j = list[slot] * kBlock + x % kBlock;
    if (j >= v.end) continue;
    const float old = score[j];
    float lost_part = low[j], w = 0.f;
    for (int r = 0; r < group; ++r) w += ex2(lg[(size_t)r * c.cap + slot * kBlock + x % kBlock] - row_base[r]);
    score[j] = add_score(old, lost_part, w);
    low[j] = lost_part;
  }
}

// The weights of several tokens' rows, added in the tokens' order: a CTA has a
// run of a head's blocks, and finds in each token's list those of them that it
// holds.
__global__ void __launch_bounds__(256) scores_kernel(const Args a, int slices) {
  const View &c = a.c;
  const int bh = blockIdx.x / slices, slice = blockIdx.x - bh * slices, b = bh / c.H, group = c.group;
  const Seq s = seq_of(a.l, b);
  const int nblk = ceil_div(s.total, kBlock);
  const int j0 = (int)((int64_t)slice * nblk / slices), j1 = (int)((int64_t)(slice + 1) * nblk / slices);
  __shared__ float base[H2O_BLOCK_MAX_ROWS];
  float *score = c.score + (size_t)bh * c.cap, *low = c.low + (size_t)bh * c.cap;
  for (int t = 0; t < s.cnt; ++t) {
    const View1 v = view_of(a, s, t);
    const int32_t *list = list_of(a, bh, t);
    auto first = [&](int j) {  // the first slot whose block is j or later
      int lo = 0, hi = v.S;
      while (lo < hi) {
        const int mid = (lo + hi) / 2;
        if (list[mid] < j)
          lo = mid + 1;
        else
          hi = mid;
      }
      return lo;
    };
    const int s0 = first(j0), s1 = first(j1);
    __syncthreads();  // the token before is done
    for (int r = threadIdx.x; r < group; r += 256) base[r] = c.part[(size_t)bh * c.max_rows + t * group + r];
    __syncthreads();
    const float *lg = logits_of(a, bh, t, 0);
    for (int x = s0 * kBlock + threadIdx.x; x < s1 * kBlock; x += 256) {
      const int j = list[x / kBlock] * kBlock + x % kBlock;
      if (j >= v.end) continue;
      const float old = score[j];
      float lost = low[j], w = 0.f;
      for (int r = 0; r < group; ++r) w += ex2(lg[(size_t)r * c.cap + x] - base[r]);
      score[j] = add_score(old, lost, w);
      low[j] = lost;
    }
  }
}

template <typename F, int D, int NR, int P>
cudaError_t sparse_p(Args a, const CUtensorMap &kmap, const CUtensorMap &vmap, cudaStream_t st) {
  const int most = (a.c.cap / kBlock + P - 1) / P;
  a.held = most < kHeldMost ? most : kHeldMost;
  const int smem = Room<D>::bytes(a.c.group, a.held);
  static SmemLimit limit;
  const void *kernel = (const void *)sparse_kernel<F, D, NR, P>;
  cudaError_t e = limit.raise(kernel, smem);
  if (e != cudaSuccess) return e;
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3((unsigned)((int64_t)a.c.B * a.c.H * a.l.n * P));
  cfg.blockDim = dim3(kThreads);
  cfg.dynamicSmemBytes = smem;
  cfg.stream = st;
  cudaLaunchAttribute at;
  at.id = cudaLaunchAttributeClusterDimension;
  at.val.clusterDim = {(unsigned)P, 1, 1};
  cfg.attrs = &at;
  cfg.numAttrs = P > 1 ? 1 : 0;
  return cudaLaunchKernelEx(&cfg, sparse_kernel<F, D, NR, P>, a, kmap, vmap);
}

template <typename F, int D, int NR>
cudaError_t sparse_n(const Args &a, const CUtensorMap &kmap, const CUtensorMap &vmap, cudaStream_t st) {
  const int64_t items = (int64_t)a.c.B * a.c.H * a.l.n;
  const int blocks = a.c.cap / kBlock;
  auto fits = [&](int p) { return items * p <= 2 * a.c.sms && blocks >= 8 * p; };
  if (fits(8)) return sparse_p<F, D, NR, 8>(a, kmap, vmap, st);
  if (fits(4)) return sparse_p<F, D, NR, 4>(a, kmap, vmap, st);
  if (fits(2)) return sparse_p<F, D, NR, 2>(a, kmap, vmap, st);
  return sparse_p<F, D, NR, 1>(a, kmap, vmap, st);
}

template <typename F, int D>
cudaError_t sparse_d(const Args &a, const CUtensorMap &kmap, const CUtensorMap &vmap, cudaStream_t st) {
  cudaError_t e = a.c.group <= 8 ? sparse_n<F, D, 1>(a, kmap, vmap, st) : sparse_n<F, D, 2>(a, kmap, vmap, st);
  if (e != cudaSuccess || !a.accumulate || a.l.n == 1) return e;
  const int64_t heads = (int64_t)a.c.B * a.c.H;
  int64_t slices = (2 * a.c.sms + heads - 1) / heads;
  if (slices > a.c.cap / kBlock) slices = a.c.cap / kBlock;
  scores_kernel<<<(unsigned)(heads * slices), 256, 0, st>>>(a, (int)slices);
  return cudaGetLastError();
}

}  // namespace

cudaError_t launch_sparse(const View &c, const Lens &l, const Rows &q, int causal, int accumulate, int n_blocks,
                          int n_first, int n_last, const Rows &out, float *lse, int32_t *blocks, const CUtensorMap &kmap,
                          const CUtensorMap &vmap, cudaStream_t st) {
  const Args a{c, l, q, out, lse, blocks, causal, accumulate, n_blocks, n_first, n_last, 0};
  if (c.kv == H2O_KV_E4M3)
    return c.d == 128 ? sparse_d<E4M3, 128>(a, kmap, vmap, st) : sparse_d<E4M3, 64>(a, kmap, vmap, st);
  return c.d == 128 ? sparse_d<I8, 128>(a, kmap, vmap, st) : sparse_d<I8, 64>(a, kmap, vmap, st);
}

}  // namespace blk
}  // namespace h2o
