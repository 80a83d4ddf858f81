// block_sparse.cu — attention of a token's query rows over the blocks of a
// block-scaled 8-bit cache that a bound on their logits chooses.
//
//   x_gi = round(q_gi / 2^e), |x| <= 127, one e for the token's group of rows
//   m_j = max_g sum_i (x_gi > 0 ? x_gi hi_ji : x_gi lo_ji)      (block_bounds.cu)
//   key_j = m_j ks_j; the first n_first and the last n_last blocks, and of the
//   rest those with the highest keys, lowest index first among equals; then as
//   in block_attend.cu over the chosen blocks' entries.
//
// The sums are whole numbers below 2^22, exact in the fp32 sums of mma.sync on
// f16, and the scales powers of two: keys are exact and the choice does not
// depend on the order of any sum.
//
// A cluster of P CTAs takes a token's rows of a cached head from the choice to
// the output.
// Keys: a warp takes 16 blocks as the rows of m16n8k16 (their bounds are 2 d
// bytes, straight from memory in 16-byte loads, the next 16 blocks' on their
// way) and 8 query rows as its columns: x's negative part against lo, the
// positive one against hi.
// Choice: of up to kLocal candidates each CTA makes all keys for itself and each
// warp finds the threshold for itself, keys in registers, a bit at a time from
// the first one that differs, so nothing but the keys crosses a barrier.  More
// candidates are shared by the cluster: radix select, 8 bits at a time, the
// digits' counts met over distributed shared memory, and the list through
// memory.
// Attention: the chosen blocks in turn over the cluster's CTAs and their warps,
// each with its own ring of TMA loads and its own partial output; the CTA's and
// then the cluster's parts meet in shared memory.
// With one token a sequence the new row is appended, and the weights are added
// to the scores, in the same launch (each CTA those of its own blocks); several
// tokens may choose the same block, so theirs are added by scores_kernel, in
// the tokens' order.
#include <cooperative_groups.h>

#include <algorithm>

#include "block_tile.cuh"

namespace h2o {
namespace blk {
namespace {

namespace cg = cooperative_groups;

constexpr int kBins = 256;
constexpr int kLocal = 512;      // candidates of which each CTA makes all keys
constexpr int kHeldMost = 4096;  // keys of a CTA that stay in shared memory
constexpr int kOwnMost = 1024;   // chosen blocks of a CTA whose list does
constexpr int kLogitsMost = 4096;  // logits of a CTA that do
constexpr int kCodesMost = 64;     // query rows of a token whose codes do

struct Args {
  View c;
  Lens l;
  Rows q, out;
  float *lse;
  int32_t *blocks;  // [B*H][n][n_blocks]
  int causal, accumulate, n_blocks, n_first, n_last;
  int fused;  // the launch appends the sequences' one new row: k, v, position
  Rows k, v;
  const int32_t *position;
  int held, own, logits;  // keys, chosen blocks and logits a CTA has room for
};

// What token t of a sequence sees: `end` entries in nb blocks, S of them chosen.
struct Sight {
  int end, nb, S;
};
__device__ __forceinline__ Sight sight_of(const Args &a, const Seq &s, int t) {
  Sight v;
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

// Four entries' scores with weights w added; entries from `left` on keep theirs.
__device__ __forceinline__ void store_scores(float *score, float *low, int left, const float4 &old, float4 less,
                                             const float4 &w) {
  const float4 sum = make_float4(add_score(old.x, less.x, w.x), add_score(old.y, less.y, w.y),
                                 add_score(old.z, less.z, w.z), add_score(old.w, less.w, w.w));
  if (left >= 4) {
    *(float4 *)score = sum;
    *(float4 *)low = less;
  } else {
    if (left > 0) score[0] = sum.x, low[0] = less.x;
    if (left > 1) score[1] = sum.y, low[1] = less.y;
    if (left > 2) score[2] = sum.z, low[2] = less.z;
  }
}

// ------------------------------------------------------------------- keys
// Bounds of blocks x0 + g and x0 + 8 + g of a run of n: the lane's chunks t,
// t + 4 .. of lo and of hi.
template <int D> struct Bounds {
  static constexpr int C = D / 64;
  uint4 w[2][2][C];
  float ks[2];
  __device__ __forceinline__ void load(const int8_t *bounds, const float *scales, int x0, int n) {
    const int lane = threadIdx.x & 31, g = lane >> 2, t = lane & 3;
#pragma unroll
    for (int r = 0; r < 2; ++r) {
      const int x = min(x0 + 8 * r + g, n - 1);
      const int8_t *p = bounds + (size_t)x * 2 * D + t * 16;
#pragma unroll
      for (int h = 0; h < 2; ++h)
#pragma unroll
        for (int i = 0; i < C; ++i) w[r][h][i] = *(const uint4 *)(p + h * D + i * 64);
      ks[r] = scales[x];
    }
  }
};

// Codes of 8 query rows as the B operand, in the order of the bounds' words.
template <int D> struct Codes {
  static constexpr int C = D / 64;
  uint32_t b[2][C][4][2];  // [lo, hi][chunk][word]
  // f: the lane's C chunks of 16 elements of row g.
  __device__ __forceinline__ void set(const float (&f)[C][16], float inv) {
#pragma unroll
    for (int i = 0; i < C; ++i)
#pragma unroll
      for (int e = 0; e < 4; ++e) {
        float x[4];
#pragma unroll
        for (int j = 0; j < 4; ++j) {
          const float y = f[i][4 * e + j] * inv;
          x[j] = y != y ? 0.f : rintf(fminf(fmaxf(y, -127.f), 127.f));
        }
        static_assert(!ToF16<I8>::kAdjacent, "pairs of a word's codes: 0 and 2, 1 and 3");
        const __half2 l0 = __floats2half2_rn(fminf(x[0], 0.f), fminf(x[2], 0.f));
        const __half2 l1 = __floats2half2_rn(fminf(x[1], 0.f), fminf(x[3], 0.f));
        const __half2 h0 = __floats2half2_rn(fmaxf(x[0], 0.f), fmaxf(x[2], 0.f));
        const __half2 h1 = __floats2half2_rn(fmaxf(x[1], 0.f), fmaxf(x[3], 0.f));
        b[0][i][e][0] = *(const uint32_t *)&l0, b[0][i][e][1] = *(const uint32_t *)&l1;
        b[1][i][e][0] = *(const uint32_t *)&h0, b[1][i][e][1] = *(const uint32_t *)&h1;
      }
  }
};
// The lane's chunks of a query row, and the largest finite magnitude among them as bits of a bf16.
template <int D> __device__ __forceinline__ unsigned query_row(const __nv_bfloat16 *p, float (&f)[D / 64][16]) {
  const int t = threadIdx.x & 3;
  unsigned top = 0;
#pragma unroll
  for (int i = 0; i < D / 64; ++i)
#pragma unroll
    for (int u = 0; u < 2; ++u) {
      const uint4 w = ld_nc16(p + (t + 4 * i) * 16 + u * 8);
      Unpack<__nv_bfloat16>::run(w, f[i] + u * 8);
#pragma unroll
      for (int e = 0; e < 4; ++e) {
        const uint32_t x = (&w.x)[e], y = x & 0x7fffu, z = (x >> 16) & 0x7fffu;
        top = max(top, max(y < 0x7f80u ? y : 0u, z < 0x7f80u ? z : 0u));
      }
    }
  return top;
}

// Largest sum of the two blocks over the 8 rows; all lanes of a quad get them.
template <int D> __device__ __forceinline__ float2 block_sums(const Bounds<D> &bd, const Codes<D> &q) {
  float c[4] = {0.f, 0.f, 0.f, 0.f};
#pragma unroll
  for (int h = 0; h < 2; ++h)
#pragma unroll
    for (int i = 0; i < D / 64; ++i)
#pragma unroll
      for (int e = 0; e < 4; ++e) {
        uint32_t a[4];
        ToF16<I8>::run((&bd.w[0][h][i].x)[e], a[0], a[2]);
        ToF16<I8>::run((&bd.w[1][h][i].x)[e], a[1], a[3]);
        mma16816(c, a, q.b[h][i][e][0], q.b[h][i][e][1]);
      }
  float2 m = make_float2(fmaxf(c[0], c[1]), fmaxf(c[2], c[3]));
#pragma unroll
  for (int o = 1; o < 4; o <<= 1) {
    m.x = fmaxf(m.x, __shfl_xor_sync(0xffffffffu, m.x, o));
    m.y = fmaxf(m.y, __shfl_xor_sync(0xffffffffu, m.y, o));
  }
  return m;
}
// Ordered like the keys.  2^-20: a key of the largest scale stays in fp32's range, one of the least a normal number.
__device__ __forceinline__ uint32_t key_bits(float m, float ks) {
  const uint32_t u = __float_as_uint(m * 0x1p-20f * ks + 0.f);
  return u & 0x80000000u ? ~u : u | 0x80000000u;
}

// The `want` highest of n <= 32 N keys, the first ones among equals, found by a
// warp alone: the largest T with count(key >= T) >= want, two bits at a time
// from the first one in which keys differ.  Those that are the warp's go to own
// and to the list.
template <int N, int P, int W>
__device__ __forceinline__ void choose(const Args &a, const uint32_t *keys, int n, unsigned want, int lo, int rank,
                                       int warp, int *own, int32_t *list) {
  const int lane = threadIdx.x & 31;
  uint32_t k[N], high = 0, low = 0xffffffffu;
#pragma unroll
  for (int i = 0; i < N; ++i) {
    const bool is = i * 32 + lane < n;
    k[i] = is ? keys[i * 32 + lane] : 0u;  // no key is 0
    high = max(high, k[i]);
    if (is) low = min(low, k[i]);
  }
  high = __reduce_max_sync(0xffffffffu, high);
  low = __reduce_min_sync(0xffffffffu, low);
  const int differ = 32 - __clz(high ^ low);  // bits below which keys differ
  int bit = (differ + 1) & ~1;                 // T is right in its bits from `bit` up
  uint32_t T = bit >= 32 ? 0u : high >> bit << bit;
  unsigned ge = (unsigned)n;
  while (bit > 0 && ge != want) {
    bit -= 2;
    const uint32_t at1 = T | 1u << bit, at2 = T | 2u << bit, at3 = T | 3u << bit;
    unsigned c1 = 0, c2 = 0, c3 = 0;
#pragma unroll
    for (int i = 0; i < N; ++i) c1 += k[i] >= at1, c2 += k[i] >= at2, c3 += k[i] >= at3;
    const unsigned sum = __reduce_add_sync(0xffffffffu, c1 | c2 << 10 | c3 << 20);  // at most 512 each
    c1 = sum & 1023u, c2 = sum >> 10 & 1023u, c3 = sum >> 20;
    if (c3 >= want)
      T = at3, ge = c3;
    else if (c2 >= want)
      T = at2, ge = c2;
    else if (c1 >= want)
      T = at1, ge = c1;
  }
  const bool exact = ge == want;  // else T is a key itself, and only the first of its equals stay
  unsigned above = 0;
  if (!exact) {
#pragma unroll
    for (int i = 0; i < N; ++i) above += k[i] > T;
    above = __reduce_add_sync(0xffffffffu, above);
  }
  const int ties = (int)(want - above);
  int taken = 0, equal = 0;
  const unsigned below = (1u << lane) - 1;
#pragma unroll
  for (int i = 0; i < N; ++i) {
    if (i * 32 >= n) break;
    bool keep = exact ? k[i] >= T : k[i] > T;
    if (!exact) {
      const unsigned eq = __ballot_sync(0xffffffffu, k[i] == T);
      keep |= k[i] == T && equal + __popc(eq & below) < ties;
      equal += __popc(eq);
    }
    if (i * 32 + lane >= n) keep = false;
    const unsigned kept = __ballot_sync(0xffffffffu, keep);
    const int slot = a.n_first + taken + __popc(kept & below);
    if (keep && slot % P == rank) {
      const int mine = slot / P;
      if (mine % W == warp) own[mine] = lo + i * 32 + lane, list[slot] = lo + i * 32 + lane;
    }
    taken += __popc(kept);
  }
}

// Shared memory of a CTA, in order: the warps' rings (later their partial
// outputs), the CTA's partial output, query codes of groups above 8, keys, the
// own blocks, logits.
template <int D, int NR, int W> struct Room {
  static constexpr int kStage = 2 * kBlock * D;
  static constexpr int kStages = D == 64 ? 4 : 2;  // blocks of a warp on their way
  static constexpr int kRing = W * kStages * kStage;
  static constexpr int kOut = 8 * NR * D * 4;
  static constexpr int kTile = sizeof(Codes<D>) * 32;  // codes of 8 rows
  __host__ __device__ static int codes(int group) { return NR == 1 || group > kCodesMost ? 0 : (group + 7) / 8 * kTile; }
  __host__ __device__ static int bytes(int group, int held, int own, int logits) {
    return 1024 + kRing + kOut + codes(group) + held * 4 + own * 4 + logits * 4;
  }
};

template <typename F, int D, int NR, int P, int W>
__global__ void __launch_bounds__(W * 32 + 32, W == 4 && NR == 1 ? 2 : 1)
    sparse_kernel(const Args a, const __grid_constant__ CUtensorMap kmap, const __grid_constant__ CUtensorMap vmap) {
  using R = Room<D, NR, W>;
  constexpr int kThreads = W * 32, OT = D / 16, kStage = R::kStage, kStages = R::kStages, kRows = 8 * NR;
  extern __shared__ uint8_t smem_raw[];
  uint8_t *smem = smem_raw + (-smem_u32(smem_raw) & 1023u);  // swizzled tiles start at multiples of 1024
  float *cta_o = (float *)(smem + R::kRing);                  // [kRows][D]
  const int group = a.c.group;
  Codes<D> *codes = (Codes<D> *)(smem + R::kRing + R::kOut);  // [tile][lane], groups above 8
  uint32_t *held = (uint32_t *)((uint8_t *)codes + R::codes(group));
  int *own = (int *)(held + a.held);
  float *held_logits = (float *)(own + a.own);
  __shared__ __align__(8) uint64_t full[W][kStages];
  __shared__ unsigned hist[2][kBins];
  __shared__ unsigned s_sum[W + 1], s_digit, s_want, s_have, s_top;
  __shared__ int s_scan[2][W + 1], s_count[2];
  __shared__ float2 part_ml[W][kRows], cta_ml[kRows];
  __shared__ float row_base[H2O_BLOCK_MAX_ROWS];
  const View &c = a.c;
  // W warps work; one more, where the launch appends, has the new row and then only meets the barriers: its tid is behind
  // every loop's end (2^25 blocks and list places of at most 2^26)
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5, g = lane >> 2, t4 = lane & 3;
  const bool works = warp < W;
  constexpr int kNone = 1 << 26;
  const int tid = works ? (int)threadIdx.x : kNone;
  const int rank = P > 1 ? (int)cg::this_cluster().block_rank() : 0;
  const int64_t item = blockIdx.x / P;
  const int bh = (int)(item / a.l.n), t = (int)(item - (int64_t)bh * a.l.n), b = bh / c.H, h = bh - b * c.H;
  const Seq s = seq_of(a.l, b);
  if (!s.ok && h == 0 && t == 0 && rank == 0 && tid == 0) atomicOr(c.err, H2O_BERR_RANGE);
  if (t >= s.cnt) return;  // the whole cluster
  const Sight v = sight_of(a, s, t);
  const Rows q{a.q.p + t * a.q.st, a.q.sb, a.q.sh, a.q.st};  // the token's rows alone
  const Seq one{s.len, 1, v.end, true};
  int32_t *list = list_of(a, bh, t);
  const size_t scales = (size_t)bh * (c.cap / kBlock);
  const bool all = v.nb <= a.n_blocks;
  const int nc = all ? 0 : v.nb - a.n_first - a.n_last;  // candidates n_first .. n_first + nc - 1
  const bool shared = P > 1 && (nc > kLocal || ceil_div(v.S, P) > a.own);  // the cluster shares the choice
  const bool local = !all && !shared && nc <= kLocal && ceil_div(v.S, P) <= a.own;
  const int share = shared ? ceil_div(nc, P) : nc;
  const int lo = a.n_first + (shared ? min(nc, rank * share) : 0);
  const int n = min(a.n_first + nc, lo + share) - lo;  // this CTA's candidates lo .. lo + n - 1
  unsigned want = all ? 0u : (unsigned)(a.n_blocks - a.n_first - a.n_last);
  const int steps = want > 0 ? ceil_div(n, 16) : 0;
  const int8_t *bounds = c.bounds + (scales + lo) * 2 * D;
  const float *ksc = c.Ksc + scales + lo;

  grid_dependency_wait();
  Bounds<D> bd;
  if (works && warp < steps) bd.load(bounds, ksc, warp * 16, n);
  if (works && lane == 0) {
    for (int i = 0; i < kStages; ++i) mbar_init(&full[warp][i], 1);
    fence_mbar_init();
  }
  // The new row: its block is the last one of the list, and no other CTA touches it.
  if (!works && rank == (v.S - 1) % P) {
    append_rows<F, D>(c, false, a.k, b, h, s.len, s.len, s.len + 1);
    append_rows<F, D>(c, true, a.v, b, h, s.len, s.len, s.len + 1);
    if (lane == 0) {
      const size_t at = (size_t)bh * c.cap + s.len;
      c.pos[at] = a.position ? a.position[b] : s.len;
      c.score[at] = 0.f;
      c.low[at] = 0.f;
    }
    __syncwarp();
    bound_block<F, D>(c, bh, s.len / kBlock, s.total);
    __threadfence();  // the codes are read back by a copy
    asm volatile("fence.proxy.async;" ::: "memory");
  }

  // ------------------------------------------------------------- the choice
  if (want > 0) {
    uint32_t *keys = n <= a.held ? held : (uint32_t *)logits_of(a, bh, t, 0) + (shared ? rank * share : 0);  // read before any logit is written
    Codes<D> qc;
    float inv;
    if constexpr (NR == 1) {  // every warp for itself; columns behind the last row repeat it
      float f[D / 64][16];
      const unsigned top = query_row<D>(q.at(b, h * group + min(g, group - 1), 0), f);
      inv = inverse_pow2(block_scale<I8>(__uint_as_float(__reduce_max_sync(0xffffffffu, top) << 16)));
      qc.set(f, inv);
    } else {
      if (tid == 0) s_top = 0;
      __syncthreads();
      const int tiles = works ? ceil_div(group, 8) : 0;
      for (int x = warp; x < tiles; x += W) {
        float f[D / 64][16];
        const unsigned top = __reduce_max_sync(0xffffffffu, query_row<D>(q.at(b, h * group + min(8 * x + g, group - 1), 0), f));
        if (lane == 0) atomicMax(&s_top, top);
      }
      __syncthreads();
      inv = inverse_pow2(block_scale<I8>(__uint_as_float(s_top << 16)));
      if (group <= kCodesMost) {
        for (int x = warp; x < tiles; x += W) {
          float f[D / 64][16];
          query_row<D>(q.at(b, h * group + min(8 * x + g, group - 1), 0), f);
          qc.set(f, inv);
          codes[x * 32 + lane] = qc;
        }
        __syncthreads();
      }
    }
    for (int x = works ? warp : steps; x < steps; x += W) {
      Bounds<D> now = bd;
      if (x + W < steps) bd.load(bounds, ksc, (x + W) * 16, n);
      float2 m;
      if constexpr (NR == 1) {
        m = block_sums<D>(now, qc);
      } else {
        m = make_float2(-INFINITY, -INFINITY);
        for (int y = 0; y < ceil_div(group, 8); ++y) {
          if (group <= kCodesMost) {
            qc = codes[y * 32 + lane];
          } else {  // made anew for each 16 blocks
            float f[D / 64][16];
            query_row<D>(q.at(b, h * group + min(8 * y + g, group - 1), 0), f);
            qc.set(f, inv);
          }
          const float2 z = block_sums<D>(now, qc);
          m = make_float2(fmaxf(m.x, z.x), fmaxf(m.y, z.y));
        }
      }
      if (t4 < 2) {
        const int j = x * 16 + t4 * 8 + g;
        if (j < n) keys[j] = t4 ? key_bits(m.y, now.ks[1]) : key_bits(m.x, now.ks[0]);
      }
    }
    __syncthreads();
    if (local) {
      if (works) {
        if (n <= 128)
          choose<4, P, W>(a, keys, n, want, lo, rank, warp, own, list);
        else
          choose<kLocal / 32, P, W>(a, keys, n, want, lo, rank, warp, own, list);
      }
    } else {
      uint32_t prefix = 0, pmask = 0;
      constexpr int kOwn = kBins / kThreads;
      unsigned have = 0;
#pragma unroll 1
      for (int pass = 0; pass < 4 && have != want; ++pass) {
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
        unsigned mine_of[kOwn], sum = 0;
        const int top = works ? kBins - kOwn * (tid + 1) : 0;
#pragma unroll
        for (int e = 0; e < kOwn; ++e) {
          mine_of[e] = 0;
          if (works) {
#pragma unroll
            for (int i = 0; i < P; ++i) mine_of[e] += *peer<P>(mine + top + e, i);
          }
          sum += mine_of[e];
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
            if (cum < want && want <= cum + mine_of[e])
              s_digit = (unsigned)(top + e), s_want = want - cum, s_have = mine_of[e];
            cum += mine_of[e];
          }
        }
        __syncthreads();
        prefix |= s_digit << shift;
        pmask |= 255u << shift;
        want = s_want;
        have = s_have;  // as many as are wanted: the digits so far decide
      }
      // each thread scans a run of consecutive candidates
      const int run = ceil_div(n, kThreads), x0 = works ? min(n, tid * run) : n, x1 = min(n, x0 + run);
      int above = 0, equal = 0;
      for (int x = x0; x < x1; ++x) above += (keys[x] & pmask) > prefix, equal += (keys[x] & pmask) == prefix;
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
        const uint32_t u = keys[x] & pmask;
        const int slot = before_a + min(before_e, (int)want);  // the first of the equal ones stay
        const bool keep = u > prefix || (u == prefix && before_e < (int)want);
        before_a += u > prefix;
        before_e += u == prefix;
        if (keep) list[a.n_first + slot] = lo + x;
      }
    }
  }
  // the list's ends, and what is behind it
  const int first = all ? v.S : a.n_first, last = all ? v.S : v.S - a.n_last;
  if (rank == 0) {
    for (int i = tid; i < first; i += kThreads) list[i] = i;
    for (int i = last + tid; i < v.S; i += kThreads) list[i] = v.nb - v.S + i;
    for (int i = v.S + tid; i < a.n_blocks; i += kThreads) list[i] = -1;
  }
  if (all || local)
    __syncthreads();  // the new row is there, every key has been read
  else
    team_sync<P>();  // the list is whole too
  auto block_of = [&](int slot) {
    if (slot < first) return slot;
    if (slot >= last) return v.nb - v.S + slot;
    return local ? own[slot / P] : list[slot];
  };

  // ----------------------------------------------------------- the attention
  // Slot rank + P (warp + W i) of the list is the i-th block of a warp.  Logits: by own blocks in shared memory, or by slots in memory.
  const bool near = a.l.n == 1 && group * ceil_div(v.S, P) * kBlock <= a.logits;
  const int64_t row_step = near ? ceil_div(v.S, P) * kBlock : c.cap;
  float *logits = near ? held_logits : logits_of(a, bh, t, 0);
  auto place = [&](int slot) { return (near ? slot / P : slot) * kBlock; };
  uint8_t *ring = smem + warp * kStages * kStage;
  const uint64_t policy = l2_policy(false);
  const int first_slot = rank + P * warp;
  bool lost = false;
  uint32_t phases = 0;
  // Scores: 8 threads to an own block, four entries each; kAhead of a thread's are on their way at once.
  constexpr int kAhead = 4;
  float *score = c.score + (size_t)bh * c.cap, *low = c.low + (size_t)bh * c.cap;
  float4 old[kAhead], less[kAhead];
  auto entry_of = [&](int y) {  // the first of the thread's y-th four, -1 behind the last
    const int slot = rank + (tid / 8 + y * (kThreads / 8)) * P;
    return works && slot < v.S ? block_of(slot) * kBlock + tid % 8 * 4 : -1;
  };
  auto load_scores = [&](int y, int at) {
    const int j = entry_of(y);
    if (j >= 0) old[at] = *(const float4 *)(score + j), less[at] = *(const float4 *)(low + j);
  };
  for (int row0 = 0; row0 < group; row0 += kRows) {
    auto fetch = [&](int i) {
      const int slot = first_slot + i * P * W;
      if (!works || slot >= v.S || lane != 0 || lost) return;
      asm volatile("fence.proxy.async;" ::: "memory");
      uint8_t *dst = ring + i % kStages * kStage;
      uint64_t *bar = &full[warp][i % kStages];
      const int row = bh * c.cap + block_of(slot) * kBlock;
      mbar_expect_tx(bar, kStage);
      tma_load_2d(dst, &kmap, bar, 0, row, policy);
      tma_load_2d(dst + kBlock * D, &vmap, bar, 0, row, policy);
    };
    for (int i = 0; i < kStages; ++i) fetch(i);
    Tile<F, D, NR, false> tl;
    if (works) tl.begin(q, group, 0, one, b, h, row0, nullptr);
    for (int i = 0; works && first_slot + i * P * W < v.S; ++i) {
      const int slot = first_slot + i * P * W, blk = block_of(slot);
      const float ks = c.Ksc[scales + blk], vs = c.Vsc[scales + blk];
      const int st = i % kStages;
      if (!lost && !mbar_wait(&full[warp][st], phases >> st & 1)) lost = true;
      if (lost) break;
      phases ^= 1u << st;
      uint8_t *kt = ring + st * kStage;
      tl.block(kt, kt + kBlock * D, ks, vs, blk, v.end - blk * kBlock, nullptr,
               [&](int r, int j, float s0, float s1, float s2, float s3) {
                 if (!a.accumulate) return;
                 float *lg = logits + (row0 + r) * row_step + place(slot) + (j - blk * kBlock);
                 lg[0] = s0, lg[8] = s1, lg[16] = s2, lg[24] = s3;
               });
      __syncwarp();  // this warp has read the stage
      fetch(i + kStages);
    }
    if (lost) {  // a copy never arrived: report, and wait for the others before the memory goes
      if (lane == 0) atomicOr(c.err, H2O_BERR_INTERNAL);
      for (int i = 0; i < kStages; ++i) mbar_wait(&full[warp][i], 0), mbar_wait(&full[warp][i], 1);
    }
    __syncthreads();  // every warp is done with its ring: the partial outputs go there
    float *po = (float *)smem;  // [W][kRows][D]
    if (works) {
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
    }
    // the own entries' scores are on their way while the parts meet
    if (row0 == 0 && a.l.n == 1 && a.accumulate) {
#pragma unroll
      for (int y = 0; y < kAhead; ++y) load_scores(y, y);
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
      meet(W, [&](int i) { return part_ml[i][r]; }, [&](int i) { return *(const float4 *)(po + (i * kRows + r) * D + d0); },
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
    if (row0 + kRows < group) team_sync<P>();  // the parts have been read
  }
  __syncwarp();
  if (P > 1) asm volatile("barrier.cluster.arrive.release.aligned;" ::: "memory");  // and the last ones too

  // -------------------------------------------------------------- the scores
  if (a.l.n == 1 && a.accumulate) {
    __syncthreads();
    for (int y0 = 0; entry_of(y0) >= 0; y0 += kAhead) {
      if (y0 > 0) {
#pragma unroll
        for (int y = 0; y < kAhead; ++y) load_scores(y0 + y, y);
      }
#pragma unroll
      for (int y = 0; y < kAhead; ++y) {
        const int j = entry_of(y0 + y);
        if (j < 0) break;
        const float *lg = logits + place(rank + (tid / 8 + (y0 + y) * (kThreads / 8)) * P) + tid % 8 * 4;
        float4 w = make_float4(0.f, 0.f, 0.f, 0.f);
#pragma unroll 4
        for (int r = 0; r < group; ++r) {
          const float4 x = *(const float4 *)(lg + r * row_step);
          const float e = row_base[r];
          w.x += ex2(x.x - e), w.y += ex2(x.y - e), w.z += ex2(x.z - e), w.w += ex2(x.w - e);
        }
        store_scores(score + j, low + j, v.end - j, old[y], less[y], w);
      }
    }
  }
  __syncwarp();
  if (P > 1) asm volatile("barrier.cluster.wait.acquire.aligned;" ::: "memory");  // a peer may still read this CTA's parts
}

// The weights of several tokens' rows, added in the tokens' order: a CTA has
// kSlice blocks of a head, four entries a thread, and finds each token's slots
// of them first (a warp a token).
constexpr int kSlice = 32, kScoreThreads = kSlice * 8;
__global__ void __launch_bounds__(kScoreThreads) scores_kernel(const Args a, int slices) {
  extern __shared__ int slot_of[];  // [n][kSlice], -1: not chosen
  const View &c = a.c;
  const int bh = blockIdx.x / slices, j0 = (blockIdx.x - bh * slices) * kSlice, b = bh / c.H, group = c.group;
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  const Seq s = seq_of(a.l, b);
  if (s.cnt == 0 || j0 * kBlock >= s.total) return;
  __shared__ float base[H2O_BLOCK_MAX_ROWS];
  float *score = c.score + (size_t)bh * c.cap, *low = c.low + (size_t)bh * c.cap;
  const int mine = threadIdx.x / 8, j = (j0 + mine) * kBlock + threadIdx.x % 8 * 4;
  grid_dependency_wait();
  const bool in = j < s.total;
  float4 old = make_float4(0.f, 0.f, 0.f, 0.f), less = old;
  if (in) old = *(const float4 *)(score + j), less = *(const float4 *)(low + j);
  for (int r = threadIdx.x; r < s.cnt * group; r += kScoreThreads) base[r] = c.part[(size_t)bh * c.max_rows + r];
  for (int t = warp; t < s.cnt; t += kScoreThreads / 32) {
    const Sight v = sight_of(a, s, t);
    const int32_t *list = list_of(a, bh, t);
    slot_of[t * kSlice + lane] = -1;
    __syncwarp();
#pragma unroll 4
    for (int i = lane; i < v.S; i += 32) {
      const int x = list[i] - j0;
      if (x >= 0 && x < kSlice) slot_of[t * kSlice + x] = i;
    }
  }
  __syncthreads();
  if (!in) return;
  bool any = false;
  for (int t = 0; t < s.cnt; ++t) {
    const int slot = slot_of[t * kSlice + mine];
    if (slot < 0) continue;
    const float *lg = logits_of(a, bh, t, 0) + slot * kBlock + threadIdx.x % 8 * 4;
    float4 w = make_float4(0.f, 0.f, 0.f, 0.f);
#pragma unroll 8
    for (int r = 0; r < group; ++r) {
      const float4 x = *(const float4 *)(lg + (size_t)r * c.cap);
      const float e = base[t * group + r];
      w.x += ex2(x.x - e), w.y += ex2(x.y - e), w.z += ex2(x.z - e), w.w += ex2(x.w - e);
    }
    old.x = add_score(old.x, less.x, w.x), old.y = add_score(old.y, less.y, w.y);
    old.z = add_score(old.z, less.z, w.z), old.w = add_score(old.w, less.w, w.w);
    any = true;
  }
  if (!any) return;
  if (j + 4 <= s.total) {
    *(float4 *)(score + j) = old;
    *(float4 *)(low + j) = less;
  } else {  // entries behind the last one keep their score
    score[j] = old.x, low[j] = less.x;
    if (j + 1 < s.total) score[j + 1] = old.y, low[j + 1] = less.y;
    if (j + 2 < s.total) score[j + 2] = old.z, low[j + 2] = less.z;
  }
}

template <typename... X>
cudaError_t launch_with(void (*kernel)(X...), unsigned ctas, int threads, int smem, int cluster, bool after,
                        cudaStream_t st, X... args) {
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3(ctas);
  cfg.blockDim = dim3(threads);
  cfg.dynamicSmemBytes = smem;
  cfg.stream = st;
  cudaLaunchAttribute at[2];
  int n = 0;
  if (cluster > 1) {
    at[n].id = cudaLaunchAttributeClusterDimension;
    at[n++].val.clusterDim = {(unsigned)cluster, 1, 1};
  }
  if (after) {
    at[n].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    at[n++].val.programmaticStreamSerializationAllowed = 1;
  }
  cfg.attrs = at;
  cfg.numAttrs = n;
  return cudaLaunchKernelEx(&cfg, kernel, args...);
}

template <typename F, int D, int NR, int P, int W>
cudaError_t sparse_p(Args a, const CUtensorMap &kmap, const CUtensorMap &vmap, cudaStream_t st) {
  const int blocks = a.c.cap / kBlock, own = (std::min(blocks, a.n_blocks) + P - 1) / P;
  const int share = std::min(blocks, std::max(kLocal, (blocks + P - 1) / P));
  a.held = (std::min(share, kHeldMost) + 3) & ~3;
  a.own = (std::min(own, kOwnMost) + 3) & ~3;
  const int64_t logits = (int64_t)a.c.group * own * kBlock;
  a.logits = a.accumulate && a.l.n == 1 && logits <= kLogitsMost ? (int)logits : 0;
  const int smem = Room<D, NR, W>::bytes(a.c.group, a.held, a.own, a.logits);
  static SmemLimit limit;
  const auto kernel = sparse_kernel<F, D, NR, P, W>;
  cudaError_t e = limit.raise((const void *)kernel, smem);
  if (e == cudaSuccess && P > 8)
    e = cudaFuncSetAttribute((const void *)kernel, cudaFuncAttributeNonPortableClusterSizeAllowed, 1);
  if (e != cudaSuccess) return e;
  const int64_t ctas = (int64_t)a.c.B * a.c.H * a.l.n * P;
  return launch_with(kernel, (unsigned)ctas, (W + a.fused) * 32, smem, P, a.l.appends && !a.fused, st, a, kmap, vmap);
}

template <typename F, int D, int NR>
cudaError_t sparse_n(const Args &a, const CUtensorMap &kmap, const CUtensorMap &vmap, cudaStream_t st) {
  const int64_t items = (int64_t)a.c.B * a.c.H * a.l.n;
  const int blocks = a.c.cap / kBlock;
  auto fits = [&](int p, int per_sm) { return items * p <= (int64_t)per_sm * a.c.sms && blocks >= 8 * p; };
  if (items * 16 <= a.c.sms && blocks >= 2048) return sparse_p<F, D, NR, 16, 8>(a, kmap, vmap, st);
  if (fits(8, 1)) return sparse_p<F, D, NR, 8, 8>(a, kmap, vmap, st);
  if (fits(4, 2)) return sparse_p<F, D, NR, 4, 4>(a, kmap, vmap, st);
  if (fits(2, 2)) return sparse_p<F, D, NR, 2, 4>(a, kmap, vmap, st);
  return sparse_p<F, D, NR, 1, 4>(a, kmap, vmap, st);
}

template <typename F, int D>
cudaError_t sparse_d(const Args &a, const CUtensorMap &kmap, const CUtensorMap &vmap, cudaStream_t st) {
  cudaError_t e = a.c.group <= 8 ? sparse_n<F, D, 1>(a, kmap, vmap, st) : sparse_n<F, D, 2>(a, kmap, vmap, st);
  if (e != cudaSuccess || !a.accumulate || a.l.n == 1) return e;
  const int64_t heads = (int64_t)a.c.B * a.c.H;
  const int slices = (a.c.cap / kBlock + kSlice - 1) / kSlice;
  return launch_with(scores_kernel, (unsigned)(heads * slices), kScoreThreads, a.l.n * kSlice * 4, 1, true, st, a, slices);
}

}  // namespace

cudaError_t launch_sparse(const View &c, const Lens &l, const Rows &q, const Rows *k, const Rows *v,
                          const int32_t *position, int causal, int accumulate, int n_blocks, int n_first, int n_last,
                          const Rows &out, float *lse, int32_t *blocks, const CUtensorMap &kmap, const CUtensorMap &vmap,
                          cudaStream_t st) {
  const Rows none{};
  const bool fused = k && l.n == 1;
  if (k && !fused) {
    cudaError_t e = launch_append(c, l, *k, *v, position, nullptr, st);
    if (e != cudaSuccess) return e;
  }
  const Args a{c, l, q, out, lse, blocks, causal, accumulate, n_blocks, n_first, n_last,
               fused, k ? *k : none, v ? *v : none, position, 0, 0, 0};
  if (c.kv == H2O_KV_E4M3)
    return c.d == 128 ? sparse_d<E4M3, 128>(a, kmap, vmap, st) : sparse_d<E4M3, 64>(a, kmap, vmap, st);
  return c.d == 128 ? sparse_d<I8, 128>(a, kmap, vmap, st) : sparse_d<I8, 64>(a, kmap, vmap, st);
}

}  // namespace blk
}  // namespace h2o
