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
// the output, each CTA a run of the list's places (slots).
// Keys: a warp takes 16 blocks as the rows of m16n8k16 (their bounds are 2 d
// bytes, straight from memory in 16-byte loads, the next 16 blocks' on their
// way) and 8 query rows as its columns: x's negative part against lo, the
// positive one against hi.
// Choice: of up to kAloneKeys candidates each CTA makes all keys and finds the
// threshold for itself (up to kWarpKeys each warp: keys in registers, two bits
// at a time from the first one that differs); of more it makes a share, and the
// cluster finds the threshold together, counting keys in bins that meet over
// distributed shared memory.
// Attention: each warp takes every W-th slot of its CTA through its own ring of
// TMA loads; the warps' and then the CTAs' parts meet in shared memory, each CTA
// joining a slice of the output that the others have handed to it.
// Weights meet V whole, as two f16 numbers each (Tile): products are not what
// bounds this kernel, and 11 bits showed in one output of fifty (a step of bf16,
// 8e-4 of the outputs' norm against 32-bit weights; now 1e-4 and less).  Second
// products cost up to 6 % (groups of 4 28.1 -> 29.0 us, long batch 56.9 -> 60.1).
// With one token a sequence the new row is appended, and the weights are added
// to the scores, in the same launch (each CTA those of its own blocks); several
// tokens may choose the same block, so theirs are added by scores_kernel, in
// the tokens' order.
//
// Bound: short runs by latency, a dozen steps from the lengths to the scores (32
// heads of 2,560 entries, 16 blocks each, 10.6 us, of it 3 to the keys, 1 for
// the choice, 2 for copy and products, 3 to join the parts, 1 for the scores);
// larger ones by memory in two of them, the keys' (4 to 5 TB/s) and the
// blocks' (6 TB/s of 4 KB pieces): 128 heads of 20,000 to 65,500 entries, 128
// blocks each, 183 MB, 60 us, where memory alone would take 27.
#include <cooperative_groups.h>

#include <algorithm>
#include <atomic>

#include "block_tile.cuh"

namespace h2o {
namespace blk {
namespace {

namespace cg = cooperative_groups;

constexpr int kMostCtas = 16;     // of a cluster
constexpr int kWarpKeys = 128, kAloneKeys = 512;
constexpr int kHeldKeys = 4096;    // of a CTA, in shared memory
constexpr int kOwnMost = 1024;    // chosen blocks of a CTA whose list stays in shared memory
constexpr int kLogitsMost = 512;  // logits of a CTA that do
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
  int P;           // CTAs of a cluster
  int own, logits;  // chosen blocks and logits a CTA has room for
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

// The cluster's barrier in two halves: what a thread wrote before its arrival, also to other CTAs' shared memory, is
// there for all behind the wait.
__device__ __forceinline__ void team_arrive() {
  __syncwarp();
  asm volatile("barrier.cluster.arrive.release.aligned;" ::: "memory");
}
__device__ __forceinline__ void team_wait() {
  __syncwarp();
  asm volatile("barrier.cluster.wait.acquire.aligned;" ::: "memory");
}
__device__ __forceinline__ void team_sync() {
  team_arrive();
  team_wait();
}
// `p` of this CTA's shared memory in CTA `rank` of the cluster.
template <typename T> __device__ __forceinline__ T *peer(T *p, int rank) {
  return cg::this_cluster().map_shared_rank(p, rank);
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
  // In shared memory: 16 bytes of each lane beside those of the next one.
  static constexpr int kFours = 4 * C;
  __device__ __forceinline__ void put(uint4 *tile) const {
#pragma unroll
    for (int i = 0; i < kFours; ++i) {
      const uint32_t *w = &b[0][0][0][0] + 4 * i;
      tile[i * 32 + (threadIdx.x & 31)] = make_uint4(w[0], w[1], w[2], w[3]);
    }
  }
  __device__ __forceinline__ void get(const uint4 *tile) {
#pragma unroll
    for (int i = 0; i < kFours; ++i) {
      uint32_t *w = &b[0][0][0][0] + 4 * i;
      const uint4 u = tile[i * 32 + (threadIdx.x & 31)];
      w[0] = u.x, w[1] = u.y, w[2] = u.z, w[3] = u.w;
    }
  }
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

// A threshold among keys that some threads hold: the largest T with count(key
// >= T) >= want, or, where a T has exactly `want` keys from it on, that one.
struct Cut {
  uint32_t T;
  unsigned want;
  bool exact;  // else T is a key itself, and of its equals only the first ones stay
};
// count(c): c[0..2] over all keys for thresholds at[0..2].
template <typename Count>
__device__ __forceinline__ Cut find_cut(uint32_t high, uint32_t low, unsigned n, unsigned want, Count count) {
  const int differ = 32 - __clz(high ^ low);  // bits below which keys differ
  int bit = (differ + 1) & ~1;                // T is right in its bits from `bit` up
  Cut c{bit >= 32 ? 0u : high >> bit << bit, want, n == want};
  while (bit > 0 && !c.exact) {
    bit -= 2;
    const uint32_t at[3] = {c.T | 1u << bit, c.T | 2u << bit, c.T | 3u << bit};
    unsigned cnt[3];
    count(at, cnt);
#pragma unroll
    for (int i = 0; i < 3; ++i)
      if (cnt[i] >= want) c.T = at[i], c.exact = cnt[i] == want;
  }
  return c;
}

// Keys of n <= 32 N candidates chosen by a warp alone; emit(slot among the chosen, candidate) in order.
template <int N, typename Emit>
__device__ __forceinline__ void choose_warp(const uint32_t *keys, int n, unsigned want, Emit emit) {
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
  const Cut c = find_cut(high, low, (unsigned)n, want, [&](const uint32_t (&at)[3], unsigned (&cnt)[3]) {
    unsigned c0 = 0, c1 = 0, c2 = 0;
#pragma unroll
    for (int i = 0; i < N; ++i) c0 += k[i] >= at[0], c1 += k[i] >= at[1], c2 += k[i] >= at[2];
    static_assert(32 * N < 1024, "three counts to a word");
    const unsigned sum = __reduce_add_sync(0xffffffffu, c0 | c1 << 10 | c2 << 20);
    cnt[0] = sum & 1023u, cnt[1] = sum >> 10 & 1023u, cnt[2] = sum >> 20;
  });
  unsigned above = 0;
  if (!c.exact) {
#pragma unroll
    for (int i = 0; i < N; ++i) above += k[i] > c.T;
    above = __reduce_add_sync(0xffffffffu, above);
  }
  const int ties = (int)(want - above);
  int taken = 0, equal = 0;
  const unsigned below = (1u << lane) - 1;
#pragma unroll
  for (int i = 0; i < N; ++i) {
    if (i * 32 >= n) break;
    bool keep = c.exact ? k[i] >= c.T : k[i] > c.T;
    if (!c.exact) {
      const unsigned eq = __ballot_sync(0xffffffffu, k[i] == c.T);
      keep |= k[i] == c.T && equal + __popc(eq & below) < ties;
      equal += __popc(eq);
    }
    if (i * 32 + lane >= n) keep = false;
    const unsigned kept = __ballot_sync(0xffffffffu, keep);
    if (keep) emit(taken + __popc(kept & below), i * 32 + lane);
    taken += __popc(kept);
  }
}

// The same by a team of P CTAs, each of W warps, each CTA with n keys of its own
// (P = 1: by a CTA alone): counts in 2^8 bins between the team's least and
// largest key, then in as many of the bin that holds the threshold, until the
// keys above it and in it are as many as are wanted, or it is one key.  The bins
// are summed over the team by every CTA, which tells it also how many chosen
// keys the CTAs before it have.
constexpr int kBins = 256;
template <int W> struct ChooseRoom {
  uint32_t high[W], low[W];
  uint32_t team_high[kMostCtas], team_low[kMostCtas];
  unsigned sum[W], bin, want, have;
  unsigned before[2][W];
  int scan[2][W];
};
template <int W, typename Emit>
__device__ __forceinline__ void choose_team(const uint32_t *keys, int n, unsigned want, int P, int rank,
                                            unsigned (*bins)[kBins], ChooseRoom<W> &room, Emit emit) {
  constexpr int kThreads = W * 32, kOwn = kBins / kThreads;
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
  const int run = (n + kThreads - 1) / kThreads * 32, x0 = warp * run + lane, x1 = min(n, (warp + 1) * run);  // the warp's keys
  auto meet = [&]() {
    if (P > 1)
      team_sync();
    else
      __syncthreads();
  };
  uint32_t high = 0, low = 0xffffffffu;
#pragma unroll 4
  for (int x = x0; x < x1; x += 32) {
    const uint32_t k = keys[x];
    high = max(high, k), low = min(low, k);
  }
  high = __reduce_max_sync(0xffffffffu, high);
  low = __reduce_min_sync(0xffffffffu, low);
  if (lane == 0) room.high[warp] = high, room.low[warp] = low;
  for (int i = tid; i < kBins; i += kThreads) bins[0][i] = 0, bins[1][i] = 0;
  __syncthreads();
#pragma unroll
  for (int w = 0; w < W; ++w) high = max(high, room.high[w]), low = min(low, room.low[w]);
  if (P > 1) {
    if (tid < P) *peer(&room.team_high[rank], tid) = high, *peer(&room.team_low[rank], tid) = low;
    team_sync();
    for (int i = 0; i < P; ++i) high = max(high, room.team_high[i]), low = min(low, room.team_low[i]);
  }
  // keys low .. low + span are counted; want of them, the highest, are kept with all above
  uint32_t span = high - low;
  int shift = max(0, 32 - __clz(span) - 8);
  bool exact = false;
  unsigned taken_before = 0, equal_before = 0;  // a thread's part of what the CTAs before this one have above the bin, and in it
#pragma unroll 1
  for (int pass = 0;; ++pass) {
    unsigned *mine = bins[pass & 1];
#pragma unroll 4
    for (int x = x0; x < x1; x += 32) {
      const uint32_t k = keys[x] - low;
      if (k <= span) atomicAdd(&mine[k >> shift], 1u);
    }
    meet();
    // thread i sums its bins over the team, the highest ones first
    unsigned own[kOwn], before[kOwn], sum = 0;
    const int top = kBins - kOwn * (tid + 1);
#pragma unroll
    for (int e = 0; e < kOwn; ++e) {
      own[e] = before[e] = 0;
#pragma unroll 4
      for (int i = 0; i < P; ++i) {
        const unsigned u = P > 1 ? *peer(mine + top + e, i) : mine[top + e];
        own[e] += u;
        if (i < rank) before[e] += u;
      }
      sum += own[e];
    }
    unsigned cum = sum;
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
      const unsigned x = __shfl_up_sync(0xffffffffu, cum, o);
      if (lane >= o) cum += x;
    }
    if (lane == 31) room.sum[warp] = cum;
    __syncthreads();
    for (int w = 0; w < warp; ++w) cum += room.sum[w];
    const unsigned upto = cum;
    cum -= sum;
    if (cum < want && want <= upto) {
#pragma unroll
      for (int e = kOwn - 1; e >= 0; --e) {
        if (cum < want && want <= cum + own[e]) room.bin = (unsigned)(top + e), room.want = want - cum, room.have = own[e];
        cum += own[e];
      }
    }
    __syncthreads();
    const int bin = (int)room.bin;
    equal_before = 0;
#pragma unroll
    for (int e = 0; e < kOwn; ++e) {
      if (top + e > bin) taken_before += before[e];
      if (top + e == bin) equal_before = before[e];
    }
    low += (uint32_t)bin << shift;
    want = room.want;
    exact = room.have == want;
    if (exact || shift == 0) break;
    span = (1u << shift) - 1u;
    shift = max(0, shift - 8);
    // read by others in the pass before the last one: its barrier is behind them
    if (pass > 0)
      for (int i = tid; i < kBins; i += kThreads) bins[(pass + 1) & 1][i] = 0;
    __syncthreads();
  }
  // kept: the keys from low on if exact, else those above it and the first `want` that equal it
  int above = 0, equal = 0;
#pragma unroll 4
  for (int x = x0; x < x1; x += 32) {
    const uint32_t k = keys[x];
    above += k > low || (exact && k == low);
    equal += !exact && k == low;
  }
  above = (int)__reduce_add_sync(0xffffffffu, (unsigned)above);
  equal = (int)__reduce_add_sync(0xffffffffu, (unsigned)equal);
  taken_before = __reduce_add_sync(0xffffffffu, taken_before);
  equal_before = __reduce_add_sync(0xffffffffu, equal_before);
  if (lane == 0) {
    room.scan[0][warp] = above, room.scan[1][warp] = equal;
    room.before[0][warp] = taken_before, room.before[1][warp] = equal_before;
  }
  __syncthreads();
  int taken = 0, seen = 0;  // by the CTAs and warps before; exact: what is in the bin is all kept
#pragma unroll
  for (int w = 0; w < W; ++w) {
    taken += room.before[0][w] + (exact ? room.before[1][w] : 0u), seen += exact ? 0u : room.before[1][w];
    if (w < warp) taken += room.scan[0][w], seen += room.scan[1][w];
  }
  taken += min(seen, (int)want);
  const unsigned below = (1u << lane) - 1;
#pragma unroll 1
  for (int x = x0; x - lane < x1; x += 32) {
    const uint32_t k = x < x1 ? keys[x] : 0u;  // no key is 0
    const unsigned eq = exact ? 0u : __ballot_sync(0xffffffffu, k == low && x < x1);
    const bool keep = x < x1 && (k > low || (k == low && (exact || seen + __popc(eq & below) < (int)want)));
    const unsigned kept = __ballot_sync(0xffffffffu, keep);
    if (keep) emit(taken + __popc(kept & below), x);
    seen += __popc(eq);
    taken += __popc(kept);
  }
}

// Shared memory of a CTA, in order: the warps' rings (before them the keys,
// after them the warps' partial outputs), the parts that the cluster's CTAs hand
// over, query codes of groups above 8, the own blocks, logits.
template <int D, int NR, int W> struct Room {
  static constexpr int kRows = 8 * NR;
  static constexpr int kStage = 2 * kBlock * D;
  static constexpr int kStages = D == 64 ? 4 : 2;  // blocks of a warp on their way
  static constexpr int kRing = W * kStages * kStage;
  static constexpr int kParts = (kRows * D / 4 + kMostCtas) * 16;
  static constexpr int kTile = sizeof(Codes<D>) * 32;  // codes of 8 rows
  static_assert(kRing >= kHeldKeys * 4 + 2 * kBins * 4, "the keys and their bins share the rings' memory");
  __host__ __device__ static int codes(int group) { return NR == 1 || group > kCodesMost ? 0 : (group + 7) / 8 * kTile; }
  __host__ __device__ static int bytes(int group, int own, int logits) {
    return 1024 + kRing + kParts + codes(group) + own * 4 + logits * 4;
  }
};

// Weights of the N parts of a row under their maximum: z[i] of each part's mean, and the whole's reference and sum.
template <int N> __device__ __forceinline__ float2 weigh(const float2 *ml, int step, float (&z)[N]) {
  float2 p[N];
  float m = -INFINITY, l = 0.f;
#pragma unroll
  for (int i = 0; i < N; ++i) p[i] = ml[i * step], m = fmaxf(m, p[i].x);
#pragma unroll
  for (int i = 0; i < N; ++i) {
    z[i] = p[i].x == -INFINITY ? p[i].y : p[i].y * ex2(p[i].x - m);
    l += z[i];
  }
  const float inv = inverse_sum(l);
#pragma unroll
  for (int i = 0; i < N; ++i) z[i] *= inv;
  return make_float2(m, l);
}

// CTAs that shared memory leaves room for on an SM (at d = 128, of 228 KB: 8 warps 140 KB and more; 4 warps 75 KB, three
// while a CTA's list is at most 688 blocks, else two; 2 warps 42 KB; above 8 rows 85 and 56 KB), so the registers that a
// thread may have: a partition's 512 x 32 among its warps, 168 for three of them and 255 for two.  At d = 128 the forms of
// 168 registers spill 80 to 140 bytes a thread, those of more than 8 rows 100 to 130 at 255 and that of 8 warps 20; at
// d = 64 it is 8 at most.
template <int NR, int W> constexpr int kResident = W == 8 ? 1 : W == 4 ? (NR == 1 ? 3 : 2) : (NR == 1 ? 5 : 4);

template <typename F, int D, int NR, int W>
__global__ void __launch_bounds__(W * 32, kResident<NR, W>)
    sparse_kernel(const Args a, const __grid_constant__ CUtensorMap kmap, const __grid_constant__ CUtensorMap vmap) {
  using R = Room<D, NR, W>;
  constexpr int kThreads = W * 32, OT = D / 16, kStage = R::kStage, kStages = R::kStages, kRows = R::kRows;
  extern __shared__ uint8_t smem_raw[];
  uint8_t *smem = smem_raw + (-smem_u32(smem_raw) & 1023u);  // swizzled tiles start at multiples of 1024
  const int group = a.c.group, P = a.P;
  uint32_t *keys = (uint32_t *)smem;
  unsigned(*bins)[kBins] = (unsigned(*)[kBins])(keys + kHeldKeys);
  float *parts = (float *)(smem + R::kRing);                     // [P][float4s of this CTA's slice]
  uint4 *codes = (uint4 *)(smem + R::kRing + R::kParts);         // [tile][kFours][lane], groups above 8
  int *own = (int *)((uint8_t *)codes + R::codes(group));
  float *held_logits = (float *)(own + a.own);
  __shared__ __align__(8) uint64_t full[W][kStages];
  __shared__ unsigned s_top;
  __shared__ ChooseRoom<W> choose_room;
  __shared__ float2 part_ml[W][kRows], team_ml[kMostCtas][kRows];
  __shared__ float row_z[kRows][kMostCtas], row_base[H2O_BLOCK_MAX_ROWS];
  const View &c = a.c;
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5, g = lane >> 2, t4 = lane & 3;
  const int64_t item = blockIdx.x / P;
  const int rank = blockIdx.x - (int)item * P;
  const int bh = (int)(item / a.l.n), t = (int)(item - (int64_t)bh * a.l.n), b = bh / c.H, h = bh - b * c.H;
  const Seq s = seq_of(a.l, b);
  if (!s.ok && h == 0 && t == 0 && rank == 0 && tid == 0) atomicOr(c.err, H2O_BERR_RANGE);
  if (t >= s.cnt) {  // the whole cluster; what comes behind this launch counts on the one before it too
    grid_dependency_wait();
    return;
  }
  if (a.l.n > 1) grid_launch_dependents();  // scores_kernel
  const Sight v = sight_of(a, s, t);
  const Rows q{a.q.p + t * a.q.st, a.q.sb, a.q.sh, a.q.st};  // the token's rows alone
  const Seq one{s.len, 1, v.end, true};
  int32_t *list = list_of(a, bh, t);
  const size_t scales = (size_t)bh * (c.cap / kBlock);
  const int per = ceil_div(v.S, P), slot0 = min(v.S, rank * per), slot1 = min(v.S, slot0 + per);  // this CTA's slots
  const bool all = v.nb <= a.n_blocks;
  const int nc = all ? 0 : v.nb - a.n_first - a.n_last;  // candidates n_first .. n_first + nc - 1
  const unsigned wanted = all ? 0u : (unsigned)(a.n_blocks - a.n_first - a.n_last);
  const bool near_list = per <= a.own;
  const bool shared = P > 1 && nc > kAloneKeys;  // each CTA has a share of the keys to make
  const int share = shared ? (ceil_div(nc, P) + 3) & ~3 : nc;
  const int lo = shared ? min(nc, rank * share) : 0;
  const int n = min(nc, lo + share) - lo;  // this CTA's candidates n_first + lo ..
  const int steps = wanted > 0 ? ceil_div(n, 16) : 0;
  const int8_t *bounds = c.bounds + (scales + a.n_first + lo) * 2 * D;
  const float *ksc = c.Ksc + scales + a.n_first + lo;
  const bool new_row = a.fused && v.S - 1 >= slot0 && v.S - 1 < slot1;  // the last slot's block

  // every CTA has begun before another one writes to its memory
  __syncwarp();
  if (P > 1) asm volatile("barrier.cluster.arrive.relaxed.aligned;" ::: "memory");
  Codes<D> qc;
  float qf[D / 64][16];
  unsigned top = 0;
  // every warp for itself; columns behind the last row repeat it
  if (NR == 1 && steps > 0) top = query_row<D>(q.at(b, h * group + min(g, group - 1), 0), qf);
  grid_dependency_wait();  // an append
  constexpr int kDeep = W > 4 ? 3 : 2;  // a warp's sixteens of blocks on their way at once
  Bounds<D> bd[kDeep];
#pragma unroll
  for (int i = 0; i < kDeep; ++i)
    if (warp + i * W < steps) bd[i].load(bounds, ksc, (warp + i * W) * 16, n);
  if (lane == 0) {
    for (int i = 0; i < kStages; ++i) mbar_init(&full[warp][i], 1);
    fence_mbar_init();
  }
  // The new row, while those loads are on their way; no other CTA touches its block.
  if (new_row && warp >= W - 2) {
    const bool is_v = warp == W - 2;
    append_rows<F, D, 1>(c, is_v, is_v ? a.v : a.k, b, h, s.len, s.len, s.len + 1);
    if (!is_v && lane == 0) {
      const size_t at = (size_t)bh * c.cap + s.len;
      c.pos[at] = a.position ? a.position[b] : s.len;
      c.score[at] = 0.f;
      c.low[at] = 0.f;
    }
    __threadfence();  // the codes are read back by a copy
    asm volatile("fence.proxy.async;" ::: "memory");
  }

  // ------------------------------------------------------------- the choice
  if (wanted > 0) {
    float inv;
    if constexpr (NR == 1) {
      inv = inverse_pow2(block_scale<I8>(__uint_as_float(__reduce_max_sync(0xffffffffu, top) << 16)));
      if (steps > 0) qc.set(qf, inv);
    } else {
      if (tid == 0) s_top = 0;
      __syncthreads();
      const int tiles = ceil_div(group, 8);
      for (int x = warp; x < tiles; x += W) {
        top = __reduce_max_sync(0xffffffffu, query_row<D>(q.at(b, h * group + min(8 * x + g, group - 1), 0), qf));
        if (lane == 0) atomicMax(&s_top, top);
      }
      __syncthreads();
      inv = inverse_pow2(block_scale<I8>(__uint_as_float(s_top << 16)));
      if (group <= kCodesMost) {
        for (int x = warp; x < tiles; x += W) {
          query_row<D>(q.at(b, h * group + min(8 * x + g, group - 1), 0), qf);
          qc.set(qf, inv);
          qc.put(codes + x * Codes<D>::kFours * 32);
        }
        __syncthreads();
      }
    }
    if (n > kHeldKeys) keys = (uint32_t *)logits_of(a, bh, t, 0) + lo;  // read before any logit is written
    for (int x0 = warp; x0 < steps; x0 += W * kDeep) {
#pragma unroll
      for (int i = 0; i < kDeep; ++i) {
        const int x = x0 + i * W;
        if (x >= steps) break;
        float2 m;
        if constexpr (NR == 1) {
          m = block_sums<D>(bd[i], qc);
        } else {
          m = make_float2(-INFINITY, -INFINITY);
          for (int y = 0; y < ceil_div(group, 8); ++y) {
            if (group <= kCodesMost) {
              qc.get(codes + y * Codes<D>::kFours * 32);
            } else {  // made anew for each 16 blocks
              query_row<D>(q.at(b, h * group + min(8 * y + g, group - 1), 0), qf);
              qc.set(qf, inv);
            }
            const float2 z = block_sums<D>(bd[i], qc);
            m = make_float2(fmaxf(m.x, z.x), fmaxf(m.y, z.y));
          }
        }
        // keys of a quad's two blocks are known to its four lanes
        const int j = x * 16 + (t4 & 1) * 8 + g;
        const uint32_t key = t4 & 1 ? key_bits(m.y, bd[i].ks[1]) : key_bits(m.x, bd[i].ks[0]);
        if (t4 < 2 && j < n) keys[j] = key;
        if (x + W * kDeep < steps) bd[i].load(bounds, ksc, (x + W * kDeep) * 16, n);
      }
    }
    __syncthreads();
    if (P > 1) team_wait();
    // Each slot's block, to the list and to the CTA that attends to it.
    if (shared) {
      choose_team<W>(keys, n, wanted, P, rank, bins, choose_room, [&](int slot, int x) {
        slot += a.n_first;
        const int to = slot / per;
        list[slot] = a.n_first + lo + x;
        if (near_list) peer(own, to)[slot - to * per] = a.n_first + lo + x;
      });
      team_sync();
    } else {
      auto mine = [&](int slot, int x) {
        slot += a.n_first;
        if (slot < slot0 || slot >= slot1) return;
        list[slot] = a.n_first + x;
        if (near_list) own[slot - slot0] = a.n_first + x;
      };
      if (nc <= kWarpKeys)  // every warp for itself, and its own slots alone
        choose_warp<kWarpKeys / 32>(keys, nc, wanted, [&](int slot, int x) {
          if ((slot + a.n_first - slot0) % W == warp) mine(slot, x);
        });
      else
        choose_team<W>(keys, nc, wanted, 1, 0, bins, choose_room, mine);
    }
  } else if (P > 1) {
    team_wait();
  }
  // the list's ends, and what is behind it
  const int first = all ? v.S : a.n_first, last = all ? v.S : v.S - a.n_last;
  if (rank == 0) {
    for (int i = tid; i < first; i += kThreads) list[i] = i;
    for (int i = last + tid; i < v.S; i += kThreads) list[i] = v.nb - v.S + i;
    for (int i = v.S + tid; i < a.n_blocks; i += kThreads) list[i] = -1;
  }
  fence_proxy_async_smem();  // copies land where the keys were
  __syncthreads();           // the new row is there, every key has been read
  if (new_row && lane == 0) asm volatile("fence.proxy.async;" ::: "memory");
  auto block_of = [&](int slot) {
    if (slot < first) return slot;
    if (slot >= last) return v.nb - v.S + slot;
    return near_list ? own[slot - slot0] : list[slot];
  };

  // ----------------------------------------------------------- the attention
  // Logits: by own blocks in shared memory, or by slots in memory.  The host made room for all of a CTA's or for none
  // (per <= its own), in 64 bits: 256 rows of 2^18 blocks are 2^31 logits.
  const bool near = a.logits > 0;
  const int64_t row_step = near ? per * kBlock : c.cap;
  float *logits = near ? held_logits : logits_of(a, bh, t, 0) + slot0 * kBlock;
  uint8_t *ring = smem + warp * kStages * kStage;
  const uint64_t policy = l2_policy(false);
  bool lost = false;
  uint32_t phases = 0;
  // Scores: 8 threads to an own block, four entries each; kAhead of a thread's are on their way at once.
  constexpr int kAhead = 4;
  const bool alone = a.l.n == 1;  // no other token's weights meet these
  float *score = c.score + (size_t)bh * c.cap, *low = c.low + (size_t)bh * c.cap;
  float4 old[kAhead], less[kAhead];
  auto entry_of = [&](int y) {  // the first of the thread's y-th four, -1 behind the last
    const int slot = slot0 + tid / 8 + y * (kThreads / 8);
    return slot < slot1 ? block_of(slot) * kBlock + tid % 8 * 4 : -1;
  };
  auto load_scores = [&](int y, int at) {
    const int j = entry_of(y);
    if (j >= 0) old[at] = *(const float4 *)(score + j), less[at] = *(const float4 *)(low + j);
  };
  for (int row0 = 0; row0 < group; row0 += kRows) {
    float ks, vs;  // the next block's scales, a block ahead
    auto scales_of = [&](int slot) {
      if (slot >= slot1) return;
      const size_t at = scales + block_of(slot);
      ks = c.Ksc[at], vs = c.Vsc[at];
    };
    auto fetch = [&](int i) {
      const int slot = slot0 + warp + i * W;
      if (slot >= slot1 || lane != 0 || lost) return;
      uint8_t *dst = ring + i % kStages * kStage;
      uint64_t *bar = &full[warp][i % kStages];
      const int row = bh * c.cap + block_of(slot) * kBlock;
      mbar_expect_tx(bar, kStage);
      tma_load_2d(dst, &kmap, bar, 0, row, policy);
      tma_load_2d(dst + kBlock * D, &vmap, bar, 0, row, policy);
    };
    for (int i = 0; i < kStages; ++i) fetch(i);
    scales_of(slot0 + warp);
    Tile<F, D, NR, false, true> tl;
    tl.begin(q, group, 0, one, b, h, row0, nullptr);
    for (int i = 0; slot0 + warp + i * W < slot1; ++i) {
      const int slot = slot0 + warp + i * W, blk = block_of(slot);
      const float ks_now = ks, vs_now = vs;
      scales_of(slot + W);
      const int st = i % kStages;
      if (!lost && !mbar_wait(&full[warp][st], phases >> st & 1)) lost = true;
      if (lost) break;
      phases ^= 1u << st;
      uint8_t *kt = ring + st * kStage;
      tl.block(kt, kt + kBlock * D, ks_now, vs_now, blk, v.end - blk * kBlock, nullptr,
               [&](int r, int j, float s0, float s1, float s2, float s3) {
                 if (!a.accumulate) return;
                 float *lg = logits + (row0 + r) * row_step + (slot - slot0) * kBlock + (j - blk * kBlock);
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
    // the own entries' scores are on their way while the parts meet
    if (row0 == 0 && alone && a.accumulate) {
#pragma unroll
      for (int y = 0; y < kAhead; ++y) load_scores(y, y);
    }
    __syncthreads();
    // The CTA's parts become one, and go to the CTA that joins their slice: four dimensions of a row to a thread.
    const int rows = min(group - row0, kRows), fours = rows * (D / 4), slice = ceil_div(fours, P);
    for (int x = tid; x < fours; x += kThreads) {
      const int r = x / (D / 4), d0 = x % (D / 4) * 4;
      float z[W];
      const float2 ml = weigh<W>(&part_ml[0][r], kRows, z);
      float4 o = make_float4(0.f, 0.f, 0.f, 0.f);
#pragma unroll
      for (int i = 0; i < W; ++i) {
        const float4 e = *(const float4 *)(po + (i * kRows + r) * D + d0);
        o.x = fmaf(e.x, z[i], o.x), o.y = fmaf(e.y, z[i], o.y), o.z = fmaf(e.z, z[i], o.z), o.w = fmaf(e.w, z[i], o.w);
      }
      const int to = x / slice;
      *(float4 *)peer(parts + (rank * slice + x - to * slice) * 4, to) = o;
      if (d0 < P * 4)  // (m, l) to every CTA, by as many threads
        for (int i = d0 / 4; i < P; i += D / 4) *peer(&team_ml[rank][r], i) = ml;
    }
    team_sync();
    // A row's parts, kMostCtas lanes to a row: their weights, the row's sum.
    for (int x = tid; x < kRows * kMostCtas; x += kThreads) {
      const int r = x / kMostCtas, i = x % kMostCtas;
      const float2 p = i < P && r < rows ? team_ml[i][r] : make_float2(-INFINITY, 0.f);
      float m = p.x;
#pragma unroll
      for (int o = 1; o < kMostCtas; o <<= 1) m = fmaxf(m, __shfl_xor_sync(0xffffffffu, m, o));
      const float z = p.x == -INFINITY ? p.y : p.y * ex2(p.x - m);
      float l = z;
#pragma unroll
      for (int o = 1; o < kMostCtas; o <<= 1) l += __shfl_xor_sync(0xffffffffu, l, o);
      const bool any = l > 0.f || l != l;
      row_z[r][i] = any ? z / l : 0.f;
      if (i == 0 && r < rows) {
        const float base = weight_base(m, l);
        const int hq = h * group + row0 + r;
        row_base[row0 + r] = base;
        if (rank == 0 && a.lse)
          a.lse[((size_t)b * c.H * group + hq) * a.l.n + t] = any ? (m + log2f(l)) * kLn2 : -INFINITY;
      }
    }
    __syncthreads();
    for (int y = tid; y < slice && rank * slice + y < fours; y += kThreads) {
      const int x = rank * slice + y, r = x / (D / 4), d0 = x % (D / 4) * 4, hq = h * group + row0 + r;
      float4 o = make_float4(0.f, 0.f, 0.f, 0.f);
#pragma unroll 4
      for (int i = 0; i < P; ++i) {
        const float4 e = *(const float4 *)(parts + (i * slice + y) * 4);
        const float z = row_z[r][i];
        o.x = fmaf(e.x, z, o.x), o.y = fmaf(e.y, z, o.y), o.z = fmaf(e.z, z, o.z), o.w = fmaf(e.w, z, o.w);
      }
      const __nv_bfloat162 p0 = __floats2bfloat162_rn(o.x * kPartUp, o.y * kPartUp),
                           p1 = __floats2bfloat162_rn(o.z * kPartUp, o.w * kPartUp);
      *(uint2 *)(const_cast<__nv_bfloat16 *>(a.out.at(b, hq, t)) + d0) =
          make_uint2(*(const uint32_t *)&p0, *(const uint32_t *)&p1);
    }
    if (row0 + kRows < group) {
      fence_proxy_async_smem();  // the next rows' copies land where the parts were
      team_sync();               // and every part has been read
    }
  }

  // -------------------------------------------------------------- the scores
  // Several tokens: the weights go where the first row's logits were, for scores_kernel.
  float *sums = logits_of(a, bh, t, 0) + slot0 * kBlock;
  if (a.accumulate) {
    for (int y0 = 0; entry_of(y0) >= 0; y0 += kAhead) {
      if (y0 > 0 && alone) {
#pragma unroll
        for (int y = 0; y < kAhead; ++y) load_scores(y0 + y, y);
      }
#pragma unroll
      for (int y = 0; y < kAhead; ++y) {
        const int j = entry_of(y0 + y);
        if (j < 0) break;
        const int x = (tid / 8 + (y0 + y) * (kThreads / 8)) * kBlock + tid % 8 * 4;
        float4 w = make_float4(0.f, 0.f, 0.f, 0.f);
#pragma unroll 8
        for (int r = 0; r < group; ++r) {
          const float4 u = *(const float4 *)(logits + x + r * row_step);
          const float e = row_base[r];
          w.x += ex2(u.x - e), w.y += ex2(u.y - e), w.z += ex2(u.z - e), w.w += ex2(u.w - e);
        }
        if (alone)
          store_scores(score + j, low + j, v.end - j, old[y], less[y], w);
        else
          *(float4 *)(sums + x) = w;
      }
    }
  }
  if (new_row && warp == W - 1) bound_block<F, D>(c, bh, s.len / kBlock, s.total);  // for the calls to come
}

// The weights of several tokens' rows, added in the tokens' order: a CTA has
// kSlice blocks of a head, four entries a thread, and finds each token's slots
// of them first (a warp a token); the rows' weights are summed already.
constexpr int kSlice = 32, kScoreThreads = kSlice * 8;
__global__ void __launch_bounds__(kScoreThreads) scores_kernel(const Args a, int slices) {
  extern __shared__ int slot_of[];  // [n][kSlice], -1: not chosen
  const View &c = a.c;
  const int bh = blockIdx.x / slices, j0 = (blockIdx.x - bh * slices) * kSlice, b = bh / c.H;
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  const Seq s = seq_of(a.l, b);
  if (s.cnt == 0 || j0 * kBlock >= s.total) {
    grid_dependency_wait();
    return;
  }
  float *score = c.score + (size_t)bh * c.cap, *low = c.low + (size_t)bh * c.cap;
  const int mine = threadIdx.x / 8, j = (j0 + mine) * kBlock + threadIdx.x % 8 * 4;
  grid_dependency_wait();
  const bool in = j < s.total;
  float4 old = make_float4(0.f, 0.f, 0.f, 0.f), less = old;
  if (in) old = *(const float4 *)(score + j), less = *(const float4 *)(low + j);
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
    const float4 w = *(const float4 *)(logits_of(a, bh, t, 0) + slot * kBlock + threadIdx.x % 8 * 4);
    const int left = sight_of(a, s, t).end - j;  // entries that the token does not see keep their score
    if (left > 0) old.x = add_score(old.x, less.x, w.x);
    if (left > 1) old.y = add_score(old.y, less.y, w.y);
    if (left > 2) old.z = add_score(old.z, less.z, w.z);
    if (left > 3) old.w = add_score(old.w, less.w, w.w);
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

struct Launch {
  cudaLaunchConfig_t cfg = {};
  cudaLaunchAttribute at[2];
  Launch(unsigned ctas, int threads, int smem, int cluster, bool after, cudaStream_t st) {
    cfg.gridDim = dim3(ctas);
    cfg.blockDim = dim3(threads);
    cfg.dynamicSmemBytes = smem;
    cfg.stream = st;
    cfg.attrs = at;
    if (cluster > 1) {
      at[cfg.numAttrs].id = cudaLaunchAttributeClusterDimension;
      at[cfg.numAttrs++].val.clusterDim = {(unsigned)cluster, 1, 1};
    }
    if (after) {
      at[cfg.numAttrs].id = cudaLaunchAttributeProgrammaticStreamSerialization;
      at[cfg.numAttrs++].val.programmaticStreamSerializationAllowed = 1;
    }
  }
};

template <typename F, int D, int NR, int W> SmemLimit &limit_of() {  // one for all launches of a kernel
  static SmemLimit limit;
  return limit;
}

template <typename F, int D, int NR, int W>
cudaError_t sparse_w(Args a, const CUtensorMap &kmap, const CUtensorMap &vmap, cudaStream_t st) {
  const int own = (std::min(a.c.cap / kBlock, a.n_blocks) + a.P - 1) / a.P;
  a.own = (std::min(own, kOwnMost) + 3) & ~3;
  const int64_t logits = (int64_t)a.c.group * own * kBlock;
  a.logits = a.accumulate && logits <= kLogitsMost ? (int)logits : 0;
  const int smem = Room<D, NR, W>::bytes(a.c.group, a.own, a.logits);
  const auto kernel = sparse_kernel<F, D, NR, W>;
  cudaError_t e = limit_of<F, D, NR, W>().raise((const void *)kernel, smem);
  if (e == cudaSuccess && a.P > 8)
    e = cudaFuncSetAttribute((const void *)kernel, cudaFuncAttributeNonPortableClusterSizeAllowed, 1);
  if (e != cudaSuccess) return e;
  const int64_t ctas = (int64_t)a.c.B * a.c.H * a.l.n * a.P;
  const Launch l((unsigned)ctas, W * 32, smem, a.P, a.l.appends && !a.fused, st);
  return cudaLaunchKernelEx(&l.cfg, kernel, a, kmap, vmap);
}

// Clusters of P CTAs of 8 warps, one an SM, that run at once: a cluster has to
// find its SMs in one GPC (16 heads of 100,000 entries: 35 us with 8 CTAs, for
// which not all find them on 152 SMs, 21 with 6; 8 heads of 262,000: 23 with 8,
// 21 with 12, 37 with 16).  Asked once for each device.
template <typename F, int D, int NR> int clusters_at_once(int P) {
  static std::atomic<int> known[SmemLimit::kDevices][kMostCtas + 1] = {};
  int dev = 0;
  if (cudaGetDevice(&dev) != cudaSuccess || dev < 0 || dev >= SmemLimit::kDevices) return 0;
  int n = known[dev][P].load(std::memory_order_relaxed);
  if (n == 0) {
    const auto kernel = sparse_kernel<F, D, NR, 8>;
    const int smem = Room<D, NR, 8>::bytes(8 * NR, kOwnMost, kLogitsMost);
    const Launch l(P, 8 * 32, smem, P, false, nullptr);
    if (P > 8) cudaFuncSetAttribute((const void *)kernel, cudaFuncAttributeNonPortableClusterSizeAllowed, 1);
    if (limit_of<F, D, NR, 8>().raise((const void *)kernel, smem) != cudaSuccess ||
        cudaOccupancyMaxActiveClusters(&n, kernel, &l.cfg) != cudaSuccess) {
      cudaGetLastError();  // no answer: no cluster
      return 0;
    }
    if (n == 0) n = -1;  // an answer too
    known[dev][P].store(n, std::memory_order_relaxed);
  }
  return n;
}

// CTAs of 8 warps, one an SM, while they all fit at once, as many to a token as
// do; more tokens than SMs: CTAs of 4 warps, three an SM (two with 9 rows and
// more, or lists above 688 blocks); more than those hold: of 2 warps, five an SM
// (four), since the way from lengths to outputs is then hidden by other tokens
// and not by more warps.  Measured, us a call (2 / 4 / 8 warps, the best P of
// each), 64 blocks a token but the last (16): 8 heads of 8,000 entries 25 / 16 /
// 13; 128 of 3,000 to 8,400 44 / 30 / 28; 192 of 4,000 to 8,000 48 / 36 / 49; 512
// of them 84 / 107 / 104; 3,584 of 700 to 2,047 142 / 163 / 284.  With the weights
// whole the last four take 29, 36, 88 (floor 45) and 146 (floor 78).
template <typename F, int D, int NR>
cudaError_t sparse_n(Args &a, const CUtensorMap &kmap, const CUtensorMap &vmap, cudaStream_t st) {
  // counts leave tokens out: half of those behind the first, on the average
  const int64_t heads = (int64_t)a.c.B * a.c.H;
  const int64_t items = a.l.counts ? heads * (a.l.n + 1) / 2 : heads * a.l.n;
  const int blocks = a.c.cap / kBlock, sms = a.c.sms;
  a.P = 1;
  if (items <= sms) {
    for (int p : {2, 3, 4, 6, 8, 10, 12, 14, 16})
      if (items * p <= sms && blocks >= 8 * p && items <= clusters_at_once<F, D, NR>(p)) a.P = p;
    return sparse_w<F, D, NR, 8>(a, kmap, vmap, st);
  }
  constexpr int kFours = NR == 1 ? 3 : 2;  // CTAs of 4 warps on an SM
  if (2 * items <= kFours * sms && blocks >= 16) a.P = 2;
  if (items > kFours * sms) return sparse_w<F, D, NR, 2>(a, kmap, vmap, st);
  return sparse_w<F, D, NR, 4>(a, kmap, vmap, st);
}

template <typename F, int D>
cudaError_t sparse_d(Args &a, const CUtensorMap &kmap, const CUtensorMap &vmap, cudaStream_t st) {
  cudaError_t e = a.c.group <= 8 ? sparse_n<F, D, 1>(a, kmap, vmap, st) : sparse_n<F, D, 2>(a, kmap, vmap, st);
  if (e != cudaSuccess || !a.accumulate || a.l.n == 1) return e;
  const int64_t heads = (int64_t)a.c.B * a.c.H;
  const int slices = (a.c.cap / kBlock + kSlice - 1) / kSlice;
  const Launch s((unsigned)(heads * slices), kScoreThreads, a.l.n * kSlice * 4, 1, true, st);
  return cudaLaunchKernelEx(&s.cfg, scores_kernel, a, slices);
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
  Args a{c, l, q, out, lse, blocks, causal, accumulate, n_blocks, n_first, n_last,
               fused, k ? *k : none, v ? *v : none, position, 1, 0, 0};
  if (c.kv == H2O_KV_E4M3)
    return c.d == 128 ? sparse_d<E4M3, 128>(a, kmap, vmap, st) : sparse_d<E4M3, 64>(a, kmap, vmap, st);
  return c.d == 128 ? sparse_d<I8, 128>(a, kmap, vmap, st) : sparse_d<I8, 64>(a, kmap, vmap, st);
}

}  // namespace blk
}  // namespace h2o
