// block_attend.cu — attention of a group's query rows over a block-scaled
// 8-bit cache, each entry's weights added to its score.
//
//   s_rj = (q_r . code_j) ks_j / sqrt(d),  j < end_r
//   LSE_r = ln sum_j exp s_rj;  O_r = sum_j exp(s_rj - LSE_r) vs_j code_j
//   score_j += sum_r exp(s_rj - LSE_r)
//
// Rows r of a cached head: r = t * group + g for query token t and query head
// g of the group.
//
// attend_kernel: the blocks of all sequences and heads, in one list, are cut
// into as many equal runs as the device has workers, so a ragged batch, one
// long sequence and many short ones keep every SM equally busy.  A worker is
// a warp for each 8 * NR rows (MT warps); it streams its run's K and V blocks
// through its own ring of TMA loads (128- or 64-byte swizzle, so the
// fragment reads below meet no bank conflict), with no barrier shared with
// other workers.  Per block of 32 entries the codes become f16 in registers
// (exact), once for all of the warp's rows, and are the A operand (16 rows of
// the matrix instruction) of both products, the query rows the 8 columns of
// B: S^T = K Q^T and O^T = V^T P^T on mma.sync m16n8k16 with fp32 sums.  A
// lane's K words hold four consecutive dimensions of an entry and its V words
// four dimensions of two entries: the instruction sums over any order of k
// and its rows may be any dimensions, so the loads stay 16 bytes wide and
// need no transpose.  P^T leaves S^T's accumulator layout for B's by one
// movmatrix for each 8 x 8.
// Where a head's blocks lie in more than one run, the partial (m, l, O) go to
// scratch memory; the runs' and heads' boundaries form a staircase, so
// (worker + head) numbers the partials without gaps or collisions.
//
// Why mma.sync and not tcgen05: a decode step has 1 to 16 rows per cached
// head, so the step is bound by the codes' bytes (2 d per entry), and the
// codes have to pass through registers anyway to become f16; tcgen05 would
// read them back from shared memory, 4 more bytes of its traffic per code.
//
// finish_kernel: joins the partials of a row to O and LSE, and turns the
// logits that the first kernel left in scratch memory into weights: 4 bytes
// written and read per row and entry, instead of K read again.
//
// head_kernel: few and short heads, a CTA each, in one launch.
//
// Bound by memory up to about 16 rows: 8 heads of 262,000 entries, 537 MB of
// codes, 85 us without scores, 93 % of the copy rate; with the logits of 8 rows
// 104 us, and about 20 us of the finishing launch.  Above, by the products'
// instructions: 32 heads of 16,384 entries, d = 128, 256 rows 364 us, 189
// TFLOP/s; each warp of a worker converts the block for itself, and above 64
// rows the codes are read once for every 64.  With scores the logits' 8 bytes a
// row and entry come on top: 64 rows 96 us without, 154 us with them.
#include "block_tile.cuh"

namespace h2o {
namespace blk {
namespace {

// ------------------------------------------------------------ runs of blocks
// Warp-collective sum over the sequences of ceil(total / unit).
__device__ __forceinline__ int sum_units(const Lens &l, int B, int unit) {
  int n = 0;
  for (int b = threadIdx.x & 31; b < B; b += 32) n += ceil_div(seq_of(l, b).total, unit);
  return __reduce_add_sync(0xffffffffu, n);
}
// Warp-collective: the sequence that holds item x of the list in which each
// sequence has H * ceil(total / unit) items; x becomes the index among its
// items and `blocks_before` the blocks of the sequences before it, per head.
__device__ __forceinline__ int find_seq(const Lens &l, int B, int H, int unit, int &x, int &blocks_before) {
  const int lane = threadIdx.x & 31;
  blocks_before = 0;
  for (int b0 = 0;; b0 += 32) {
    const int total = b0 + lane < B ? seq_of(l, b0 + lane).total : 0;
    int items = H * ceil_div(total, unit), blocks = ceil_div(total, kBlock);
    const int mine = items, mine_blocks = blocks;
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
      const int a = __shfl_up_sync(0xffffffffu, items, o), z = __shfl_up_sync(0xffffffffu, blocks, o);
      if (lane >= o) items += a, blocks += z;
    }
    const unsigned here = __ballot_sync(0xffffffffu, x < items);
    if (here || b0 + 32 >= B) {
      const int src = here ? __ffs(here) - 1 : 31;
      x -= __shfl_sync(0xffffffffu, items - mine, src);
      blocks_before += __shfl_sync(0xffffffffu, blocks - mine_blocks, src);
      return b0 + src;
    }
    x -= __shfl_sync(0xffffffffu, items, 31);
    blocks_before += __shfl_sync(0xffffffffu, blocks, 31);
  }
}
// Workers of a list: no run is empty, so the partials of a head are those of
// every worker between its first and its last block's.
__device__ __forceinline__ int run_start(int w, int blocks, int workers) {
  return (int)((int64_t)w * blocks / workers);
}
// The worker whose run holds block x.
__device__ __forceinline__ int worker_of(int x, int blocks, int workers) {
  return (int)((((int64_t)x + 1) * workers - 1) / blocks);
}

// A place in the list of blocks.
struct Cursor {
  int b, h, blk, nblk;
  Seq s;
  __device__ __forceinline__ void seek(const Lens &l, int B, int H, int x) {
    int before;
    b = find_seq(l, B, H, kBlock, x, before);
    s = seq_of(l, b);
    nblk = ceil_div(s.total, kBlock);
    h = x / nblk;
    blk = x - h * nblk;
  }
  __device__ __forceinline__ void next(const Lens &l, int B, int H) {
    if (++blk < nblk) return;
    blk = 0;
    if (++h < H) return;
    h = 0;
    do {
      if (++b >= B) return;
      s = seq_of(l, b);
      nblk = ceil_div(s.total, kBlock);
    } while (nblk == 0);
  }
};

// A worker's rows: MT warps of NR tiles of 8 rows.  Up to 8 rows one warp has
// one tile (D / 4 registers of O); more rows are tiles of 16, on up to four
// warps that share the worker's ring.  8 to 16 warps and 96 to 192 KB of ring
// to an SM; Q is in registers where a worker is one warp.  At d = 128 twelve
// warps of 168 registers, at d = 64 also sixteen of 128, measured faster than
// the other: 32 heads of 16,384 entries, d = 128, 32 rows 60 / 89 us, 64 rows
// 96 / 139 us; d = 64, 32 rows 37 / 38 us, 64 rows (sixteen) 60 / 60 us.  From
// 17 rows on at d = 128 the 168 registers spill about 140 bytes.
template <int D, int NR, int MT> struct Cfg {
  static constexpr int kTeams = MT == 2 ? 6 : MT == 4 && D == 128 ? 3 : 4;  // workers of a CTA, mostly of 12 warps in all
  static constexpr int kWarps = kTeams * MT;
  static constexpr int kCtas = NR == 1 ? (D == 64 ? 4 : 3) : MT == 1 ? 2 : 1;  // per SM
  static constexpr int kStage = 2 * kBlock * D;
  static constexpr bool kQSmem = MT > 1;
  static constexpr int kRing = MT == 4 && D == 64 ? 131072 : MT > 1 ? 147456 : NR == 2 ? 98304 : kCtas == 4 ? 49152 : 65536;
  static constexpr int kStages = kRing / (kTeams * kStage);
  static constexpr int kQBytes = kQSmem ? kWarps * NR * D * 16 : 0;
  static constexpr int kSmem = 1024 + kTeams * kStages * kStage + kQBytes + kTeams * kStages * 16;
};
constexpr int kMaxWorkers = 16;  // of an SM

struct Args {
  View c;
  Lens l;
  Rows q, out;
  float *lse;
  float2 *ml;  // [workers + B*H][max_rows]  partial reference and sum
  float *po;   // [workers + B*H][max_rows][d]  partial output, normalised, times kPartDown
  int causal, accumulate, workers;
  int rows;  // n * group: rows of a head in this call
  int streams;  // the codes pass through L2 once: they make way first
};

template <typename F, int D, int NR, int MT>
__global__ void __launch_bounds__(Cfg<D, NR, MT>::kWarps * 32, Cfg<D, NR, MT>::kCtas)
    attend_kernel(const Args a, const __grid_constant__ CUtensorMap kmap, const __grid_constant__ CUtensorMap vmap) {
  using G = Cfg<D, NR, MT>;
  constexpr int KS = D / 16, OT = D / 16;
  constexpr int S = G::kStages;
  extern __shared__ uint8_t smem_raw[];
  uint8_t *smem = smem_raw + (-smem_u32(smem_raw) & 1023u);  // swizzled tiles start at multiples of 1024
  const View &c = a.c;
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  const int team = warp / MT, tile = warp - team * MT;
  const int g = lane >> 2, t = lane & 3;
  uint8_t *ring = smem + team * S * G::kStage;
  uint4 *qs = (uint4 *)(smem + G::kTeams * S * G::kStage) + (G::kQSmem ? warp * NR * (KS / 2) * 32 : 0);
  uint64_t *full = (uint64_t *)(smem + G::kTeams * S * G::kStage + G::kQBytes) + team * 2 * S, *empty = full + S;
  const int worker = team * gridDim.x + blockIdx.x;  // few runs: one for each CTA first

  if (tile == 0 && lane == 0) {
    for (int i = 0; i < S; ++i) {
      mbar_init(full + i, 1);
      mbar_init(empty + i, MT);
    }
    fence_mbar_init();
  }
  __syncthreads();

  const int blocks = c.H * sum_units(a.l, c.B, kBlock);
  const int workers = min(a.workers, blocks);
  const int x0 = worker < workers ? run_start(worker, blocks, workers) : 0;
  const int count = worker < workers ? run_start(worker + 1, blocks, workers) - x0 : 0;
  if (worker == 0 && tile == 0 && blockIdx.y == 0)  // refused sequences are reported once
    for (int b = lane; b < c.B; b += 32)
      if (!seq_of(a.l, b).ok) atomicOr(c.err, H2O_BERR_RANGE);
  if (count == 0) {
    grid_dependency_wait();
    return;
  }

  Cursor cur, ld;
  cur.seek(a.l, c.B, c.H, x0);
  ld = cur;
  int issued = 0, put = 0;
  const uint64_t policy = l2_policy(a.streams);
  auto issue = [&]() {  // the run's next block into its stage (leader warp)
    if (lane == 0) {
      uint8_t *dst = ring + put * G::kStage;
      const int row = (ld.b * c.H + ld.h) * c.cap + ld.blk * kBlock;
      mbar_expect_tx(full + put, G::kStage);
      tma_load_2d(dst, &kmap, full + put, 0, row, policy);
      tma_load_2d(dst + kBlock * D, &vmap, full + put, 0, row, policy);
    }
    ++issued;
    put = put + 1 == S ? 0 : put + 1;
    ld.next(a.l, c.B, c.H);
  };
  // Blocks that the append before this launch does not change are on their way while it still runs.
  if (tile == 0)
    while (issued < S && issued < count && (ld.blk + 1) * kBlock <= ld.s.len) issue();
  grid_dependency_wait();
  grid_launch_dependents();
  if (tile == 0)
    while (issued < S && issued < count) issue();

  const int row0 = (blockIdx.y * MT + tile) * (8 * NR);  // the warp's rows of the head
  const int nsc = c.cap / kBlock;
  Tile<F, D, NR, G::kQSmem, false> tl;
  int first_blk = 0;
  bool open = false, busy = true, lost = false;
  float ks, vs;
  {
    const size_t sc = (size_t)(cur.b * c.H + cur.h) * nsc + cur.blk;
    ks = c.Ksc[sc];
    vs = c.Vsc[sc];
  }

  int st = 0;
  uint32_t phase = 0;
  for (int i = 0; i < count; ++i) {
    const int bh = cur.b * c.H + cur.h;
    if (!open) {  // a head begins
      open = true;
      first_blk = cur.blk;
      if (MT > 1) busy = row0 < cur.s.cnt * c.group;  // else the warp has no row of this head
      if (busy) tl.begin(a.q, c.group, a.causal, cur.s, cur.b, cur.h, row0, qs);
    }
    const float ks_now = ks, vs_now = vs;
    const int blk = cur.blk, rest = cur.s.total - blk * kBlock;
    const int ab = cur.b, ah = cur.h;
    const bool last_blk = blk + 1 == cur.nblk;
    cur.next(a.l, c.B, c.H);
    if (i + 1 < count) {  // the next block's scales, a block ahead
      const size_t sc = (size_t)(cur.b * c.H + cur.h) * nsc + cur.blk;
      ks = c.Ksc[sc];
      vs = c.Vsc[sc];
    }
    uint8_t *kt = ring + st * G::kStage, *vt = kt + kBlock * D;
    if (!mbar_wait(full + st, phase)) {
      lost = true;
      break;
    }
    if (MT > 1 && tile == 0 && i > 0 && issued < count) {  // the stage of block i - 1, once every warp has read it
      if (!mbar_wait(empty + put, st == 0 ? phase ^ 1 : phase)) {
        lost = true;
        break;
      }
      issue();
    }
    if (busy)
      tl.block(kt, vt, ks_now, vs_now, blk, rest, qs, [&](int r, int j, float s0, float s1, float s2, float s3) {
        if (!a.accumulate) return;
        float *lg = c.logits + ((size_t)bh * c.max_rows + row0 + r) * c.cap + j;
        lg[0] = s0, lg[8] = s1, lg[16] = s2, lg[24] = s3;
      });
    // this warp has read the stage
    __syncwarp();
    if (MT > 1) {
      if (lane == 0) mbar_arrive(empty + st);
    } else if (issued < count) {
      issue();
    }
    if (++st == S) st = 0, phase ^= 1;
    if (i + 1 < count && !last_blk) continue;
    open = false;
    if (!busy) continue;
    const bool whole = first_blk == 0 && last_blk;  // no other worker holds a part of this head
    const size_t slot = ((size_t)worker + bh) * c.max_rows;
    const float back = tl.unit(), part = back * kPartDown;
#pragma unroll
    for (int n = 0; n < NR; ++n)
#pragma unroll
      for (int u = 0; u < 2; ++u) {
        const float l = tl.sum(n, u);
        if (!(tl.live >> (2 * n + u) & 1)) continue;
        const int r = row0 + 8 * n + 2 * t + u;
        if (g == 0) a.ml[slot + r] = make_float2(tl.m[n][u], l);
        // the lane's D/8 dimensions: g D/8 + 2 j (accumulator u) and + 1 (2 + u)
        if (whole) {
          const int tok = r / c.group, hq = ah * c.group + r % c.group;
          const bool any = l > 0.f || l != l;
          const float inv = any ? 1.f / l : 0.f;
          uint32_t *dst = (uint32_t *)(const_cast<__nv_bfloat16 *>(a.out.at(ab, hq, tok)) + g * (D / 8));
          uint32_t w[OT];
#pragma unroll
          for (int j = 0; j < OT; ++j) {
            const __nv_bfloat162 b2 = __floats2bfloat162_rn(tl.o[n][j][u] * inv * back, tl.o[n][j][2 + u] * inv * back);
            w[j] = *(const uint32_t *)&b2;
          }
#pragma unroll
          for (int j = 0; j < OT; j += 4) *(uint4 *)(dst + j) = make_uint4(w[j], w[j + 1], w[j + 2], w[j + 3]);
          if (a.lse && g == 0)
            a.lse[((size_t)ab * c.H * c.group + hq) * a.l.n + tok] = any ? (tl.m[n][u] + log2f(l)) * kLn2 : -INFINITY;
        } else {
          const float inv = inverse_sum(l);
          float *dst = a.po + (slot + r) * D + g * (D / 8);
#pragma unroll
          for (int j = 0; j < OT; j += 2)
            *(float4 *)(dst + 2 * j) = make_float4(tl.o[n][j][u] * inv * part, tl.o[n][j][2 + u] * inv * part,
                                                   tl.o[n][j + 1][u] * inv * part, tl.o[n][j + 1][2 + u] * inv * part);
        }
      }
  }
  if (lost) {  // a copy never arrived: report, and let what is in flight land before the memory goes
    if (lane == 0) atomicOr(c.err, H2O_BERR_INTERNAL);
    if (tile == 0)
      for (int i = 0; i < S; ++i) mbar_wait(full + i, i >= st ? phase : phase ^ 1);
  }
}

// --------------------------------------------------------- one CTA per head
constexpr int kHeadCap = 512;  // entries

// A head of at most kHeadCap entries and 8 rows in one CTA, and with it the
// append of a step, where the heads fit the device at once: one launch instead
// of three that depend on each other.  Measured, us a step of 50 in a graph, this
// form / the other: 32 heads of 256 entries 6.3 / 8.5, of 512 7.9 / 9.4, of
// 1024 11.6 / 9.0; 128 cached heads x 4, 300 entries 8.6 / 11.8; 256 heads of
// 512 12.5 / 14.9; 1024 heads of 512 47.3 / 31.0.  Each warp takes every W-th block through two stages of its
// own; the warp of a block that receives new rows quantises them first.  The
// logits stay in shared memory; when every warp is done the CTA joins the
// rows' outputs and adds the weights to the scores.
template <typename F, int D, int W>
__global__ void __launch_bounds__(W * 32, W == 4 ? 3 : 1)
    head_kernel(const Args a, const Rows k, const Rows v, const int32_t *__restrict__ position,
                const __grid_constant__ CUtensorMap kmap, const __grid_constant__ CUtensorMap vmap) {
  constexpr int S = 2, OT = D / 16, kStage = 2 * kBlock * D;
  extern __shared__ uint8_t smem_raw[];
  uint8_t *smem = smem_raw + (-smem_u32(smem_raw) & 1023u);  // swizzled tiles start at multiples of 1024
  float *logits = (float *)(smem + W * S * kStage);          // [rows][cap]
  __shared__ uint64_t full[W][S];
  __shared__ float2 part_ml[W][8];
  __shared__ float row_lse[8];
  const View &c = a.c;
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5, g = lane >> 2, t = lane & 3;
  const int bh = blockIdx.x, b = bh / c.H, h = bh - b * c.H;
  const Seq s = seq_of(a.l, b);
  if (!s.ok && h == 0 && threadIdx.x == 0) atomicOr(c.err, H2O_BERR_RANGE);
  if (s.cnt == 0) return;  // neither rows nor queries
  if (lane == 0) {
    for (int i = 0; i < S; ++i) mbar_init(&full[warp][i], 1);
    fence_mbar_init();
  }
  __syncwarp();
  const int nblk = ceil_div(s.total, kBlock);
  uint8_t *ring = smem + warp * S * kStage;
  const uint64_t policy = l2_policy(a.streams);
  auto fetch = [&](int i) {  // the warp's i-th block into its stage
    const int blk = warp + i * W, base = blk * kBlock;
    if (blk >= nblk) return;
    if (a.l.appends && base + kBlock > s.len) {
      const int lo = max(s.len, base), hi = min(s.total, base + kBlock);
      append_rows<F, D>(c, false, k, b, h, s.len, lo, hi);
      append_rows<F, D>(c, true, v, b, h, s.len, lo, hi);
      if (c.bounds) {
        __syncwarp();  // the codes are there
        bound_block<F, D>(c, bh, blk, s.total);
      }
      const int j = base + lane;
      if (j >= lo && j < hi) {
        c.pos[(size_t)bh * c.cap + j] = (position ? position[b] : s.len) + (j - s.len);
        c.score[(size_t)bh * c.cap + j] = 0.f;
        c.low[(size_t)bh * c.cap + j] = 0.f;
      }
      // the codes are read back by the copy below
      __threadfence();
      asm volatile("fence.proxy.async;" ::: "memory");
      __syncwarp();
    }
    if (lane == 0) {
      asm volatile("fence.proxy.async;" ::: "memory");
      uint8_t *dst = ring + i % S * kStage;
      uint64_t *bar = &full[warp][i % S];
      mbar_expect_tx(bar, kStage);
      tma_load_2d(dst, &kmap, bar, 0, bh * c.cap + base, policy);
      tma_load_2d(dst + kBlock * D, &vmap, bar, 0, bh * c.cap + base, policy);
    }
  };
  for (int i = 0; i < S; ++i) fetch(i);

  Tile<F, D, 1, false, false> tl;
  tl.begin(a.q, c.group, a.causal, s, b, h, 0, nullptr);
  const size_t scales = (size_t)bh * (c.cap / kBlock);
  bool lost = false;
  for (int i = 0; warp + i * W < nblk; ++i) {
    const int blk = warp + i * W;
    const float ks = c.Ksc[scales + blk], vs = c.Vsc[scales + blk];
    if (!mbar_wait(&full[warp][i % S], i / S & 1)) {
      lost = true;
      break;
    }
    uint8_t *kt = ring + i % S * kStage;
    tl.block(kt, kt + kBlock * D, ks, vs, blk, s.total - blk * kBlock, nullptr,
             [&](int r, int j, float s0, float s1, float s2, float s3) {
               float *lg = logits + r * c.cap + j;
               lg[0] = s0, lg[8] = s1, lg[16] = s2, lg[24] = s3;
             });
    __syncwarp();  // this warp has read the stage
    fetch(i + S);
  }
  if (lost) {  // a copy never arrived: report, and wait for the other one before the memory goes
    if (lane == 0) atomicOr(c.err, H2O_BERR_INTERNAL);
    for (int i = 0; i < S; ++i) mbar_wait(&full[warp][i], 0), mbar_wait(&full[warp][i], 1);
  }
  __syncthreads();  // every warp is done with its ring: the partial outputs go there
  float *po = (float *)smem;  // [W][8][D]
  const float part = tl.unit() * kPartDown;
#pragma unroll
  for (int u = 0; u < 2; ++u) {
    const float l = tl.sum(0, u);
    const int r = 2 * t + u;
    if (g == 0) part_ml[warp][r] = make_float2(tl.m[0][u], l);
    const float inv = inverse_sum(l);
    float *dst = po + (warp * 8 + r) * D + g * (D / 8);
#pragma unroll
    for (int j = 0; j < OT; j += 2)
      *(float4 *)(dst + 2 * j) = make_float4(tl.o[0][j][u] * inv * part, tl.o[0][j][2 + u] * inv * part,
                                             tl.o[0][j + 1][u] * inv * part, tl.o[0][j + 1][2 + u] * inv * part);
  }
  __syncthreads();
  const int rows = s.cnt * c.group;
  for (int x = threadIdx.x; x < rows * (D / 4); x += W * 32) {
    const int r = x / (D / 4), d0 = x % (D / 4) * 4, tok = r / c.group, hq = h * c.group + r % c.group;
    float m = -INFINITY, l = 0.f;
    float4 o = make_float4(0.f, 0.f, 0.f, 0.f);
#pragma unroll
    for (int w = 0; w < W; ++w) m = fmaxf(m, part_ml[w][r].x);
    float z[W];  // the parts' sums of weights, under the row's maximum
#pragma unroll
    for (int w = 0; w < W; ++w) {
      const float2 p = part_ml[w][r];
      z[w] = p.x == -INFINITY ? p.y : p.y * ex2(p.x - m);
      l += z[w];
    }
    const bool any = l > 0.f || l != l;
    const float inv = any ? 1.f / l : 0.f;
#pragma unroll
    for (int w = 0; w < W; ++w) {
      const float4 e = *(const float4 *)(po + (w * 8 + r) * D + d0);
      const float x = z[w] * inv;
      o.x = fmaf(e.x, x, o.x), o.y = fmaf(e.y, x, o.y), o.z = fmaf(e.z, x, o.z), o.w = fmaf(e.w, x, o.w);
    }
    const __nv_bfloat162 p0 = __floats2bfloat162_rn(o.x * kPartUp, o.y * kPartUp),
                         p1 = __floats2bfloat162_rn(o.z * kPartUp, o.w * kPartUp);
    *(uint2 *)(const_cast<__nv_bfloat16 *>(a.out.at(b, hq, tok)) + d0) =
        make_uint2(*(const uint32_t *)&p0, *(const uint32_t *)&p1);
    if (d0 == 0) {
      row_lse[r] = weight_base(m, l);
      if (a.lse) a.lse[((size_t)b * c.H * c.group + hq) * a.l.n + tok] = any ? (m + log2f(l)) * kLn2 : -INFINITY;
    }
  }
  if (!a.accumulate) return;
  __syncthreads();
  float *sc = c.score + (size_t)bh * c.cap, *low = c.low + (size_t)bh * c.cap;
  for (int j = threadIdx.x; j < s.total; j += W * 32) {
    const float old = sc[j];
    float lost = low[j], w = 0.f;
    for (int r = 0; r < rows; ++r) w += ex2(logits[r * c.cap + j] - row_lse[r]);
    sc[j] = add_score(old, lost, w);
    low[j] = lost;
  }
}

// ------------------------------------------------------------------- finish
constexpr int kFinWarps = 8;

// (m, l) of two parts of a row, base 2.
__device__ __forceinline__ void join(float &m, float &l, float om, float ol) {
  const float mn = fmaxf(m, om);
  l = (m == -INFINITY ? l : l * ex2(m - mn)) + (om == -INFINITY ? ol : ol * ex2(om - mn));
  m = mn;
}

// Items of a CTA, the longer ones first.  Scores: W warps gather the LSE of a
// head's rows, and each lane adds the rows' weights of V fours of entries, in
// the rows' order.  Then a row's output to each warp, where its head lies in
// several runs: the lanes take its partials in turn.
// W = 8 where the parts and rows to gather are many, so that they are gathered
// once for 1024 V entries; else W = 1, eight items of 128 V entries to a CTA,
// which need no barrier.  Deep: few heads in many runs, whose rows' outputs
// then take a CTA each, its warps in turn for the partials.
template <int D, int W, int V, bool Deep>
__global__ void __launch_bounds__(kFinWarps * 32, 3) finish_kernel(const Args a) {
  constexpr int kChunk = 128 * W * V;              // entries of a score item
  constexpr int kPer = kFinWarps / W;              // score items of a CTA
  constexpr int kLanes = D / 4;                                     // lanes of an output row, 4 dimensions each
  constexpr int kGroups = (Deep ? kFinWarps : 1) * (32 / kLanes);   // groups of lanes that take the partials in turn
  const View &c = a.c;
  __shared__ float2 part_ml[W == 1 ? 1 : W][W == 1 ? 1 : H2O_BLOCK_MAX_ROWS];
  __shared__ float4 part_o[Deep ? kFinWarps : 1][kLanes];
  __shared__ float row_lse[kPer][H2O_BLOCK_MAX_ROWS];
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  const int blocks = c.H * sum_units(a.l, c.B, kBlock);
  const int workers = min(a.workers, blocks);
  const int64_t outs = (int64_t)c.B * c.H * a.rows;
  const int out_ctas = (int)(Deep ? outs : (outs + kFinWarps - 1) / kFinWarps);
  const int chunks = a.accumulate ? c.H * sum_units(a.l, c.B, kChunk) : 0;
  const int score_ctas = (chunks + kPer - 1) / kPer, ctas = score_ctas + out_ctas;
  // Where an item lies follows from the lengths alone; the first one is found while the launch before still runs.
  struct Item {
    int b, h, bh, r, j0, w0, w1, nblk;  // r: row of an output; j0: first entry of the item's scores; w0 .. w1: parts
    Seq s;
    bool some;
  };
  auto find = [&](int cta) {
    Item it;
    it.some = false;
    if (cta >= ctas) return it;
    int before = 0;
    if (cta >= score_ctas) {
      const int64_t item = Deep ? cta - score_ctas : (int64_t)(cta - score_ctas) * kFinWarps + warp;
      if (item >= outs) return it;
      it.r = (int)(item % a.rows), it.bh = (int)(item / a.rows), it.b = it.bh / c.H, it.h = it.bh - it.b * c.H;
      it.s = seq_of(a.l, it.b);
      for (int i = lane; i < it.b; i += 32) before += ceil_div(seq_of(a.l, i).total, kBlock);
      before = __reduce_add_sync(0xffffffffu, before);
      it.some = it.r / c.group < it.s.cnt;
    } else {
      int x = cta * kPer + warp / W;
      if (x >= chunks) return it;  // W = 8 has no such item
      it.b = find_seq(a.l, c.B, c.H, kChunk, x, before);
      it.s = seq_of(a.l, it.b);
      const int nch = ceil_div(it.s.total, kChunk);
      it.h = x / nch, it.bh = it.b * c.H + it.h, it.j0 = (x - it.h * nch) * kChunk;
      it.some = true;
    }
    it.nblk = ceil_div(it.s.total, kBlock);
    if (it.nblk > 0) {
      const int start = c.H * before + it.h * it.nblk;
      it.w0 = worker_of(start, blocks, workers), it.w1 = worker_of(start + it.nblk - 1, blocks, workers);
    }
    return it;
  };
  Item it = find(blockIdx.x);
  grid_dependency_wait();
  for (int cta = blockIdx.x; cta < ctas; cta += gridDim.x) {
    if (cta != blockIdx.x) it = find(cta);
    if (!it.some) continue;
    const int b = it.b, h = it.h, bh = it.bh, w0 = it.w0, w1 = it.w1;
    const Seq s = it.s;
    if (cta >= score_ctas) {
      const int r = it.r, tok = r / c.group, hq = h * c.group + r % c.group;
      const int d0 = lane % kLanes * 4;
      const bool writes = lane < kLanes && (!Deep || warp == 0);
      __nv_bfloat16 *dst = const_cast<__nv_bfloat16 *>(a.out.at(b, hq, tok)) + d0;
      float *lse = a.lse ? a.lse + ((size_t)b * c.H * c.group + hq) * a.l.n + tok : nullptr;
      if (it.nblk == 0) {  // no entry at all
        if (writes) *(uint2 *)dst = make_uint2(0u, 0u);
        if (lse && writes && lane == 0) *lse = -INFINITY;
        continue;
      }
      if (w0 == w1) continue;  // written by its worker
      const float2 *ml = a.ml + (size_t)bh * c.max_rows + r;
      const float *po = a.po + ((size_t)bh * c.max_rows + r) * D + d0;
      // Each group weighs its partials by its own maximum, then the groups meet; o is the weighted mean so far.
      constexpr int kBatch = Deep ? 8 : 4;  // partials on their way at once
      float m = -INFINITY, l = 0.f;
      float4 o = make_float4(0.f, 0.f, 0.f, 0.f);
      for (int wb = w0 + (Deep ? warp * (32 / kLanes) : 0) + lane / kLanes; wb <= w1; wb += kGroups * kBatch) {
        float4 v[kBatch];
        float2 p[kBatch];
        float mn = m;
#pragma unroll
        for (int i = 0; i < kBatch; ++i) {
          const size_t w = min(wb + i * kGroups, w1);  // the last one again counts as unseen
          p[i] = ml[w * c.max_rows];
          v[i] = *(const float4 *)(po + w * c.max_rows * D);
        }
#pragma unroll
        for (int i = 0; i < kBatch; ++i) {
          if (wb + i * kGroups > w1) p[i] = make_float2(-INFINITY, 0.f), v[i] = make_float4(0.f, 0.f, 0.f, 0.f);
          mn = fmaxf(mn, p[i].x);
        }
        const float own = m == -INFINITY ? l : l * ex2(m - mn);
        m = mn;
        l = own;
#pragma unroll
        for (int i = 0; i < kBatch; ++i) {
          if (p[i].x != -INFINITY) p[i].y *= ex2(p[i].x - m);
          l += p[i].y;
        }
        const float inv = inverse_sum(l), f = own * inv;
        o.x *= f, o.y *= f, o.z *= f, o.w *= f;
#pragma unroll
        for (int i = 0; i < kBatch; ++i) {
          const float z = p[i].y * inv;
          o.x = fmaf(v[i].x, z, o.x), o.y = fmaf(v[i].y, z, o.y), o.z = fmaf(v[i].z, z, o.z), o.w = fmaf(v[i].w, z, o.w);
        }
      }
      auto meet = [&](float om, float ol, float4 oo) {
        const float mn = fmaxf(m, om);
        float f = m == -INFINITY ? l : l * ex2(m - mn), z = om == -INFINITY ? ol : ol * ex2(om - mn);
        l = f + z;
        const float inv = inverse_sum(l);
        f *= inv, z *= inv;
        o.x = o.x * f + oo.x * z, o.y = o.y * f + oo.y * z, o.z = o.z * f + oo.z * z, o.w = o.w * f + oo.w * z;
        m = mn;
      };
#pragma unroll
      for (int off = kLanes; off < 32; off <<= 1)
        meet(__shfl_xor_sync(0xffffffffu, m, off), __shfl_xor_sync(0xffffffffu, l, off),
             make_float4(__shfl_xor_sync(0xffffffffu, o.x, off), __shfl_xor_sync(0xffffffffu, o.y, off),
                         __shfl_xor_sync(0xffffffffu, o.z, off), __shfl_xor_sync(0xffffffffu, o.w, off)));
      if constexpr (Deep) {  // every warp of the CTA is here: the item is the CTA's
        if (lane < kLanes) {
          part_o[warp][lane] = o;
          if (lane == 0) part_ml[warp][0] = make_float2(m, l);
        }
        __syncthreads();
        if (warp == 0)
          for (int i = 1; i < kFinWarps; ++i) meet(part_ml[i][0].x, part_ml[i][0].y, part_o[i][lane % kLanes]);
        __syncthreads();
      }
      const bool any = l > 0.f || l != l;
      if (writes) {
        const __nv_bfloat162 p0 = __floats2bfloat162_rn(o.x * kPartUp, o.y * kPartUp),
                             p1 = __floats2bfloat162_rn(o.z * kPartUp, o.w * kPartUp);
        *(uint2 *)dst = make_uint2(*(const uint32_t *)&p0, *(const uint32_t *)&p1);
        if (lse && lane == 0) *lse = any ? (m + log2f(l)) * kLn2 : -INFINITY;
      }
      continue;
    }
    const int j0 = it.j0 + warp % W * (128 * V) + lane * 4, rows = s.cnt * c.group;
    constexpr int kRows = 8 / V;  // rows whose logits are on their way at once
    const int j_last = max(0, s.total - 1) & ~3;
    const float *lg = c.logits + (size_t)bh * c.max_rows * c.cap;
    float *sc = c.score + (size_t)bh * c.cap, *low = c.low + (size_t)bh * c.cap;
    float4 w[V], old[V], lost[V], v[kRows][V];
    auto load = [&](int r0) {
#pragma unroll
      for (int i = 0; i < kRows; ++i)
#pragma unroll
        for (int y = 0; y < V; ++y)
          v[i][y] = *(const float4 *)(lg + (size_t)min(r0 + i, rows - 1) * c.cap + min(j0 + y * 128, j_last));
    };
    auto first = [&]() {
#pragma unroll
      for (int y = 0; y < V; ++y) {
        w[y] = make_float4(0.f, 0.f, 0.f, 0.f);
        old[y] = *(const float4 *)(sc + min(j0 + y * 128, j_last));
      }
      if (V == 1) load(0);
    };
    // One four a lane (many rows): its first loads are on their way while the LSE is gathered (draft tokens, a step of 50
    // in a graph: 44.5 us without, 37.8 us with it); four of them would not fit the registers beside that.
    if (V == 1) first();
    // Eight rows to a warp, a lane of each group of eight for one; the four groups, and the warps that have the same
    // rows, take the parts in turn.
    const float2 *ml = a.ml + (size_t)bh * c.max_rows;
    const int tiles = (rows + 7) / 8, sharing = W == 1 || tiles >= W ? 1 : W / max(tiles, 1);
    for (int tile = warp % W; tile < tiles * sharing; tile += W) {
      const int r = tile % tiles * 8 + (lane & 7), turn = tile / tiles;
      float m = -INFINITY, l = 0.f;
      if (r < rows)
        for (int wb = w0 + turn * 4 + (lane >> 3); wb <= w1; wb += sharing * 16) {
          float2 p[4];
#pragma unroll
          for (int i = 0; i < 4; ++i) p[i] = ml[(size_t)min(wb + i * sharing * 4, w1) * c.max_rows + r];
#pragma unroll
          for (int i = 0; i < 4; ++i)
            if (wb + i * sharing * 4 <= w1) join(m, l, p[i].x, p[i].y);
        }
#pragma unroll
      for (int off = 8; off < 32; off <<= 1)
        join(m, l, __shfl_xor_sync(0xffffffffu, m, off), __shfl_xor_sync(0xffffffffu, l, off));
      if (lane < 8 && r < rows) {
        if constexpr (W == 1)
          row_lse[warp][r] = weight_base(m, l);
        else
          part_ml[turn][r] = make_float2(m, l);
      }
    }
    if constexpr (W > 1) {
      __syncthreads();
      for (int r = threadIdx.x; r < rows; r += kFinWarps * 32) {
        float m = -INFINITY, l = 0.f;
        for (int i = 0; i < sharing; ++i) join(m, l, part_ml[i][r].x, part_ml[i][r].y);
        row_lse[0][r] = weight_base(m, l);
      }
      __syncthreads();
    } else {
      __syncwarp();
    }
    if (V > 1) first();
    else lost[0] = *(const float4 *)(low + min(j0, j_last));
    for (int r0 = 0; r0 < rows; r0 += kRows) {
      if (V > 1 || r0 > 0) load(r0);
#pragma unroll
      for (int i = 0; i < kRows; ++i) {
        if (r0 + i >= rows) break;
        const float e = row_lse[warp / W][r0 + i];
#pragma unroll
        for (int y = 0; y < V; ++y) {
          w[y].x += ex2(v[i][y].x - e), w[y].y += ex2(v[i][y].y - e);
          w[y].z += ex2(v[i][y].z - e), w[y].w += ex2(v[i][y].w - e);
        }
      }
    }
    if (V > 1)  // no registers for them before (72 bytes of spills)
#pragma unroll
      for (int y = 0; y < V; ++y) lost[y] = *(const float4 *)(low + min(j0 + y * 128, j_last));
#pragma unroll
    for (int y = 0; y < V; ++y) {
      const int j = j0 + y * 128;
      const float4 sum = make_float4(add_score(old[y].x, lost[y].x, w[y].x), add_score(old[y].y, lost[y].y, w[y].y),
                                     add_score(old[y].z, lost[y].z, w[y].z), add_score(old[y].w, lost[y].w, w[y].w));
      if (j + 4 <= s.total) {
        *(float4 *)(sc + j) = sum;
        *(float4 *)(low + j) = lost[y];
      } else {  // entries behind the last one keep their score
        if (j < s.total) sc[j] = sum.x, low[j] = lost[y].x;
        if (j + 1 < s.total) sc[j + 1] = sum.y, low[j + 1] = lost[y].y;
        if (j + 2 < s.total) sc[j + 2] = sum.z, low[j + 2] = lost[y].z;
      }
    }
    __syncwarp();  // before the next item's row_lse (W = 8: the barriers above keep it back)
  }
}

template <typename... P>
cudaError_t launch_after(void (*kernel)(P...), dim3 grid, int threads, int smem, cudaStream_t st, P... args) {
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = grid;
  cfg.blockDim = dim3(threads);
  cfg.dynamicSmemBytes = smem;
  cfg.stream = st;
  cudaLaunchAttribute at;
  at.id = cudaLaunchAttributeProgrammaticStreamSerialization;
  at.val.programmaticStreamSerializationAllowed = 1;
  cfg.attrs = &at;
  cfg.numAttrs = 1;
  return cudaLaunchKernelEx(&cfg, kernel, args...);
}

template <typename F, int D, int NR, int MT>
cudaError_t attend_t(Args a, const CUtensorMap &kmap, const CUtensorMap &vmap, cudaStream_t st) {
  using G = Cfg<D, NR, MT>;
  const int ctas = a.c.sms * G::kCtas;
  a.workers = ctas * G::kTeams;
  const dim3 grid(ctas, (a.rows + 8 * NR * MT - 1) / (8 * NR * MT));
  static SmemLimit limit;
  cudaError_t e = limit.raise((const void *)attend_kernel<F, D, NR, MT>, G::kSmem);
  if (e != cudaSuccess) return e;
  if (a.l.appends) {
    e = launch_after(attend_kernel<F, D, NR, MT>, grid, G::kWarps * 32, G::kSmem, st, a, kmap, vmap);
  } else {
    attend_kernel<F, D, NR, MT><<<grid, G::kWarps * 32, G::kSmem, st>>>(a, kmap, vmap);
    e = cudaGetLastError();
  }
  if (e != cudaSuccess) return e;
  // Parts of a head, about, and what a warp can gather at once of them and its rows.
  const int64_t heads = (int64_t)a.c.B * a.c.H, parts = a.workers / heads + 1;
  const bool deep = parts > 48, many = deep || parts * a.rows > 64;
  const bool wide = !many || heads * ((a.c.cap + 4095) / 4096) >= 2 * a.c.sms;  // enough items of four fours a lane
  const int chunk = (many ? 1024 : 128) * (wide ? 4 : 1), per = many ? 1 : 8;
  const int64_t items = (deep ? heads * a.rows : (heads * a.rows + kFinWarps - 1) / kFinWarps) +
                        (a.accumulate ? (heads * ((a.c.cap + chunk - 1) / chunk) + per - 1) / per : 0);
  const dim3 fin((unsigned)(items < a.c.sms * 8 ? items : a.c.sms * 8));
  const auto kernel = !many  ? finish_kernel<D, 1, 4, false>
                      : deep ? (wide ? finish_kernel<D, 8, 4, true> : finish_kernel<D, 8, 1, true>)
                             : (wide ? finish_kernel<D, 8, 4, false> : finish_kernel<D, 8, 1, false>);
  return launch_after(kernel, fin, kFinWarps * 32, 0, st, a);
}

template <typename F, int D>
cudaError_t attend_d(const Args &a, const CUtensorMap &kmap, const CUtensorMap &vmap, cudaStream_t st) {
  if (a.rows <= 8) return attend_t<F, D, 1, 1>(a, kmap, vmap, st);
  if (a.rows <= 16) return attend_t<F, D, 2, 1>(a, kmap, vmap, st);
  if (a.rows <= 32) return attend_t<F, D, 2, 2>(a, kmap, vmap, st);
  if (a.rows <= 48) return attend_t<F, D, 2, 3>(a, kmap, vmap, st);
  return attend_t<F, D, 2, 4>(a, kmap, vmap, st);
}

template <typename F, int D, int W>
cudaError_t head_t(const Args &a, const Rows &k, const Rows &v, const int32_t *position, const CUtensorMap &kmap,
                   const CUtensorMap &vmap, cudaStream_t st) {
  const int smem = 1024 + W * 2 * 2 * kBlock * D + a.rows * a.c.cap * 4;
  static SmemLimit limit;
  const cudaError_t e = limit.raise((const void *)head_kernel<F, D, W>, smem);
  if (e != cudaSuccess) return e;
  head_kernel<F, D, W><<<a.c.B * a.c.H, W * 32, smem, st>>>(a, k, v, position, kmap, vmap);
  return cudaGetLastError();
}

template <typename F, int D>
cudaError_t head_d(const Args &a, const Rows &k, const Rows &v, const int32_t *position, const CUtensorMap &kmap,
                   const CUtensorMap &vmap, cudaStream_t st) {
  return a.c.B * a.c.H <= a.c.sms ? head_t<F, D, 8>(a, k, v, position, kmap, vmap, st)
                                  : head_t<F, D, 4>(a, k, v, position, kmap, vmap, st);
}

Args args_of(const View &c, const Lens &l, const Rows &q, int causal, int accumulate, const Rows &out, float *lse) {
  Args a;
  a.c = c;
  a.l = l;
  a.q = q;
  a.out = out;
  a.lse = lse;
  a.causal = causal;
  a.accumulate = accumulate;
  a.workers = 0;
  a.rows = l.n * c.group;
  // Codes of more than L2's size evict each other before the next call reads them; the logits, which are read again
  // in this one, then stay.  8 heads of 262,000 entries: 129 us a step, 134 without the hint; 56 heads, 1.3 GB of codes:
  // 246 both.
  a.streams = 2 * (int64_t)c.B * c.H * c.cap * c.d > (int64_t)c.l2_bytes;
  a.po = nullptr;
  a.ml = nullptr;
  return a;
}

size_t partial_slots(int B, int H, int sms) { return (size_t)sms * kMaxWorkers + (size_t)B * H; }

}  // namespace

size_t attend_scratch_bytes(int B, int H, int d, int max_rows, int sms) {
  return partial_slots(B, H, sms) * max_rows * (sizeof(float2) + d * sizeof(float));
}

cudaError_t launch_attend(const View &c, const Lens &l, const Rows &q, int causal, int accumulate, const Rows &out,
                          float *lse, const CUtensorMap &kmap, const CUtensorMap &vmap, cudaStream_t st) {
  Args a = args_of(c, l, q, causal, accumulate, out, lse);
  const size_t rows = partial_slots(c.B, c.H, c.sms) * c.max_rows;
  a.po = c.part;
  a.ml = (float2 *)(c.part + rows * c.d);
  if (c.kv == H2O_KV_E4M3)
    return c.d == 128 ? attend_d<E4M3, 128>(a, kmap, vmap, st) : attend_d<E4M3, 64>(a, kmap, vmap, st);
  return c.d == 128 ? attend_d<I8, 128>(a, kmap, vmap, st) : attend_d<I8, 64>(a, kmap, vmap, st);
}

bool head_fits(const View &c, int n) {
  return n <= kFewRows && n * c.group <= 8 && c.cap <= kHeadCap && (int64_t)c.B * c.H <= 2 * c.sms;
}

cudaError_t launch_head(const View &c, const Lens &l, const Rows &q, const Rows *k, const Rows *v,
                        const int32_t *position, int causal, int accumulate, const Rows &out, float *lse,
                        const CUtensorMap &kmap, const CUtensorMap &vmap, cudaStream_t st) {
  const Args a = args_of(c, l, q, causal, accumulate, out, lse);
  const Rows none{};
  if (c.kv == H2O_KV_E4M3)
    return c.d == 128 ? head_d<E4M3, 128>(a, k ? *k : none, v ? *v : none, position, kmap, vmap, st)
                      : head_d<E4M3, 64>(a, k ? *k : none, v ? *v : none, position, kmap, vmap, st);
  return c.d == 128 ? head_d<I8, 128>(a, k ? *k : none, v ? *v : none, position, kmap, vmap, st)
                    : head_d<I8, 64>(a, k ? *k : none, v ? *v : none, position, kmap, vmap, st);
}

}  // namespace blk
}  // namespace h2o
