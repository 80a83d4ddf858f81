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
// one warp for each 16 rows (MT warps); it streams its run's K and V blocks
// through its own ring of TMA loads (128- or 64-byte swizzle, so the
// fragment reads below meet no bank conflict), with no barrier shared with
// other workers.  Per block of 32 entries: codes become f16 in registers
// (exact), S = Q K^T and P V run on mma.sync m16n8k16 with fp32 sums, softmax
// is online.  A lane's K words hold four consecutive dimensions of a row and
// its V words four dimensions of two entries: the matrix instruction sums
// over any order of k, so the loads stay 16 bytes wide and need no transpose.
// Where a head's blocks lie in more than one run, the partial (m, l, O) go to
// scratch memory; the runs' and heads' boundaries form a staircase, so
// (worker + head) numbers the partials without gaps or collisions.
//
// Why mma.sync and not tcgen05: a decode step has 1 to 64 rows per cached
// head, so the step is bound by the codes' bytes (2 d per entry), and the
// codes have to pass through registers anyway to become f16; tcgen05 would
// read them back from shared memory, 4 more bytes of its traffic per code.
//
// finish_kernel: joins the partials to O and LSE, and turns the logits the
// first kernel left in scratch memory into weights, once LSE is known:
// 4 bytes written and read per row and entry, instead of K read again.
#include <cuda.h>

#include "block_cache.cuh"
#include "sm100.cuh"

namespace h2o {
namespace blk {
namespace {

using namespace sm100;

// ------------------------------------------------------------ runs of blocks
__device__ __forceinline__ int ceil_div(int a, int b) { return (a + b - 1) / b; }

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

// ------------------------------------------------------------------- formats
// Two code pairs of a word as f16x2 (exact).
template <typename F> __device__ __forceinline__ void to_f16(uint32_t w, uint32_t &a, uint32_t &z);
template <> __device__ __forceinline__ void to_f16<E4M3>(uint32_t w, uint32_t &a, uint32_t &z) {
  a = e4m3x2_to_f16x2(w);
  z = e4m3x2_to_f16x2(w >> 16);
}
// code + 128 in the low bits of the f16 number 1024, less 1152.
template <> __device__ __forceinline__ void to_f16<I8>(uint32_t w, uint32_t &a, uint32_t &z) {
  w ^= 0x80808080u;
  a = __byte_perm(w, 0x64646464u, 0x4140);
  z = __byte_perm(w, 0x64646464u, 0x4342);
  const __half2 bias = __halves2half2(__ushort_as_half(0x6480), __ushort_as_half(0x6480));
  const __half2 x = __hsub2(*(const __half2 *)&a, bias), y = __hsub2(*(const __half2 *)&z, bias);
  a = *(const uint32_t *)&x;
  z = *(const uint32_t *)&y;
}

__device__ __forceinline__ void mma16816(float (&c)[4], const uint32_t (&a)[4], uint32_t b0, uint32_t b1) {
  asm("mma.sync.aligned.m16n8k16.row.col.f32.f16.f16.f32 {%0,%1,%2,%3}, {%4,%5,%6,%7}, {%8,%9}, {%0,%1,%2,%3};"
      : "+f"(c[0]), "+f"(c[1]), "+f"(c[2]), "+f"(c[3])
      : "r"(a[0]), "r"(a[1]), "r"(a[2]), "r"(a[3]), "r"(b0), "r"(b1));
}

__device__ __forceinline__ void tma_load_2d(void *dst, const CUtensorMap *map, uint64_t *bar, int c0, int c1) {
  asm volatile(
      "cp.async.bulk.tensor.2d.shared::cluster.global.mbarrier::complete_tx::bytes [%0], [%1, {%3, %4}], [%2];" ::"r"(
          smem_u32(dst)),
      "l"(map), "r"(smem_u32(bar)), "r"(c0), "r"(c1)
      : "memory");
}

__device__ __forceinline__ void grid_dependency_wait() { asm volatile("griddepcontrol.wait;" ::: "memory"); }
__device__ __forceinline__ void grid_launch_dependents() { asm volatile("griddepcontrol.launch_dependents;"); }

// Byte offset of 16-byte chunk `chunk` of row `row` in a swizzled block.
template <int D> __device__ __forceinline__ int chunk_at(int row, int chunk) {
  return row * D + ((D == 128 ? chunk ^ (row & 7) : chunk ^ ((row >> 1) & 3)) << 4);
}

constexpr int kTeams = 4;  // workers of a CTA

// MT row tiles of 16 (warps) per worker.  One to two tiles leave a warp 255
// registers, so its Q stays there; four tiles run 16 warps of 128 registers
// and keep Q in shared memory.  Ring: about 192 KB per SM for one and two
// tiles, 128 KB (and 64 KB of Q) for four.
template <int D, int MT> struct Cfg {
  static constexpr int kWarps = kTeams * MT;
  static constexpr int kCtas = MT == 1 ? 2 : 1;  // per SM
  static constexpr int kStage = 2 * kBlock * D;
  static constexpr int kStages = (MT == 1 ? 98304 : MT == 2 ? 196608 : 131072) / (kTeams * kStage);
  static constexpr bool kQSmem = MT == 4;
  static constexpr int kQBytes = kQSmem ? kWarps * D * 32 : 0;
  static constexpr int kSmem = 1024 + kTeams * kStages * kStage + kQBytes + kTeams * kStages * 16;
};

struct Args {
  View c;
  Lens l;
  Rows q, out;
  float *lse;
  float2 *ml;  // [workers + B*H][max_rows]  partial maximum and sum
  float *po;   // [workers + B*H][max_rows][d]  partial output
  int causal, accumulate, workers;
  int rows;  // n * group: rows of a head in this call
};

template <typename F, int D, int MT>
__global__ void __launch_bounds__(Cfg<D, MT>::kWarps * 32, Cfg<D, MT>::kCtas)
    attend_kernel(const Args a, const __grid_constant__ CUtensorMap kmap, const __grid_constant__ CUtensorMap vmap) {
  using G = Cfg<D, MT>;
  constexpr int KS = D / 16;  // k steps of S, words of a lane's K row
  constexpr int NT = D / 8;   // n tiles of O
  constexpr int S = G::kStages;
  extern __shared__ uint8_t smem_raw[];
  uint8_t *smem = (uint8_t *)(((uintptr_t)smem_raw + 1023) & ~(uintptr_t)1023);
  const View &c = a.c;
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  const int team = warp / MT, tile = warp - team * MT;
  const int g = lane >> 2, t = lane & 3;
  uint8_t *ring = smem + team * S * G::kStage;
  uint4 *qs = (uint4 *)(smem + kTeams * S * G::kStage) + (G::kQSmem ? warp * KS * 32 : 0);
  uint64_t *full = (uint64_t *)(smem + kTeams * S * G::kStage + G::kQBytes) + team * 2 * S, *empty = full + S;
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
  grid_dependency_wait();  // the append before this launch
  grid_launch_dependents();
  if (count == 0) return;

  Cursor cur, ld;
  cur.seek(a.l, c.B, c.H, x0);
  ld = cur;
  auto issue = [&](int i) {  // block i of the run into its stage (leader warp)
    if (lane == 0) {
      uint8_t *dst = ring + (i % S) * G::kStage;
      uint64_t *bar = full + i % S;
      const int row = (ld.b * c.H + ld.h) * c.cap + ld.blk * kBlock;
      mbar_expect_tx(bar, G::kStage);
      tma_load_2d(dst, &kmap, bar, 0, row);
      tma_load_2d(dst + kBlock * D, &vmap, bar, 0, row);
    }
    ld.next(a.l, c.B, c.H);
  };
  int issued = 0;
  if (tile == 0)
    for (; issued < S && issued < count; ++issued) issue(issued);

  const int row0 = (blockIdx.y * MT + tile) * 16 + g;  // rows row0 and row0 + 8 of the head
  const bool idle = (blockIdx.y * MT + tile) * 16 >= a.rows;
  const int nsc = c.cap / kBlock;
  float o[NT][4], m[2], lsum[2], crow[2];
  int end[2];
  bool live[2];
  uint32_t qr[G::kQSmem ? 1 : KS][4];
  float *lg[2];
  int first_blk = 0, min_end = 0;
  bool open = false, lost = false;
  float ks = 0.f, vs = 0.f;
  {
    const size_t sc = (size_t)(cur.b * c.H + cur.h) * nsc + cur.blk;
    ks = c.Ksc[sc];
    vs = c.Vsc[sc];
  }

  for (int i = 0; i < count; ++i) {
    const int bh = cur.b * c.H + cur.h;
    if (!open) {  // a head begins
      open = true;
      first_blk = cur.blk;
      min_end = a.causal ? cur.s.total - cur.s.cnt + 1 : cur.s.total;
#pragma unroll
      for (int j = 0; j < NT; ++j) o[j][0] = o[j][1] = o[j][2] = o[j][3] = 0.f;
      uint32_t qh[2][KS * 2];
#pragma unroll
      for (int u = 0; u < 2; ++u) {
        const int r = row0 + 8 * u, tok = r / c.group;
        live[u] = tok < cur.s.cnt;
        end[u] = live[u] && a.causal ? cur.s.total - cur.s.cnt + tok + 1 : cur.s.total;
        m[u] = -INFINITY;
        lsum[u] = 0.f;
        lg[u] = c.logits + ((size_t)bh * c.max_rows + r) * c.cap + 2 * t;
        // the lane's D/4 dimensions of the row
        uint4 w[D / 32];
        const __nv_bfloat16 *p = a.q.at(cur.b, cur.h * c.group + r % c.group, tok) + t * (D / 4);
#pragma unroll
        for (int e = 0; e < D / 32; ++e) w[e] = live[u] ? ld_nc16(p + e * 8) : make_uint4(0u, 0u, 0u, 0u);
        float f[D / 4], top = 0.f;
#pragma unroll
        for (int e = 0; e < D / 32; ++e) Unpack<__nv_bfloat16>::run(w[e], f + e * 8);
#pragma unroll
        for (int e = 0; e < D / 4; ++e) top = fmaxf(top, fabsf(f[e]));
        top = fmaxf(top, __shfl_xor_sync(0xffffffffu, top, 1));
        top = fmaxf(top, __shfl_xor_sync(0xffffffffu, top, 2));
        // q to f16: a power of two brings the row's largest element to 2^13 .. 2^14; bf16's 8 bits then fit, and
        // only elements 2^-27 of the largest and below lose bits
        int ex = 0;
        frexpf(top, &ex);
        const int sh = top > 0.f && top < INFINITY ? min(14 - ex, 100) : 0;
        const float up = ldexpf(1.f, sh);
        crow[u] = ldexpf(rsqrtf((float)D) * kLog2e, -sh);
#pragma unroll
        for (int e = 0; e < D / 8; ++e) {
          const __half2 h2 = __floats2half2_rn(f[2 * e] * up, f[2 * e + 1] * up);
          qh[u][e] = *(const uint32_t *)&h2;
        }
      }
      if (G::kQSmem) {
        __syncwarp();
#pragma unroll
        for (int k = 0; k < KS; ++k)
          qs[k * 32 + lane] = make_uint4(qh[0][2 * k], qh[1][2 * k], qh[0][2 * k + 1], qh[1][2 * k + 1]);
        __syncwarp();
      } else {
#pragma unroll
        for (int k = 0; k < KS; ++k) {
          qr[G::kQSmem ? 0 : k][0] = qh[0][2 * k];
          qr[G::kQSmem ? 0 : k][1] = qh[1][2 * k];
          qr[G::kQSmem ? 0 : k][2] = qh[0][2 * k + 1];
          qr[G::kQSmem ? 0 : k][3] = qh[1][2 * k + 1];
        }
      }
    }
    const float ks_now = ks, vs_now = vs;
    const int blk = cur.blk, total = cur.s.total;
    const Cursor at = cur;
    cur.next(a.l, c.B, c.H);
    const bool closes = i + 1 == count || cur.blk == 0;
    if (i + 1 < count) {  // the next block's scales, a block ahead
      const size_t sc = (size_t)(cur.b * c.H + cur.h) * nsc + cur.blk;
      ks = c.Ksc[sc];
      vs = c.Vsc[sc];
    }
    uint8_t *kt = ring + (i % S) * G::kStage, *vt = kt + kBlock * D;
    if (!mbar_wait(full + i % S, (i / S) & 1)) {
      lost = true;
      break;
    }
    if (MT > 1 && tile == 0 && i > 0 && issued < count) {  // the stage of block i - 1, once every warp has read it
      if (!mbar_wait(empty + (i - 1) % S, ((i - 1) / S) & 1)) {
        lost = true;
        break;
      }
      issue(issued++);
    }
    if (!idle) {
      // S = Q K^T of 16 rows and 32 entries
      float s[4][4];
      {
        uint32_t kw[4][KS];
#pragma unroll
        for (int n = 0; n < 4; ++n) {
          s[n][0] = s[n][1] = s[n][2] = s[n][3] = 0.f;
#pragma unroll
          for (int e = 0; e < KS / 4; ++e) {
            const uint4 u = *(const uint4 *)(kt + chunk_at<D>(n * 8 + g, t * (KS / 4) + e));
            kw[n][4 * e] = u.x, kw[n][4 * e + 1] = u.y, kw[n][4 * e + 2] = u.z, kw[n][4 * e + 3] = u.w;
          }
        }
#pragma unroll
        for (int k = 0; k < KS; ++k) {
          uint32_t qa[4];
          if (G::kQSmem) {
            const uint4 u = qs[k * 32 + lane];
            qa[0] = u.x, qa[1] = u.y, qa[2] = u.z, qa[3] = u.w;
          } else {
#pragma unroll
            for (int e = 0; e < 4; ++e) qa[e] = qr[G::kQSmem ? 0 : k][e];
          }
#pragma unroll
          for (int n = 0; n < 4; ++n) {
            uint32_t b0, b1;
            to_f16<F>(kw[n][k], b0, b1);
            mma16816(s[n], qa, b0, b1);
          }
        }
      }
      const int j0 = blk * kBlock + 2 * t;
      const float f0 = crow[0] * ks_now, f1 = crow[1] * ks_now;
      const bool edge = blk * kBlock + kBlock > min_end;
#pragma unroll
      for (int n = 0; n < 4; ++n) {
        s[n][0] *= f0, s[n][1] *= f0, s[n][2] *= f1, s[n][3] *= f1;
        if (edge) {
          const int j = j0 + n * 8;
          if (j >= end[0]) s[n][0] = -INFINITY;
          if (j + 1 >= end[0]) s[n][1] = -INFINITY;
          if (j >= end[1]) s[n][2] = -INFINITY;
          if (j + 1 >= end[1]) s[n][3] = -INFINITY;
        }
      }
      if (a.accumulate) {
#pragma unroll
        for (int u = 0; u < 2; ++u)
          if (live[u]) {
            float *p = lg[u] + blk * kBlock;
#pragma unroll
            for (int n = 0; n < 4; ++n) *(float2 *)(p + n * 8) = make_float2(s[n][2 * u], s[n][2 * u + 1]);
          }
      }
      float top[2];
#pragma unroll
      for (int u = 0; u < 2; ++u) {
        top[u] = fmaxf(fmaxf(fmaxf(s[0][2 * u], s[0][2 * u + 1]), fmaxf(s[1][2 * u], s[1][2 * u + 1])),
                       fmaxf(fmaxf(s[2][2 * u], s[2][2 * u + 1]), fmaxf(s[3][2 * u], s[3][2 * u + 1])));
        top[u] = fmaxf(top[u], __shfl_xor_sync(0xffffffffu, top[u], 1));
        top[u] = fmaxf(top[u], __shfl_xor_sync(0xffffffffu, top[u], 2));
      }
      // The running maximum moves only when it is passed by more than 2^8: weights then stay below 2^8, in f16's range
      if (__any_sync(0xffffffffu, top[0] > m[0] + 8.f || top[1] > m[1] + 8.f || m[0] == -INFINITY || m[1] == -INFINITY)) {
#pragma unroll
        for (int u = 0; u < 2; ++u) {
          const float mn = fmaxf(m[u], top[u]);
          const float f = m[u] == -INFINITY ? 0.f : ex2(m[u] - mn);
          m[u] = mn;
          lsum[u] *= f;
#pragma unroll
          for (int j = 0; j < NT; ++j) o[j][2 * u] *= f, o[j][2 * u + 1] *= f;
        }
      }
      const float mu0 = m[0] == -INFINITY ? 0.f : m[0], mu1 = m[1] == -INFINITY ? 0.f : m[1];
      uint32_t p[2][4];  // P as the A operand of two k steps of 16 entries
#pragma unroll
      for (int n = 0; n < 4; ++n) {
        const float e0 = ex2(s[n][0] - mu0), e1 = ex2(s[n][1] - mu0), e2 = ex2(s[n][2] - mu1), e3 = ex2(s[n][3] - mu1);
        lsum[0] += e0 + e1;
        lsum[1] += e2 + e3;
        // 16 bits for the product with V: f16's 2^-11 per weight, an eighth of the output's own rounding
        const __half2 a0 = __floats2half2_rn(e0, e1), a1 = __floats2half2_rn(e2, e3);
        p[n >> 1][(n & 1) * 2] = *(const uint32_t *)&a0;
        p[n >> 1][(n & 1) * 2 + 1] = *(const uint32_t *)&a1;
      }
      const int rest = total - blk * kBlock;
      if (rest < kBlock) {  // codes behind the last entry may be anything, also NaN: weight 0 needs a finite code
        for (int z = rest * D + lane * 16; z < kBlock * D; z += 512) *(uint4 *)(vt + z) = make_uint4(0u, 0u, 0u, 0u);
        fence_proxy_async_smem();
        __syncwarp();
      }
      // O += vs (P V): a fresh product per block, added in fp32 under the block's scale
      constexpr int VW = D / 32;  // words of a lane's V row: D/8 dimensions
      constexpr int HALF = G::kQSmem && VW == 4 ? 2 : VW;  // words at a time (registers)
#pragma unroll
      for (int hw = 0; hw < VW; hw += HALF) {
        uint32_t vw[8][HALF];
#pragma unroll
        for (int e = 0; e < 8; ++e) {
          const int r = (e >> 1) * 8 + 2 * t + (e & 1);
          if constexpr (HALF == 4) {
            const uint4 u = *(const uint4 *)(vt + chunk_at<D>(r, g));
            vw[e][0] = u.x, vw[e][1] = u.y, vw[e][2 % HALF] = u.z, vw[e][3 % HALF] = u.w;
          } else {
            const uint8_t *src = D == 128 ? vt + chunk_at<D>(r, g) + hw * 4 : vt + chunk_at<D>(r, g >> 1) + (g & 1) * 8;
            const uint2 u = *(const uint2 *)src;
            vw[e][0] = u.x, vw[e][1] = u.y;
          }
        }
#pragma unroll
        for (int w = 0; w < HALF; ++w) {
          float acc[4][4];
#pragma unroll
          for (int j = 0; j < 4; ++j) acc[j][0] = acc[j][1] = acc[j][2] = acc[j][3] = 0.f;
#pragma unroll
          for (int k = 0; k < 2; ++k) {
            uint32_t b0[4], b1[4];
            const uint32_t x = vw[4 * k][w], y = vw[4 * k + 1][w], z = vw[4 * k + 2][w], v = vw[4 * k + 3][w];
            to_f16<F>(__byte_perm(x, y, 0x5140), b0[0], b0[1]);
            to_f16<F>(__byte_perm(x, y, 0x7362), b0[2], b0[3]);
            to_f16<F>(__byte_perm(z, v, 0x5140), b1[0], b1[1]);
            to_f16<F>(__byte_perm(z, v, 0x7362), b1[2], b1[3]);
#pragma unroll
            for (int j = 0; j < 4; ++j) mma16816(acc[j], p[k], b0[j], b1[j]);
          }
#pragma unroll
          for (int j = 0; j < 4; ++j)
#pragma unroll
            for (int e = 0; e < 4; ++e) o[(hw + w) * 4 + j][e] = fmaf(acc[j][e], vs_now, o[(hw + w) * 4 + j][e]);
        }
      }
    }
    // this warp has read the stage
    __syncwarp();
    if (MT > 1) {
      if (lane == 0) mbar_arrive(empty + i % S);
    } else if (issued < count) {
      issue(issued++);
    }
    if (!closes) continue;
    open = false;
    if (idle) continue;
    const int hb = at.b * c.H + at.h;
    const bool whole = first_blk == 0 && blk + 1 == at.nblk;  // no other worker holds a part of this head
    const size_t slot = ((size_t)worker + hb) * c.max_rows;
#pragma unroll
    for (int u = 0; u < 2; ++u) {
      float l = lsum[u];
      l += __shfl_xor_sync(0xffffffffu, l, 1);
      l += __shfl_xor_sync(0xffffffffu, l, 2);
      if (!live[u]) continue;
      const int r = row0 + 8 * u, tok = r / c.group, hq = at.h * c.group + r % c.group;
      if (t == 0) a.ml[slot + r] = make_float2(m[u], l);
      if (whole) {
        const float inv = l > 0.f || l != l ? 1.f / l : 0.f;
        __nv_bfloat16 *dst = const_cast<__nv_bfloat16 *>(a.out.at(at.b, hq, tok)) + t * (D / 4);
#pragma unroll
        for (int e = 0; e < 2; ++e)
#pragma unroll
          for (int j = 0; j < NT; j += 8) {
            uint4 w;
#pragma unroll
            for (int y = 0; y < 4; ++y) {
              const __nv_bfloat162 b2 = __floats2bfloat162_rn(o[j + 2 * y][2 * u + e] * inv, o[j + 2 * y + 1][2 * u + e] * inv);
              (&w.x)[y] = *(const uint32_t *)&b2;
            }
            *(uint4 *)(dst + e * (D / 8) + j) = w;
          }
        if (a.lse && t == 0)
          a.lse[((size_t)at.b * c.H * c.group + hq) * a.l.n + tok] = l > 0.f || l != l ? (m[u] + log2f(l)) * kLn2 : -INFINITY;
      } else {
        float *dst = a.po + (slot + r) * D + t * (D / 4);
#pragma unroll
        for (int e = 0; e < 2; ++e)
#pragma unroll
          for (int j = 0; j < NT; j += 4)
            *(float4 *)(dst + e * (D / 8) + j) =
                make_float4(o[j][2 * u + e], o[j + 1][2 * u + e], o[j + 2][2 * u + e], o[j + 3][2 * u + e]);
      }
    }
  }
  if (lost) {  // a copy never arrived: report, and let what is in flight land before the memory goes
    if (lane == 0) atomicOr(c.err, H2O_BERR_INTERNAL);
    if (tile == 0)
      for (int i = max(0, issued - S); i < issued; ++i) mbar_wait(full + i % S, (i / S) & 1);
  }
}

// ------------------------------------------------------------------- finish
constexpr int kChunk = 256;  // entries of one score item
constexpr int kFinishWarps = 8;

// One item per warp: first D/32 items for each row of a head that lies in
// several runs (32 output dimensions each: four groups of eight lanes take
// the partials in turn), then kChunk entries' scores each.
template <int D>
__global__ void __launch_bounds__(kFinishWarps * 32) finish_kernel(const Args a) {
  const View &c = a.c;
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  __shared__ float row_lse[kFinishWarps][H2O_BLOCK_MAX_ROWS];
  const int blocks = c.H * sum_units(a.l, c.B, kBlock);
  const int workers = min(a.workers, blocks);
  const int chunks = a.accumulate ? c.H * sum_units(a.l, c.B, kChunk) : 0;
  const int64_t outs = (int64_t)c.B * c.H * a.rows * (D / 32);
  grid_dependency_wait();
  for (int64_t item = (int64_t)blockIdx.x * kFinishWarps + warp; item < outs + chunks;
       item += (int64_t)gridDim.x * kFinishWarps) {
    if (item < outs) {
      const int part = (int)(item % (D / 32));
      const int64_t hr = item / (D / 32);
      const int r = (int)(hr % a.rows), bh = (int)(hr / a.rows), b = bh / c.H, h = bh - b * c.H;
      const Seq s = seq_of(a.l, b);
      const int tok = r / c.group, hq = h * c.group + r % c.group;
      if (tok >= s.cnt) continue;
      __nv_bfloat16 *dst = const_cast<__nv_bfloat16 *>(a.out.at(b, hq, tok)) + part * 32 + (lane & 7) * 4;
      float *lse = a.lse ? a.lse + ((size_t)b * c.H * c.group + hq) * a.l.n + tok : nullptr;
      const int nblk = ceil_div(s.total, kBlock);
      if (nblk == 0) {  // no entry at all
        if (lane < 8) *(uint2 *)dst = make_uint2(0u, 0u);
        if (lse && part == 0 && lane == 0) *lse = -INFINITY;
        continue;
      }
      int before = 0;
      for (int i = lane; i < b; i += 32) before += ceil_div(seq_of(a.l, i).total, kBlock);
      const int x = c.H * __reduce_add_sync(0xffffffffu, before) + h * nblk;
      const int w0 = worker_of(x, blocks, workers), w1 = worker_of(x + nblk - 1, blocks, workers);
      if (w0 == w1) continue;  // written by its worker
      float m = -INFINITY, l = 0.f;
      float4 o = make_float4(0.f, 0.f, 0.f, 0.f);
      for (int w = w0 + (lane >> 3); w <= w1; w += 4) {
        const size_t at = ((size_t)w + bh) * c.max_rows + r;
        const float2 p = a.ml[at];
        const float4 v = *(const float4 *)(a.po + at * D + part * 32 + (lane & 7) * 4);
        if (p.x == -INFINITY && p.y == 0.f) continue;  // this run saw nothing of the row
        const float mn = fmaxf(m, p.x), f = m == -INFINITY ? 0.f : ex2(m - mn), z = ex2(p.x - mn);
        m = mn;
        l = l * f + p.y * z;
        o.x = o.x * f + v.x * z, o.y = o.y * f + v.y * z, o.z = o.z * f + v.z * z, o.w = o.w * f + v.w * z;
      }
#pragma unroll
      for (int off = 8; off < 32; off <<= 1) {
        const float om = __shfl_xor_sync(0xffffffffu, m, off), ol = __shfl_xor_sync(0xffffffffu, l, off);
        const float4 oo = make_float4(__shfl_xor_sync(0xffffffffu, o.x, off), __shfl_xor_sync(0xffffffffu, o.y, off),
                                      __shfl_xor_sync(0xffffffffu, o.z, off), __shfl_xor_sync(0xffffffffu, o.w, off));
        const float mn = fmaxf(m, om);
        const float f = m == -INFINITY ? 0.f : ex2(m - mn), z = om == -INFINITY ? 0.f : ex2(om - mn);
        m = mn;
        l = l * f + ol * z;
        o.x = o.x * f + oo.x * z, o.y = o.y * f + oo.y * z, o.z = o.z * f + oo.z * z, o.w = o.w * f + oo.w * z;
      }
      const bool any = l > 0.f || l != l;
      const float inv = any ? 1.f / l : 0.f;
      if (lane < 8) {
        const __nv_bfloat162 p0 = __floats2bfloat162_rn(o.x * inv, o.y * inv), p1 = __floats2bfloat162_rn(o.z * inv, o.w * inv);
        *(uint2 *)dst = make_uint2(*(const uint32_t *)&p0, *(const uint32_t *)&p1);
      }
      if (lse && part == 0 && lane == 0) *lse = any ? (m + log2f(l)) * kLn2 : -INFINITY;
      continue;
    }
    int x = (int)(item - outs), before;
    const int b = find_seq(a.l, c.B, c.H, kChunk, x, before);
    const Seq s = seq_of(a.l, b);
    const int nch = ceil_div(s.total, kChunk), nblk = ceil_div(s.total, kBlock);
    const int h = x / nch, j0 = (x - h * nch) * kChunk, bh = b * c.H + h;
    const int rows = s.cnt * c.group;
    const int start = c.H * before + h * nblk;
    const int w0 = worker_of(start, blocks, workers), w1 = worker_of(start + nblk - 1, blocks, workers);
    // log-sum-exp (base 2) of each row; +infinity where nothing was seen, so that its weights are 0
    if (w1 - w0 < 4) {
      for (int r = lane; r < rows; r += 32) {
        float m = -INFINITY, l = 0.f;
        for (int w = w0; w <= w1; ++w) {
          const float2 p = a.ml[((size_t)w + bh) * c.max_rows + r];
          if (p.x == -INFINITY && p.y == 0.f) continue;
          const float mn = fmaxf(m, p.x);
          l = (m == -INFINITY ? 0.f : l * ex2(m - mn)) + p.y * ex2(p.x - mn);
          m = mn;
        }
        row_lse[warp][r] = l > 0.f || l != l ? m + log2f(l) : INFINITY;
      }
    } else {
      for (int r = 0; r < rows; ++r) {
        float m = -INFINITY, l = 0.f;
        for (int w = w0 + lane; w <= w1; w += 32) {
          const float2 p = a.ml[((size_t)w + bh) * c.max_rows + r];
          if (p.x == -INFINITY && p.y == 0.f) continue;
          const float mn = fmaxf(m, p.x);
          l = (m == -INFINITY ? 0.f : l * ex2(m - mn)) + p.y * ex2(p.x - mn);
          m = mn;
        }
        const float mn = warp_max(m);
        l = warp_sum(m == -INFINITY ? (l != l ? l : 0.f) : l * ex2(m - mn));
        if (lane == 0) row_lse[warp][r] = l > 0.f || l != l ? mn + log2f(l) : INFINITY;
      }
    }
    __syncwarp();
    const float *lg = c.logits + (size_t)bh * c.max_rows * c.cap + j0 + lane * 4;
    float *sc = c.score + (size_t)bh * c.cap + j0 + lane * 4;
#pragma unroll
    for (int y = 0; y < kChunk / 128; ++y) {
      const int j = j0 + y * 128 + lane * 4;
      if (j >= s.total) continue;
      float4 w = make_float4(0.f, 0.f, 0.f, 0.f);
#pragma unroll 4
      for (int r = 0; r < rows; ++r) {
        const float4 v = *(const float4 *)(lg + (size_t)r * c.cap + y * 128);
        const float e = row_lse[warp][r];
        w.x += ex2(v.x - e), w.y += ex2(v.y - e), w.z += ex2(v.z - e), w.w += ex2(v.w - e);
      }
      if (j + 4 <= s.total) {
        float4 v = *(float4 *)(sc + y * 128);
        v.x += w.x, v.y += w.y, v.z += w.z, v.w += w.w;
        *(float4 *)(sc + y * 128) = v;
      } else {  // entries behind the last one keep their score
        for (int e = 0; j + e < s.total; ++e) sc[y * 128 + e] += (&w.x)[e];
      }
    }
    __syncwarp();
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

template <typename F, int D, int MT>
cudaError_t attend_t(Args a, const CUtensorMap &kmap, const CUtensorMap &vmap, cudaStream_t st) {
  using G = Cfg<D, MT>;
  const int ctas = a.c.sms * G::kCtas;
  a.workers = ctas * kTeams;
  const int tiles = (a.rows + 15) / 16;
  cudaError_t e = cudaFuncSetAttribute(attend_kernel<F, D, MT>, cudaFuncAttributeMaxDynamicSharedMemorySize, G::kSmem);
  if (e != cudaSuccess) return e;
  if (a.l.appends) {
    e = launch_after(attend_kernel<F, D, MT>, dim3(ctas, (tiles + MT - 1) / MT), G::kWarps * 32, G::kSmem, st, a, kmap, vmap);
  } else {
    attend_kernel<F, D, MT><<<dim3(ctas, (tiles + MT - 1) / MT), G::kWarps * 32, G::kSmem, st>>>(a, kmap, vmap);
    e = cudaGetLastError();
  }
  if (e != cudaSuccess) return e;
  return launch_after(finish_kernel<D>, dim3(a.c.sms * 8), kFinishWarps * 32, 0, st, a);
}

template <typename F, int D>
cudaError_t attend_d(const Args &a, const CUtensorMap &kmap, const CUtensorMap &vmap, cudaStream_t st) {
  if (a.rows <= 16) return attend_t<F, D, 1>(a, kmap, vmap, st);
  if (a.rows <= 32) return attend_t<F, D, 2>(a, kmap, vmap, st);
  return attend_t<F, D, 4>(a, kmap, vmap, st);
}

}  // namespace

size_t attend_scratch_bytes(int B, int H, int d, int max_rows, int sms) {
  const size_t slots = (size_t)sms * Cfg<128, 1>::kCtas * kTeams + (size_t)B * H;
  return slots * max_rows * (sizeof(float2) + d * sizeof(float));
}

cudaError_t launch_attend(const View &c, const Lens &l, const Rows &q, int causal, int accumulate, const Rows &out,
                          float *lse, const CUtensorMap &kmap, const CUtensorMap &vmap, cudaStream_t st) {
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
  const size_t slots = (size_t)c.sms * Cfg<128, 1>::kCtas * kTeams + (size_t)c.B * c.H;
  a.po = c.part;
  a.ml = (float2 *)(c.part + slots * c.max_rows * c.d);
  if (c.kv == H2O_KV_E4M3)
    return c.d == 128 ? attend_d<E4M3, 128>(a, kmap, vmap, st) : attend_d<E4M3, 64>(a, kmap, vmap, st);
  return c.d == 128 ? attend_d<I8, 128>(a, kmap, vmap, st) : attend_d<I8, 64>(a, kmap, vmap, st);
}

}  // namespace blk
}  // namespace h2o
