// block_copy.cu — sequences of a block-scaled 8-bit cache copied to other rows
// of it, or into another cache.
//
// Row b receives row parent[b]: blocks that hold entries, whole, with scales,
// positions, scores (and what their sums have lost) and bounds.  In place any
// map is fine (permutations, a row to several): a CTA takes the same bytes of
// every row that is read, brings them to shared memory, and writes them only
// when all are there; no two CTAs share bytes.  So each row that is read is
// read once, however many receive it, and nothing is copied twice.
//
// Copies in both directions are bulk ones, a few KB each; the scales, whose
// rows may start at any multiple of 4 bytes, go through registers.
#include "block_cache.cuh"
#include "sm100.cuh"

namespace h2o {
namespace blk {
namespace {

using namespace sm100;

constexpr int kThreads = 256;
constexpr int kBulk = 6, kArrays = 8;  // K, V, pos, score, low, bounds; then the scales

struct Args {
  const uint8_t *from[kArrays];
  uint8_t *to[kArrays];
  int per_block[kArrays];             // bytes of a block of 32 entries
  int64_t from_head[kArrays], to_head[kArrays];  // bytes of a head
  const int32_t *parent, *from_lengths, *lengths;
  int32_t *new_lengths;
  int *err;
  int H, to_rows, from_rows, from_cap, to_cap;
  int same;    // the rows are those of one cache
  int arrays;  // kBulk, or one less without bounds
  int chunk;   // bytes of a row that a CTA takes at a time, at most: a power of two
  int room;    // bytes for the rows' pieces
};

__device__ __forceinline__ void bulk_store(void *dst, const void *src, uint32_t bytes) {
  asm volatile("cp.async.bulk.global.shared::cta.bulk_group [%0], [%1], %2;" ::"l"(dst), "r"(smem_u32(src)), "r"(bytes)
               : "memory");
}

// Shared memory: the pieces; slot_of [from_rows] (a read row's place among the
// pieces, -1); blocks [from_rows] (their lengths first); the read rows and the
// rows that receive something, in order; parent [to_rows].
__global__ void __launch_bounds__(kThreads) copy_kernel(const Args a) {
  extern __shared__ __align__(128) uint8_t smem[];
  int *slot_of = (int *)(smem + a.room), *blocks = slot_of + a.from_rows;
  int *source = blocks + a.from_rows;  // of a piece
  int *dest = source + a.from_rows, *parent = dest + a.to_rows;
  __shared__ __align__(8) uint64_t bar;
  __shared__ int s_sources, s_moves, s_most, s_warp[kThreads / 32], s_lost;
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
  if (tid == 0) {
    s_sources = s_moves = s_most = s_lost = 0;
    mbar_init(&bar, 1);
    fence_mbar_init();
  }
  for (int p = tid; p < a.from_rows; p += kThreads) slot_of[p] = -1, blocks[p] = a.from_lengths[p];
  for (int b = tid; b < a.to_rows; b += kThreads) parent[b] = a.parent[b];
  __syncthreads();
  for (int b0 = 0; b0 < a.to_rows; b0 += kThreads) {
    const int b = b0 + tid;
    const int p = b < a.to_rows ? parent[b] : -1;
    const bool known = p >= 0 && p < a.from_rows;
    const int len = known ? blocks[p] : 0;
    const bool fits = known && len >= 0 && len <= a.from_cap && len <= a.to_cap;
    const bool is = fits && !(a.same && p == b);  // it moves
    if (b < a.to_rows && blockIdx.x == 0) {
      if (p != -1 && !fits) atomicOr(a.err, H2O_BERR_RANGE);
      a.new_lengths[b] = fits ? len : a.lengths[b];
    }
    if (is) slot_of[p] = 0;
    // the moves in the order of their rows
    const unsigned ballot = __ballot_sync(0xffffffffu, is);
    if (lane == 0) s_warp[warp] = __popc(ballot);
    __syncthreads();
    int at = s_moves + __popc(ballot & ((1u << lane) - 1));
    for (int w = 0; w < warp; ++w) at += s_warp[w];
    if (is) dest[at] = b;
    __syncthreads();
    if (tid == kThreads - 1) s_moves = at + (is ? 1 : 0);
    __syncthreads();
  }
  for (int p0 = 0; p0 < a.from_rows; p0 += kThreads) {
    const int p = p0 + tid;
    const bool is = p < a.from_rows && slot_of[p] == 0;
    const unsigned ballot = __ballot_sync(0xffffffffu, is);
    if (lane == 0) s_warp[warp] = __popc(ballot);
    __syncthreads();
    int at = s_sources + __popc(ballot & ((1u << lane) - 1));
    for (int w = 0; w < warp; ++w) at += s_warp[w];
    if (is) {
      slot_of[p] = at, source[at] = p;
      blocks[p] = (blocks[p] + kBlock - 1) / kBlock;
      atomicMax(&s_most, blocks[p]);
    }
    __syncthreads();
    if (tid == kThreads - 1) s_sources = at + (is ? 1 : 0);
    __syncthreads();
  }
  const int sources = s_sources, n_moves = s_moves, most = s_most;
  if (n_moves == 0 || most == 0) return;
  int chunk = a.chunk;
  while (chunk > 16 && (int64_t)chunk * sources > a.room) chunk >>= 1;

  // Items: (head, array, chunk), then the scales.
  int64_t items_of[kArrays], items = 0;
#pragma unroll
  for (int x = 0; x < kArrays; ++x) {
    const bool none = x == kBulk - 1 && a.arrays < kBulk;
    items_of[x] = none ? 0 : ((int64_t)most * a.per_block[x] + chunk - 1) / chunk * a.H;
    items += items_of[x];
  }
  uint32_t phase = 0;
  for (int64_t item = blockIdx.x; item < items; item += gridDim.x) {
    int x = 0;
    int64_t i = item;
    while (i >= items_of[x]) i -= items_of[x++];
    const int64_t pieces = items_of[x] / a.H;  // neighbours in a row to neighbouring CTAs
    const int h = (int)(i / pieces);
    const int64_t at = (i - h * pieces) * chunk;  // the chunk's first byte of a row's
    auto bytes_of = [&](int p) {
      const int64_t left = (int64_t)blocks[p] * a.per_block[x] - at;
      return (int)(left < 0 ? 0 : left < chunk ? left : chunk);
    };
    const uint8_t *from = a.from[x] + h * a.from_head[x] + at;
    uint8_t *to = a.to[x] + h * a.to_head[x] + at;
    const int64_t from_row = a.from_head[x] * a.H, to_row = a.to_head[x] * a.H;
    if (x < kBulk) {
      if (warp == 0 && !s_lost) {
        // the last item's pieces have left shared memory
        asm volatile("cp.async.bulk.wait_group.read 0;" ::: "memory");
        __syncwarp();
        int total = 0;
        for (int s = lane; s < sources; s += 32) total += bytes_of(source[s]);
        total = __reduce_add_sync(0xffffffffu, total);
        if (lane == 0) mbar_expect_tx(&bar, total);
        __syncwarp();
        for (int s = lane; s < sources; s += 32) {
          const int n = bytes_of(source[s]);
          if (n) bulk_load(smem + s * chunk, from + source[s] * from_row, n, &bar);
        }
        if (!mbar_wait(&bar, phase)) {  // a copy never arrived: report, wait once more, and move nothing else
          if (lane == 0) atomicOr(a.err, H2O_BERR_INTERNAL), s_lost = 1;
          mbar_wait(&bar, phase);
          __syncwarp();
          continue;
        }
        phase ^= 1;
        for (int m = lane; m < n_moves; m += 32) {
          const int b = dest[m], p = parent[b], n = bytes_of(p);
          if (n) bulk_store(to + b * to_row, smem + slot_of[p] * chunk, n);
        }
        asm volatile("cp.async.bulk.commit_group;" ::: "memory");
      }
      continue;
    }
    // scales: words of 4 bytes
    if (warp == 0) asm volatile("cp.async.bulk.wait_group.read 0;" ::: "memory");
    __syncthreads();
    if (s_lost) continue;
    const int words = chunk / 4;
    for (int z = tid; z < sources * words; z += kThreads) {
      const int s = z / words, w = z % words;
      if (w * 4 < bytes_of(source[s])) ((float *)smem)[z] = *(const float *)(from + source[s] * from_row + w * 4);
    }
    __syncthreads();
    for (int z = tid; z < n_moves * words; z += kThreads) {
      const int b = dest[z / words], w = z % words, p = parent[b];
      if (w * 4 < bytes_of(p)) *(float *)(to + b * to_row + w * 4) = ((const float *)smem)[slot_of[p] * words + w];
    }
    __syncthreads();
  }
  if (warp == 0) asm volatile("cp.async.bulk.wait_group 0;" ::: "memory");
}

}  // namespace

cudaError_t launch_copy(const View &to, const View &from, const int32_t *parent, const int32_t *from_lengths,
                        const int32_t *lengths, int32_t *new_lengths, cudaStream_t st) {
  Args a = {};
  const void *const src[kArrays] = {from.K, from.V, from.pos, from.score, from.low, from.bounds, from.Ksc, from.Vsc};
  void *const dst[kArrays] = {to.K, to.V, to.pos, to.score, to.low, to.bounds, to.Ksc, to.Vsc};
  const int per[kArrays] = {kBlock * to.d, kBlock * to.d, kBlock * 4, kBlock * 4, kBlock * 4, 2 * to.d, 4, 4};
  for (int x = 0; x < kArrays; ++x) {
    a.from[x] = (const uint8_t *)src[x], a.to[x] = (uint8_t *)dst[x], a.per_block[x] = per[x];
    a.from_head[x] = (int64_t)(from.cap / kBlock) * per[x], a.to_head[x] = (int64_t)(to.cap / kBlock) * per[x];
  }
  a.parent = parent, a.from_lengths = from_lengths, a.lengths = lengths, a.new_lengths = new_lengths;
  a.err = to.err;
  a.H = to.H, a.to_rows = to.B, a.from_rows = from.B, a.from_cap = from.cap, a.to_cap = to.cap;
  a.same = to.K == from.K;
  a.arrays = to.bounds && from.bounds ? kBulk : kBulk - 1;
  const int lists = (3 * from.B + 2 * to.B) * 4;
  // Four CTAs an SM.  Large caches: several waves of them and larger pieces (64 rows of 56 heads 309 -> 306 us, prompt forks
  // 194 -> 177; four beams of 255 entries would take 18 us for 9).  Room for fewer and larger pieces, 98 KB of two CTAs an
  // SM, 315 and 190; the next item's reads under this one's writes, with half the pieces' size, 312 and 192 at best.
  const bool large = 2 * (int64_t)to.B * to.H * to.cap * to.d >= 256 << 20;
  a.chunk = large ? 8192 : 4096;
  a.room = 16 * from.B > 49152 ? 16 * from.B : 49152;
  const int smem = a.room + lists;
  static SmemLimit limit;
  const cudaError_t e = limit.raise((const void *)copy_kernel, smem);
  if (e != cudaSuccess) return e;
  copy_kernel<<<to.sms * (large ? 16 : 4), kThreads, smem, st>>>(a);
  return cudaGetLastError();
}

}  // namespace blk
}  // namespace h2o
