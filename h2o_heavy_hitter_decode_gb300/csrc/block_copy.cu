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
// Copies in both directions are bulk ones, a few KB each, by one warp of a CTA;
// the scales, whose rows may start at any multiple of 4 bytes, go through the
// registers of the others meanwhile.
//
// Bound by memory: beams of 64 rows of 56 heads, 700 to 2,047 entries, 1,771
// MB, 283 us, 92 % of the copy rate; two prompts of 8,000 tokens forked into 13
// rows, 1,065 MB, 175 us, 90 %.  Four beams of 255 entries by latency: 7 us, the
// maps' way through shared memory, one piece a CTA in and out.
//
// All rows that are read share the pieces' 48 KB: of more rows the pieces are
// smaller, and from some 200 on their number bounds it.  Beams of 1,593 MB in
// all (e4m3, bounds; memory alone 235 us): 128 rows x 32 heads 278 us, 256 x 16
// 569, 512 x 8 1,058, 1,024 x 4 2,039, 4,096 x 1 21,570, which is 16 bytes a piece.
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
  int words;   // and words for those of scales: a power of two
};

__device__ __forceinline__ void bulk_store(void *dst, const void *src, uint32_t bytes) {
  asm volatile("cp.async.bulk.global.shared::cta.bulk_group [%0], [%1], %2;" ::"l"(dst), "r"(smem_u32(src)), "r"(bytes)
               : "memory");
}

// Shared memory: the bulk copies' pieces; slot_of [from_rows] (a read row's place among the
// pieces, -1); blocks [from_rows] (their lengths first); the read rows and the
// rows that receive something, in order; parent [to_rows]; the scales' pieces.
__global__ void __launch_bounds__(kThreads) copy_kernel(const Args a) {
  extern __shared__ __align__(128) uint8_t smem[];
  int *slot_of = (int *)(smem + a.room), *blocks = slot_of + a.from_rows;
  int *source = blocks + a.from_rows;  // of a piece
  int *dest = source + a.from_rows, *parent = dest + a.to_rows;
  __shared__ __align__(8) uint64_t bar;
  __shared__ int s_sources, s_moves, s_most, s_warp[kThreads / 32];
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
  if (tid == 0) {
    s_sources = s_moves = s_most = 0;
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
  int words = a.words;  // of a row's scales
  while (words > 1 && words * sources > a.words) words >>= 1;

  // Items: (array, head, chunk); warp 0 has the bulk copies, the others the scales.
  int64_t items_of[kArrays];
#pragma unroll
  for (int x = 0; x < kArrays; ++x) {
    const bool none = x == kBulk - 1 && a.arrays < kBulk;
    const int piece = x < kBulk ? chunk : words * 4;
    items_of[x] = none ? 0 : ((int64_t)most * a.per_block[x] + piece - 1) / piece * a.H;
  }
  struct Item {
    int x, h;
    int64_t at;  // the first byte of a row's
  };
  auto item_at = [&](int64_t i, int x, int piece) {  // the i-th from array x on
    Item it;
    it.x = x;
    while (i >= items_of[it.x]) i -= items_of[it.x++];
    const int64_t pieces = items_of[it.x] / a.H;  // neighbours in a row to neighbouring CTAs
    it.h = (int)(i / pieces);
    it.at = (i - it.h * pieces) * piece;
    return it;
  };
  auto bytes_of = [&](const Item &it, int p, int piece) {
    const int64_t left = (int64_t)blocks[p] * a.per_block[it.x] - it.at;
    return (int)(left < 0 ? 0 : left < piece ? left : piece);
  };
  auto from_of = [&](const Item &it, int p) {
    return a.from[it.x] + ((int64_t)p * a.H + it.h) * a.from_head[it.x] + it.at;
  };
  auto to_of = [&](const Item &it, int b) {
    return a.to[it.x] + ((int64_t)b * a.H + it.h) * a.to_head[it.x] + it.at;
  };
  int64_t bulk = 0;
#pragma unroll
  for (int x = 0; x < kBulk; ++x) bulk += items_of[x];
  if (warp == 0) {
    uint32_t phase = 0;
    for (int64_t item = blockIdx.x; item < bulk; item += gridDim.x) {
      const Item it = item_at(item, 0, chunk);
      int total = 0;
      for (int s = lane; s < sources; s += 32) total += bytes_of(it, source[s], chunk);
      total = __reduce_add_sync(0xffffffffu, total);
      if (lane == 0) mbar_expect_tx(&bar, total);
      // the last item's pieces have left shared memory
      asm volatile("cp.async.bulk.wait_group.read 0;" ::: "memory");
      __syncwarp();
      for (int s = lane; s < sources; s += 32) {
        const int n = bytes_of(it, source[s], chunk);
        if (n) bulk_load(smem + s * chunk, from_of(it, source[s]), n, &bar);
      }
      if (!mbar_wait(&bar, phase)) {  // a copy never arrived: report, wait once more, and move nothing else
        if (lane == 0) atomicOr(a.err, H2O_BERR_INTERNAL);
        mbar_wait(&bar, phase);
        break;
      }
      phase ^= 1;
      for (int m = lane; m < n_moves; m += 32) {
        const int b = dest[m], p = parent[b], n = bytes_of(it, p, chunk);
        if (n) bulk_store(to_of(it, b), smem + slot_of[p] * chunk, n);
      }
      asm volatile("cp.async.bulk.commit_group;" ::: "memory");
    }
    __syncwarp();
    asm volatile("cp.async.bulk.wait_group 0;" ::: "memory");
    return;
  }
  float *held = (float *)(parent + a.to_rows);  // [sources][words]
  auto others = [&]() { asm volatile("bar.sync 1, %0;" ::"n"(kThreads - 32) : "memory"); };
  // from the last CTA down: those have the fewer bulk items
  const int64_t scales = items_of[kBulk] + items_of[kBulk + 1];
  for (int64_t item = gridDim.x - 1 - blockIdx.x; item < scales; item += gridDim.x) {
    const Item it = item_at(item, kBulk, words * 4);
    for (int z = tid - 32; z < sources * words; z += kThreads - 32) {
      const int s = z / words, w = z % words;
      if (w * 4 < bytes_of(it, source[s], words * 4)) held[z] = *(const float *)(from_of(it, source[s]) + w * 4);
    }
    others();
    for (int z = tid - 32; z < n_moves * words; z += kThreads - 32) {
      const int b = dest[z / words], w = z % words, p = parent[b];
      if (w * 4 < bytes_of(it, p, words * 4)) *(float *)(to_of(it, b) + w * 4) = held[slot_of[p] * words + w];
    }
    others();
  }
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
  a.words = 1024;
  while (a.words < from.B) a.words *= 2;
  const int lists = (3 * from.B + 2 * to.B + a.words) * 4;
  // Four CTAs an SM.  Large caches: several waves of them and larger pieces (64 rows of 56 heads 309 -> 306 us, prompt forks
  // 194 -> 177 when it was measured; four beams of 255 entries would take 18 us for 9).  Fewer and larger pieces, 98 KB
  // for two CTAs an SM, took 315 and 190; the next item's reads under this one's writes, in pieces of half the size, 312
  // and 192 at best.
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
