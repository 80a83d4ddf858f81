// block_api.cu — the C ABI of the block-scaled 8-bit caches (h2o_bcache_* in
// include/h2o.h): argument checks, the workspace carve-up and the launches.
#include <cudaTypedefs.h>

#include <cstdint>
#include <new>

#include "block_cache.cuh"
#include "rows.h"

using namespace h2o;

struct h2o_bcache {
  blk::View view;
  CUtensorMap kmap, vmap;
  int max_queries;
  int device;
  cudaStream_t stream;
};

namespace {

constexpr size_t kAlign = 256;

size_t align_up(size_t x) { return (x + kAlign - 1) & ~(kAlign - 1); }

h2o_status fail(cudaError_t e) {
  note_cuda_error(e);
  return H2O_ECUDA;
}

// Makes the cache's device current for the launches of one call.
struct OnDevice {
  int before = -1;
  cudaError_t err;
  explicit OnDevice(int device) {
    err = cudaGetDevice(&before);
    if (err == cudaSuccess && before != device)
      err = cudaSetDevice(device);
    else
      before = -1;
  }
  ~OnDevice() {
    if (before >= 0) cudaSetDevice(before);
  }
};

bool shape_ok(int B, int H, int d, int64_t capacity, int group, int max_queries, h2o_kv8 kv) {
  if (B < 1 || H < 1 || (int64_t)B * H > (1LL << 24) || d < 1) return false;
  if (capacity < H2O_BLOCK || capacity % H2O_BLOCK || capacity > (1LL << 30)) return false;
  if ((int64_t)B * H * capacity > 0x7fffffffLL) return false;
  if (group < 1 || max_queries < 1 || group > H2O_BLOCK_MAX_ROWS || max_queries > H2O_BLOCK_MAX_ROWS) return false;
  if (group * max_queries > H2O_BLOCK_MAX_ROWS) return false;
  return kv == H2O_KV_E4M3 || kv == H2O_KV_INT8;
}
bool d_supported(int d) { return d == 64 || d == 128; }

struct Layout {
  size_t K, V, Ksc, Vsc, pos, score, low, logits, part, err, total;
};
Layout layout(int B, int H, int d, int64_t cap, int rows, int sms) {
  const size_t nh = (size_t)B * H, entries = nh * (size_t)cap, scales = entries / H2O_BLOCK * sizeof(float);
  Layout l;
  size_t o = 0;
  l.K = o;       o = align_up(o + entries * d);
  l.V = o;       o = align_up(o + entries * d);
  l.Ksc = o;     o = align_up(o + scales);
  l.Vsc = o;     o = align_up(o + scales);
  l.pos = o;     o = align_up(o + entries * sizeof(int32_t));
  l.score = o;   o = align_up(o + entries * sizeof(float));
  l.low = o;     o = align_up(o + entries * sizeof(float));
  l.logits = o;  o = align_up(o + entries * rows * sizeof(float));
  l.part = o;    o = align_up(o + blk::attend_scratch_bytes(B, H, d, rows, sms));
  l.err = o;     o = align_up(o + sizeof(int));
  l.total = o;
  return l;
}

bool rows_ok(const h2o_rows *r) { return rows_fit(r, 8); }
blk::Rows rows_of(const h2o_rows *r) {
  return blk::Rows{(const __nv_bfloat16 *)r->data, r->stride_b, r->stride_h, r->stride_t};
}

// The codes as a matrix of d-byte rows in boxes of one block, with the widest
// swizzle a row allows.
bool code_map(CUtensorMap *m, const void *base, int d, int64_t entries) {
  void *p = nullptr;
  cudaDriverEntryPointQueryResult q;
  if (cudaGetDriverEntryPointByVersion("cuTensorMapEncodeTiled", &p, 12000, cudaEnableDefault, &q) != cudaSuccess ||
      q != cudaDriverEntryPointSuccess)
    return false;
  const cuuint64_t dims[2] = {(cuuint64_t)d, (cuuint64_t)entries}, strides[1] = {(cuuint64_t)d};
  const cuuint32_t box[2] = {(cuuint32_t)d, H2O_BLOCK}, step[2] = {1, 1};
  return ((PFN_cuTensorMapEncodeTiled_v12000)p)(
             m, CU_TENSOR_MAP_DATA_TYPE_UINT8, 2, const_cast<void *>(base), dims, strides, box, step,
             CU_TENSOR_MAP_INTERLEAVE_NONE, d == 128 ? CU_TENSOR_MAP_SWIZZLE_128B : CU_TENSOR_MAP_SWIZZLE_64B,
             CU_TENSOR_MAP_L2_PROMOTION_L2_128B, CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) == CUDA_SUCCESS;
}

bool ints_ok(const int32_t *p, bool may_be_null) { return p ? aligned(p, 4) : may_be_null; }

// A choice of blocks holds the last one, whose bounds need not be current.
bool choice_ok(const h2o_bcache *c, int n, int n_blocks, int n_first, int n_last, const int32_t *blocks) {
  if (n_first < 0 || n_last < 1 || (int64_t)n_first + n_last > n_blocks || n_blocks > H2O_SPARSE_MAX_BLOCKS) return false;
  if (!ints_ok(blocks, false)) return false;
  return (int64_t)c->view.B * c->view.H * n <= 0x7fffffffLL;  // a grid
}

bool overlap(const int32_t *x, int nx, const int32_t *y, int ny) {
  const uintptr_t a = (uintptr_t)x, z = (uintptr_t)y;
  return a < z + (uintptr_t)ny * sizeof(int32_t) && z < a + (uintptr_t)nx * sizeof(int32_t);
}

}  // namespace

extern "C" {

size_t h2o_bcache_workspace_bytes(int B, int H, int d, int64_t capacity, int group, int max_queries, h2o_kv8 kv) {
  if (!shape_ok(B, H, d, capacity, group, max_queries, kv) || !d_supported(d)) return 0;
  const int sms = num_sms_current_device();
  if (sms <= 0) return 0;
  return layout(B, H, d, capacity, group * max_queries, sms).total;
}

h2o_status h2o_bcache_create(int B, int H, int d, int64_t capacity, int group, int max_queries, h2o_kv8 kv,
                             void *workspace, void *cuda_stream, h2o_bcache_t *out) {
  if (!out) return H2O_EINVAL;
  *out = nullptr;
  if (!shape_ok(B, H, d, capacity, group, max_queries, kv)) return H2O_EINVAL;
  if (!d_supported(d)) return H2O_EUNSUPPORTED;
  if (!workspace || !aligned(workspace, kAlign)) return H2O_EINVAL;
  const int sms = num_sms_current_device();
  if (sms <= 0) return fail(cudaGetLastError());
  h2o_bcache *c = new (std::nothrow) h2o_bcache();
  if (!c) return H2O_ENOMEM;
  c->max_queries = max_queries;
  c->stream = (cudaStream_t)cuda_stream;
  const Layout l = layout(B, H, d, capacity, group * max_queries, sms);
  char *w = (char *)workspace;
  blk::View &v = c->view;
  v.B = B; v.H = H; v.d = d; v.cap = (int)capacity; v.group = group; v.max_rows = group * max_queries;
  v.kv = (int)kv; v.sms = sms;
  v.K = (uint8_t *)w + l.K; v.V = (uint8_t *)w + l.V;
  v.Ksc = (float *)(w + l.Ksc); v.Vsc = (float *)(w + l.Vsc);
  v.pos = (int32_t *)(w + l.pos); v.score = (float *)(w + l.score);
  v.low = (float *)(w + l.low);
  v.logits = (float *)(w + l.logits); v.kept = (int32_t *)(w + l.logits);
  v.part = (float *)(w + l.part);
  v.err = (int *)(w + l.err);
  const int64_t entries = (int64_t)B * H * capacity;
  if (!code_map(&c->kmap, v.K, d, entries) || !code_map(&c->vmap, v.V, d, entries)) {
    delete c;
    return fail(cudaErrorNotSupported);
  }
  cudaError_t e = cudaGetDevice(&c->device);
  if (e == cudaSuccess) e = cudaDeviceGetAttribute(&v.l2_bytes, cudaDevAttrL2CacheSize, c->device);
  if (e == cudaSuccess) e = cudaMemsetAsync(w + l.K, 0, l.pos - l.K, c->stream);  // codes and scales
  if (e == cudaSuccess) e = cudaMemsetAsync(v.pos, 0xff, l.score - l.pos, c->stream);
  if (e == cudaSuccess) e = cudaMemsetAsync(v.score, 0, l.logits - l.score, c->stream);  // and what they lose
  if (e == cudaSuccess) e = cudaMemsetAsync(v.err, 0, sizeof(int), c->stream);
  if (e != cudaSuccess) {
    delete c;
    return fail(e);
  }
  *out = c;
  return H2O_OK;
}

h2o_status h2o_bcache_destroy(h2o_bcache_t c) {
  delete c;
  return H2O_OK;
}

h2o_status h2o_bcache_set_stream(h2o_bcache_t c, void *s) {
  if (!c) return H2O_EINVAL;
  c->stream = (cudaStream_t)s;
  return H2O_OK;
}

h2o_status h2o_bcache_arrays(h2o_bcache_t c, void **K, void **V, float **K_scale, float **V_scale, int32_t **pos,
                             float **score) {
  if (!c) return H2O_EINVAL;
  if (K) *K = c->view.K;
  if (V) *V = c->view.V;
  if (K_scale) *K_scale = c->view.Ksc;
  if (V_scale) *V_scale = c->view.Vsc;
  if (pos) *pos = c->view.pos;
  if (score) *score = c->view.score;
  return H2O_OK;
}

h2o_status h2o_bcache_append(h2o_bcache_t c, int n, const h2o_rows *k, const h2o_rows *v, const int32_t *lengths,
                             const int32_t *counts, const int32_t *position, const float *score) {
  if (!c || n < 1 || n > c->view.cap || !rows_ok(k) || !rows_ok(v)) return H2O_EINVAL;
  if (!ints_ok(lengths, false) || !ints_ok(counts, true) || !ints_ok(position, true) || !aligned(score, 4))
    return H2O_EINVAL;
  OnDevice on(c->device);
  if (on.err != cudaSuccess) return fail(on.err);
  const blk::Lens l{lengths, counts, n, 1, c->view.cap};
  const cudaError_t e = blk::launch_append(c->view, l, rows_of(k), rows_of(v), position, score, c->stream);
  return e == cudaSuccess ? H2O_OK : fail(e);
}

h2o_status h2o_bcache_attend(h2o_bcache_t c, int n, const h2o_rows *q, const int32_t *lengths,
                             const int32_t *counts, int causal, int accumulate, const h2o_rows *out, float *lse) {
  if (!c || n < 1 || n > c->max_queries || !rows_ok(q) || !rows_ok(out)) return H2O_EINVAL;
  if (!ints_ok(lengths, false) || !ints_ok(counts, true) || !aligned(lse, 4)) return H2O_EINVAL;
  if (!rows_apart(out, c->view.B, c->view.H * c->view.group, n, c->view.d)) return H2O_EINVAL;
  OnDevice on(c->device);
  if (on.err != cudaSuccess) return fail(on.err);
  const blk::Lens l{lengths, counts, n, 0, c->view.cap};
  const cudaError_t e =
      blk::head_fits(c->view, n)
          ? blk::launch_head(c->view, l, rows_of(q), nullptr, nullptr, nullptr, causal != 0, accumulate != 0, rows_of(out),
                             lse, c->kmap, c->vmap, c->stream)
          : blk::launch_attend(c->view, l, rows_of(q), causal != 0, accumulate != 0, rows_of(out), lse, c->kmap, c->vmap,
                               c->stream);
  return e == cudaSuccess ? H2O_OK : fail(e);
}

h2o_status h2o_bcache_step(h2o_bcache_t c, int n, const h2o_rows *q, const h2o_rows *k, const h2o_rows *v,
                           const int32_t *lengths, const int32_t *counts, const int32_t *position, int accumulate,
                           const h2o_rows *out, float *lse) {
  if (!c || n < 1 || n > c->max_queries || n > c->view.cap) return H2O_EINVAL;
  if (!rows_ok(q) || !rows_ok(k) || !rows_ok(v) || !rows_ok(out)) return H2O_EINVAL;
  if (!ints_ok(lengths, false) || !ints_ok(counts, true) || !ints_ok(position, true) || !aligned(lse, 4))
    return H2O_EINVAL;
  if (!rows_apart(out, c->view.B, c->view.H * c->view.group, n, c->view.d)) return H2O_EINVAL;
  OnDevice on(c->device);
  if (on.err != cudaSuccess) return fail(on.err);
  const blk::Lens l{lengths, counts, n, 1, c->view.cap};
  if (blk::head_fits(c->view, n)) {
    const blk::Rows kr = rows_of(k), vr = rows_of(v);
    const cudaError_t e = blk::launch_head(c->view, l, rows_of(q), &kr, &vr, position, 1, accumulate != 0, rows_of(out),
                                           lse, c->kmap, c->vmap, c->stream);
    return e == cudaSuccess ? H2O_OK : fail(e);
  }
  cudaError_t e = blk::launch_append(c->view, l, rows_of(k), rows_of(v), position, nullptr, c->stream);
  if (e == cudaSuccess)
    e = blk::launch_attend(c->view, l, rows_of(q), 1, accumulate != 0, rows_of(out), lse, c->kmap, c->vmap, c->stream);
  return e == cudaSuccess ? H2O_OK : fail(e);
}

h2o_status h2o_bcache_evict(h2o_bcache_t c, const int32_t *lengths, int k_heavy, int k_local, int n_sink,
                            int score_mode, const int32_t *position, int32_t *new_lengths) {
  if (!c || k_heavy < 0 || k_local < 0 || (int64_t)k_heavy + k_local < 1 || (int64_t)k_heavy + k_local > 0x7fffffffLL)
    return H2O_EINVAL;
  if (n_sink < 0 || n_sink > k_heavy || (score_mode != 0 && score_mode != 1)) return H2O_EINVAL;
  if (!ints_ok(lengths, false) || !ints_ok(new_lengths, false) || !ints_ok(position, true)) return H2O_EINVAL;
  // heads still read the lengths and positions when the first ones write the new lengths
  if (overlap(lengths, c->view.B, new_lengths, c->view.B) ||
      (position && overlap(position, c->view.B, new_lengths, c->view.B)))
    return H2O_EINVAL;
  OnDevice on(c->device);
  if (on.err != cudaSuccess) return fail(on.err);
  cudaError_t e = blk::launch_evict(c->view, lengths, k_heavy, k_local, n_sink, score_mode, position, new_lengths,
                                    c->stream);
  if (e == cudaSuccess && c->view.bounds)
    e = blk::launch_bound(c->view, blk::Lens{new_lengths, nullptr, 1, 0, c->view.cap}, 2, c->stream);
  return e == cudaSuccess ? H2O_OK : fail(e);
}

h2o_status h2o_bcache_copy(h2o_bcache_t c, h2o_bcache_t source, const int32_t *parent, const int32_t *source_lengths,
                           const int32_t *lengths, int32_t *new_lengths) {
  if (!c || !ints_ok(parent, false) || !ints_ok(lengths, false) || !ints_ok(new_lengths, false)) return H2O_EINVAL;
  const bool same = !source || source == c;
  if (same) source = c;
  if (same ? source_lengths != nullptr : !ints_ok(source_lengths, false)) return H2O_EINVAL;
  const blk::View &to = c->view, &from = source->view;
  if (source->device != c->device || to.H != from.H || to.d != from.d || to.kv != from.kv) return H2O_EINVAL;
  // rows still read the lengths when the first ones write the new lengths
  if (overlap(lengths, to.B, new_lengths, to.B) || overlap(parent, to.B, new_lengths, to.B) ||
      (!same && overlap(source_lengths, from.B, new_lengths, to.B)))
    return H2O_EINVAL;
  if (to.B > blk::kCopyRows || from.B > blk::kCopyRows) return H2O_EUNSUPPORTED;
  OnDevice on(c->device);
  if (on.err != cudaSuccess) return fail(on.err);
  cudaError_t e = blk::launch_copy(to, from, parent, same ? lengths : source_lengths, lengths, new_lengths, c->stream);
  if (e == cudaSuccess && to.bounds && !from.bounds)
    e = blk::launch_bound(to, blk::Lens{new_lengths, nullptr, 1, 0, to.cap}, 2, c->stream);
  return e == cudaSuccess ? H2O_OK : fail(e);
}

size_t h2o_bcache_bounds_bytes(h2o_bcache_t c) {
  return c ? (size_t)c->view.B * c->view.H * (c->view.cap / H2O_BLOCK) * 2 * c->view.d : 0;
}

h2o_status h2o_bcache_set_bounds(h2o_bcache_t c, void *bounds) {
  if (!c || !aligned(bounds, 16)) return H2O_EINVAL;
  c->view.bounds = (int8_t *)bounds;
  return H2O_OK;
}

h2o_status h2o_bcache_bound(h2o_bcache_t c, const int32_t *lengths) {
  if (!c || !ints_ok(lengths, false)) return H2O_EINVAL;
  if (!c->view.bounds) return H2O_ESTATE;
  OnDevice on(c->device);
  if (on.err != cudaSuccess) return fail(on.err);
  const cudaError_t e = blk::launch_bound(c->view, blk::Lens{lengths, nullptr, 1, 0, c->view.cap}, 1, c->stream);
  return e == cudaSuccess ? H2O_OK : fail(e);
}

h2o_status h2o_bcache_attend_sparse(h2o_bcache_t c, int n, const h2o_rows *q, const int32_t *lengths,
                                    const int32_t *counts, int causal, int accumulate, int n_blocks, int n_first,
                                    int n_last, const h2o_rows *out, float *lse, int32_t *blocks) {
  if (!c || n < 1 || n > c->max_queries || !rows_ok(q) || !rows_ok(out)) return H2O_EINVAL;
  if (!ints_ok(lengths, false) || !ints_ok(counts, true) || !aligned(lse, 4)) return H2O_EINVAL;
  if (!rows_apart(out, c->view.B, c->view.H * c->view.group, n, c->view.d)) return H2O_EINVAL;
  if (!choice_ok(c, n, n_blocks, n_first, n_last, blocks)) return H2O_EINVAL;
  if (!c->view.bounds) return H2O_ESTATE;
  OnDevice on(c->device);
  if (on.err != cudaSuccess) return fail(on.err);
  const blk::Lens l{lengths, counts, n, 0, c->view.cap};
  const cudaError_t e =
      blk::launch_sparse(c->view, l, rows_of(q), nullptr, nullptr, nullptr, causal != 0, accumulate != 0, n_blocks, n_first,
                         n_last, rows_of(out), lse, blocks, c->kmap, c->vmap, c->stream);
  return e == cudaSuccess ? H2O_OK : fail(e);
}

h2o_status h2o_bcache_step_sparse(h2o_bcache_t c, int n, const h2o_rows *q, const h2o_rows *k, const h2o_rows *v,
                                  const int32_t *lengths, const int32_t *counts, const int32_t *position,
                                  int accumulate, int n_blocks, int n_first, int n_last, const h2o_rows *out, float *lse,
                                  int32_t *blocks) {
  if (!c || n < 1 || n > c->max_queries || n > c->view.cap) return H2O_EINVAL;
  if (!rows_ok(q) || !rows_ok(k) || !rows_ok(v) || !rows_ok(out)) return H2O_EINVAL;
  if (!ints_ok(lengths, false) || !ints_ok(counts, true) || !ints_ok(position, true) || !aligned(lse, 4))
    return H2O_EINVAL;
  if (!rows_apart(out, c->view.B, c->view.H * c->view.group, n, c->view.d)) return H2O_EINVAL;
  if (!choice_ok(c, n, n_blocks, n_first, n_last, blocks)) return H2O_EINVAL;
  if (!c->view.bounds) return H2O_ESTATE;
  OnDevice on(c->device);
  if (on.err != cudaSuccess) return fail(on.err);
  const blk::Lens l{lengths, counts, n, 1, c->view.cap};
  const blk::Rows kr = rows_of(k), vr = rows_of(v);
  const cudaError_t e =
      blk::launch_sparse(c->view, l, rows_of(q), &kr, &vr, position, 1, accumulate != 0, n_blocks, n_first, n_last,
                         rows_of(out), lse, blocks, c->kmap, c->vmap, c->stream);
  return e == cudaSuccess ? H2O_OK : fail(e);
}

h2o_status h2o_bcache_get_error(h2o_bcache_t c, int *bits) {
  if (!c) return H2O_EINVAL;
  OnDevice on(c->device);
  if (on.err != cudaSuccess) return fail(on.err);
  int flag = 0;
  cudaError_t e = cudaMemcpyAsync(&flag, c->view.err, sizeof(int), cudaMemcpyDeviceToHost, c->stream);
  if (e == cudaSuccess) e = cudaStreamSynchronize(c->stream);
  if (e != cudaSuccess) return fail(e);
  if (bits) *bits = flag;
  return flag ? H2O_EDEVICE : H2O_OK;
}

}  // extern "C"
