// C ABI of the paged-cache operators: argument checks, then one launcher each.
#include <cmath>
#include <cstdint>

#include "fa_cache.h"
#include "fa_internal.h"

namespace {

bool aligned(const void* p, uintptr_t to) { return p != nullptr && (reinterpret_cast<uintptr_t>(p) & (to - 1)) == 0; }

// log2 of a page size the cache takes (a power of two, 8..1024), -1 otherwise.
int page_shift_of(int page_size) {
  for (int s = 3; s <= 10; ++s)
    if (page_size == (1 << s)) return s;
  return -1;
}

bool stride_ok(long long s) { return s > 0 && s % 8 == 0 && s < (1ll << 38); }

// Rows of d elements, `count` of them `stride` apart, do not overlap (what is written must not).
bool apart(long long stride, long long count, int d) { return count <= 1 || stride >= d; }

fa_status check_cache(const fa_kv_cache* c) {
  if (c == nullptr || !aligned(c->k, 16) || !aligned(c->v, 16)) return FA_ERR_INVALID_ARG;
  if (c->dtype != FA_FP16 && c->dtype != FA_BF16) return FA_ERR_INVALID_ARG;
  if (c->num_pages < 1 || c->H_kv < 1 || c->d < 1 || page_shift_of(c->page_size) < 0) return FA_ERR_INVALID_ARG;
  if (!stride_ok(c->page_stride) || !stride_ok(c->head_stride) || !stride_ok(c->row_stride)) return FA_ERR_INVALID_ARG;
  if (!fa::head_dim_supported(c->d) || c->H_kv > 65535) return FA_ERR_UNSUPPORTED;
  if (static_cast<long long>(c->num_pages) * c->page_size > 0x7FFFFFFFll) return FA_ERR_UNSUPPORTED;
  if (!apart(c->page_stride, c->num_pages, c->d) || !apart(c->head_stride, c->H_kv, c->d) ||
      !apart(c->row_stride, c->page_size, c->d))
    return FA_ERR_INVALID_ARG;
  return FA_OK;
}

bool rows_ok(const fa_rows* r) {
  return r != nullptr && aligned(r->data, 16) && r->row_stride >= 0 && r->row_stride % 8 == 0 &&
         r->head_stride >= 0 && r->head_stride % 8 == 0;
}

bool written_rows_ok(const fa_rows* r, int rows, int heads, int d) {
  return rows_ok(r) && apart(r->row_stride, rows, d) && apart(r->head_stride, heads, d);
}

fa_status check_batch(int B, int rows, int max_pages) {
  if (B < 1 || rows < 0 || max_pages < 1) return FA_ERR_INVALID_ARG;
  if (B > fa::kCacheMaxB) return FA_ERR_UNSUPPORTED;
  if (static_cast<long long>(B) * max_pages > 0x7FFFFFFFll) return FA_ERR_UNSUPPORTED;
  return FA_OK;
}

fa_status check_rope_tables(int n_axes, int rot, int d, const int32_t* positions, long long pos_axis_stride,
                            const float* inv_freq, const uint8_t* axis) {
  if (rot < 0 || rot > d || rot % 16 != 0) return FA_ERR_INVALID_ARG;
  if (rot == 0) return FA_OK;
  if (n_axes < 1 || n_axes > 8 || pos_axis_stride < 0) return FA_ERR_INVALID_ARG;
  if (!aligned(positions, 4) || !aligned(inv_freq, 4) || axis == nullptr) return FA_ERR_INVALID_ARG;
  return FA_OK;
}

fa_status done(int cuda_status) { return cuda_status == 0 ? FA_OK : FA_ERR_CUDA; }

fa_status tree_impl(const fa_kv_cache* cache, const fa_rows* q, const fa_rows* o, float* lse, int B, int rows, int max_q,
                    int Hq, int max_pages, const int32_t* block_table, const int32_t* cu_q, const int32_t* seq_len,
                    const uint64_t* tree_mask, float softmax_scale, void* workspace, uint64_t withhold_timeout_ns,
                    cudaStream_t stream) {
  fa_status s = check_cache(cache);
  if (s != FA_OK) return s;
  s = check_batch(B, rows, max_pages);
  if (s != FA_OK) return s;
  if (max_q < 1 || Hq < 1 || Hq % cache->H_kv != 0 || !std::isfinite(softmax_scale)) return FA_ERR_INVALID_ARG;
  if (Hq > 65535 || (tree_mask != nullptr && max_q > FA_TREE_MAX)) return FA_ERR_UNSUPPORTED;
  if (static_cast<long long>(rows) * Hq > 0x7FFFFFFFll) return FA_ERR_UNSUPPORTED;
  if (rows == 0) return FA_OK;
  if (!rows_ok(q) || !written_rows_ok(o, rows, Hq, cache->d) || !aligned(lse, 4)) return FA_ERR_INVALID_ARG;
  if (!aligned(block_table, 4) || !aligned(cu_q, 4) || !aligned(seq_len, 4)) return FA_ERR_INVALID_ARG;
  if (tree_mask != nullptr && !aligned(tree_mask, 8)) return FA_ERR_INVALID_ARG;
  if (!aligned(workspace, 256)) return FA_ERR_INVALID_ARG;
  fa::TreeArgs a{};
  a.cache = *cache;
  a.q = *q;
  a.o = *o;
  a.lse = lse;
  a.B = B;
  a.rows = rows;
  a.max_q = max_q;
  a.Hq = Hq;
  a.max_pages = max_pages;
  a.page_shift = page_shift_of(cache->page_size);
  a.words = (max_q + 63) / 64;
  a.block_table = block_table;
  a.cu_q = cu_q;
  a.seq_len = seq_len;
  a.tree_mask = reinterpret_cast<const unsigned long long*>(tree_mask);
  a.scale = softmax_scale;
  a.workspace = workspace;
  if (withhold_timeout_ns != 0) {
    a.withhold = 1;
    a.timeout_ns = withhold_timeout_ns;
  }
  a.status = fa::device_status_word();
  if (a.status == nullptr) return FA_ERR_CUDA;
  return done(fa::launch_tree_fwd(a, stream));
}

}  // namespace

extern "C" {

fa_status fa_cache_plan(int B, int rows, int max_new, int page_size, int num_pages, int max_pages,
                        const int32_t* ctx_len, const int32_t* cu_new, const int32_t* parent, int32_t* block_table,
                        int32_t* n_pages, int32_t* free_list, int32_t* free_count, int32_t* seq_len, int32_t* slot,
                        int32_t* position, uint64_t* tree_mask, cudaStream_t stream) {
  const fa_status s = check_batch(B, rows, max_pages);
  if (s != FA_OK) return s;
  const int shift = page_shift_of(page_size);
  if (max_new < 1 || shift < 0 || num_pages < 1) return FA_ERR_INVALID_ARG;
  if ((parent == nullptr) != (tree_mask == nullptr)) return FA_ERR_INVALID_ARG;
  if (static_cast<long long>(num_pages) * page_size > 0x7FFFFFFFll) return FA_ERR_UNSUPPORTED;
  if (parent != nullptr && max_new > FA_TREE_MAX) return FA_ERR_UNSUPPORTED;
  const void* needed[] = {ctx_len, cu_new, block_table, n_pages, free_list, free_count, seq_len};
  for (const void* p : needed)
    if (!aligned(p, 4)) return FA_ERR_INVALID_ARG;
  if (rows > 0 && (!aligned(slot, 4) || !aligned(position, 4))) return FA_ERR_INVALID_ARG;
  if (parent != nullptr && (!aligned(parent, 4) || !aligned(tree_mask, 8))) return FA_ERR_INVALID_ARG;
  fa::PlanArgs a{};
  a.B = B;
  a.rows = rows;
  a.max_new = max_new;
  a.page_shift = shift;
  a.num_pages = num_pages;
  a.max_pages = max_pages;
  a.words = (max_new + 63) / 64;
  a.ctx_len = ctx_len;
  a.cu_new = cu_new;
  a.parent = parent;
  a.block_table = block_table;
  a.n_pages = n_pages;
  a.free_list = free_list;
  a.free_count = free_count;
  a.seq_len = seq_len;
  a.slot = slot;
  a.position = position;
  a.tree_mask = reinterpret_cast<unsigned long long*>(tree_mask);
  return done(fa::launch_cache_plan(a, stream));
}

fa_status fa_rope(fa_dtype dtype, const void* x, void* out, int B, int H, int N, int d, const long long x_strides[3],
                  const long long out_strides[3], const int32_t* positions, long long pos_axis_stride,
                  long long pos_b_stride, int n_axes, const float* inv_freq, const uint8_t* axis, int rot, int inverse,
                  int pairs, cudaStream_t stream) {
  if (dtype != FA_FP16 && dtype != FA_BF16) return FA_ERR_INVALID_ARG;
  if (B < 1 || H < 1 || N < 1 || d < 1 || x_strides == nullptr || out_strides == nullptr) return FA_ERR_INVALID_ARG;
  if (!fa::head_dim_supported(d)) return FA_ERR_UNSUPPORTED;
  if (static_cast<long long>(B) * N > 0x7FFFFFFFll || H > 65535) return FA_ERR_UNSUPPORTED;
  if (!aligned(x, 16) || !aligned(out, 16) || rot < 16 || pos_b_stride < 0) return FA_ERR_INVALID_ARG;
  for (int i = 0; i < 3; ++i)
    if (x_strides[i] < 0 || x_strides[i] % 8 != 0 || out_strides[i] < 0 || out_strides[i] % 8 != 0)
      return FA_ERR_INVALID_ARG;
  if (!apart(out_strides[0], B, d) || !apart(out_strides[1], H, d) || !apart(out_strides[2], N, d))
    return FA_ERR_INVALID_ARG;
  const fa_status s = check_rope_tables(n_axes, rot, d, positions, pos_axis_stride, inv_freq, axis);
  if (s != FA_OK) return s;
  fa::RopeArgs a{};
  fa::RopePart& r = a.part[0];
  r.src = static_cast<const uint16_t*>(x);
  r.dst = static_cast<uint16_t*>(out);
  r.src_b = x_strides[0];
  r.src_h = x_strides[1];
  r.src_n = x_strides[2];
  r.dst_b = out_strides[0];
  r.dst_h = out_strides[1];
  r.dst_n = out_strides[2];
  r.heads = H;
  r.rotate = 1;
  a.n_parts = 1;
  a.bf16 = dtype == FA_BF16;
  a.B = B;
  a.N = N;
  a.d = d;
  a.rot = rot;
  a.n_axes = n_axes;
  a.inverse = inverse != 0;
  a.pairs = pairs != 0;
  a.positions = positions;
  a.pos_axis = pos_axis_stride;
  a.pos_b = pos_b_stride;
  a.inv_freq = inv_freq;
  a.axis = axis;
  return done(fa::launch_rope(a, stream));
}

fa_status fa_rope_append(const fa_kv_cache* cache, int rows, int Hq, const fa_rows* q, const fa_rows* k,
                         const fa_rows* v, const fa_rows* q_out, const int32_t* slot, const int32_t* positions,
                         long long pos_axis_stride, int n_axes, const float* inv_freq, const uint8_t* axis, int rot,
                         int pairs, cudaStream_t stream) {
  fa_status s = check_cache(cache);
  if (s != FA_OK) return s;
  if (rows < 0 || (q == nullptr) != (q_out == nullptr)) return FA_ERR_INVALID_ARG;
  if (rows == 0) return FA_OK;
  if (!rows_ok(k) || !rows_ok(v) || !aligned(slot, 4)) return FA_ERR_INVALID_ARG;
  if (q != nullptr && (Hq < 1 || !rows_ok(q) || !written_rows_ok(q_out, rows, Hq, cache->d))) return FA_ERR_INVALID_ARG;
  if (q != nullptr && Hq > 65535) return FA_ERR_UNSUPPORTED;
  s = check_rope_tables(n_axes, rot, cache->d, positions, pos_axis_stride, inv_freq, axis);
  if (s != FA_OK) return s;
  fa::RopeArgs a{};
  a.n_parts = 0;
  if (q != nullptr) {
    fa::RopePart& r = a.part[a.n_parts++];
    r.src = static_cast<const uint16_t*>(q->data);
    r.dst = static_cast<uint16_t*>(q_out->data);
    r.src_n = q->row_stride;
    r.src_h = q->head_stride;
    r.dst_n = q_out->row_stride;
    r.dst_h = q_out->head_stride;
    r.heads = Hq;
    r.rotate = 1;
  }
  const fa_rows* from[2] = {k, v};
  void* to[2] = {cache->k, cache->v};
  for (int i = 0; i < 2; ++i) {
    fa::RopePart& r = a.part[a.n_parts++];
    r.src = static_cast<const uint16_t*>(from[i]->data);
    r.dst = static_cast<uint16_t*>(to[i]);
    r.src_n = from[i]->row_stride;
    r.src_h = from[i]->head_stride;
    r.dst_b = cache->page_stride;
    r.dst_h = cache->head_stride;
    r.dst_n = cache->row_stride;
    r.heads = cache->H_kv;
    r.rotate = i == 0;
    r.to_cache = 1;
  }
  a.bf16 = cache->dtype == FA_BF16;
  a.B = 1;
  a.N = rows;
  a.d = cache->d;
  a.rot = rot;
  a.n_axes = n_axes;
  a.pairs = pairs != 0;
  a.positions = positions;
  a.pos_axis = pos_axis_stride;
  a.inv_freq = inv_freq;
  a.axis = axis;
  a.slot = slot;
  a.page_shift = page_shift_of(cache->page_size);
  a.cache_rows = static_cast<long long>(cache->num_pages) * cache->page_size;
  return done(fa::launch_rope(a, stream));
}

size_t fa_tree_fwd_workspace_size(int B, int rows, int max_q, int Hq, int H_kv, int d) {
  if (B < 1 || rows < 0 || max_q < 1 || H_kv < 1 || Hq < 1 || Hq % H_kv != 0 || !fa::head_dim_supported(d)) return 0;
  return fa::tree_fwd_workspace(B, rows, max_q, Hq, H_kv, d);
}

fa_status fa_tree_fwd(const fa_kv_cache* cache, const fa_rows* q, const fa_rows* o, float* lse, int B, int rows,
                      int max_q, int Hq, int max_pages, const int32_t* block_table, const int32_t* cu_q,
                      const int32_t* seq_len, const uint64_t* tree_mask, float softmax_scale, void* workspace,
                      cudaStream_t stream) {
  return tree_impl(cache, q, o, lse, B, rows, max_q, Hq, max_pages, block_table, cu_q, seq_len, tree_mask, softmax_scale,
                   workspace, 0, stream);
}

fa_status fa_debug_tree_withhold(const fa_kv_cache* cache, const fa_rows* q, const fa_rows* o, float* lse, int B,
                                 int rows, int max_q, int Hq, int max_pages, const int32_t* block_table,
                                 const int32_t* cu_q, const int32_t* seq_len, const uint64_t* tree_mask,
                                 float softmax_scale, void* workspace, int timeout_ms, cudaStream_t stream) {
  if (timeout_ms < 1 || timeout_ms > 5000) return FA_ERR_INVALID_ARG;
  return tree_impl(cache, q, o, lse, B, rows, max_q, Hq, max_pages, block_table, cu_q, seq_len, tree_mask, softmax_scale,
                   workspace, static_cast<uint64_t>(timeout_ms) * 1000000ull, stream);
}

fa_status fa_cache_commit(const fa_kv_cache* cache, int B, int max_pages, int max_accept, const int32_t* block_table,
                          const int32_t* ctx_len, const int32_t* accepted, const int32_t* n_accepted,
                          int32_t* new_len, cudaStream_t stream) {
  fa_status s = check_cache(cache);
  if (s != FA_OK) return s;
  s = check_batch(B, 0, max_pages);
  if (s != FA_OK) return s;
  if (max_accept < 1) return FA_ERR_INVALID_ARG;
  const void* needed[] = {block_table, ctx_len, accepted, n_accepted, new_len};
  for (const void* p : needed)
    if (!aligned(p, 4)) return FA_ERR_INVALID_ARG;
  fa::CommitArgs a{};
  a.k = static_cast<uint16_t*>(cache->k);
  a.v = static_cast<uint16_t*>(cache->v);
  a.page_stride = cache->page_stride;
  a.head_stride = cache->head_stride;
  a.row_stride = cache->row_stride;
  a.num_pages = cache->num_pages;
  a.page_shift = page_shift_of(cache->page_size);
  a.H_kv = cache->H_kv;
  a.d = cache->d;
  a.B = B;
  a.max_pages = max_pages;
  a.max_accept = max_accept;
  a.block_table = block_table;
  a.ctx_len = ctx_len;
  a.accepted = accepted;
  a.n_accepted = n_accepted;
  a.new_len = new_len;
  return done(fa::launch_cache_commit(a, stream));
}

}  // extern "C"
