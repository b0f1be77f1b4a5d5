// extern "C" entry points of the paged 8-bit cache: argument checks on the
// host, before anything is launched, and dispatch.
#include <cuda_runtime.h>
#include <nvtx3/nvToolsExt.h>

#include <algorithm>
#include <cmath>
#include <vector>

#include "kvq_overlap.h"
#include "kvq_pages.h"

namespace {

// An entry point's NVTX range (for Nsight timelines and ncu --nvtx filters).
// The other entry points get theirs in the binding; these calls are short
// enough for that to be a tenth of them.
struct Range {
  explicit Range(const char* name) { nvtxRangePushA(name); }
  ~Range() { nvtxRangePop(); }
};

bool aligned(const void* p, unsigned a) { return (reinterpret_cast<uintptr_t>(p) & (a - 1u)) == 0; }

kvq_status check_geometry(const kvq_pages* p) {
  if (p == nullptr) return KVQ_ERR_INVALID_ARG;
  if (p->layers < 1 || p->n_pages < 1 || p->kv_heads < 1) return KVQ_ERR_INVALID_ARG;
  if (p->head_dim != 64 && p->head_dim != 128) return KVQ_ERR_UNSUPPORTED;
  if (p->page_tokens != 16 && p->page_tokens != 32 && p->page_tokens != 64 && p->page_tokens != 128)
    return KVQ_ERR_UNSUPPORTED;
  const long long blocks = (long long)p->n_pages * p->kv_heads;
  if (blocks >= (1LL << 31) || blocks > (1LL << 44) / p->layers) return KVQ_ERR_INVALID_ARG;
  return KVQ_OK;
}

kvq_status check_pool(const kvq_pages* p) {
  const kvq_status st = check_geometry(p);
  if (st != KVQ_OK) return st;
  if (!p->k_codes || !p->v_codes || !p->k_scale || !p->v_scale) return KVQ_ERR_INVALID_ARG;
  if (!aligned(p->k_codes, 16) || !aligned(p->v_codes, 16) || !aligned(p->k_scale, 2) ||
      !aligned(p->v_scale, 2))
    return KVQ_ERR_ALIGNMENT;
  return KVQ_OK;
}

kvq_status check_sequences(const kvq_sequences* s, int page_tokens) {
  if (s == nullptr || s->batch < 0 || s->width < 0 || s->rows < 0) return KVQ_ERR_INVALID_ARG;
  if (s->offsets == nullptr && s->rows != s->batch) return KVQ_ERR_INVALID_ARG;
  if (s->batch > (1 << 24)) return KVQ_ERR_INVALID_ARG;
  if ((long long)s->width * page_tokens > (1LL << 30) || s->rows > (1 << 30)) return KVQ_ERR_TOO_LARGE;
  if (s->rows == 0) return KVQ_OK;
  if (s->batch < 1 || s->kv_lens == nullptr) return KVQ_ERR_INVALID_ARG;
  if (s->width > 0 && s->table == nullptr) return KVQ_ERR_INVALID_ARG;
  if (s->batch > 1 && s->table_stride < s->width) return KVQ_ERR_INVALID_ARG;
  if (!aligned(s->table, 4) || !aligned(s->kv_lens, 4) || !aligned(s->offsets, 4))
    return KVQ_ERR_ALIGNMENT;
  return KVQ_OK;
}

int shift_of(int page) { return page == 16 ? 4 : page == 32 ? 5 : page == 64 ? 6 : 7; }

kvq::PageLayer layer_of(const kvq_pages* p, int layer) {
  const long long blocks = (long long)layer * p->n_pages * p->kv_heads;
  kvq::PageLayer l{};
  l.codes[0] = p->k_codes + blocks * p->page_tokens * p->head_dim;
  l.codes[1] = p->v_codes + blocks * p->page_tokens * p->head_dim;
  l.scale[0] = p->k_scale + blocks;
  l.scale[1] = p->v_scale + blocks;
  l.n_pages = p->n_pages;
  l.heads = p->kv_heads;
  l.d = p->head_dim;
  l.page = p->page_tokens;
  l.shift = shift_of(p->page_tokens);
  return l;
}

kvq::PageSeqs seqs_of(const kvq_sequences* s) {
  return kvq::PageSeqs{s->table, s->kv_lens, s->offsets, s->table_stride, s->batch, s->width, s->rows};
}

kvq::PagePool pool_of(const kvq_pages* p) {
  kvq::PagePool o{};
  o.codes[0] = p->k_codes;
  o.codes[1] = p->v_codes;
  o.scale[0] = p->k_scale;
  o.scale[1] = p->v_scale;
  o.layers = p->layers;
  o.n_pages = p->n_pages;
  o.heads = p->kv_heads;
  o.page_bytes = (long long)p->kv_heads * p->page_tokens * p->head_dim;
  return o;
}

// rows of 16-byte vectors at these strides
bool bad_stride(int64_t s) { return s < 0 || (s & 7) != 0; }

kvq_status check_rope(const kvq_rope_table* t, int head_dim) {
  if (t == nullptr || t->cos_sin == nullptr || t->n_positions < 1) return KVQ_ERR_INVALID_ARG;
  if (t->pairs < 8 || t->pairs % 8 != 0 || t->pairs > kvq::kRopeMaxPairs || 2 * t->pairs > head_dim) return KVQ_ERR_INVALID_ARG;
  if (t->axes < 1 || t->axes > kvq::kRopeMaxAxes) return KVQ_ERR_INVALID_ARG;
  for (int p = 0; p < t->pairs; ++p)
    if (t->axis[p] >= t->axes) return KVQ_ERR_INVALID_ARG;
  if (!aligned(t->cos_sin, 16)) return KVQ_ERR_ALIGNMENT;
  return KVQ_OK;
}

kvq::RopeTab rope_of(const kvq_rope_table* t) {
  kvq::RopeTab o{};
  o.cs = reinterpret_cast<const float2*>(t->cos_sin);
  o.n = t->n_positions;
  o.pairs = t->pairs;
  o.axes = t->axes;
  o.interleaved = t->interleaved != 0;
  o.none = -0.f;
  for (int k = 0; k < t->pairs; ++k) o.axis[k >> 4] |= (uint32_t)t->axis[k] << (2 * (k & 15));
  return o;
}

// The checks and arguments that the appends share; *done where there is
// nothing to append.
kvq_status append_args(const kvq_pages* pages, int32_t layer, const uint16_t* k_new, int64_t k_row_stride,
                       int64_t k_head_stride, const uint16_t* v_new, int64_t v_row_stride, int64_t v_head_stride,
                       const kvq_sequences* seqs, kvq::AppendArgs* out, bool* done) {
  *done = false;
  kvq_status st = check_pool(pages);
  if (st != KVQ_OK) return st;
  if (layer < 0 || layer >= pages->layers) return KVQ_ERR_INVALID_ARG;
  st = check_sequences(seqs, pages->page_tokens);
  if (st != KVQ_OK) return st;
  if (seqs->rows == 0) {
    *done = true;
    return KVQ_OK;
  }
  if (k_new == nullptr || v_new == nullptr) return KVQ_ERR_INVALID_ARG;
  if (bad_stride(k_row_stride) || bad_stride(k_head_stride) || bad_stride(v_row_stride) ||
      bad_stride(v_head_stride) || !aligned(k_new, 16) || !aligned(v_new, 16))
    return KVQ_ERR_ALIGNMENT;
  kvq::AppendArgs a{};
  a.p = layer_of(pages, layer);
  a.s = seqs_of(seqs);
  if (((long long)(seqs->rows >> a.p.shift) + 2LL * seqs->batch) * pages->kv_heads >= (1LL << 30))
    return KVQ_ERR_TOO_LARGE;
  a.x[0] = k_new;
  a.x[1] = v_new;
  a.row_stride[0] = k_row_stride;
  a.row_stride[1] = v_row_stride;
  a.head_stride[0] = k_head_stride;
  a.head_stride[1] = v_head_stride;
  *out = a;
  return KVQ_OK;
}

// The checks and arguments that the attention calls share; *done where there
// are no rows.
kvq_status attention_args(const kvq_pages* pages, int32_t layer, const uint16_t* q, int64_t q_row_stride,
                          int64_t q_head_stride, int32_t q_heads, const kvq_sequences* seqs, int32_t max_q, float scale,
                          int32_t causal, int32_t window, void* workspace, size_t workspace_bytes, uint16_t* out,
                          float* lse, kvq::PagedAttnArgs* out_args, bool* done) {
  *done = false;
  kvq_status st = check_pool(pages);
  if (st != KVQ_OK) return st;
  if (layer < 0 || layer >= pages->layers) return KVQ_ERR_INVALID_ARG;
  if (q_heads < 1 || q_heads % pages->kv_heads != 0) return KVQ_ERR_INVALID_ARG;
  st = check_sequences(seqs, pages->page_tokens);
  if (st != KVQ_OK) return st;
  if (!std::isfinite(scale) || scale <= 0.f || window < 0 || max_q < 0) return KVQ_ERR_INVALID_ARG;
  if (seqs->rows == 0) {
    *done = true;
    return KVQ_OK;
  }
  if (max_q < 1 || q == nullptr || out == nullptr) return KVQ_ERR_INVALID_ARG;
  if (bad_stride(q_row_stride) || bad_stride(q_head_stride) || !aligned(q, 16) || !aligned(out, 16) ||
      !aligned(lse, 4) || !aligned(workspace, 16))
    return KVQ_ERR_ALIGNMENT;
  if (max_q > seqs->rows) max_q = seqs->rows;
  if (seqs->offsets == nullptr) max_q = 1;
  const size_t need = kvq::paged_attention_workspace(
      pages->kv_heads, q_heads, pages->head_dim, seqs->batch,
      (long long)seqs->width * pages->page_tokens, seqs->rows, max_q);
  if (need > 16 && (workspace == nullptr || workspace_bytes < need)) return KVQ_ERR_INVALID_ARG;
  kvq::PagedAttnArgs a{};
  a.p = layer_of(pages, layer);
  a.s = seqs_of(seqs);
  a.q = q;
  a.q_row_stride = q_row_stride;
  a.q_head_stride = q_head_stride;
  a.q_heads = q_heads;
  a.group = q_heads / pages->kv_heads;
  a.max_q = max_q;
  a.causal = causal != 0;
  a.window = std::min(window, 1 << 30);   // no sequence is longer; t - window stays in 32 bits
  a.scale = scale;
  a.out = out;
  a.lse = lse;
  a.ws = workspace;
  a.ws_bytes = workspace_bytes;
  a.status = kvq::status_ptr();
  a.bounds_site = kvq::bounds_site_ptr();
  a.wait_limit_ns = kvq::wait_limit_ns();
  if (a.status == nullptr) return KVQ_ERR_CUDA;
  *out_args = a;
  return KVQ_OK;
}

}  // namespace

extern "C" {

kvq_status kvq_pages_bytes(const kvq_pages* pages, size_t* codes_bytes, size_t* scale_bytes) {
  const kvq_status st = check_geometry(pages);
  if (st != KVQ_OK) return st;
  const size_t blocks = (size_t)pages->layers * pages->n_pages * pages->kv_heads;
  if (codes_bytes) *codes_bytes = blocks * pages->page_tokens * pages->head_dim;
  if (scale_bytes) *scale_bytes = blocks * 2;
  return KVQ_OK;
}

kvq_status kvq_pages_append(const kvq_pages* pages, int32_t layer, const uint16_t* k_new,
                            int64_t k_row_stride, int64_t k_head_stride, const uint16_t* v_new,
                            int64_t v_row_stride, int64_t v_head_stride, const kvq_sequences* seqs,
                            void* stream) {
  const Range range("kvq_pages_append");
  kvq::AppendArgs a;
  bool done;
  const kvq_status st = append_args(pages, layer, k_new, k_row_stride, k_head_stride, v_new, v_row_stride, v_head_stride,
                                    seqs, &a, &done);
  if (st != KVQ_OK || done) return st;
  a.status = kvq::status_ptr();
  a.bounds_site = kvq::bounds_site_ptr();
  if (a.status == nullptr) return KVQ_ERR_CUDA;
  return kvq::launch_pages_append(a, static_cast<cudaStream_t>(stream)) == cudaSuccess ? KVQ_OK
                                                                                      : KVQ_ERR_CUDA;
}

kvq_status kvq_rope_fill(const kvq_rope_table* table, const double* frequency, double factor, void* stream) {
  const Range range("kvq_rope_fill");
  const kvq_status st = check_rope(table, 2 * kvq::kRopeMaxPairs);
  if (st != KVQ_OK) return st;
  if (frequency == nullptr || !std::isfinite(factor)) return KVQ_ERR_INVALID_ARG;
  for (int p = 0; p < table->pairs; ++p)
    if (!std::isfinite(frequency[p])) return KVQ_ERR_INVALID_ARG;
  return kvq::launch_rope_fill(table->cos_sin, table->n_positions, table->pairs, frequency, factor,
                               static_cast<cudaStream_t>(stream)) == cudaSuccess
             ? KVQ_OK
             : KVQ_ERR_CUDA;
}

kvq_status kvq_rope(const kvq_rope_table* table, const int32_t* positions, int64_t pos_batch_stride,
                    int64_t pos_row_stride, int64_t pos_axis_stride, int32_t batch, int32_t rows, int32_t head_dim,
                    int32_t inverse, const kvq_rope_tensor* tensors, int32_t n_tensors, void* stream) {
  const Range range("kvq_rope");
  if (head_dim != 64 && head_dim != 128) return KVQ_ERR_UNSUPPORTED;
  const kvq_status st = check_rope(table, head_dim);
  if (st != KVQ_OK) return st;
  if (batch < 0 || rows < 0 || tensors == nullptr || n_tensors < 1 || n_tensors > 2) return KVQ_ERR_INVALID_ARG;
  kvq::RopeArgs a{};
  long long heads = 0, blocks = 0;
  for (int i = 0; i < n_tensors; ++i) {
    const kvq_rope_tensor& t = tensors[i];
    if (t.heads < 0) return KVQ_ERR_INVALID_ARG;
    heads += t.heads;
    a.x[i] = kvq::RopeTensor{t.x, t.y, t.x_batch_stride, t.x_row_stride, t.x_head_stride,
                             t.y_batch_stride, t.y_row_stride, t.y_head_stride, t.heads};
  }
  const long long all = (long long)batch * rows;
  if (all > 0x7fffffffLL || heads > 0x7fffffffLL || (all > 0 && heads > (1LL << 35) / all)) return KVQ_ERR_TOO_LARGE;
  for (int i = 0; i < n_tensors; ++i) blocks += batch * kvq::rope_blocks(rows, tensors[i].heads, 16);
  if (blocks > 0x7fffffffLL) return KVQ_ERR_TOO_LARGE;
  if (all == 0 || heads == 0) return KVQ_OK;
  if (positions == nullptr) return KVQ_ERR_INVALID_ARG;
  if (!aligned(positions, 4)) return KVQ_ERR_ALIGNMENT;
  for (int i = 0; i < n_tensors; ++i) {
    const kvq_rope_tensor& t = tensors[i];
    if (t.heads == 0) continue;
    if (t.x == nullptr || t.y == nullptr) return KVQ_ERR_INVALID_ARG;
    if (!aligned(t.x, 16) || !aligned(t.y, 16) || bad_stride(t.x_batch_stride) || bad_stride(t.x_row_stride) ||
        bad_stride(t.x_head_stride) || bad_stride(t.y_batch_stride) || bad_stride(t.y_row_stride) ||
        bad_stride(t.y_head_stride))
      return KVQ_ERR_ALIGNMENT;
    // in place means place by place
    if (t.x == t.y && ((batch > 1 && t.x_batch_stride != t.y_batch_stride) ||
                       (rows > 1 && t.x_row_stride != t.y_row_stride) ||
                       (t.heads > 1 && t.x_head_stride != t.y_head_stride)))
      return KVQ_ERR_INVALID_ARG;
  }
  // nothing else is written that the call reads or writes
  auto x_of = [&](int i) {
    const kvq_rope_tensor& t = tensors[i];
    return kvq::Strided{t.x, t.x_batch_stride, t.x_row_stride, t.x_head_stride, batch, rows, t.heads, head_dim};
  };
  auto y_of = [&](int i) {
    const kvq_rope_tensor& t = tensors[i];
    return kvq::Strided{t.y, t.y_batch_stride, t.y_row_stride, t.y_head_stride, batch, rows, t.heads, head_dim};
  };
  for (int i = 0; i < n_tensors; ++i)
    if ((tensors[i].x != tensors[i].y && kvq::overlap(x_of(i), y_of(i))) || kvq::repeats(y_of(i))) return KVQ_ERR_INVALID_ARG;
  if (n_tensors == 2 && (kvq::overlap(y_of(0), x_of(1)) || kvq::overlap(y_of(0), y_of(1)) || kvq::overlap(y_of(1), x_of(0))))
    return KVQ_ERR_INVALID_ARG;
  a.t = rope_of(table);
  a.pos = positions;
  a.pb = pos_batch_stride;
  a.pr = pos_row_stride;
  a.pa = pos_axis_stride;
  a.batch = batch;
  a.rows = rows;
  a.d = head_dim;
  a.inverse = inverse != 0;
  a.status = kvq::status_ptr();
  a.bounds_site = kvq::bounds_site_ptr();
  if (a.status == nullptr) return KVQ_ERR_CUDA;
  return kvq::launch_rope(a, static_cast<cudaStream_t>(stream)) == cudaSuccess ? KVQ_OK : KVQ_ERR_CUDA;
}

kvq_status kvq_pages_append_rope(const kvq_pages* pages, int32_t layer, const kvq_rope_table* table,
                                 const int32_t* positions, int64_t pos_row_stride, const uint16_t* k_new,
                                 int64_t k_row_stride, int64_t k_head_stride, const uint16_t* v_new,
                                 int64_t v_row_stride, int64_t v_head_stride, const uint16_t* q, int64_t q_row_stride,
                                 int64_t q_head_stride, int32_t q_heads, uint16_t* q_out, int64_t q_out_row_stride,
                                 int64_t q_out_head_stride, const kvq_sequences* seqs, void* stream) {
  const Range range("kvq_pages_append_rope");
  kvq::AppendRopeArgs p{};
  bool done;
  kvq_status st = check_pool(pages);
  if (st != KVQ_OK) return st;
  st = check_rope(table, pages->head_dim);
  if (st != KVQ_OK) return st;
  if (q_heads < 0 || (q == nullptr) != (q_heads == 0) || (q_out == nullptr) != (q_heads == 0)) return KVQ_ERR_INVALID_ARG;
  if (positions == nullptr && table->axes != 1) return KVQ_ERR_INVALID_ARG;
  if (!aligned(positions, 4) || !aligned(q, 16) || !aligned(q_out, 16) || bad_stride(q_row_stride) ||
      bad_stride(q_head_stride) || bad_stride(q_out_row_stride) || bad_stride(q_out_head_stride))
    return KVQ_ERR_ALIGNMENT;
  st = append_args(pages, layer, k_new, k_row_stride, k_head_stride, v_new, v_row_stride, v_head_stride, seqs, &p.a, &done);
  if (st != KVQ_OK || done) return st;
  if ((long long)seqs->rows * q_heads > (1LL << 32) || kvq::append_rope_blocks(p.a.s, p.a.p, q_heads) > 0x7fffffffLL)
    return KVQ_ERR_TOO_LARGE;
  // queries in place are so place by place, and nothing else that the call reads is written
  if (q != nullptr) {
    auto rows_of = [&](const uint16_t* x, int64_t row, int64_t head, int32_t heads) {
      return kvq::Strided{x, 0, row, head, 1, seqs->rows, heads, pages->head_dim};
    };
    const kvq::Strided out = rows_of(q_out, q_out_row_stride, q_out_head_stride, q_heads);
    if (q == q_out ? (seqs->rows > 1 && q_row_stride != q_out_row_stride) || (q_heads > 1 && q_head_stride != q_out_head_stride)
                   : kvq::overlap(out, rows_of(q, q_row_stride, q_head_stride, q_heads)))
      return KVQ_ERR_INVALID_ARG;
    if (kvq::repeats(out) || kvq::overlap(out, rows_of(k_new, k_row_stride, k_head_stride, pages->kv_heads)) ||
        kvq::overlap(out, rows_of(v_new, v_row_stride, v_head_stride, pages->kv_heads)))
      return KVQ_ERR_INVALID_ARG;
  }
  p.a.status = kvq::status_ptr();
  p.a.bounds_site = kvq::bounds_site_ptr();
  if (p.a.status == nullptr) return KVQ_ERR_CUDA;
  p.t = rope_of(table);
  p.pos = positions;
  p.pr = pos_row_stride;
  p.q = kvq::RopeTensor{q, q_out, 0, q_row_stride, q_head_stride, 0, q_out_row_stride, q_out_head_stride, q_heads};
  return kvq::launch_pages_append_rope(p, static_cast<cudaStream_t>(stream)) == cudaSuccess ? KVQ_OK : KVQ_ERR_CUDA;
}

size_t kvq_paged_workspace_bytes(const kvq_pages* pages, int32_t q_heads, int32_t batch,
                                 int32_t width, int32_t rows, int32_t max_q) {
  if (check_geometry(pages) != KVQ_OK) return 0;
  if (q_heads < 1 || q_heads % pages->kv_heads != 0 || batch < 0 || width < 0 || rows < 0 || max_q < 0) return 0;
  return kvq::paged_attention_workspace(pages->kv_heads, q_heads, pages->head_dim, batch,
                                        (long long)width * pages->page_tokens, rows, max_q);
}

kvq_status kvq_paged_attention(const kvq_pages* pages, int32_t layer, const uint16_t* q,
                               int64_t q_row_stride, int64_t q_head_stride, int32_t q_heads,
                               const kvq_sequences* seqs, int32_t max_q, float scale,
                               int32_t causal, int32_t window, void* workspace,
                               size_t workspace_bytes, uint16_t* out, float* lse, void* stream) {
  const Range range("kvq_paged_attention");
  kvq::PagedAttnArgs a;
  bool done;
  const kvq_status st = attention_args(pages, layer, q, q_row_stride, q_head_stride, q_heads, seqs, max_q, scale, causal,
                                       window, workspace, workspace_bytes, out, lse, &a, &done);
  if (st != KVQ_OK || done) return st;
  return kvq::launch_paged_attention(a, static_cast<cudaStream_t>(stream));
}

kvq_status kvq_paged_attention_scored(const kvq_pages* pages, int32_t layer, const uint16_t* q,
                                      int64_t q_row_stride, int64_t q_head_stride, int32_t q_heads,
                                      const kvq_sequences* seqs, int32_t max_q, float scale,
                                      int32_t causal, int32_t window, const kvq_scores* scores, void* workspace,
                                      size_t workspace_bytes, uint16_t* out, float* lse, void* stream) {
  const Range range("kvq_paged_attention_scored");
  const bool capped = scores != nullptr && scores->softcap != 0.f;
  if (capped && !(scores->softcap >= 9.5367431640625e-07f && scores->softcap <= 1048576.f)) return KVQ_ERR_INVALID_ARG;
  if (scores != nullptr && (!aligned(scores->slopes, 4) || !aligned(scores->prefix, 4) || !aligned(scores->ranges, 8)))
    return KVQ_ERR_ALIGNMENT;
  kvq::PagedAttnArgs a;
  bool done;
  const kvq_status st = attention_args(pages, layer, q, q_row_stride, q_head_stride, q_heads, seqs, max_q, scale, causal,
                                       window, workspace, workspace_bytes, out, lse, &a, &done);
  if (st != KVQ_OK || done) return st;
  if (!capped && (scores == nullptr || (!scores->slopes && !scores->prefix && !scores->ranges)))
    return kvq::launch_paged_attention(a, static_cast<cudaStream_t>(stream));
  a.shape = kvq::ScoreShape{scores->softcap, scores->slopes, scores->prefix, scores->ranges};
  return kvq::launch_paged_attention_scored(a, static_cast<cudaStream_t>(stream));
}

kvq_status kvq_pages_copy(const kvq_pages* pages, const int32_t* src, const int32_t* dst, int32_t n,
                          void* stream) {
  const Range range("kvq_pages_copy");
  const kvq_status st = check_pool(pages);
  if (st != KVQ_OK) return st;
  if (n < 0) return KVQ_ERR_INVALID_ARG;
  if (n == 0) return KVQ_OK;
  if (src == nullptr || dst == nullptr) return KVQ_ERR_INVALID_ARG;
  // ids in the pool, dst distinct, none of them a src: the call's number is
  // noted beside every dst (scratch of this thread, never cleared)
  try {
    static thread_local std::vector<uint32_t> seen;
    static thread_local uint32_t call = 0;
    if (seen.size() < (size_t)pages->n_pages) seen.resize(pages->n_pages, 0u);
    if (++call == 0) {
      std::fill(seen.begin(), seen.end(), 0u);
      call = 1;
    }
    const uint32_t most = (uint32_t)pages->n_pages;
    for (int32_t i = 0; i < n; ++i) {
      if ((uint32_t)src[i] >= most || (uint32_t)dst[i] >= most || seen[dst[i]] == call)
        return KVQ_ERR_INVALID_ARG;
      seen[dst[i]] = call;
    }
    for (int32_t i = 0; i < n; ++i)
      if (seen[src[i]] == call) return KVQ_ERR_INVALID_ARG;
  } catch (...) {
    return KVQ_ERR_TOO_LARGE;   // no host memory for the check
  }
  return kvq::launch_pages_copy(pool_of(pages), src, dst, n, static_cast<cudaStream_t>(stream)) ==
                 cudaSuccess
             ? KVQ_OK
             : KVQ_ERR_CUDA;
}

size_t kvq_pages_compact_workspace_bytes(const kvq_pages* pages) {
  if (check_geometry(pages) != KVQ_OK || pages->n_pages > kvq::kCompactMaxPages) return 0;
  return 16 + 3 * (size_t)pages->n_pages * 4;
}

kvq_status kvq_pages_compact(const kvq_pages* pages, const int32_t* table, int32_t batch,
                             int32_t width, int64_t table_stride, int32_t* table_out,
                             int64_t table_out_stride, int32_t* n_live, void* workspace,
                             size_t workspace_bytes, void* stream) {
  const Range range("kvq_pages_compact");
  const kvq_status st = check_pool(pages);
  if (st != KVQ_OK) return st;
  if (pages->n_pages > kvq::kCompactMaxPages) return KVQ_ERR_TOO_LARGE;
  if (batch < 0 || width < 0 || n_live == nullptr || workspace == nullptr) return KVQ_ERR_INVALID_ARG;
  if (batch > 0 && width > 0 && (table == nullptr || table_out == nullptr)) return KVQ_ERR_INVALID_ARG;
  if (batch > 1 && (table_stride < width || table_out_stride < width)) return KVQ_ERR_INVALID_ARG;
  if (table == table_out && batch > 1 && table_stride != table_out_stride) return KVQ_ERR_INVALID_ARG;
  if (!aligned(table, 4) || !aligned(table_out, 4) || !aligned(n_live, 4) || !aligned(workspace, 16))
    return KVQ_ERR_ALIGNMENT;
  if (workspace_bytes < kvq_pages_compact_workspace_bytes(pages)) return KVQ_ERR_INVALID_ARG;
  kvq::CompactArgs a{};
  a.pool = pool_of(pages);
  a.table = table;
  a.table_out = table_out;
  a.stride = table_stride;
  a.out_stride = table_out_stride;
  a.batch = batch;
  a.width = width;
  a.n_live = n_live;
  a.ws = static_cast<int32_t*>(workspace);
  a.status = kvq::status_ptr();
  if (a.status == nullptr) return KVQ_ERR_CUDA;
  return kvq::launch_pages_compact(a, static_cast<cudaStream_t>(stream)) == cudaSuccess ? KVQ_OK
                                                                                       : KVQ_ERR_CUDA;
}

}  // extern "C"
