// extern "C" entry points of the paged 8-bit cache: argument checks on the
// host, before anything is launched, and dispatch.
#include <cuda_runtime.h>
#include <nvtx3/nvToolsExt.h>

#include <algorithm>
#include <cmath>
#include <vector>

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
  kvq_status st = check_pool(pages);
  if (st != KVQ_OK) return st;
  if (layer < 0 || layer >= pages->layers) return KVQ_ERR_INVALID_ARG;
  st = check_sequences(seqs, pages->page_tokens);
  if (st != KVQ_OK) return st;
  if (seqs->rows == 0) return KVQ_OK;
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
  a.status = kvq::status_ptr();
  a.bounds_site = kvq::bounds_site_ptr();
  if (a.status == nullptr) return KVQ_ERR_CUDA;
  return kvq::launch_pages_append(a, static_cast<cudaStream_t>(stream)) == cudaSuccess ? KVQ_OK
                                                                                      : KVQ_ERR_CUDA;
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
  kvq_status st = check_pool(pages);
  if (st != KVQ_OK) return st;
  if (layer < 0 || layer >= pages->layers) return KVQ_ERR_INVALID_ARG;
  if (q_heads < 1 || q_heads % pages->kv_heads != 0) return KVQ_ERR_INVALID_ARG;
  st = check_sequences(seqs, pages->page_tokens);
  if (st != KVQ_OK) return st;
  if (!std::isfinite(scale) || scale <= 0.f || window < 0 || max_q < 0) return KVQ_ERR_INVALID_ARG;
  if (seqs->rows == 0) return KVQ_OK;
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
  return kvq::launch_paged_attention(a, static_cast<cudaStream_t>(stream));
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
