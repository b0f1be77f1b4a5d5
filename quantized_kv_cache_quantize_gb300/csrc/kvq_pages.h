// Host-side declarations of the paged 8-bit cache's kernels.
#pragma once

#include "kvq_internal.h"

namespace kvq {

constexpr int kPageExpMin = -60, kPageExpMax = 60;   // scale exponents
constexpr int kCompactMaxPages = 1 << 20;            // the plan's bitmap fits shared memory

// One layer of a pool.
struct PageLayer {
  uint8_t* codes[2];     // K, V: [n_pages][kv_heads][page][d]
  uint16_t* scale[2];    // [n_pages][kv_heads]
  int n_pages, heads, d;
  int page, shift;       // tokens per page = 1 << shift
};

// The sequences of a call (device arrays).
struct PageSeqs {
  const int32_t* table;
  const int32_t* lens;
  const int32_t* offsets;   // null: one row per sequence
  long long stride;
  int batch, width, rows;
};

struct AppendArgs {
  PageLayer p;
  PageSeqs s;
  const uint16_t* x[2];                        // K, V rows
  long long row_stride[2], head_stride[2];     // elements
  int* status;
  int* bounds_site;
};

struct PagedAttnArgs {
  PageLayer p;
  PageSeqs s;
  const uint16_t* q;
  long long q_row_stride, q_head_stride;
  int q_heads, group;    // group = q_heads / kv_heads
  int max_q, causal, window;
  float scale;
  uint16_t* out;
  float* lse;
  void* ws;
  size_t ws_bytes;
  int* status;
  int* bounds_site;
  unsigned long long wait_limit_ns;
};

// Pages of all layers, for copies.
struct PagePool {
  uint8_t* codes[2];
  uint16_t* scale[2];
  int layers, n_pages, heads;
  long long page_bytes;   // codes of one page and layer: heads * page * d
};

struct CompactArgs {
  PagePool pool;
  const int32_t* table;
  int32_t* table_out;
  long long stride, out_stride;
  int batch, width;
  int32_t* n_live;
  int32_t* ws;       // [1] number of moves, padded to 4; src, dst, to: n_pages each
  int* status;
};

cudaError_t launch_pages_append(const AppendArgs& a, cudaStream_t stream);
kvq_status launch_paged_attention(const PagedAttnArgs& a, cudaStream_t stream);
// bytes, 16 where none are needed
size_t paged_attention_workspace(int kv_heads, int q_heads, int d, int batch, long long keys, int rows, int max_q);
cudaError_t launch_pages_copy(const PagePool& p, const int32_t* src, const int32_t* dst, int n,
                              cudaStream_t stream);
cudaError_t launch_pages_compact(const CompactArgs& a, cudaStream_t stream);

int sm_count_current();   // SMs of the current device, 0 on an error

}  // namespace kvq
