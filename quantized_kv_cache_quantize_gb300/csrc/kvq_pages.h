// Host-side declarations of the paged 8-bit cache's kernels.
#pragma once

#include "kvq_internal.h"

namespace kvq {

constexpr int kPageExpMin = -60, kPageExpMax = 60;   // scale exponents
constexpr int kRopeMaxPairs = 64, kRopeMaxAxes = 4;
constexpr int kRopeHeads = 8;                        // of one block of a rotation
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

// A table of rotations: (cos, sin) of pair p at a position, and the pair's axis.
struct RopeTab {
  const float2* cs;   // [n][pairs]
  int n, pairs, axes, interleaved;
  float none;         // -0
  uint32_t axis[4];   // of each pair, two bits
};

// One tensor that is rotated, [batch][row][head][d] at strides in elements.
struct RopeTensor {
  const uint16_t* x;
  uint16_t* y;
  long long xb, xr, xh, yb, yr, yh;
  int heads;
};

// Blocks of a rotation of rows x heads, `tile` rows and kRopeHeads heads each.  (In
// 64 bits: a call may have 2^31 - 1 rows, or heads.)
inline long long rope_blocks(long long rows, long long heads, int tile) {
  return (rows + tile - 1) / tile * ((heads + kRopeHeads - 1) / kRopeHeads);
}

struct RopeArgs {
  RopeTab t;
  const int32_t* pos;
  long long pb, pr, pa;   // strides of batch entries, rows, axes
  RopeTensor x[2];
  int batch, rows, d, inverse;
  int* status;
  int* bounds_site;
};

// Pages that an append with offsets looks at (see append_item), and the rows of a
// block of queries beside it (a page of 16 tokens has too few threads for 16).
inline long long append_items(long long rows, long long batch, int shift) { return (rows >> shift) + 2 * batch; }
inline int append_query_rows(bool one_token, int page) { return one_token || page == 16 ? 4 : 16; }
// Blocks of an append that rotates, at most: keys and values a page and head, queries.
inline long long append_rope_blocks(const PageSeqs& s, const PageLayer& p, long long q_heads) {
  return append_items(s.rows, s.batch, p.shift) * p.heads * 2 +
         rope_blocks(s.rows, q_heads, append_query_rows(s.offsets == nullptr, p.page));
}

struct AppendRopeArgs {
  AppendArgs a;
  RopeTab t;
  const int32_t* pos;     // null: a token's place in its sequence
  long long pr;
  RopeTensor q;           // heads = 0: none
};

// Shapes of scores and masks beyond causal and window (kvq_scores).
struct ScoreShape {
  float cap;              // 0: none
  const float* slopes;    // null: none
  const int32_t* prefix;
  const int32_t* ranges;
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
  ScoreShape shape;      // of the scored call
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
cudaError_t launch_rope_fill(float* cos_sin, int n, int pairs, const double* frequency, double factor,
                             cudaStream_t stream);
cudaError_t launch_rope(const RopeArgs& a, cudaStream_t stream);
cudaError_t launch_pages_append_rope(const AppendRopeArgs& a, cudaStream_t stream);
kvq_status launch_paged_attention(const PagedAttnArgs& a, cudaStream_t stream);
kvq_status launch_paged_attention_scored(const PagedAttnArgs& a, cudaStream_t stream);
kvq_status launch_paged_biased(const PagedAttnArgs& a, cudaStream_t stream);
kvq_status launch_paged_capped(const PagedAttnArgs& a, cudaStream_t stream);
// CTAs per item of the decoding form, 0 for the line of all keys
int decode_by_item(int sms, int d, long long items, long long keys);
// bytes, 16 where none are needed
size_t paged_attention_workspace(int kv_heads, int q_heads, int d, int batch, long long keys, int rows, int max_q);
cudaError_t launch_pages_copy(const PagePool& p, const int32_t* src, const int32_t* dst, int n,
                              cudaStream_t stream);
cudaError_t launch_pages_compact(const CompactArgs& a, cudaStream_t stream);

int sm_count_current();   // SMs of the current device, 0 on an error

}  // namespace kvq
