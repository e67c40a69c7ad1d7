// paged.cuh — parameters and launch interface of the kernels around the paged
// key/value cache (host side).
#pragma once
#include <cuda.h>
#include <cuda_runtime.h>
#include <cstdint>

#include "kernels.cuh"

namespace nwc {

// A tensor [tokens, heads, dim] read or written by the kernels: the last
// dimension contiguous, the others at any stride (in elements).
struct HeadsView {
  void* data;
  int64_t token_stride, head_stride;
};

// The cache: K and V pages of page_size tokens x kv_heads x dim BF16.
struct CacheView {
  uint16_t* k;
  uint16_t* v;
  int64_t k_page, k_token, k_head;  // strides in elements
  int64_t v_page, v_token, v_head;
  int64_t pages;
  int32_t page_shift;               // log2(page_size)
  uint32_t* err;                    // device: the cache's error word
};

// The batch's tables (all int32 on the device).
struct BatchView {
  int32_t sequences, chunk;         // rows of the batch: sequences x chunk
  const int32_t* table;             // own pages, [sequences] rows of table_width
  int64_t table_stride;
  int32_t table_width;
  const int32_t* lens;              // own tokens, the new ones among them
  const int32_t* q_lens;            // new tokens of each sequence; null: chunk
  int32_t groups;                   // shared prefixes; 0: none
  const int32_t* group_start;       // [groups + 1]
  const int32_t* prefix_table;
  int64_t prefix_stride;
  int32_t prefix_width;
  const int32_t* prefix_lens;       // [groups]
};

enum : int32_t { kTypeBf16 = 0, kTypeF32 = 1 };

// Norms and rotation of heads, and where they go: to output tensors
// (append == false, positions given) or q to its tensor and k, v to the cache.
struct RopeParams {
  HeadsView q, k, v;          // inputs; q.data or k.data may be null
  HeadsView q_out, k_out;     // outputs of the same shapes
  int32_t tokens, heads, kv_heads, dim;
  int32_t rotary;             // leading elements of a head that rotate; 0: none
  int32_t interleaved;        // pairs (2i, 2i + 1), else (i, i + rotary / 2)
  const double* freq;         // [rotary / 2] radians a position
  const void* q_weight;       // [dim] or null: no norm
  const void* k_weight;
  int32_t weight_f32;
  float eps;
  const void* positions;      // [tokens] int32 or int64 (append == false)
  int32_t positions_64;
  int32_t append;
  CacheView cache;
  BatchView batch;
};
cudaError_t launch_rope(const RopeParams& p, int in_type, int out_type, int sm_count,
                        cudaStream_t stream);

// Attention.  The work is cut into tiles of kKvTile tokens.  A segment is a
// prefix with the rows of all its sequences, or a sequence's own tokens with its
// rows; an item is a segment's rows of one key head, up to kPairRows of them;
// the items' tiles lie end to end on one axis (segments, blocks of rows, key
// heads, tiles), which the CTAs share out equally.  What a CTA does of an item is
// a part; each of its two softmax teams leaves the part's running maximum, sum
// and weighted values in the workspace, and a second kernel joins them.
constexpr int kKvShift = 7;
constexpr int kKvTile = 1 << kKvShift;
constexpr int kTeamRows = 128;
constexpr int kPairRows = 2 * kTeamRows;
constexpr int kFewRows = 16;  // rows of a segment that are multiplied without TMEM
// Heads that a tile of such a segment holds (16 tokens of one head a warp), so it
// has 128 / that tokens: the largest power of two up to 8 that divides the heads.
inline int few_heads_of(int kv_heads) {
  int n = 8;
  while (kv_heads % n) n /= 2;
  return n;
}

// The workspace: which CTAs have an item's parts, then the parts' results,
// prefixes' and own.
struct AttentionWorkspace {
  uint64_t far_spans, own_spans;  // int32 [items][2]: first and last CTA
  uint64_t items;         // int32 [groups + 1]: first item of a prefix
  uint64_t far_ml, far_o; // prefixes: float2 [slots][256], float [slots][256][dim]
  uint64_t own_ml, own_o; // own: the same with own_rows rows
  int64_t far_slots, own_slots;
  int32_t own_rows;       // rows a slot of an own part holds: both teams', or all heads'
  int32_t seq_rows;       // rows of a sequence for a key head, where they are few
  int32_t own_items;      // items of a sequence's own segment
  uint64_t bytes;
};
AttentionWorkspace attention_workspace(int sequences, int chunk, int groups, int heads,
                                       int kv_heads, int dim, int ctas);

struct AttentionParams {
  HeadsView q, out;           // BF16 [rows][heads][dim]
  int32_t heads, kv_heads, dim;
  float scale;
  float* lse;                 // [rows][heads] or null
  CacheView cache;
  BatchView batch;
  uint8_t* workspace;
  AttentionWorkspace ws;
  int32_t ctas;
  int32_t gq, seq_rows;       // heads / kv_heads; rows of a sequence for a key head
  int32_t few_heads, few_tokens;  // of a tile of a segment of few rows
  int32_t few_shift, few_items;   // log2 of its tokens; kv_heads / few_heads
  uint32_t wait_limit;        // polls before a bounded wait gives up (0: default)
};
// The pages of K and V as [pages][kv_heads][page_size][dim], 128-byte swizzle: with
// a box of 64 elements x min(page_size, 128) tokens, then with one of 64 x
// min(page_size, few_tokens) x few_heads.
struct PageMaps {
  CUtensorMap map[4];
};
cudaError_t launch_attention(const AttentionParams& p, const PageMaps& maps, cudaStream_t stream);

}  // namespace nwc
