// paged_api.cu — the C ABI of the calls around the projections (include/nwc.h):
// argument checks on the host, then one launch path each.
#include <cuda_runtime.h>

#include <cmath>
#include <cstring>

#include "../../include/nwc.h"
#include "nwc_device.h"
#include "paged.cuh"

namespace {

constexpr int32_t kMaxTokens = 1 << 24;
constexpr int32_t kMaxHeads = 1 << 12;
constexpr int64_t kMaxRows = 1 << 30;  // of attention: tokens x query heads of a key head
constexpr int32_t kMaxDim = 256;
constexpr int32_t kMaxPageSize = 1 << 20;
constexpr int64_t kMaxStride = 1ll << 39;  // elements: products with 2^24 stay in 64 bits

bool aligned_to(const void* p, uintptr_t a) { return (reinterpret_cast<uintptr_t>(p) % a) == 0; }

// A heads tensor of the given type (any of the two when type < 0).
bool good_heads(const nwc_heads* h, int type) {
  if (!h || h->struct_size != sizeof(nwc_heads) || !h->d_data) return false;
  if (h->type > NWC_TYPE_F32 || (type >= 0 && (int)h->type != type)) return false;
  return aligned_to(h->d_data, h->type == NWC_TYPE_F32 ? 4 : 2) && h->token_stride >= 0 &&
         h->head_stride >= 0 && h->token_stride <= kMaxStride && h->head_stride <= kMaxStride;
}
// BF16 rows that are moved 16 bytes at a time.
bool wide_heads(const nwc_heads* h) {
  return good_heads(h, NWC_TYPE_BF16) && aligned_to(h->d_data, 16) && h->token_stride % 8 == 0 &&
         h->head_stride % 8 == 0;
}
nwc::HeadsView view(const nwc_heads* h) {
  return h ? nwc::HeadsView{h->d_data, h->token_stride, h->head_stride}
           : nwc::HeadsView{nullptr, 0, 0};
}

bool good_dims(int32_t heads, int32_t kv_heads, int32_t dim) {
  return heads >= 1 && heads <= kMaxHeads && kv_heads >= 1 && kv_heads <= kMaxHeads && dim >= 8 &&
         dim <= kMaxDim && dim % 8 == 0;
}

bool good_rope(const nwc_rope* r, int32_t dim) {
  if (!r || r->struct_size != sizeof(nwc_rope)) return false;
  if (r->rotary_dim < 0 || r->rotary_dim > dim || r->rotary_dim % 8) return false;
  if (r->rotary_dim && (!r->d_freq || !aligned_to(r->d_freq, 8))) return false;
  if (r->weight_type > NWC_TYPE_F32) return false;
  const uintptr_t unit = r->weight_type == NWC_TYPE_F32 ? 4 : 2;
  if (!aligned_to(r->d_q_weight, unit) || !aligned_to(r->d_k_weight, unit)) return false;
  return r->eps >= 0.f && std::isfinite(r->eps);
}

bool good_stride(int64_t s) { return s >= 0 && s <= kMaxStride && s % 8 == 0; }

bool good_cache(const nwc_kv_cache* c) {
  if (!c || c->struct_size != sizeof(nwc_kv_cache) || !c->d_k || !c->d_v || !c->d_error)
    return false;
  if (!aligned_to(c->d_k, 16) || !aligned_to(c->d_v, 16) || !aligned_to(c->d_error, 4))
    return false;
  if (c->page_size < 8 || c->page_size > kMaxPageSize || (c->page_size & (c->page_size - 1)))
    return false;
  if (!good_dims(1, c->kv_heads, c->dim) || c->pages < 1 || c->pages > 0x7FFFFFFF) return false;
  return good_stride(c->k_page_stride) && good_stride(c->k_token_stride) &&
         good_stride(c->k_head_stride) && good_stride(c->v_page_stride) &&
         good_stride(c->v_token_stride) && good_stride(c->v_head_stride);
}

bool good_batch(const nwc_kv_batch* b) {
  if (!b || b->struct_size != sizeof(nwc_kv_batch)) return false;
  if (b->sequences < 0 || b->new_tokens < 1 ||
      (int64_t)b->sequences * b->new_tokens > kMaxTokens)
    return false;
  if (b->groups < 0 || b->groups > b->sequences) return false;
  if (b->sequences == 0) return true;
  if (b->table_width < 0 || (b->table_width && !b->d_block_table) || !b->d_seq_lens ||
      b->table_stride < 0 || b->table_stride > kMaxStride)
    return false;
  if (!aligned_to(b->d_block_table, 4) || !aligned_to(b->d_seq_lens, 4) ||
      !aligned_to(b->d_q_lens, 4))
    return false;
  if (b->groups == 0) return true;
  return b->d_group_start && b->d_prefix_lens && b->prefix_width >= 0 &&
         (b->d_prefix_table || !b->prefix_width) && b->prefix_stride >= 0 && b->prefix_stride <= kMaxStride &&
         aligned_to(b->d_group_start, 4) && aligned_to(b->d_prefix_table, 4) &&
         aligned_to(b->d_prefix_lens, 4);
}

nwc::CacheView view(const nwc_kv_cache& c) {
  nwc::CacheView v;
  v.k = c.d_k, v.v = c.d_v;
  v.k_page = c.k_page_stride, v.k_token = c.k_token_stride, v.k_head = c.k_head_stride;
  v.v_page = c.v_page_stride, v.v_token = c.v_token_stride, v.v_head = c.v_head_stride;
  v.pages = c.pages;
  v.page_shift = 0;
  while ((1 << v.page_shift) < c.page_size) ++v.page_shift;
  v.err = c.d_error;
  return v;
}

nwc::BatchView view(const nwc_kv_batch& b) {
  return nwc::BatchView{b.sequences,    b.new_tokens,  b.d_block_table, b.table_stride,
                        b.table_width,  b.d_seq_lens,  b.d_q_lens,      b.groups,
                        b.d_group_start, b.d_prefix_table, b.prefix_stride, b.prefix_width,
                        b.d_prefix_lens};
}

void set_rope(nwc::RopeParams* p, const nwc_rope& r) {
  p->rotary = r.rotary_dim;
  p->interleaved = r.interleaved != 0;
  p->freq = r.d_freq;
  p->q_weight = r.d_q_weight;
  p->k_weight = r.d_k_weight;
  p->weight_f32 = r.weight_type == NWC_TYPE_F32;
  p->eps = r.eps;
}

nwc_status run_rope(const nwc::RopeParams& p, int in_type, int out_type, nwc_stream_t stream) {
  int dev, sms;
  size_t smem;
  const nwc_status st = nwc::current_device(&dev, &sms, &smem);
  if (st != NWC_OK) return st;
  return nwc::launch_rope(p, in_type, out_type, sms, reinterpret_cast<cudaStream_t>(stream)) ==
                 cudaSuccess
             ? NWC_OK
             : NWC_ERR_CUDA;
}

// The TMA descriptor of a cache's K or V pages.  Strides of dimensions of one
// element play no part but have to be valid.
bool page_map(const nwc_kv_cache& c, uint16_t* base, int64_t page_stride, int64_t token_stride,
              int64_t head_stride, int tokens, int heads, CUtensorMap* map) {
  PFN_cuTensorMapEncodeTiled_v12000 encode = nwc::tensor_map_encoder();
  if (!encode) return false;
  const int32_t rows = c.page_size < tokens ? c.page_size : tokens;
  const cuuint64_t dims[4] = {(cuuint64_t)c.dim, (cuuint64_t)c.page_size, (cuuint64_t)c.kv_heads,
                              (cuuint64_t)c.pages};
  const cuuint64_t strides[3] = {(cuuint64_t)token_stride * 2, (cuuint64_t)head_stride * 2,
                                 (cuuint64_t)page_stride * 2};
  const cuuint32_t box[4] = {64, (cuuint32_t)rows, (cuuint32_t)heads, 1};
  const cuuint32_t elem[4] = {1, 1, 1, 1};
  return encode(map, CU_TENSOR_MAP_DATA_TYPE_BFLOAT16, 4, base, dims, strides, box, elem,
                CU_TENSOR_MAP_INTERLEAVE_NONE, CU_TENSOR_MAP_SWIZZLE_128B,
                CU_TENSOR_MAP_L2_PROMOTION_L2_256B,
                CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) == CUDA_SUCCESS;
}

bool attention_shape(const nwc_kv_cache* c, const nwc_kv_batch* b, int32_t heads) {
  return good_cache(c) && good_batch(b) && heads >= 1 && heads <= kMaxHeads &&
         heads % c->kv_heads == 0 &&
         (int64_t)b->sequences * b->new_tokens * (heads / c->kv_heads) <= kMaxRows;
}

}  // namespace

extern "C" {

nwc_status nwc_qk_norm_rope(const nwc_heads* q, const nwc_heads* k, const nwc_heads* q_out,
                            const nwc_heads* k_out, int32_t tokens, int32_t heads,
                            int32_t kv_heads, int32_t dim, const void* d_positions,
                            int32_t positions_64, const nwc_rope* rope, nwc_stream_t stream) {
  if ((!q && !k) || !q != !q_out || !k != !k_out) return NWC_ERR_INVALID_ARG;
  const int in = (int)(q ? q : k)->type, out = (int)(q ? q_out : k_out)->type;
  if (q && !(good_heads(q, in) && good_heads(q_out, out))) return NWC_ERR_INVALID_ARG;
  if (k && !(good_heads(k, in) && good_heads(k_out, out))) return NWC_ERR_INVALID_ARG;
  if (tokens < 0 || tokens > kMaxTokens || !good_dims(q ? heads : 1, k ? kv_heads : 1, dim) ||
      !good_rope(rope, dim) || !d_positions || !aligned_to(d_positions, positions_64 ? 8 : 4))
    return NWC_ERR_INVALID_ARG;
  if (tokens == 0) return NWC_OK;
  nwc::RopeParams p;
  std::memset(&p, 0, sizeof(p));
  p.q = view(q), p.k = view(k), p.q_out = view(q_out), p.k_out = view(k_out);
  p.tokens = tokens, p.heads = heads, p.kv_heads = kv_heads, p.dim = dim;
  set_rope(&p, *rope);
  p.positions = d_positions;
  p.positions_64 = positions_64 != 0;
  return run_rope(p, in, out, stream);
}

nwc_status nwc_kv_append(const nwc_kv_cache* cache, const nwc_kv_batch* batch,
                         const nwc_heads* q, const nwc_heads* q_out, int32_t heads,
                         const nwc_heads* k, const nwc_heads* v, const nwc_rope* rope,
                         nwc_stream_t stream) {
  if (!good_cache(cache) || !good_batch(batch) || !k || !v || !q != !q_out)
    return NWC_ERR_INVALID_ARG;
  const int in = (int)k->type;
  if (!good_heads(k, in) || !good_heads(v, in)) return NWC_ERR_INVALID_ARG;
  if (q && !(good_heads(q, in) && good_heads(q_out, NWC_TYPE_BF16))) return NWC_ERR_INVALID_ARG;
  if (!good_dims(q ? heads : 1, cache->kv_heads, cache->dim) || !good_rope(rope, cache->dim))
    return NWC_ERR_INVALID_ARG;
  if (batch->sequences == 0) return NWC_OK;
  nwc::RopeParams p;
  std::memset(&p, 0, sizeof(p));
  p.q = view(q), p.k = view(k), p.v = view(v), p.q_out = view(q_out);
  p.tokens = batch->sequences * batch->new_tokens;
  p.heads = heads, p.kv_heads = cache->kv_heads, p.dim = cache->dim;
  set_rope(&p, *rope);
  p.append = 1;
  p.cache = view(*cache);
  p.batch = view(*batch);
  return run_rope(p, in, NWC_TYPE_BF16, stream);
}

nwc_status nwc_kv_attention_workspace(const nwc_kv_cache* cache, const nwc_kv_batch* batch,
                                      int32_t heads, uint64_t* bytes) {
  if (!bytes || !attention_shape(cache, batch, heads)) return NWC_ERR_INVALID_ARG;
  if (cache->dim != 64 && cache->dim != 128) return NWC_ERR_UNSUPPORTED;
  int dev, sms;
  size_t smem;
  const nwc_status st = nwc::current_device(&dev, &sms, &smem);
  if (st != NWC_OK) return st;
  *bytes = nwc::attention_workspace(batch->sequences, batch->new_tokens, batch->groups, heads,
                                    cache->kv_heads, cache->dim, sms)
               .bytes;
  return NWC_OK;
}

nwc_status nwc_kv_attention(const nwc_kv_cache* cache, const nwc_kv_batch* batch,
                            const nwc_heads* q, int32_t heads, float scale,
                            const nwc_heads* out, float* d_lse, void* d_workspace,
                            uint64_t workspace_bytes, nwc_stream_t stream) {
  if (!attention_shape(cache, batch, heads) || !wide_heads(q) || !wide_heads(out) ||
      !std::isfinite(scale * 1.4426950408889634f) || !aligned_to(d_lse, 4))
    return NWC_ERR_INVALID_ARG;   // (the kernels' scores are in units of log2)
  if (cache->dim != 64 && cache->dim != 128) return NWC_ERR_UNSUPPORTED;
  if (batch->sequences == 0) return NWC_OK;
  int dev, sms;
  size_t smem;
  const nwc_status st = nwc::current_device(&dev, &sms, &smem);
  if (st != NWC_OK) return st;
  nwc::AttentionParams p;
  std::memset(&p, 0, sizeof(p));
  p.ctas = sms;
  p.ws = nwc::attention_workspace(batch->sequences, batch->new_tokens, batch->groups, heads,
                                  cache->kv_heads, cache->dim, sms);
  if (!d_workspace || workspace_bytes < p.ws.bytes || !aligned_to(d_workspace, 256))
    return NWC_ERR_INVALID_ARG;
  p.q = view(q), p.out = view(out);
  p.heads = heads, p.kv_heads = cache->kv_heads, p.dim = cache->dim;
  p.scale = scale;
  p.lse = d_lse;
  p.cache = view(*cache);
  p.batch = view(*batch);
  p.workspace = static_cast<uint8_t*>(d_workspace);
  p.wait_limit = nwc::wait_limit();
  p.few_heads = nwc::few_heads_of(cache->kv_heads);
  p.few_tokens = nwc::kKvTile / p.few_heads;
  for (p.few_shift = 0; (1 << p.few_shift) < p.few_tokens;) ++p.few_shift;
  p.few_items = cache->kv_heads / p.few_heads;
  p.gq = heads / cache->kv_heads;
  p.seq_rows = batch->new_tokens * p.gq;
  nwc::PageMaps maps;
  for (int i = 0; i < 4; ++i) {
    const int tokens = i < 2 ? nwc::kKvTile : p.few_tokens, per = i < 2 ? 1 : p.few_heads;
    const bool ok =
        i % 2 == 0 ? page_map(*cache, cache->d_k, cache->k_page_stride, cache->k_token_stride,
                              cache->k_head_stride, tokens, per, &maps.map[i])
                   : page_map(*cache, cache->d_v, cache->v_page_stride, cache->v_token_stride,
                              cache->v_head_stride, tokens, per, &maps.map[i]);
    if (!ok) return NWC_ERR_UNSUPPORTED;
  }
  return nwc::launch_attention(p, maps, reinterpret_cast<cudaStream_t>(stream)) == cudaSuccess
             ? NWC_OK
             : NWC_ERR_CUDA;
}

nwc_status nwc_kv_get_error(const nwc_kv_cache* cache, nwc_stream_t stream, uint32_t* word) {
  if (!cache || cache->struct_size != sizeof(nwc_kv_cache) || !cache->d_error)
    return NWC_ERR_INVALID_ARG;
  cudaStream_t cs = reinterpret_cast<cudaStream_t>(stream);
  uint32_t w = 0;
  cudaError_t e = cudaMemcpyAsync(&w, cache->d_error, sizeof(w), cudaMemcpyDeviceToHost, cs);
  if (e == cudaSuccess) e = cudaStreamSynchronize(cs);
  if (e == cudaSuccess && w) {
    e = cudaMemsetAsync(cache->d_error, 0, sizeof(w), cs);
    if (e == cudaSuccess) e = cudaStreamSynchronize(cs);
  }
  if (e != cudaSuccess) return NWC_ERR_CUDA;
  if (word) *word = w;
  if (w & nwc::kErrTimeout) return NWC_ERR_DEVICE_TIMEOUT;
  if (w & nwc::kErrRange) return NWC_ERR_INVALID_ARG;
  if (w & nwc::kErrLayout) return NWC_ERR_UNSUPPORTED;
  return NWC_OK;
}

}  // extern "C"
