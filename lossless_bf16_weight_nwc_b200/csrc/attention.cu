// attention.cu — attention of a batch's new tokens over a paged cache, with
// prefixes that several sequences share.
//
// out = sum_j e^(s_j - m) v_j / sum_j e^(s_j - m), s_j = scale q . k_j, over the
// row's prefix and its own tokens, in one pass with the running maximum m.
#include <cuda_bf16.h>
#include <cuda_runtime.h>

#include <cmath>
#include <cstdint>

#include "paged.cuh"
#include "ptx.cuh"

namespace nwc {

namespace {

constexpr unsigned kAll = 0xFFFFFFFFu;
constexpr int kWarps = 4;

// One CTA a row and head; its warps take the tokens in turn.
template <int DIM>
__global__ void __launch_bounds__(kWarps * 32) attention_kernel(
    const __grid_constant__ AttentionParams p) {
  constexpr int E = DIM / 32;
  __shared__ float part[kWarps][DIM + 2];
  allow_dependents();
  wait_prerequisites();
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  const int row = blockIdx.x / p.heads, head = blockIdx.x % p.heads;
  const int kvh = head / (p.heads / p.kv_heads);
  const BatchView& b = p.batch;
  const int seq = row / b.chunk, i = row - seq * b.chunk;
  const int fresh = b.q_lens ? min(max(b.q_lens[seq], 0), b.chunk) : b.chunk;
  const bool real = i < fresh;
  const int64_t own_cap = (int64_t)b.table_width << p.cache.page_shift;
  int own = real ? max(max(b.lens[seq], 0) - fresh + i + 1, 0) : 0;
  if (own > own_cap) {
    own = (int)own_cap;
    atomicOr(p.cache.err, kErrRange);
  }
  int prefix = 0, group = -1;
  for (int g = 0; real && g < b.groups; ++g)
    if (b.group_start[g] <= seq && seq < b.group_start[g + 1]) group = g;
  if (group >= 0) {
    const int64_t cap = (int64_t)b.prefix_width << p.cache.page_shift;
    prefix = max(b.prefix_lens[group], 0);
    if (prefix > cap) {
      prefix = (int)cap;
      atomicOr(p.cache.err, kErrRange);
    }
  }
  const __nv_bfloat16* q = static_cast<const __nv_bfloat16*>(p.q.data) +
                           (int64_t)row * p.q.token_stride + (int64_t)head * p.q.head_stride;
  float qv[E], acc[E];
#pragma unroll
  for (int e = 0; e < E; ++e) qv[e] = __bfloat162float(q[lane * E + e]) * p.scale, acc[e] = 0.f;
  float m = -INFINITY, l = 0.f;
  for (int64_t j = warp; j < (int64_t)prefix + own; j += kWarps) {
    const bool far = j < prefix;
    const int t = (int)(far ? j : j - prefix);
    const int n = t >> p.cache.page_shift, slot = t & ((1 << p.cache.page_shift) - 1);
    const int64_t page = far ? b.prefix_table[(int64_t)group * b.prefix_stride + n]
                             : b.table[(int64_t)seq * b.table_stride + n];
    const bool there = page >= 0 && page < p.cache.pages;
    if (!there && lane == 0) atomicOr(p.cache.err, kErrRange);
    const __nv_bfloat16* k = reinterpret_cast<const __nv_bfloat16*>(p.cache.k) +
                             page * p.cache.k_page + slot * p.cache.k_token + kvh * p.cache.k_head;
    const __nv_bfloat16* v = reinterpret_cast<const __nv_bfloat16*>(p.cache.v) +
                             page * p.cache.v_page + slot * p.cache.v_token + kvh * p.cache.v_head;
    float s = 0.f;
#pragma unroll
    for (int e = 0; e < E; ++e)
      s += there ? qv[e] * __bfloat162float(k[lane * E + e]) : 0.f;
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) s += __shfl_xor_sync(kAll, s, o);
    const float top = fmaxf(m, s);
    const float old = top == -INFINITY ? 0.f : expf(m - top);
    const float w = top == -INFINITY ? 0.f : expf(s - top);
    l = l * old + w;
#pragma unroll
    for (int e = 0; e < E; ++e)
      acc[e] = acc[e] * old + (there ? w * __bfloat162float(v[lane * E + e]) : 0.f);
    m = top;
  }
#pragma unroll
  for (int e = 0; e < E; ++e) part[warp][lane * E + e] = acc[e];
  if (lane == 0) part[warp][DIM] = m, part[warp][DIM + 1] = l;
  __syncthreads();
  float top = -INFINITY, sum = 0.f;
  for (int w = 0; w < kWarps; ++w) top = fmaxf(top, part[w][DIM]);
  for (int w = 0; w < kWarps; ++w)
    sum += part[w][DIM + 1] > 0.f ? part[w][DIM + 1] * expf(part[w][DIM] - top) : 0.f;
  __nv_bfloat16* out = static_cast<__nv_bfloat16*>(p.out.data) +
                       (int64_t)row * p.out.token_stride + (int64_t)head * p.out.head_stride;
  for (int e = threadIdx.x; e < DIM; e += kWarps * 32) {
    float a = 0.f;
    for (int w = 0; w < kWarps; ++w)
      a += part[w][DIM + 1] > 0.f ? part[w][e] * expf(part[w][DIM] - top) : 0.f;
    out[e] = __float2bfloat16_rn(sum > 0.f ? a / sum : 0.f);
  }
  if (p.lse && threadIdx.x == 0)
    p.lse[(int64_t)row * p.heads + head] = sum > 0.f ? top + logf(sum) : -INFINITY;
}

}  // namespace

uint64_t attention_workspace(int, int, int, int, int, int, int) { return 256; }

cudaError_t launch_attention(const AttentionParams& p, int, cudaStream_t stream) {
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3((unsigned)(p.batch.sequences * p.batch.chunk * p.heads));
  cfg.blockDim = dim3(kWarps * 32);
  cfg.stream = stream;
  cudaLaunchAttribute attr[1];
  attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[0].val.programmaticStreamSerializationAllowed = 1;
  cfg.attrs = attr;
  cfg.numAttrs = 1;
  return p.dim == 64 ? cudaLaunchKernelEx(&cfg, attention_kernel<64>, p)
                     : cudaLaunchKernelEx(&cfg, attention_kernel<128>, p);
}

}  // namespace nwc
