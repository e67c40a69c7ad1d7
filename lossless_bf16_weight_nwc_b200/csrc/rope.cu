// rope.cu — per-head RMS norm and position rotation of q and k in one pass, to
// tensors or (k and v) straight into a paged cache.
//
// y = x / sqrt(mean(x^2) + eps) * w over a head, then every pair (a, b) of the
// leading `rotary` elements becomes (a cos t - b sin t, b cos t + a sin t) with
// t = position * freq_i.  Sums and products are FP32 and there is one rounding,
// on the store.  The angle is reduced to turns in 64 bits: at position 10^6 an
// FP32 product would already be off by 0.06 rad.
//
// A head takes dim / 8 lanes (padded to 8, 16 or 32), each holding the two quads of
// elements that rotate into each other, so that the rotation needs no exchange and
// the norm one butterfly.  A block takes a few tokens: it works out their places and
// each angle once, into shared memory, then its warps run over the tokens' heads,
// loading the next while they turn the last.  A prompt is bound by its 18 warps an SM
// (what registers leave) at 2.6 instructions a cycle, 0.6 of a copy's rate; a few tokens
// by the chain of loads, so those get a block for every four warps' heads.
//
// B200, 32 + 8 heads of 128: q and k of 8192 tokens from BF16 42 us (168 MB, 4.0 TB/s);
// appending 4 x 1024 rows of which 2519 are real 20.5 us; 64 tokens 3.8 us, one 3.2 us.
// From FP32 70 us (252 MB, 3.6 TB/s); in the general form half of each head 54 us, heads
// of 96 53 us (126 MB).
// Five blocks an SM measured best (four 45 us, six 46), as did four tokens a block (eight
// 48 us; twelve 41, but 40 for the ragged append), and eight elements a lane (sixteen,
// with fewer instructions and fewer warps: 43).
#include <cuda_bf16.h>
#include <cuda_runtime.h>

#include <cstdint>

#include "paged.cuh"
#include "ptx.cuh"

namespace nwc {

namespace {

constexpr unsigned kAll = 0xFFFFFFFFu;
constexpr int kRopeWarps = 4;
constexpr int kMaxDim = 256;

// Four elements as they lie in memory, and as FP32.
struct Raw32 {
  float v[4];
};
struct Raw16 {
  uint32_t v[2];
};
template <typename T>
struct RawOf {
  using type = Raw32;
};
template <>
struct RawOf<__nv_bfloat16> {
  using type = Raw16;
};
__device__ __forceinline__ Raw32 load_raw(const float* p, bool vec) {
  Raw32 r;
  if (vec) {
    const float4 f = *reinterpret_cast<const float4*>(p);
    r.v[0] = f.x, r.v[1] = f.y, r.v[2] = f.z, r.v[3] = f.w;
  } else {
#pragma unroll
    for (int i = 0; i < 4; ++i) r.v[i] = p[i];
  }
  return r;
}
__device__ __forceinline__ Raw16 load_raw(const __nv_bfloat16* p, bool vec) {
  Raw16 r;
  if (vec) {
    const uint2 u = *reinterpret_cast<const uint2*>(p);
    r.v[0] = u.x, r.v[1] = u.y;
  } else {
    const uint16_t* h = reinterpret_cast<const uint16_t*>(p);
    r.v[0] = h[0] | (uint32_t)h[1] << 16;
    r.v[1] = h[2] | (uint32_t)h[3] << 16;
  }
  return r;
}
__device__ __forceinline__ void widen(const Raw32& r, float (&v)[4]) {
#pragma unroll
  for (int i = 0; i < 4; ++i) v[i] = r.v[i];
}
__device__ __forceinline__ void widen(const Raw16& r, float (&v)[4]) {
#pragma unroll
  for (int i = 0; i < 2; ++i) {
    v[2 * i] = __uint_as_float(r.v[i] << 16);
    v[2 * i + 1] = __uint_as_float(r.v[i] & 0xFFFF0000u);
  }
}
template <typename T>
__device__ __forceinline__ void load4(const T* p, bool vec, float (&v)[4]) {
  widen(load_raw(p, vec), v);
}
__device__ __forceinline__ void store4(float* p, bool vec, const float (&v)[4]) {
  if (vec) {
    *reinterpret_cast<float4*>(p) = make_float4(v[0], v[1], v[2], v[3]);
  } else {
#pragma unroll
    for (int i = 0; i < 4; ++i) p[i] = v[i];
  }
}
__device__ __forceinline__ void store4(__nv_bfloat16* p, bool vec, const float (&v)[4]) {
  if (vec) {
    __nv_bfloat162 a = __floats2bfloat162_rn(v[0], v[1]), b = __floats2bfloat162_rn(v[2], v[3]);
    uint2 u;
    u.x = *reinterpret_cast<uint32_t*>(&a), u.y = *reinterpret_cast<uint32_t*>(&b);
    *reinterpret_cast<uint2*>(p) = u;
  } else {
#pragma unroll
    for (int i = 0; i < 4; ++i) p[i] = __float2bfloat16_rn(v[i]);
  }
}
// Row `row` of the batch as a token of its sequence.
struct Place {
  bool real;         // a new token (not padding)
  int64_t position;  // in the whole text: prefix + own index
  int64_t slot_page; // its page, or -1 when it has none or the tables do not hold it
  int32_t slot;      // its place in the page
};
__device__ __forceinline__ Place place_of(const CacheView& c, const BatchView& b, int row,
                                          int lane) {
  Place at;
  const int seq = row / b.chunk, i = row - seq * b.chunk;
  const int len = max(b.lens[seq], 0);
  const int fresh = b.q_lens ? min(max(b.q_lens[seq], 0), b.chunk) : b.chunk;
  const int j = len - fresh + i;
  at.real = i < fresh;
  int64_t base = 0;
  for (int g0 = 0; g0 < b.groups; g0 += 32) {  // the group that holds the sequence
    const int g = g0 + lane;
    const bool in = g < b.groups && b.group_start[g] <= seq && seq < b.group_start[g + 1];
    const unsigned hit = __ballot_sync(kAll, in);
    if (hit) {
      base = max(b.prefix_lens[g0 + __ffs(hit) - 1], 0);
      break;
    }
  }
  at.position = base + j;
  at.slot = j & ((1 << c.page_shift) - 1);
  at.slot_page = -1;
  if (at.real && j >= 0) {   // before the sequence's start there is no place
    const int n = j >> c.page_shift;
    if (n < b.table_width && j < (1 << 30)) at.slot_page = b.table[(int64_t)seq * b.table_stride + n];
    if (at.slot_page < 0 || at.slot_page >= c.pages) {
      at.slot_page = -1;
      if (lane == 0) atomicOr(c.err, kErrRange);
    }
  }
  return at;
}

constexpr int kMaxTokens = 4;   // of a block
constexpr int kBlocks = 5;      // an SM, for prompts

// What a warp does with one kind of a token's heads.
struct Turn {
  bool norm, rotate, interleaved;
  float inv_dim, eps;
  float c[4], s[4];         // of the lane's pairs
  float wa[4], wb[4];       // weights of its quads
};

// Heads come in groups of 32 / G; a warp has groups first, first + step, ....  EXACT:
// the lanes fill the heads, the groups the number of heads, and whole heads rotate,
// so that nothing is left to a lane to ask.
template <int G, bool EXACT>
struct Groups {
  int first, step, count, heads;
  bool on;                  // the lane has elements
  __device__ __forceinline__ bool has(int g) const {
    if (EXACT) return g < count;
    return on && g * (32 / G) + (int)(threadIdx.x & 31) / G < heads;
  }
};

// The raw quads of U groups.
template <typename TIn, int U>
struct Batch {
  typename RawOf<TIn>::type q[U][2];
};
// src: the lane's first quad in group 0, its second `quad` elements on.
template <typename TIn, int G, int U, bool VEC, bool EXACT>
__device__ __forceinline__ void load_groups(Batch<TIn, U>& raw, const Groups<G, EXACT>& of,
                                            int from, const TIn* src, int64_t group, int quad) {
  const TIn* p = src + from * group;
#pragma unroll
  for (int j = 0; j < U; ++j, p += of.step * group)
    if (of.has(from + j * of.step)) {
      raw.q[j][0] = load_raw(p, VEC);
      raw.q[j][1] = load_raw(p + quad, VEC);
    }
}
template <typename TOut, int G, bool VEC, bool EXACT>
__device__ __forceinline__ void zero_groups(const Groups<G, EXACT>& of, TOut* dst, int64_t group,
                                            int quad) {
  const float none[4] = {0.f, 0.f, 0.f, 0.f};
  for (int g = of.first; g < of.count; g += of.step)
    if (of.has(g)) {
      store4(dst + g * group, VEC, none);
      store4(dst + g * group + quad, VEC, none);
    }
}

// Turns the groups of this warp, U at a time.  The first U are in `raw`; where `next`
// is given, those of the next token replace them as they are used.  INTER is the
// pairing where EXACT holds.
template <typename TIn, typename TOut, int G, int U, bool VEC_IN, bool VEC_OUT, bool EXACT,
          bool INTER>
__device__ __forceinline__ void turn_heads(const Turn& k, Batch<TIn, U>& raw,
                                           const Groups<G, EXACT>& of, const TIn* src,
                                           int64_t src_group, const TIn* next, TOut* dst,
                                           int64_t dst_group, int quad) {
#pragma unroll 1
  for (int g0 = of.first; g0 < of.count; g0 += U * of.step) {
    if (g0 != of.first)
      load_groups<TIn, G, U, VEC_IN, EXACT>(raw, of, g0, src, src_group, quad);
    const bool last = g0 + U * of.step >= of.count;
    TOut* to = dst + g0 * dst_group;
    const TIn* ahead = next + of.first * src_group;
#pragma unroll
    for (int j = 0; j < U; ++j) {
      float a[4], b[4];
      widen(raw.q[j][0], a);
      widen(raw.q[j][1], b);
      if (next && last && of.has(of.first + j * of.step)) {
        raw.q[j][0] = load_raw(ahead, VEC_IN);
        raw.q[j][1] = load_raw(ahead + quad, VEC_IN);
      }
      ahead += of.step * src_group;
      if (k.norm) {
        float sum = 0.f;
#pragma unroll
        for (int i = 0; i < 4; ++i) sum += a[i] * a[i] + b[i] * b[i];
#pragma unroll
        for (int o = G / 2; o > 0; o >>= 1) sum += __shfl_xor_sync(kAll, sum, o);
        const float r = rsqrtf(sum * k.inv_dim + k.eps);
#pragma unroll
        for (int i = 0; i < 4; ++i) a[i] *= r * k.wa[i], b[i] *= r * k.wb[i];
      }
      if (EXACT || k.rotate) {
        if (EXACT ? INTER : k.interleaved) {
          // The lane's eight elements are pairs 4u .. 4u + 3 in order.
#pragma unroll
          for (int i = 0; i < 4; ++i) {
            float& e = i < 2 ? a[2 * i] : b[2 * i - 4];
            float& o = i < 2 ? a[2 * i + 1] : b[2 * i - 3];
            const float e0 = e, o0 = o;
            e = e0 * k.c[i] - o0 * k.s[i];
            o = o0 * k.c[i] + e0 * k.s[i];
          }
        } else {
#pragma unroll
          for (int i = 0; i < 4; ++i) {
            const float a0 = a[i], b0 = b[i];
            a[i] = a0 * k.c[i] - b0 * k.s[i];
            b[i] = b0 * k.c[i] + a0 * k.s[i];
          }
        }
      }
      if (of.has(g0 + j * of.step)) {
        store4(to, VEC_OUT, a);
        store4(to + quad, VEC_OUT, b);
      }
      to += of.step * dst_group;
    }
  }
}
// V's heads: only rounded.
template <typename TIn, int G, bool VEC, bool EXACT>
__device__ __forceinline__ void copy_heads(Batch<TIn, 1>& raw, const Groups<G, EXACT>& of,
                                           const TIn* src, int64_t src_group, const TIn* next,
                                           __nv_bfloat16* dst, int64_t dst_group, bool place) {
  for (int g = of.first; g < of.count; g += of.step) {
    if (g != of.first) load_groups<TIn, G, 1, VEC, EXACT>(raw, of, g, src, src_group, 4);
    float a[4], b[4];
    widen(raw.q[0][0], a);
    widen(raw.q[0][1], b);
    if (next && g + of.step >= of.count)
      load_groups<TIn, G, 1, VEC, EXACT>(raw, of, of.first, next, src_group, 4);
    if (place && of.has(g)) {
      store4(dst + g * dst_group, true, a);
      store4(dst + g * dst_group + 4, true, b);
    }
  }
}

// G lanes a head; VEC: all quads are aligned for whole loads and stores.  Blocks are
// token blocks x `splits`, the latter sharing a token's heads.
template <typename TIn, typename TOut, int G, int U, bool VEC, bool EXACT, bool INTER>
__global__ void __launch_bounds__(kRopeWarps * 32, U != 4 ? 1 : EXACT ? kBlocks : 4) rope_kernel(
    const __grid_constant__ RopeParams p, int block_tokens, int splits, int groups_q,
    int groups_k) {
  __shared__ float2 turn[kMaxTokens][kMaxDim / 2];   // cosine and sine of each pair
  __shared__ Place places[kMaxTokens];
  allow_dependents();
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  const int split = (int)(blockIdx.x % (unsigned)splits);
  const int token0 = (int)(blockIdx.x / (unsigned)splits) * block_tokens;
  const int tokens = min(block_tokens, p.tokens - token0);
  constexpr int kHeads = 32 / G;
  const int u = lane % G, in_group = lane / G;
  const bool on = EXACT || u * 8 < p.dim;
  // The two quads of this lane, in a head that rotates; else 8 u and the next.
  const int half = p.rotary / 2;
  Turn k;
  k.rotate = EXACT || u * 8 < p.rotary;
  k.interleaved = EXACT ? INTER : p.interleaved != 0;
  k.inv_dim = 1.f / (float)p.dim;
  k.eps = p.eps;
  const bool apart = k.rotate && !k.interleaved;
  const int oa = apart ? 4 * u : 8 * u, quad = apart ? half : 4;
  const int first = split * kRopeWarps + warp, step = splits * kRopeWarps;
  // Few k and v heads: of the warps behind the last with q, and with k, first.
  const int first_k = (first + step - groups_q % step) % step;
  const int first_v = (first_k + step - groups_k % step) % step;
  const Groups<G, EXACT> of_q{first, step, groups_q, p.heads, on};
  const Groups<G, EXACT> of_k{first_k, step, groups_k, p.kv_heads, on};
  const Groups<G, EXACT> of_v{first_v, step, groups_k, p.kv_heads, on};
  const int64_t q_group = kHeads * p.q.head_stride, k_group = kHeads * p.k.head_stride,
                v_group = kHeads * p.v.head_stride;
  const TIn* q_src = static_cast<const TIn*>(p.q.data) + (int64_t)token0 * p.q.token_stride +
                     in_group * p.q.head_stride + oa;
  const TIn* k_src = static_cast<const TIn*>(p.k.data) + (int64_t)token0 * p.k.token_stride +
                     in_group * p.k.head_stride + oa;
  const TIn* v_src = static_cast<const TIn*>(p.v.data) + (int64_t)token0 * p.v.token_stride +
                     in_group * p.v.head_stride + 8 * u;
  wait_prerequisites();

  // The first token's heads are on their way while the places and angles are found.
  Batch<TIn, U> raw_q = {};
  Batch<TIn, 1> raw_k = {}, raw_v = {};
  auto bring = [&](int t) {
    if (p.q.data)
      load_groups<TIn, G, U, VEC, EXACT>(raw_q, of_q, first, q_src + t * p.q.token_stride,
                                         q_group, quad);
    if (p.k.data)
      load_groups<TIn, G, 1, VEC, EXACT>(raw_k, of_k, first_k, k_src + t * p.k.token_stride,
                                         k_group, quad);
    if (p.append)
      load_groups<TIn, G, 1, VEC, EXACT>(raw_v, of_v, first_v, v_src + t * p.v.token_stride,
                                         v_group, 4);
  };
  bring(0);
  for (int t = warp; t < tokens; t += kRopeWarps) {
    Place at;
    if (p.append) {
      at = place_of(p.cache, p.batch, token0 + t, lane);
    } else {
      at.real = true;
      at.slot_page = at.slot = 0;
      at.position = p.positions_64
                        ? static_cast<const int64_t*>(p.positions)[token0 + t]
                        : (int64_t)static_cast<const int32_t*>(p.positions)[token0 + t];
    }
    if (lane == 0) places[t] = at;
  }
  float w[2][2][4];   // weights of q and of k for the lane's quads
#pragma unroll
  for (int j = 0; j < 2; ++j) {
    const void* weight = j == 0 ? p.q_weight : p.k_weight;
#pragma unroll
    for (int i = 0; i < 4; ++i) w[j][0][i] = w[j][1][i] = 0.f;
    if (!weight || !on) continue;
    if (p.weight_f32) {
      load4(static_cast<const float*>(weight) + oa, VEC, w[j][0]);
      load4(static_cast<const float*>(weight) + oa + quad, VEC, w[j][1]);
    } else {
      load4(static_cast<const __nv_bfloat16*>(weight) + oa, VEC, w[j][0]);
      load4(static_cast<const __nv_bfloat16*>(weight) + oa + quad, VEC, w[j][1]);
    }
  }
  __syncthreads();
  for (int t = 0; t < tokens; ++t) {
    const double position = (double)places[t].position;
    for (int i = threadIdx.x; i < half; i += kRopeWarps * 32) {
      const double angle = position * p.freq[i] * 0.15915494309189533577;
      float2 cs;   // the angle in turns, of which the fraction counts
      sincospif(2.f * (float)(angle - rint(angle)), &cs.y, &cs.x);
      turn[t][i] = cs;
    }
  }
  __syncthreads();

#pragma unroll 1
  for (int t = 0; t < tokens; ++t) {
    const Place at = places[t];
    const int64_t token = token0 + t;
    const bool more = t + 1 < tokens && places[t + 1].real;
    TOut* q_dst = static_cast<TOut*>(p.q_out.data) + token * p.q_out.token_stride +
                  in_group * p.q_out.head_stride + oa;
    if (!at.real) {   // padding
      if (p.q.data)
        zero_groups<TOut, G, VEC, EXACT>(of_q, q_dst, kHeads * p.q_out.head_stride, quad);
      if (more) bring(t + 1);
      continue;
    }
    if (k.rotate) {
      const float4 lo = *reinterpret_cast<const float4*>(&turn[t][4 * u]);
      const float4 hi = *reinterpret_cast<const float4*>(&turn[t][4 * u + 2]);
      k.c[0] = lo.x, k.c[1] = lo.z, k.c[2] = hi.x, k.c[3] = hi.z;
      k.s[0] = lo.y, k.s[1] = lo.w, k.s[2] = hi.y, k.s[3] = hi.w;
    }
    if (p.q.data) {
      k.norm = p.q_weight != nullptr;
#pragma unroll
      for (int i = 0; i < 4; ++i) k.wa[i] = w[0][0][i], k.wb[i] = w[0][1][i];
      const TIn* src = q_src + t * p.q.token_stride;
      turn_heads<TIn, TOut, G, U, VEC, VEC, EXACT, INTER>(
          k, raw_q, of_q, src, q_group, more ? src + p.q.token_stride : nullptr, q_dst,
          kHeads * p.q_out.head_stride, quad);
    }
    if (!p.k.data) continue;
    k.norm = p.k_weight != nullptr;
#pragma unroll
    for (int i = 0; i < 4; ++i) k.wa[i] = w[1][0][i], k.wb[i] = w[1][1][i];
    const TIn* src = k_src + t * p.k.token_stride;
    const TIn* next = more ? src + p.k.token_stride : nullptr;
    if (!p.append) {
      turn_heads<TIn, TOut, G, 1, VEC, VEC, EXACT, INTER>(
          k, raw_k, of_k, src, k_group, next,
          static_cast<TOut*>(p.k_out.data) + token * p.k_out.token_stride +
              in_group * p.k_out.head_stride + oa,
          kHeads * p.k_out.head_stride, quad);
      continue;
    }
    // Pages are 16-byte aligned with strides of 8 elements (checked on the host).
    const CacheView& cv = p.cache;
    const bool place = at.slot_page >= 0;
    const TIn* v = v_src + t * p.v.token_stride;
    const TIn* next_v = more ? v + p.v.token_stride : nullptr;
    if (place) {
      turn_heads<TIn, __nv_bfloat16, G, 1, VEC, true, EXACT, INTER>(
          k, raw_k, of_k, src, k_group, next,
          reinterpret_cast<__nv_bfloat16*>(cv.k) + at.slot_page * cv.k_page +
              at.slot * cv.k_token + in_group * cv.k_head + oa,
          kHeads * cv.k_head, quad);
    } else if (next) {
      load_groups<TIn, G, 1, VEC, EXACT>(raw_k, of_k, first_k, next, k_group, quad);
    }
    copy_heads<TIn, G, VEC, EXACT>(
        raw_v, of_v, v, v_group, next_v,
        reinterpret_cast<__nv_bfloat16*>(cv.v) + (place ? at.slot_page : 0) * cv.v_page +
            at.slot * cv.v_token + in_group * cv.v_head + 8 * u,
        kHeads * cv.v_head, place);
  }
}

bool quads_aligned(const HeadsView& v, int type) {
  const uintptr_t unit = type == kTypeF32 ? 16 : 8;
  return !v.data || ((reinterpret_cast<uintptr_t>(v.data) % unit) == 0 &&
                     v.token_stride % 4 == 0 && v.head_stride % 4 == 0);
}

template <typename TIn, typename TOut, int G, bool VEC>
cudaError_t launch_t(const RopeParams& p, int sm_count, cudaStream_t stream) {
  constexpr int kHeads = 32 / G;
  const int groups_q = p.q.data ? (p.heads + kHeads - 1) / kHeads : 0;
  const int groups_k = p.k.data ? (p.kv_heads + kHeads - 1) / kHeads : 0;
  const int groups = groups_q + groups_k * (p.append ? 2 : 1);
  // Four tokens a block share the work on angles; until such blocks fill the device
  // a token each, its heads over as many blocks as it takes for a head group a warp.
  const bool large = p.tokens >= sm_count * 2 * kMaxTokens;
  const int block_tokens = large ? kMaxTokens : 1;
  const int splits = large ? 1 : (groups + kRopeWarps - 1) / kRopeWarps;
  const int64_t blocks = ((int64_t)p.tokens + block_tokens - 1) / block_tokens * splits;
  if (blocks > 0x7FFFFFFF) return cudaErrorInvalidValue;
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3((unsigned)blocks);
  cfg.blockDim = dim3(kRopeWarps * 32);
  cfg.stream = stream;
  cudaLaunchAttribute attr[1];
  attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[0].val.programmaticStreamSerializationAllowed = 1;
  cfg.attrs = attr;
  cfg.numAttrs = 1;
  // Four head groups of q in flight a warp where it has as many.
  auto run = [&](auto kernel) {
    return cudaLaunchKernelEx(&cfg, kernel, p, block_tokens, splits, groups_q, groups_k);
  };
  if (!large) return run(rope_kernel<TIn, TOut, G, 1, VEC, false, false>);
  const bool exact = VEC && p.dim == 8 * G && p.rotary == p.dim &&
                     (!p.q.data || p.heads % kHeads == 0) &&
                     (!p.k.data || p.kv_heads % kHeads == 0);
  if (!exact) return run(rope_kernel<TIn, TOut, G, 4, VEC, false, false>);
  return p.interleaved ? run(rope_kernel<TIn, TOut, G, 4, true, true, true>)
                       : run(rope_kernel<TIn, TOut, G, 4, true, true, false>);
}

template <typename TIn, typename TOut, bool VEC>
cudaError_t launch_g(const RopeParams& p, int sm_count, cudaStream_t stream) {
  if (p.dim <= 64) return launch_t<TIn, TOut, 8, VEC>(p, sm_count, stream);
  if (p.dim <= 128) return launch_t<TIn, TOut, 16, VEC>(p, sm_count, stream);
  return launch_t<TIn, TOut, 32, VEC>(p, sm_count, stream);
}

template <typename TIn, typename TOut>
cudaError_t launch_v(const RopeParams& p, bool vec, int sm_count, cudaStream_t stream) {
  return vec ? launch_g<TIn, TOut, true>(p, sm_count, stream)
             : launch_g<TIn, TOut, false>(p, sm_count, stream);
}

}  // namespace

cudaError_t launch_rope(const RopeParams& p, int in_type, int out_type, int sm_count,
                        cudaStream_t stream) {
  const uintptr_t unit = p.weight_f32 ? 16 : 8;
  const bool vec = quads_aligned(p.q, in_type) && quads_aligned(p.k, in_type) &&
                   quads_aligned(p.v, in_type) && quads_aligned(p.q_out, out_type) &&
                   quads_aligned(p.k_out, out_type) &&
                   (reinterpret_cast<uintptr_t>(p.q_weight) % unit) == 0 &&
                   (reinterpret_cast<uintptr_t>(p.k_weight) % unit) == 0;
  if (in_type == kTypeF32)
    return out_type == kTypeF32 ? launch_v<float, float>(p, vec, sm_count, stream)
                                : launch_v<float, __nv_bfloat16>(p, vec, sm_count, stream);
  return out_type == kTypeF32 ? launch_v<__nv_bfloat16, float>(p, vec, sm_count, stream)
                              : launch_v<__nv_bfloat16, __nv_bfloat16>(p, vec, sm_count, stream);
}

}  // namespace nwc
