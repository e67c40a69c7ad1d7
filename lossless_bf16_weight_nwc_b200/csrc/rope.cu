// rope.cu — per-head RMS norm and position rotation of q and k in one pass, to
// tensors or (k and v) straight into a paged cache.
//
// y = x / sqrt(mean(x^2) + eps) * w over a head, then every pair (a, b) of the
// leading `rotary` elements becomes (a cos t - b sin t, b cos t + a sin t) with
// t = position * freq_i.  Sums and products are FP32 and there is one rounding,
// on the store.  The angle is reduced to turns in 64 bits: at position 10^6 an
// FP32 product would already be off by 0.06 rad.
//
// A head takes dim / 8 lanes (padded to 8, 16 or 32), each holding the two
// quads of elements that rotate into each other, so that the rotation needs no
// exchange and the norm one butterfly; a warp holds 32 / G heads times U, all of
// one token and one kind (q, k or v), and evaluates the angles once for them.
#include <cuda_bf16.h>
#include <cuda_runtime.h>

#include <cstdint>

#include "paged.cuh"
#include "ptx.cuh"

namespace nwc {

namespace {

constexpr unsigned kAll = 0xFFFFFFFFu;
constexpr int kRopeWarps = 4;

__device__ __forceinline__ void load4(const float* p, bool vec, float (&v)[4]) {
  if (vec) {
    const float4 f = *reinterpret_cast<const float4*>(p);
    v[0] = f.x, v[1] = f.y, v[2] = f.z, v[3] = f.w;
  } else {
#pragma unroll
    for (int i = 0; i < 4; ++i) v[i] = p[i];
  }
}
__device__ __forceinline__ void load4(const __nv_bfloat16* p, bool vec, float (&v)[4]) {
  if (vec) {
    const uint2 u = *reinterpret_cast<const uint2*>(p);
    v[0] = __uint_as_float(u.x << 16), v[1] = __uint_as_float(u.x & 0xFFFF0000u);
    v[2] = __uint_as_float(u.y << 16), v[3] = __uint_as_float(u.y & 0xFFFF0000u);
  } else {
#pragma unroll
    for (int i = 0; i < 4; ++i) v[i] = __bfloat162float(p[i]);
  }
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
__device__ __forceinline__ void load_weights(const void* w, bool f32, int oa, int ob,
                                             float (&wa)[4], float (&wb)[4]) {
  if (f32) {
    load4(static_cast<const float*>(w) + oa, false, wa);
    load4(static_cast<const float*>(w) + ob, false, wb);
  } else {
    load4(static_cast<const __nv_bfloat16*>(w) + oa, false, wa);
    load4(static_cast<const __nv_bfloat16*>(w) + ob, false, wb);
  }
}

struct Quads {
  float a[4], b[4];
};

// Row `row` of the batch as a token of its sequence.
struct Place {
  bool real;         // a new token (not padding)
  int64_t position;  // in the whole text: prefix + own index
  int64_t slot_page; // its page, or -1 when the tables do not hold it
  int32_t slot;      // its place in the page
};
__device__ __forceinline__ Place place_of(const CacheView& c, const BatchView& b, int row,
                                          int lane) {
  Place at;
  const int seq = row / b.chunk, i = row - seq * b.chunk;
  const int len = max(b.lens[seq], 0);
  const int fresh = b.q_lens ? min(max(b.q_lens[seq], 0), b.chunk) : b.chunk;
  const int j = len - fresh + i;
  at.real = i < fresh && j >= 0;
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
  if (at.real) {
    const int n = j >> c.page_shift;
    if (n < b.table_width && j < (1 << 30)) at.slot_page = b.table[(int64_t)seq * b.table_stride + n];
    if (at.slot_page < 0 || at.slot_page >= c.pages) {
      at.slot_page = -1;
      if (lane == 0) atomicOr(c.err, kErrRange);
    }
  }
  return at;
}

// G lanes a head, U heads a group of lanes; vec_in, vec_out: quads are aligned
// for whole loads and stores.
template <typename TIn, typename TOut, int G, int U>
__global__ void __launch_bounds__(kRopeWarps * 32) rope_kernel(
    const __grid_constant__ RopeParams p, bool vec_in, bool vec_out, int jobs_q, int jobs_k,
    int jobs) {
  allow_dependents();
  const int lane = threadIdx.x & 31;
  const int64_t w = (int64_t)blockIdx.x * kRopeWarps + (threadIdx.x >> 5);
  const int64_t token64 = w / jobs;
  const int job = (int)(w - token64 * jobs);
  if (token64 >= p.tokens) return;
  const int token = (int)token64;
  const int kind = job < jobs_q ? 0 : job < jobs_q + jobs_k ? 1 : 2;
  constexpr int kHeads = 32 / G;
  const int head0 = (kind == 0 ? job : kind == 1 ? job - jobs_q : job - jobs_q - jobs_k) *
                        (kHeads * U) + lane / G;
  const int heads = kind == 0 ? p.heads : p.kv_heads;
  const int u = lane % G;
  const bool on = u * 8 < p.dim;
  // The two quads of this lane, and whether they rotate.
  const int half = p.rotary / 2;
  const bool rot = kind < 2 && on && u * 8 < p.rotary;
  const int oa = rot && !p.interleaved ? 4 * u : 8 * u;
  const int ob = rot && !p.interleaved ? half + 4 * u : 8 * u + 4;
  wait_prerequisites();

  Place at;
  at.real = true;
  at.slot_page = -1;
  at.slot = 0;
  if (p.append) {
    at = place_of(p.cache, p.batch, token, lane);
  } else {
    at.position = p.positions_64 ? static_cast<const int64_t*>(p.positions)[token]
                                 : (int64_t)static_cast<const int32_t*>(p.positions)[token];
  }
  const bool to_cache = p.append && kind > 0;
  if (to_cache && at.slot_page < 0) return;

  const HeadsView& in = kind == 0 ? p.q : kind == 1 ? p.k : p.v;
  const TIn* src = static_cast<const TIn*>(in.data) + (int64_t)token * in.token_stride;
  Quads x[U];
#pragma unroll
  for (int k = 0; k < U; ++k) {
    const int h = head0 + k * kHeads;
#pragma unroll
    for (int i = 0; i < 4; ++i) x[k].a[i] = x[k].b[i] = 0.f;
    if (on && at.real && h < heads) {
      load4(src + (int64_t)h * in.head_stride + oa, vec_in, x[k].a);
      load4(src + (int64_t)h * in.head_stride + ob, vec_in, x[k].b);
    }
  }
  if (at.real) {
    float c[4], s[4];
    if (rot) {
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        // Pair i of the lane: (a_i, b_i), or neighbours when interleaved.
        const double turns =
            (double)at.position * p.freq[4 * u + i] * 0.15915494309189533577;  // 1 / (2 pi)
        sincospif(2.f * (float)(turns - rint(turns)), &s[i], &c[i]);
      }
    }
    const void* weight = kind == 0 ? p.q_weight : kind == 1 ? p.k_weight : nullptr;
    if (weight) {
      float wa[4] = {}, wb[4] = {};
      if (on) load_weights(weight, p.weight_f32 != 0, oa, ob, wa, wb);
#pragma unroll
      for (int k = 0; k < U; ++k) {
        float sum = 0.f;
#pragma unroll
        for (int i = 0; i < 4; ++i) sum += x[k].a[i] * x[k].a[i] + x[k].b[i] * x[k].b[i];
#pragma unroll
        for (int o = G / 2; o > 0; o >>= 1) sum += __shfl_xor_sync(kAll, sum, o);
        const float r = rsqrtf(sum / (float)p.dim + p.eps);
#pragma unroll
        for (int i = 0; i < 4; ++i) {
          x[k].a[i] *= r * wa[i];
          x[k].b[i] *= r * wb[i];
        }
      }
    }
    if (rot) {
#pragma unroll
      for (int k = 0; k < U; ++k) {
        float* a = x[k].a;
        float* b = x[k].b;
        if (p.interleaved) {
          // The lane's eight elements are pairs 4u .. 4u + 3 in order.
#pragma unroll
          for (int i = 0; i < 4; ++i) {
            float& e = i < 2 ? a[2 * i] : b[2 * i - 4];
            float& o = i < 2 ? a[2 * i + 1] : b[2 * i - 3];
            const float e0 = e, o0 = o;
            e = e0 * c[i] - o0 * s[i];
            o = o0 * c[i] + e0 * s[i];
          }
        } else {
#pragma unroll
          for (int i = 0; i < 4; ++i) {
            const float a0 = a[i], b0 = b[i];
            a[i] = a0 * c[i] - b0 * s[i];
            b[i] = b0 * c[i] + a0 * s[i];
          }
        }
      }
    }
  }
  if (!on) return;
#pragma unroll
  for (int k = 0; k < U; ++k) {
    const int h = head0 + k * kHeads;
    if (h >= heads) continue;
    if (to_cache) {
      const CacheView& cv = p.cache;
      __nv_bfloat16* d =
          kind == 1 ? reinterpret_cast<__nv_bfloat16*>(cv.k) + at.slot_page * cv.k_page +
                          at.slot * cv.k_token + h * cv.k_head
                    : reinterpret_cast<__nv_bfloat16*>(cv.v) + at.slot_page * cv.v_page +
                          at.slot * cv.v_token + h * cv.v_head;
      // Pages are 16-byte aligned with strides of 8 elements (checked on the host).
      store4(d + oa, true, x[k].a);
      store4(d + ob, true, x[k].b);
    } else {
      const HeadsView& o = kind == 0 ? p.q_out : p.k_out;
      TOut* d = static_cast<TOut*>(o.data) + (int64_t)token * o.token_stride +
                (int64_t)h * o.head_stride;
      store4(d + oa, vec_out, x[k].a);
      store4(d + ob, vec_out, x[k].b);
    }
  }
}

bool quads_aligned(const HeadsView& v, int type) {
  const uintptr_t unit = type == kTypeF32 ? 16 : 8;
  return !v.data || ((reinterpret_cast<uintptr_t>(v.data) % unit) == 0 &&
                     v.token_stride % 4 == 0 && v.head_stride % 4 == 0);
}

template <typename TIn, typename TOut, int G, int U>
cudaError_t launch_t(const RopeParams& p, bool vi, bool vo, cudaStream_t stream) {
  constexpr int per = 32 / G * U;
  const int jobs_q = p.q.data ? (p.heads + per - 1) / per : 0;
  const int jobs_k = p.k.data ? (p.kv_heads + per - 1) / per : 0;
  const int jobs = jobs_q + jobs_k * (p.append ? 2 : 1);
  const int64_t blocks = ((int64_t)p.tokens * jobs + kRopeWarps - 1) / kRopeWarps;
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
  return cudaLaunchKernelEx(&cfg, rope_kernel<TIn, TOut, G, U>, p, vi, vo, jobs_q, jobs_k,
                            jobs);
}

template <typename TIn, typename TOut, int G>
cudaError_t launch_u(const RopeParams& p, bool vi, bool vo, int sm_count,
                     cudaStream_t stream) {
  // One head a lane group until that fills the device with warps twice over;
  // then four, which share their angles and keep four times the loads in flight.
  const int64_t warps =
      ((int64_t)p.tokens * (p.heads + 2 * p.kv_heads) * G + 31) / 32;
  if (warps < (int64_t)sm_count * 128) return launch_t<TIn, TOut, G, 1>(p, vi, vo, stream);
  return launch_t<TIn, TOut, G, 4>(p, vi, vo, stream);
}

template <typename TIn, typename TOut>
cudaError_t launch_g(const RopeParams& p, bool vi, bool vo, int sm_count,
                     cudaStream_t stream) {
  if (p.dim <= 64) return launch_u<TIn, TOut, 8>(p, vi, vo, sm_count, stream);
  if (p.dim <= 128) return launch_u<TIn, TOut, 16>(p, vi, vo, sm_count, stream);
  return launch_u<TIn, TOut, 32>(p, vi, vo, sm_count, stream);
}

}  // namespace

cudaError_t launch_rope(const RopeParams& p, int in_type, int out_type, int sm_count,
                        cudaStream_t stream) {
  const bool vi = quads_aligned(p.q, in_type) && quads_aligned(p.k, in_type) &&
                  quads_aligned(p.v, in_type);
  const bool vo = quads_aligned(p.q_out, out_type) && quads_aligned(p.k_out, out_type);
  if (in_type == kTypeF32)
    return out_type == kTypeF32 ? launch_g<float, float>(p, vi, vo, sm_count, stream)
                                : launch_g<float, __nv_bfloat16>(p, vi, vo, sm_count, stream);
  return out_type == kTypeF32
             ? launch_g<__nv_bfloat16, float>(p, vi, vo, sm_count, stream)
             : launch_g<__nv_bfloat16, __nv_bfloat16>(p, vi, vo, sm_count, stream);
}

}  // namespace nwc
