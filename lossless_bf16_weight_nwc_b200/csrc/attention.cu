// attention.cu — attention of a batch's new tokens over a paged cache, with
// prefixes that several sequences share.
//
// out = sum_j e^(s_j - m) v_j / sum_j e^(s_j - m), s_j = scale q . k_j, over the
// row's prefix and its own tokens, in one pass with the running maximum m.
//
// A decode batch reads each K and V once and multiplies it with few rows: what
// bounds it is memory, so the key axis is cut into equal shares for all SMs and
// every tile is multiplied on the tensor cores with up to 128 rows at once (the
// rows of a prefix's whole group times the query heads of a key head; a
// sequence's own tokens fill only a few of the 128, which costs nothing while
// memory is the bound).  One persistent CTA an SM:
//   * a producer warp brings K and V tiles of 128 tokens page by page with TMA
//     into a ring;
//   * one thread issues S = Q K^T and O += P V (tcgen05, M = 128), with S, P and O
//     in TMEM: P takes S's place as BF16 and is the A operand;
//   * two teams of 128 softmax threads, a row each: a team holds its own 128 rows
//     when an item has more than 128 (both then use each K and V tile), else the
//     teams take the tiles in turn, so that one team's exponentials run under
//     the other's products.
// The maximum that scales P follows the running one only when that has grown by
// more than 2^8, so O is rarely rescaled; P stays below 2^8 and the sums are FP32.
// A second kernel joins the parts' results in a fixed order.
#include <cuda_bf16.h>
#include <cuda_runtime.h>

#include <cmath>
#include <cstdint>

#include "paged.cuh"
#include "ptx.cuh"

namespace nwc {

namespace {

constexpr unsigned kAll = 0xFFFFFFFFu;
constexpr int kTeamThreads = 128;
constexpr int kProducerWarp = 8;
constexpr int kIssuerWarp = 9;
constexpr int kThreads = 10 * 32;
constexpr int kMaxRing = 12;
constexpr uint32_t kRingBytes = 163840;  // K and V tiles: 5 of dim 128, 10 of dim 64
constexpr uint32_t kBarBytes = 1024;
constexpr float kLazy = 8.f;             // growth of the maximum (log2) that rescales O

template <int DIM>
struct Layout {
  static constexpr uint32_t kTile = kKvTile * DIM * 2;   // bytes of a K, V or Q tile
  static constexpr int kRing = (int)(kRingBytes / kTile);
  static constexpr uint32_t kRingOff = 0;
  static constexpr uint32_t kQOff = kRing * kTile;
  static constexpr uint32_t kBarOff = kQOff + 2 * kTile;
  static constexpr uint32_t kBytes = kBarOff + kBarBytes;
};
static_assert(Layout<64>::kRing <= kMaxRing && Layout<128>::kBytes <= 232448, "shared memory");

struct Bars {
  uint64_t full[kMaxRing];   // a tile's bytes landed
  uint64_t empty[kMaxRing];  // the products that read the tile are done (2 arrivals)
  uint64_t qfull[2];         // the team's Q is in place
  uint64_t sfull[2];         // the team's S is in TMEM (and its P V before that is done)
  uint64_t pfull[2];         // the team's P is in TMEM (and V's tail is zeroed)
  uint64_t ofull[2];         // the last P V of the team's part is done
  uint64_t drain;
  uint32_t tmem;
  uint32_t abort;
  int32_t seg;               // where this CTA's share starts
  int64_t off;
  int64_t warp_flat[kThreads / 32];
  int32_t warp_items[kThreads / 32];
};
static_assert(sizeof(Bars) <= kBarBytes, "barriers");

// ---- segments, items and parts ---------------------------------------------

struct Segment {
  int seq0;    // first sequence
  int rows;    // rows (token x query head of a key head)
  int len;     // tokens
  int tiles;
  int items;
  bool far;    // a prefix
};

__device__ __forceinline__ int fresh_of(const BatchView& b, int seq) {
  return b.q_lens ? min(max(b.q_lens[seq], 0), b.chunk) : b.chunk;
}
__device__ __forceinline__ int own_len(const AttentionParams& p, int seq) {
  const int64_t cap = (int64_t)p.batch.table_width << p.cache.page_shift;
  return (int)min((int64_t)max(p.batch.lens[seq], 0), cap);
}
__device__ __forceinline__ int far_len(const AttentionParams& p, int g) {
  const int64_t cap = (int64_t)p.batch.prefix_width << p.cache.page_shift;
  return (int)min((int64_t)max(p.batch.prefix_lens[g], 0), cap);
}
__device__ __forceinline__ Segment segment(const AttentionParams& p, int s) {
  const BatchView& b = p.batch;
  Segment r;
  const int gq = p.heads / p.kv_heads;
  if (s < b.groups) {
    r.far = true;
    r.seq0 = min(max(b.group_start[s], 0), b.sequences);
    const int end = min(max(b.group_start[s + 1], r.seq0), b.sequences);
    r.rows = (end - r.seq0) * b.chunk * gq;
    r.len = r.rows ? far_len(p, s) : 0;
  } else {
    r.far = false;
    r.seq0 = s - b.groups;
    r.rows = b.chunk * gq;
    r.len = fresh_of(b, r.seq0) ? own_len(p, r.seq0) : 0;
  }
  r.tiles = (r.len + kKvTile - 1) / kKvTile;
  r.items = (r.rows + kPairRows - 1) / kPairRows * p.kv_heads;
  return r;
}
// CTAs that share `total` tiles out, and the first tile of CTA c.
__device__ __forceinline__ int sharers(const AttentionParams& p, int64_t total) {
  return (int)min((int64_t)p.ctas, max(total, (int64_t)1));
}
__device__ __forceinline__ int64_t first_tile(int64_t total, int c, int ctas) {
  return total * c / ctas;
}
__device__ __forceinline__ int owner(int64_t total, int64_t tile, int ctas) {
  return (int)(((tile + 1) * ctas - 1) / total);
}

struct Part {
  Segment seg;
  int s;           // segment
  int block, kvh;  // block of kPairRows rows, key head
  int rows;        // of the block
  bool both;       // more than kTeamRows: each team has its own rows
  int tile0, n;    // tiles [tile0, tile0 + n) of the segment
  int item;        // within the segment
};

// The parts of a CTA in order.
struct Walk {
  int s;
  int64_t off, left;
  __device__ __forceinline__ bool next(const AttentionParams& p, Part& part) {
    const int segments = p.batch.groups + p.batch.sequences;
    while (left > 0 && s < segments) {
      part.seg = segment(p, s);
      const int64_t flat = (int64_t)part.seg.tiles * part.seg.items;
      if (off >= flat) {
        ++s;
        off = 0;
        continue;
      }
      part.s = s;
      part.item = (int)(off / part.seg.tiles);
      part.tile0 = (int)(off - (int64_t)part.item * part.seg.tiles);
      part.n = (int)min((int64_t)(part.seg.tiles - part.tile0), left);
      part.block = part.item / p.kv_heads;
      part.kvh = part.item - part.block * p.kv_heads;
      part.rows = min(part.seg.rows - part.block * kPairRows, kPairRows);
      part.both = part.rows > kTeamRows;
      off += part.n;
      left -= part.n;
      return true;
    }
    return false;
  }
};

// The slot of a part's results for a team: item + CTA is different for any two
// parts, as each next part has a later item, a later CTA or both.
__device__ __forceinline__ int64_t slot_of(const AttentionParams& p, int s, int item, int cta,
                                           int team) {
  const int64_t first =
      s < p.batch.groups
          ? reinterpret_cast<const int32_t*>(p.workspace + p.ws.items)[s]
          : (int64_t)(s - p.batch.groups) * p.ws.own_items;
  return (first + item + cta) * 2 + team;
}

// ---- waits -------------------------------------------------------------------

struct Ctl {
  uint32_t* err;
  uint32_t limit;
  volatile uint32_t* abort;
};
// False (and every role leaves) when a wait gave up here or elsewhere.
__device__ __noinline__ bool wait_on(uint64_t* bar, uint32_t parity, const Ctl& c) {
  for (uint32_t it = 0; it < c.limit; ++it) {
    if (mbar_try_wait(bar, parity)) return true;
    if (*c.abort) return false;
  }
  *c.abort = 1u;
  atomicOr(c.err, kErrTimeout);
  return false;
}
__device__ __forceinline__ bool wait(uint64_t* bar, uint32_t parity, const Ctl& c) {
  return mbar_try_wait(bar, parity) || wait_on(bar, parity, c);
}

// ---- roles ---------------------------------------------------------------------

// Brings tile after tile: K at place 2n of the ring's sequence, V at 2n + 1.
template <int DIM>
__device__ void produce_kv(const AttentionParams& p, const CUtensorMap* k_map,
                           const CUtensorMap* v_map, uint8_t* smem, Bars* bars, Walk walk,
                           const Ctl& ctl) {
  using L = Layout<DIM>;
  constexpr int kHalves = DIM / 64;
  const int lane = threadIdx.x & 31;
  const int page = 1 << p.cache.page_shift;
  const int box = min(page, kKvTile);
  const int mine = lane / kHalves, half = lane % kHalves;   // this lane's box and half of it
  const BatchView& b = p.batch;
  uint32_t seq = 0;
  Part part;
  bool ok = true;
  while (ok && walk.next(p, part)) {
    const int32_t* row = part.seg.far ? b.prefix_table + (int64_t)part.s * b.prefix_stride
                                      : b.table + (int64_t)part.seg.seq0 * b.table_stride;
    for (int t = 0; t < part.n; ++t) {
      const int t0 = (part.tile0 + t) * kKvTile;
      const int boxes = (min(kKvTile, part.seg.len - t0) + box - 1) / box;
      const bool on = mine < boxes;
      const int token = t0 + mine * box;
      int32_t id = 0;
      if (on) {
        id = row[token >> p.cache.page_shift];
        if (id < 0 || id >= p.cache.pages) {      // outside: TMA fills zeros
          id = (int32_t)p.cache.pages;
          if (half == 0) atomicOr(p.cache.err, kErrRange);
        }
      }
#pragma unroll
      for (int kv = 0; kv < 2; ++kv, ++seq) {
        const uint32_t slot = seq % L::kRing, turn = seq / L::kRing;
        if (turn) ok = wait(&bars->empty[slot], (turn - 1) & 1u, ctl);
        ok = __all_sync(kAll, ok);
        if (!ok) break;
        if (lane == 0) mbar_expect_tx(&bars->full[slot], (uint32_t)(boxes * box * DIM * 2));
        __syncwarp();
        if (on)
          tma_load_4d(smem_u32(smem + L::kRingOff + slot * L::kTile) +
                          (uint32_t)(half * kKvTile + mine * box) * 128u,
                      kv ? v_map : k_map, half * 64, token & (page - 1), part.kvh, id,
                      &bars->full[slot]);
      }
      if (!ok) break;
    }
  }
  // No CTA leaves while its copies run.
  const WaitCtl dc = drain_ctl_default(p.cache.err);
  if (lane == 0)
    for (uint32_t k = seq > (uint32_t)L::kRing ? seq - L::kRing : 0u; k < seq; ++k)
      wait_bounded(&bars->full[k % L::kRing], (k / L::kRing) & 1u, dc);
}

// One team's use of one tile, in the order the products are issued: teams in turn.
struct Unit {
  uint32_t tile;   // of the CTA
  bool first;      // the team's first of a part
  bool last;       // the team's last of a part
};
struct Units {
  Walk walk;
  uint32_t tile = 0, team = 0;
  int left = 0, begun = 0;  // uses left of the part, teams that have begun it (bits)
  bool both = false;
  int next_n = 0;           // tiles of the part after it, 0: none
  bool next_both = false;
  __device__ __forceinline__ void look_ahead(const AttentionParams& p) {
    Part part;
    next_n = walk.next(p, part) ? part.n : 0;
    next_both = part.both;
  }
  __device__ __forceinline__ bool next(const AttentionParams& p, Unit& u, uint32_t& team_out) {
    if (left == 0) {
      if (next_n == 0) return false;
      both = next_both;
      left = both ? 2 * next_n : next_n;
      begun = 0;
      look_ahead(p);
    }
    team_out = team;
    u.tile = tile;
    u.first = !(begun >> team & 1);
    begun |= 1 << team;
    --left;
    u.last = left < 2;
    if (!both || (left & 1) == 0) ++tile;
    team ^= 1;
    return true;
  }
};

// Issues every product of the CTA (a whole warp, its first lane in effect).  A
// commit costs the issuer about as much as two products, so there is one a unit:
// it follows a team's P V and the S of its next unit, and the team passes the
// tiles it has then done with back to the producer.
template <int DIM>
__device__ void issue_products(const AttentionParams& p, uint8_t* smem, Bars* bars, Walk walk,
                               const Ctl& ctl) {
  using L = Layout<DIM>;
  const uint32_t leader = (threadIdx.x & 31) == 0;
  const uint32_t tmem = bars->tmem;
  const uint32_t ring = smem_u32(smem + L::kRingOff), q = smem_u32(smem + L::kQOff);
  constexpr uint32_t id_s = umma_idesc_bf16(kTeamRows, kKvTile);
  constexpr uint32_t id_o = umma_idesc_bf16_bmn(kTeamRows, DIM);
  uint32_t q_turn[2] = {0, 0}, p_turn[2] = {0, 0};
  Units units;
  units.walk = walk;
  units.look_ahead(p);

  auto issue_s = [&](const Unit& u, uint32_t w) -> bool {
    if (u.first && !wait(&bars->qfull[w], q_turn[w]++ & 1u, ctl)) return false;
    const uint32_t seq = 2 * u.tile, slot = seq % L::kRing;
    if (!wait(&bars->full[slot], (seq / L::kRing) & 1u, ctl)) return false;
    tc_fence_after();
    const uint64_t a = umma_desc_sw128(q + w * L::kTile);
    const uint64_t b = umma_desc_sw128(ring + slot * L::kTile);
#pragma unroll
    for (int k = 0; k < DIM / 16; ++k) {
      const uint32_t off = ((uint32_t)(k / 4) * (kKvTile * 128u) + (uint32_t)(k % 4) * 32u) >> 4;
      umma_bf16_by(leader, tmem + w * 128u, a + off, b + off, id_s, k > 0);
    }
    umma_commit_by(leader, &bars->sfull[w]);
    return true;
  };
  auto issue_o = [&](const Unit& u, uint32_t w) -> bool {
    if (!wait(&bars->pfull[w], p_turn[w]++ & 1u, ctl)) return false;
    const uint32_t seq = 2 * u.tile + 1, slot = seq % L::kRing;
    if (!wait(&bars->full[slot], (seq / L::kRing) & 1u, ctl)) return false;
    tc_fence_after();
    const uint64_t b = umma_desc_mn_sw128(ring + slot * L::kTile, kKvTile * 128u);
#pragma unroll
    for (int k = 0; k < kKvTile / 16; ++k)
      umma_bf16_ts_by(leader, tmem + 256u + w * 128u, tmem + w * 128u + 8u * k,
                      b + ((uint32_t)k * 2048u >> 4), id_o, !u.first || k > 0);
    if (u.last) umma_commit_by(leader, &bars->ofull[w]);
    return true;
  };

  Unit a, b, c;
  uint32_t wa = 0, wb = 0, wc = 0;
  bool has_a = units.next(p, a, wa) && issue_s(a, wa);
  bool has_b = has_a && units.next(p, b, wb) && issue_s(b, wb);
  while (has_a) {
    if (!issue_o(a, wa)) break;
    const bool has_c = has_b && units.next(p, c, wc) && issue_s(c, wc);
    a = b, wa = wb, has_a = has_b;
    b = c, wb = wc, has_b = has_c;
  }
  umma_commit_by(leader, &bars->drain);
  wait_bounded(&bars->drain, 0, drain_ctl_default(p.cache.err));
}

__device__ __forceinline__ float exp2_approx(float x) {
  float y;
  asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
  return y;
}
__device__ __forceinline__ uint32_t pack_bf16(float lo, float hi) {
  const __nv_bfloat162 v = __floats2bfloat162_rn(lo, hi);
  return *reinterpret_cast<const uint32_t*>(&v);
}

__device__ __forceinline__ uint64_t pack_f32x2(float lo, float hi) {
  uint64_t v;
  asm("mov.b64 %0, {%1, %2};" : "=l"(v) : "f"(lo), "f"(hi));
  return v;
}
__device__ __forceinline__ void unpack_f32x2(uint64_t v, float& lo, float& hi) {
  asm("mov.b64 {%0, %1}, %2;" : "=f"(lo), "=f"(hi) : "l"(v));
}
__device__ __forceinline__ uint64_t fma_f32x2(uint64_t a, uint64_t b, uint64_t c) {
  uint64_t d;
  asm("fma.rn.f32x2 %0, %1, %2, %3;" : "=l"(d) : "l"(a), "l"(b), "l"(c));
  return d;
}
__device__ __forceinline__ uint64_t add_f32x2(uint64_t a, uint64_t b) {
  uint64_t d;
  asm("add.rn.f32x2 %0, %1, %2;" : "=l"(d) : "l"(a), "l"(b));
  return d;
}
// Two probabilities (not negative) to BF16, to nearest with ties up: adds and a
// byte permute, as the conversion instruction shares the exponential's unit,
// which bounds the softmax.  A NaN is lost here but not in the row's sum, which
// every value of the row is divided by.
__device__ __forceinline__ uint32_t round_bf16x2(float lo, float hi) {
  return __byte_perm(__float_as_uint(lo) + 0x8000u, __float_as_uint(hi) + 0x8000u, 0x7632);
}

// A softmax team: thread r has row r of the team's rows.
template <int DIM>
__device__ void softmax_team(const AttentionParams& p, uint8_t* smem, Bars* bars, Walk walk,
                             const Ctl& ctl, uint32_t w) {
  using L = Layout<DIM>;
  const int r = threadIdx.x % kTeamThreads;
  const uint32_t lane_base = (uint32_t)(r & ~31) << 16;
  const uint32_t ts = bars->tmem + w * 128u + lane_base;         // S and P
  const uint32_t to = bars->tmem + 256u + w * 128u + lane_base;  // O
  const BatchView& b = p.batch;
  const int gq = p.heads / p.kv_heads;
  // Scores in units of log2; a negative scale turns Q's sign, which is exact, and
  // one of zero is replaced by one that leaves every finite score at zero (so that
  // masked scores of -inf stay what they are).
  const float c = fmaxf(fabsf(p.scale) * 1.4426950408889634f, 1e-38f);
  const uint32_t flip = p.scale < 0.f ? 0x80008000u : 0u;
  uint32_t turn = 0;       // this team's uses of tiles so far
  uint32_t done = 0;       // and its parts with at least one
  uint32_t uses = 0;       // both teams' uses so far
  uint32_t tiles = 0;      // tiles of the CTA so far
  Part part;
  bool more = walk.next(p, part);
  while (more) {
    // This thread's row: how many of the segment's tokens it sees.
    const int base = part.block * kPairRows + (part.both ? (int)w * kTeamRows : 0);
    const int team_rows = min(part.seg.rows - base, kTeamRows);
    const int first = part.both ? 0 : (int)((uses ^ w) & 1u);    // the team's first tile
    const int step = part.both ? 1 : 2;
    const int last = first + (part.n - 1 - first) / step * step;  // (when first < part.n)
    const bool zeroes = !part.both || w == (uses & 1u);          // the tile's first user
    const bool begins = first < part.n;
    const int per = b.chunk * gq;
    if (begins) {
      // Q's rows into the team's buffer: 16-byte pieces, 128-byte swizzle.  Rows
      // behind the last keep what is there: no row's result meets another's.
      constexpr int kPieces = DIM / 8, kStep = kTeamThreads / kPieces;
      const int piece = r % kPieces;
      const uint32_t dst = smem_u32(smem + L::kQOff + w * L::kTile) +
                           (uint32_t)(piece / 8) * (kTeamRows * 128u);
#pragma unroll 4
      for (int row = r / kPieces; row < team_rows; row += kStep) {
        const int sl = (base + row) / per, rest = base + row - sl * per, i = rest / gq;
        const uint4 v = reinterpret_cast<const uint4*>(
            static_cast<const uint16_t*>(p.q.data) +
            (int64_t)((part.seg.seq0 + sl) * b.chunk + i) * p.q.token_stride +
            (int64_t)(part.kvh * gq + rest - i * gq) * p.q.head_stride)[piece];
        sts128(dst + (uint32_t)row * 128u + (uint32_t)((piece % 8) ^ (row & 7)) * 16u, v.x ^ flip,
               v.y ^ flip, v.z ^ flip, v.w ^ flip);
      }
      fence_proxy_async_smem();
      tc_fence_before();
      mbar_arrive(&bars->qfull[w]);
    }
    int limit = 0;
    if (r < team_rows) {
      const int sl = (base + r) / per, i = (base + r - sl * per) / gq;
      const int seq = part.seg.seq0 + sl, fresh = fresh_of(b, seq);
      if (i < fresh)
        limit = part.seg.far ? part.seg.len
                             : min(max(max(b.lens[seq], 0) - fresh + i + 1, 0), part.seg.len);
    }
    Part next;
    more = walk.next(p, next);   // while the first scores are on their way
    float m = -INFINITY, l = 0.f;
    const bool warp_live = __any_sync(kAll, limit > 0);
    for (int t = first; t < part.n; t += step, ++turn) {
      const int t0 = (part.tile0 + t) * kKvTile;
      if (!__all_sync(kAll, wait(&bars->sfull[w], turn & 1u, ctl))) return;
      tc_fence_after();
      if (r == 0) {   // S is there: K has been read, and the V of the unit before
        mbar_arrive_n(&bars->empty[2 * (tiles + (uint32_t)t) % L::kRing], part.both ? 1 : 2);
        if (t != first)
          mbar_arrive_n(&bars->empty[(2 * (tiles + (uint32_t)(t - step)) + 1) % L::kRing],
                        part.both ? 1 : 2);
      }
      if (warp_live) {
        // Rows that are not there need no mask: nothing of theirs is read.
        const int cols = r < team_rows ? limit - t0 : kKvTile;
        const bool tail = __any_sync(kAll, cols < kKvTile);
        // The maximum first, then the scores once more for the exponentials, in
        // rolled halves: as straight code the two passes do not fit the
        // instruction cache, which cost a lone warp twice the time.
        float top[4] = {m, m, m, m};
#pragma unroll 1
        for (int h = 0; h < kKvTile; h += 64) {
          float x[64];
          tmem_load32(ts + (uint32_t)h, x);
          tmem_load32(ts + (uint32_t)h + 32u, x + 32);
          tmem_wait_load();
          tmem_tie<64>(x);
          if (tail) {
#pragma unroll
            for (int j = 0; j < 64; ++j) x[j] = j < cols - h ? x[j] : -INFINITY;
          }
#pragma unroll
          for (int j = 0; j < 64; j += 8)
#pragma unroll
            for (int k = 0; k < 4; ++k) top[k] = fmaxf(fmaxf(top[k], x[j + k]), x[j + k + 4]);
        }
        const float now = fmaxf(fmaxf(top[0], top[1]), fmaxf(top[2], top[3]));
        const bool grow = now > m && !((now - m) * c <= kLazy);
        if (__any_sync(kAll, grow)) {
          const float keep = m == -INFINITY ? 0.f : exp2_approx((m - now) * c);
          const float f = grow ? keep : 1.f;
          if (t != first) {
#pragma unroll 1
            for (int k = 0; k < DIM; k += 16) {
              float o[16];
              tmem_load<16>(to + (uint32_t)k, o);
              uint32_t u[16];
#pragma unroll
              for (int j = 0; j < 16; ++j) u[j] = __float_as_uint(o[j] * f);
              tmem_store16(to + (uint32_t)k, u);
            }
          }
          l *= f;
          if (grow) m = now;
        }
        const float shift = m == -INFINITY ? 0.f : m * c;
        const uint64_t c2 = pack_f32x2(c, c), shift2 = pack_f32x2(-shift, -shift);
        uint64_t sum[2] = {0, 0};
#pragma unroll 1
        for (int h = 0; h < kKvTile; h += 64) {
          float x[64];
          tmem_load32(ts + (uint32_t)h, x);
          tmem_load32(ts + (uint32_t)h + 32u, x + 32);
          tmem_wait_load();
          tmem_tie<64>(x);
          if (tail) {
#pragma unroll
            for (int j = 0; j < 64; ++j) x[j] = j < cols - h ? x[j] : -INFINITY;
          }
#pragma unroll
          for (int k = 0; k < 2; ++k) {
            uint32_t u[16];
#pragma unroll
            for (int j = 0; j < 16; ++j) {
              float a, d;
              unpack_f32x2(
                  fma_f32x2(pack_f32x2(x[32 * k + 2 * j], x[32 * k + 2 * j + 1]), c2, shift2), a,
                  d);
              a = exp2_approx(a);
              d = exp2_approx(d);
              sum[j & 1] = add_f32x2(sum[j & 1], pack_f32x2(a, d));
              u[j] = round_bf16x2(a, d);
            }
            // P over S: columns h / 2 .. h / 2 + 31, whose scores have been read.
            tmem_store16(ts + (uint32_t)h / 2 + 16u * k, u);
          }
        }
        float s0, s1;
        unpack_f32x2(add_f32x2(sum[0], sum[1]), s0, s1);
        l += s0 + s1;
        tmem_wait_store();
      }
      // Tokens behind the segment's last: whatever the pages hold there, V is zero.
      const int there = part.seg.len - t0;
      if (there < kKvTile && zeroes) {
        const uint32_t seq = 2 * (tiles + (uint32_t)t) + 1, slot = seq % L::kRing;
        if (!__all_sync(kAll, wait(&bars->full[slot], (seq / L::kRing) & 1u, ctl))) return;
        const uint32_t v = smem_u32(smem + L::kRingOff + slot * L::kTile);
        const int pieces = (kKvTile - there) * 8;
        for (int k = r; k < pieces; k += kTeamThreads)
#pragma unroll
          for (int h = 0; h < DIM / 64; ++h)
            sts128(v + (uint32_t)(h * kKvTile + there) * 128u + (uint32_t)k * 16u, 0, 0, 0, 0);
        fence_proxy_async_smem();
      }
      tc_fence_before();
      mbar_arrive(&bars->pfull[w]);
    }
    // The part's results.
    const int64_t slot = slot_of(p, part.s, part.item, (int)blockIdx.x, (int)w);
    const int slot_rows = part.seg.far ? kTeamRows : p.ws.own_rows;
    const bool room = slot < (part.seg.far ? p.ws.far_slots : p.ws.own_slots);
    const bool writes = r < team_rows && room;
    float* o_at = reinterpret_cast<float*>(p.workspace +
                                           (part.seg.far ? p.ws.far_o : p.ws.own_o)) +
                  (slot * slot_rows + r) * DIM;
    if (writes)
      reinterpret_cast<float2*>(p.workspace + (part.seg.far ? p.ws.far_ml : p.ws.own_ml))
          [slot * slot_rows + r] = make_float2(m * c, l);
    if (begins) {
      if (!__all_sync(kAll, wait(&bars->ofull[w], done++ & 1u, ctl))) return;
      tc_fence_after();
      if (r == 0)
        mbar_arrive_n(&bars->empty[(2 * (tiles + (uint32_t)last) + 1) % L::kRing],
                      part.both ? 1 : 2);
      if (warp_live) {
#pragma unroll 1
        for (int k = 0; k < DIM; k += 32) {
          float o[32];
          tmem_load32(to + (uint32_t)k, o);
          tmem_wait_load();
          tmem_tie<32>(o);
          if (writes) {
#pragma unroll
            for (int j = 0; j < 8; ++j)
              reinterpret_cast<float4*>(o_at + k)[j] =
                  make_float4(o[4 * j], o[4 * j + 1], o[4 * j + 2], o[4 * j + 3]);
          }
        }
      }
      tc_fence_before();
    }
    if (!room && r == 0) atomicOr(p.cache.err, kErrRange);
    uses += (uint32_t)(part.both ? 2 * part.n : part.n);
    tiles += (uint32_t)part.n;
    part = next;
  }
}

// First tile and first item of every segment, by a scan of the whole CTA; finds
// this CTA's share.  CTA 0 writes them down for the kernel that joins the parts.
__device__ Walk share_out(const AttentionParams& p, Bars* bars) {
  const int segments = p.batch.groups + p.batch.sequences;
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  int64_t* starts = reinterpret_cast<int64_t*>(p.workspace + p.ws.starts);
  int32_t* items = reinterpret_cast<int32_t*>(p.workspace + p.ws.items);
  int64_t run = 0, mine = 0, mine_flat = 0;
  int32_t run_items = 0;
  auto scan = [&](int base, int64_t& before, int64_t& flat, int32_t& before_items) {
    const int s = base + (int)threadIdx.x;
    int32_t n = 0;
    flat = 0;
    if (s < segments) {
      const Segment g = segment(p, s);
      flat = (int64_t)g.tiles * g.items;
      n = g.items;
    }
    int64_t f = flat;
    int32_t m = n;
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
      const int64_t f2 = __shfl_up_sync(kAll, f, o);
      const int32_t m2 = __shfl_up_sync(kAll, m, o);
      if (lane >= o) f += f2, m += m2;
    }
    __syncthreads();
    if (lane == 31) bars->warp_flat[warp] = f, bars->warp_items[warp] = m;
    __syncthreads();
    int64_t all = 0, low = 0;
    int32_t all_items = 0, low_items = 0;
#pragma unroll
    for (int k = 0; k < kThreads / 32; ++k) {
      if (k == warp) low = all, low_items = all_items;
      all += bars->warp_flat[k];
      all_items += bars->warp_items[k];
    }
    before = run + low + f - flat;
    before_items = run_items + low_items + m - n;
    run += all;
    run_items += all_items;
  };
  for (int base = 0; base < segments; base += kThreads) {
    int32_t mine_items;
    scan(base, mine, mine_flat, mine_items);
    const int s = base + (int)threadIdx.x;
    if (s < segments) {
      // Every CTA needs its prefixes' first items for its slots: all write the
      // same values.
      if (s < p.batch.groups) items[s] = mine_items;
      if (blockIdx.x == 0) {
        starts[s] = mine;
        const bool over = s < p.batch.groups
                              ? p.batch.prefix_lens[s] > far_len(p, s) && p.batch.prefix_lens[s] > 0
                              : p.batch.lens[s - p.batch.groups] > 0 &&
                                    p.batch.lens[s - p.batch.groups] >
                                        own_len(p, s - p.batch.groups);
        if (over) atomicOr(p.cache.err, kErrRange);
      }
    }
  }
  const int64_t total = run;
  if (blockIdx.x == 0 && threadIdx.x == 0) starts[segments] = total;
  const int ctas = sharers(p, total);
  Walk walk;
  walk.s = 0;
  walk.off = walk.left = 0;
  if ((int)blockIdx.x >= ctas || total == 0) return walk;
  const int64_t f0 = first_tile(total, (int)blockIdx.x, ctas);
  const int64_t f1 = first_tile(total, (int)blockIdx.x + 1, ctas);
  if (segments <= kThreads) {
    if (mine <= f0 && f0 < mine + mine_flat) bars->seg = (int)threadIdx.x, bars->off = f0 - mine;
  } else {
    run = 0;
    run_items = 0;
    for (int base = 0; base < segments && run <= f0; base += kThreads) {
      int32_t unused;
      scan(base, mine, mine_flat, unused);
      if (mine <= f0 && f0 < mine + mine_flat)
        bars->seg = base + (int)threadIdx.x, bars->off = f0 - mine;
    }
  }
  __syncthreads();
  walk.s = bars->seg;
  walk.off = bars->off;
  walk.left = f1 - f0;
  return walk;
}

template <int DIM>
__global__ void __launch_bounds__(kThreads, 1)
    attention_kernel(const __grid_constant__ AttentionParams p,
                     const __grid_constant__ CUtensorMap k_map,
                     const __grid_constant__ CUtensorMap v_map) {
  extern __shared__ __align__(1024) uint8_t smem_attention[];
  uint8_t* smem = smem_attention;
  using L = Layout<DIM>;
  allow_dependents();
  if (smem_u32(smem) & 1023u) {  // the swizzled tiles need 1024-byte alignment
    if (threadIdx.x == 0) atomicOr(p.cache.err, kErrLayout);
    return;
  }
  Bars* bars = reinterpret_cast<Bars*>(smem + L::kBarOff);
  const int warp = threadIdx.x >> 5;
  if (threadIdx.x == 0) {
    for (int k = 0; k < L::kRing; ++k) {
      mbar_init(&bars->full[k], 1);
      mbar_init(&bars->empty[k], 2);
    }
    for (int w = 0; w < 2; ++w) {
      mbar_init(&bars->qfull[w], kTeamThreads);
      mbar_init(&bars->sfull[w], 1);
      mbar_init(&bars->pfull[w], kTeamThreads);
      mbar_init(&bars->ofull[w], 1);
    }
    mbar_init(&bars->drain, 1);
    bars->abort = 0u;
  }
  if (warp == kIssuerWarp) {
    asm volatile("tcgen05.alloc.cta_group::1.sync.aligned.shared::cta.b32 [%0], 512;" ::"r"(
        smem_u32(&bars->tmem)));
    asm volatile("tcgen05.relinquish_alloc_permit.cta_group::1.sync.aligned;" ::: "memory");
  }
  fence_barrier_init();
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  wait_prerequisites();
  const Walk walk = share_out(p, bars);
  const Ctl ctl{p.cache.err, p.wait_limit ? p.wait_limit : kDefaultWaitLimit, &bars->abort};
  if (warp < 8) {
    softmax_team<DIM>(p, smem, bars, walk, ctl, (uint32_t)(warp >> 2));
  } else if (warp == kProducerWarp) {
    produce_kv<DIM>(p, &k_map, &v_map, smem, bars, walk, ctl);
  } else {
    issue_products<DIM>(p, smem, bars, walk, ctl);
  }
  __syncwarp();
  tc_fence_before();
  __syncthreads();
  if (warp == kIssuerWarp)
    asm volatile("tcgen05.dealloc.cta_group::1.sync.aligned.b32 %0, 512;" ::"r"(bars->tmem));
}

// ---- joining the parts ------------------------------------------------------------

constexpr int kJoinWarps = 4;

// One warp a row and query head: over the parts of its prefix and its own tokens,
// out = sum 2^(m_i - M) O_i / sum 2^(m_i - M) l_i, in order.
template <int DIM>
__global__ void __launch_bounds__(kJoinWarps * 32)
    join_kernel(const __grid_constant__ AttentionParams p) {
  constexpr int E = DIM / 32;
  allow_dependents();
  const int lane = threadIdx.x & 31;
  const int64_t id = (int64_t)blockIdx.x * kJoinWarps + (threadIdx.x >> 5);
  const BatchView& b = p.batch;
  const int64_t rows = (int64_t)b.sequences * b.chunk;
  if (id >= rows * p.heads) return;
  const int token = (int)(id / p.heads), head = (int)(id - (int64_t)token * p.heads);
  const int seq = token / b.chunk, i = token - seq * b.chunk;
  const int gq = p.heads / p.kv_heads, kvh = head / gq, h = head - kvh * gq;
  wait_prerequisites();
  const int64_t* starts = reinterpret_cast<const int64_t*>(p.workspace + p.ws.starts);
  const int segments = b.groups + b.sequences;
  const int64_t total = starts[segments];
  const int ctas = sharers(p, total);
  int group = -1;
  for (int g0 = 0; g0 < b.groups; g0 += 32) {
    const int g = g0 + lane;
    const bool in = g < b.groups && b.group_start[g] <= seq && seq < b.group_start[g + 1];
    const unsigned hit = __ballot_sync(kAll, in);
    if (hit) {
      group = g0 + __ffs(hit) - 1;
      break;
    }
  }
  float top = -INFINITY, sum = 0.f, acc[E];
#pragma unroll
  for (int e = 0; e < E; ++e) acc[e] = 0.f;
  const bool real = i < fresh_of(b, seq);
  for (int side = 0; real && side < 2; ++side) {
    const int s = side == 0 ? group : b.groups + seq;
    if (s < 0) continue;
    const Segment seg = segment(p, s);
    if (seg.tiles == 0) continue;
    const int row = ((seq - seg.seq0) * b.chunk + i) * gq + h;
    const int block = row / kPairRows, in_block = row - block * kPairRows;
    const bool both = min(seg.rows - block * kPairRows, kPairRows) > kTeamRows;
    const int item = block * p.kv_heads + kvh;
    const int64_t t0 = starts[s] + (int64_t)item * seg.tiles;
    const int c0 = owner(total, t0, ctas), c1 = owner(total, t0 + seg.tiles - 1, ctas);
    const int teams = both ? 1 : 2, team0 = both ? in_block / kTeamRows : 0;
    const int slot_rows = seg.far ? kTeamRows : p.ws.own_rows;
    const int64_t slots = seg.far ? p.ws.far_slots : p.ws.own_slots;
    const float2* ml =
        reinterpret_cast<const float2*>(p.workspace + (seg.far ? p.ws.far_ml : p.ws.own_ml));
    const float* o =
        reinterpret_cast<const float*>(p.workspace + (seg.far ? p.ws.far_o : p.ws.own_o));
    const int at = both ? in_block - team0 * kTeamRows : in_block;
    const int parts = (c1 - c0 + 1) * teams;
    for (int k0 = 0; k0 < parts; k0 += 32) {
      const int k = k0 + lane;
      float2 v = make_float2(-INFINITY, 0.f);
      int64_t place = 0;
      if (k < parts) {
        const int64_t slot =
            slot_of(p, s, item, c0 + k / teams, both ? team0 : k - k / teams * teams);
        place = slot * slot_rows + at;
        if (slot < slots) v = ml[place];
      }
      float t = v.x;
#pragma unroll
      for (int d = 16; d > 0; d >>= 1) t = fmaxf(t, __shfl_xor_sync(kAll, t, d));
      const float now = fmaxf(top, t);
      const float base = now == -INFINITY ? 0.f : now;
      const float keep = exp2f(top - base);
      sum *= keep;
#pragma unroll
      for (int e = 0; e < E; ++e) acc[e] *= keep;
      top = now;
      // A part without weight is not read (its values were not written).
      const float f = v.y != 0.f ? exp2f(v.x - base) : 0.f;
      unsigned live = __ballot_sync(kAll, v.y != 0.f);
      while (live) {
        const int j = __ffs(live) - 1;
        live &= live - 1;
        const float fj = __shfl_sync(kAll, f, j);
        sum += fj * __shfl_sync(kAll, v.y, j);
        const int64_t pj = __shfl_sync(kAll, place, j);
        const float* src = o + pj * DIM + lane * E;
        if (E == 4) {
          const float4 x = *reinterpret_cast<const float4*>(src);
          acc[0] += fj * x.x, acc[1] += fj * x.y, acc[2 % E] += fj * x.z, acc[3 % E] += fj * x.w;
        } else {
          const float2 x = *reinterpret_cast<const float2*>(src);
          acc[0] += fj * x.x, acc[1] += fj * x.y;
        }
      }
    }
  }
  const float inv = sum != 0.f ? 1.f / sum : 0.f;
  uint16_t* out = static_cast<uint16_t*>(p.out.data) + (int64_t)token * p.out.token_stride +
                  (int64_t)head * p.out.head_stride + lane * E;
#pragma unroll
  for (int e = 0; e < E; e += 2)
    *reinterpret_cast<uint32_t*>(out + e) = pack_bf16(acc[e] * inv, acc[e + 1] * inv);
  if (p.lse && lane == 0)
    p.lse[id] = sum != 0.f ? (top + log2f(sum)) * 0.69314718055994531f : -INFINITY;
}

template <int DIM>
cudaError_t launch_dim(const AttentionParams& p, const CUtensorMap& k_map,
                       const CUtensorMap& v_map, cudaStream_t stream) {
  static bool configured[64] = {};
  int dev = 0;
  cudaError_t e = cudaGetDevice(&dev);
  if (e != cudaSuccess) return e;
  if (dev < 0 || dev >= 64) return cudaErrorInvalidDevice;
  if (!configured[dev]) {
    e = cudaFuncSetAttribute(attention_kernel<DIM>, cudaFuncAttributeMaxDynamicSharedMemorySize,
                             (int)Layout<DIM>::kBytes);
    if (e != cudaSuccess) return e;
    configured[dev] = true;
  }
  const int64_t warps = (int64_t)p.batch.sequences * p.batch.chunk * p.heads;
  const int64_t blocks = (warps + kJoinWarps - 1) / kJoinWarps;
  if (blocks > 0x7FFFFFFF) return cudaErrorInvalidValue;
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3((unsigned)p.ctas);
  cfg.blockDim = dim3(kThreads);
  cfg.dynamicSmemBytes = Layout<DIM>::kBytes;
  cfg.stream = stream;
  cudaLaunchAttribute attr[1];
  attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[0].val.programmaticStreamSerializationAllowed = 1;
  cfg.attrs = attr;
  cfg.numAttrs = 1;
  e = cudaLaunchKernelEx(&cfg, attention_kernel<DIM>, p, k_map, v_map);
  if (e != cudaSuccess) return e;
  cfg.gridDim = dim3((unsigned)blocks);
  cfg.blockDim = dim3(kJoinWarps * 32);
  cfg.dynamicSmemBytes = 0;
  return cudaLaunchKernelEx(&cfg, join_kernel<DIM>, p);
}

uint64_t up256(uint64_t x) { return (x + 255) & ~255ull; }

}  // namespace

AttentionWorkspace attention_workspace(int sequences, int chunk, int groups, int heads,
                                       int kv_heads, int dim, int ctas) {
  AttentionWorkspace w;
  const int64_t seq_rows = (int64_t)chunk * (heads / kv_heads);
  const int64_t far_items =
      groups ? ((seq_rows * sequences + kPairRows - 1) / kPairRows + groups) * kv_heads : 0;
  w.own_rows = (int32_t)(seq_rows < kTeamRows ? seq_rows : kTeamRows);
  w.own_items = (int32_t)((seq_rows + kPairRows - 1) / kPairRows * kv_heads);
  w.far_slots = groups ? 2 * (far_items + ctas) : 0;
  w.own_slots = 2 * ((int64_t)sequences * w.own_items + ctas);
  uint64_t at = 0;
  auto take = [&](uint64_t bytes) {
    const uint64_t here = at;
    at += up256(bytes);
    return here;
  };
  w.starts = take(8ull * ((uint64_t)groups + sequences + 1));
  w.items = take(4ull * ((uint64_t)groups + 1));
  w.far_ml = take(8ull * w.far_slots * kTeamRows);
  w.far_o = take(4ull * w.far_slots * kTeamRows * dim);
  w.own_ml = take(8ull * w.own_slots * w.own_rows);
  w.own_o = take(4ull * w.own_slots * w.own_rows * dim);
  w.bytes = at;
  return w;
}

cudaError_t launch_attention(const AttentionParams& p, const CUtensorMap& k_map,
                             const CUtensorMap& v_map, cudaStream_t stream) {
  return p.dim == 64 ? launch_dim<64>(p, k_map, v_map, stream)
                     : launch_dim<128>(p, k_map, v_map, stream);
}

}  // namespace nwc
