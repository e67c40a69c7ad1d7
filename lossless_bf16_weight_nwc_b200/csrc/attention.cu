// attention.cu — attention of a batch's new tokens over a paged cache, with
// prefixes that several sequences share.
//
// out = sum_j e^(s_j - m) v_j / sum_j e^(s_j - m), s_j = scale q . k_j, over the
// row's prefix and its own tokens, in one pass with the running maximum m.
//
// A decode batch reads each K and V once and multiplies it with few rows: what
// bounds it is memory, so the key axis is cut into equal shares for all SMs.  One
// persistent CTA an SM:
//   * a producer warp works out the CTA's parts, announces each to the others
//     through a short queue in shared memory, and brings its K and V tiles page by
//     page with TMA into a ring;
//   * where more than 16 rows share the tokens (a prefix's group, times the query
//     heads of a key head; a chunk), one warp issues S = Q K^T and O += P V
//     (tcgen05, 128 rows x 128 tokens), with S, P and O in TMEM: P takes S's place
//     as BF16 and is the A operand.  Two teams of 128 softmax threads, a row each:
//     a team has its own 128 rows when a block has more than 128 (both then use each
//     tile), else the teams take the tiles in turn, so that one team's exponentials
//     run under the other's products;
//   * with up to 16 rows those threads multiply themselves (few_part).
// The maximum that scales P follows the running one only when that has grown by
// more than 2^8, so O is rarely rescaled; P stays below 2^8 and the sums are FP32.
// A second kernel joins the parts' results in a fixed order.
//
// B200, 32 query heads over 8 key heads of 128: 64 sequences of 100 to 1900 own tokens
// behind 32768 shared ones take 91 us in a burst (406 MB, 4.5 TB/s, 0.68 of a copy's
// rate), 97 to 100 in loops that last, where the power cap lowers the clock; the 64
// without a prefix 52 us (0.67), of 2000 to 6000 tokens each 174 us (0.96); 64 rows of
// one sequence over 16400 tokens 41 us (420 TFLOP/s): 13 us of a start, Q and results
// around 7 tiles a CTA; one row over 1003 tokens 12 us, of which 4 in the second kernel.
// A prompt taken in one call also multiplies the tiles that its rows do not see (4096
// rows: 557 us, 247 TFLOP/s of what they see).
#include <cuda_bf16.h>
#include <cuda_runtime.h>

#include <atomic>
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
constexpr int kQueue = 5;                // parts announced ahead
constexpr uint32_t kRingBytes = 163840;  // K and V tiles: 5 of dim 128, 10 of dim 64
constexpr uint32_t kBarBytes = 3 * 1024;
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

enum Kind : int32_t { kFew, kOne, kBoth };  // rows: the segment <= kFewRows; <= kTeamRows; more

// A part as the producer announces it.
struct Part {
  int32_t n;       // tiles, 0: no more parts
  int32_t kind;
  int32_t far;     // of a prefix
  int32_t seq0;    // first sequence of the segment
  int32_t len;     // tokens of the segment
  int32_t rows;    // of the block
  int32_t base;    // first row of the block
  int32_t kvh;     // key head, or the first of kFew's
  int32_t tile0;   // tiles [tile0, tile0 + n) of the segment
  int64_t place;   // first row of its results; negative: none
  int32_t* spans;  // its item's first and last CTA
  bool first, last;  // whether this is the one
};
struct Announced {
  Part part;
  int32_t limit[kFewRows];  // kFew: tokens of the segment that each row sees
  int64_t q[kFewRows];      // and where its Q is (elements)
};

struct Bars {
  uint64_t full[kMaxRing];   // a tile's bytes landed
  uint64_t empty[kMaxRing];  // the tile has been read (8 arrivals, one a softmax warp)
  uint64_t told[kQueue];     // a part is announced
  uint64_t heard[kQueue];    // all have read it (9 arrivals: the softmax warps, the issuer)
  uint64_t qfull[2];         // the team's Q is in place
  uint64_t sfull[2];         // the team's S is in TMEM (and its P V before that is done)
  uint64_t pfull[2];         // the team's P is in TMEM (and V's tail is zeroed)
  uint64_t ofull[2];         // the last P V of the team's part is done
  uint64_t team[2];          // the team's warps meet
  uint64_t drain;
  uint32_t tmem;
  uint32_t abort;
  float2 ml[2][4][kFewRows]; // maximum and sum of each warp's rows in a part of few rows
  Announced queue[kQueue];
};
static_assert(sizeof(Bars) <= kBarBytes, "barriers");

constexpr int64_t kMaxTokens = 1ll << 30;  // of a segment: indexes stay in 31 bits

// ---- segments, items and parts ---------------------------------------------

struct Segment {
  int seq0;    // first sequence
  int rows;    // rows (token x query head of a key head)
  int len;     // tokens
  int tiles;
  int items;
  bool few;    // at most kFewRows rows
  Kind kind;   // of its first block of rows
  int cost;    // of a tile on the axis that is shared out
  int lead;    // of an item's start
  bool far;    // a prefix
};

// What a tile costs by the kind of its segment, and what each item adds at its start
// (a part's end and the next one's beginning), in units of about 400 cycles: fitted
// to the times of CTAs with different parts.  (Selects: a table would be a load.)
constexpr int kCostMost = 10;
__device__ __forceinline__ int cost_of(Kind kind, bool wide) {
  return kind == kFew ? (wide ? 4 : 3) : kind == kOne ? (wide ? 9 : 6) : (wide ? 10 : 9);
}
__device__ __forceinline__ int lead_of(Kind kind, bool wide) {
  return kind == kFew ? (wide ? 9 : 8) : kind == kOne ? (wide ? 8 : 7) : (wide ? 33 : 14);
}

__device__ __forceinline__ int fresh_of(const BatchView& b, int seq) {
  return b.q_lens ? min(max(b.q_lens[seq], 0), b.chunk) : b.chunk;
}
__device__ __forceinline__ int capped(const AttentionParams& p, int len, int width) {
  const int64_t cap = min((int64_t)width << p.cache.page_shift, kMaxTokens);
  return (int)min((int64_t)max(len, 0), cap);
}

// What the tables say of segment s.
struct Raw {
  int len, first, end;   // first sequence of a prefix and the one behind its last; or
                         // 0 and the sequence's new tokens
};
// dry: made up, nothing is read.
__device__ __forceinline__ Raw raw_segment(const BatchView& b, int s, bool in, bool dry) {
  const bool far = s < b.groups;
  const int seq = far ? 0 : s - b.groups;
  Raw r;
  r.len = in && dry ? 3 * kKvTile : 0;
  r.first = 0;
  r.end = 1;
  in = in && !dry;
  if (in) r.len = *(far ? b.prefix_lens + s : b.lens + seq);
  if (in && far) r.first = b.group_start[s];
  if (in && (far || b.q_lens)) r.end = *(far ? b.group_start + s + 1 : b.q_lens + seq);
  return r;
}
// cap: the most that an item's lead may cost; negative: every tile costs 1 and a
// lead nothing.  (No divisions or branches here: a part's announcement is on the way
// to its first byte.)
__device__ __forceinline__ void price(const AttentionParams& p, Segment& g, int cap) {
  g.cost = cap < 0 ? 1 : cost_of(g.kind, p.dim == 128);
  g.lead = cap < 0 ? 0 : min(lead_of(g.kind, p.dim == 128), cap);
}
__device__ __forceinline__ Segment segment_of(const AttentionParams& p, int s, const Raw& raw) {
  const BatchView& b = p.batch;
  Segment r;
  r.far = s < b.groups;
  const int first = min(max(raw.first, 0), b.sequences);
  const int end = min(max(raw.end, first), b.sequences);
  r.seq0 = r.far ? first : s - b.groups;
  r.rows = r.far ? (end - first) * p.seq_rows : p.seq_rows;
  r.len = capped(p, raw.len, r.far ? b.prefix_width : b.table_width);
  if (r.far ? r.rows == 0 : raw.end <= 0) r.len = 0;
  r.few = r.rows <= kFewRows;
  r.kind = r.few ? kFew : r.rows <= kTeamRows ? kOne : kBoth;
  const int shift = r.few ? p.few_shift : kKvShift;
  r.tiles = (int)(((uint32_t)r.len + (1u << shift) - 1) >> shift);
  r.items = r.few ? (r.rows > 0 ? p.few_items : 0)
                  : (r.rows + kPairRows - 1) / kPairRows * p.kv_heads;
  r.cost = r.lead = 0;
  return r;
}
// The tiles lie on an axis of costs; of the CTAs that share it, c has those that start in
// [share(c), share(c + 1)).  (Divisions of 64 bits are long: 32 where they do.)
__device__ __forceinline__ int64_t divide(int64_t a, int64_t b) {
  return ((a | b) >> 32) == 0 ? (int64_t)((uint32_t)a / (uint32_t)b) : a / b;
}
__device__ __forceinline__ int64_t share(int64_t total, int c, int ctas) {
  return divide(total * c, ctas);
}

// The first and last CTA of an item (counted over the prefixes' or over the own).
__device__ __forceinline__ int32_t* spans_of(const AttentionParams& p, int s, int64_t item) {
  return reinterpret_cast<int32_t*>(p.workspace +
                                    (s < p.batch.groups ? p.ws.far_spans : p.ws.own_spans)) +
         2 * item;
}

// A segment's items on the axis: each a lead, then its tiles.
__device__ __forceinline__ int64_t item_span(const Segment& g) {
  return g.tiles ? g.lead + (int64_t)g.tiles * g.cost : 0;
}
// The first tile that starts at or behind `at` (>= 0) of its part of the axis: item and
// tile of the item.
struct At {
  int item, tile;
};
__device__ __forceinline__ At tile_from(const Segment& g, int64_t at) {
  const int64_t span = item_span(g), item = divide(at, span), in = at - item * span - g.lead;
  At r;
  r.item = (int)item;
  r.tile = in > 0 ? (int)divide(in + g.cost - 1, g.cost) : 0;
  return r;   // r.tile may be g.tiles: the item has none behind `at`
}

// The parts of a CTA in order: those of the tiles that start in [from, to) of the
// axis, from segment s, which starts at `start`.
struct Walk {
  int s, cap;
  int64_t start, from, to;
  int64_t item0;     // the segment's first item, counted over the prefixes' or the own
  bool open;         // the segment has been looked up
  Segment g;
  At at, end;        // its tiles left
  bool dry;          // a rehearsal: see raw_segment
  __device__ __forceinline__ bool next(const AttentionParams& p, Part& part) {
    const int segments = p.batch.groups + p.batch.sequences;
    for (;;) {
      if (!open) {
        if (s >= segments || start >= to) return false;
        g = segment_of(p, s, raw_segment(p.batch, s, true, dry));
        price(p, g, cap);
        at.item = at.tile = 0;
        end.item = g.tiles ? g.items : 0;
        end.tile = 0;
        const int64_t span = item_span(g) * g.items;
        if (span > 0 && from > start) at = tile_from(g, from - start);
        if (span > 0 && to - start < span) end = tile_from(g, to - start);
        start += span;
        open = true;
      }
      if (at.tile >= g.tiles) ++at.item, at.tile = 0;
      if (g.tiles && (at.item < end.item || (at.item == end.item && at.tile < end.tile))) break;
      open = false;
      item0 = ++s == p.batch.groups ? 0 : item0 + g.items;
    }
    part.tile0 = at.tile;
    part.n = (at.item == end.item ? end.tile : g.tiles) - at.tile;
    const int block = g.few || at.item < p.kv_heads ? 0 : at.item / p.kv_heads;
    part.kvh = g.few ? at.item * p.few_heads : at.item - block * p.kv_heads;
    part.base = block * kPairRows;
    part.rows = min(g.rows - part.base, kPairRows);
    part.kind = g.few ? kFew : part.rows <= kTeamRows ? kOne : kBoth;
    part.far = g.far;
    part.seq0 = g.seq0;
    part.len = g.len;
    // The slot of its results: item + CTA is different for any two parts, as each
    // next part has a later item, a later CTA or both.
    const int64_t item = item0 + at.item, slot = item + blockIdx.x;
    const bool room = item < (g.far ? p.ws.far_slots : p.ws.own_slots) - p.ctas;
    part.place = room ? slot * (g.far ? kPairRows : p.ws.own_rows) : -1;
    part.spans = spans_of(p, s, item);
    part.first = part.tile0 == 0;
    part.last = part.tile0 + part.n == g.tiles;
    at.tile += part.n;
    return true;
  }
};

// ---- waits -------------------------------------------------------------------

struct Ctl {
  uint32_t* err;
  uint32_t limit;
  bool test;   // a limit set by a test: polls that do not themselves wait
  volatile uint32_t* abort;
};
// False (and every role leaves) when a wait gave up here or elsewhere.
__device__ __noinline__ bool wait_on(uint64_t* bar, uint32_t parity, const Ctl& c) {
  for (uint32_t it = 0; it < c.limit; ++it) {
    if (c.test ? mbar_test_wait(bar, parity) : mbar_try_wait(bar, parity)) return true;
    if (*c.abort) return false;
  }
  *c.abort = 1u;
  atomicOr(c.err, kErrTimeout);
  return false;
}
__device__ __forceinline__ bool wait(uint64_t* bar, uint32_t parity, const Ctl& c) {
  return (!c.test && mbar_try_wait(bar, parity)) || wait_on(bar, parity, c);
}

// ---- roles ---------------------------------------------------------------------

// The row of a part's block: which sequence, token and query head, and how many
// of the segment's tokens it sees (0: padding).
struct Row {
  int64_t q;   // where its Q is (elements)
  int limit;
};
__device__ __forceinline__ Row row_of(const AttentionParams& p, const Part& part, int r) {
  const BatchView& b = p.batch;
  const int at = part.base + r;
  const int sl = at / p.seq_rows, rest = at - sl * p.seq_rows, i = rest / p.gq;
  const int seq = part.seq0 + sl, fresh = fresh_of(b, seq);
  Row row;
  row.q = (int64_t)(seq * b.chunk + i) * p.q.token_stride +
          (int64_t)(part.kvh * p.gq + rest - i * p.gq) * p.q.head_stride;
  row.limit = 0;
  if (i < fresh)
    row.limit =
        part.far ? part.len : min(max(max(b.lens[seq], 0) - fresh + i + 1, 0), part.len);
  return row;
}

// A sum over the warp of values below 2^52.
__device__ __forceinline__ int64_t warp_sum(int64_t v) {
  const uint32_t lo = __reduce_add_sync(kAll, (uint32_t)v & 0x3FFFFFFu);
  const uint32_t hi = __reduce_add_sync(kAll, (uint32_t)(v >> 26));
  return ((int64_t)hi << 26) + lo;
}

// Where this CTA's share of the axis starts: the producer warp sums the segments,
// up to four consecutive ones a lane, for the totals, then for the segment in which the
// share starts (from registers where there are up to 128).  Of an item's CTAs none
// may be without a tile (the join counts on it), so a share is at least as long as
// the widest gap between two tiles' starts, the most that a tile costs plus a lead:
// leads are capped for it, and where that leaves none every tile costs 1.
__device__ __forceinline__ Walk share_out(const AttentionParams& p, bool dry) {
  const BatchView& b = p.batch;
  const int segments = b.groups + b.sequences;
  const int lane = threadIdx.x & 31;
  const int per = min((segments + 31) / 32, 4);   // segments of a lane
  const int chunks = dry ? 1 : (segments + 127) / 128;
  Segment g[4];
  auto take = [&](int s0) {
    Raw raw[4];
#pragma unroll
    for (int j = 0; j < 4; ++j)
      if (j < per) raw[j] = raw_segment(b, s0 + j, s0 + j < segments, dry);
#pragma unroll
    for (int j = 0; j < 4; ++j) {
      if (j < per) g[j] = segment_of(p, s0 + j, raw[j]);
      if (j >= per || s0 + j >= segments) {
        g[j].tiles = g[j].items = g[j].cost = g[j].lead = 0;
        g[j].kind = kFew;
      }
    }
  };
  int64_t tiles = 0, cost = 0;
  int of_kind[3] = {0, 0, 0};   // items of each kind
#pragma unroll 1
  for (int t = 0; t < chunks; ++t) {
    take(t * 128 + per * lane);
#pragma unroll
    for (int j = 0; j < 4; ++j) {
      if (j >= per) break;
      const int64_t all = (int64_t)g[j].tiles * g[j].items;
      tiles += all;
      cost += all * cost_of(g[j].kind, p.dim == 128);
#pragma unroll
      for (int k = 0; k < 3; ++k) of_kind[k] += all > 0 && g[j].kind == k ? g[j].items : 0;
    }
  }
  tiles = warp_sum(tiles);
  cost = warp_sum(cost);
#pragma unroll
  for (int k = 0; k < 3; ++k) of_kind[k] = __reduce_add_sync(kAll, of_kind[k]);
  Walk walk;
  const int64_t each = divide(cost, p.ctas) - kCostMost;
  walk.cap = each < 0 ? -1 : (int)min(each, (int64_t)1024);
  int64_t total = walk.cap < 0 ? tiles : cost;
#pragma unroll
  for (int k = 0; k < 3; ++k)
    total += walk.cap < 0
                 ? 0
                 : (int64_t)of_kind[k] * min(lead_of((Kind)k, p.dim == 128), walk.cap);
  const int ctas = (int)min((int64_t)p.ctas, max(total, (int64_t)1));
  const int c = (int)blockIdx.x;
  walk.from = c < ctas ? share(total, c, ctas) : total;
  walk.to = c < ctas ? share(total, c + 1, ctas) : total;
  walk.s = segments;
  walk.start = walk.item0 = 0;
  walk.open = false;
  walk.dry = dry;
  int64_t run = 0;
  int32_t run_items = 0;
#pragma unroll 1
  for (int t = 0; t < chunks && run <= walk.from; ++t) {
    const int s0 = t * 128 + per * lane;
    if (chunks > 1) take(s0);
    int64_t span[4], sum = 0;
    int32_t n = 0;
#pragma unroll
    for (int j = 0; j < 4; ++j) {
      span[j] = 0;
      if (j >= per) break;
      price(p, g[j], walk.cap);
      span[j] = item_span(g[j]) * g[j].items;
      sum += span[j];
      n += g[j].items;
    }
    int64_t at = sum;
    int32_t item0 = n;
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
      const int64_t a = __shfl_up_sync(kAll, at, o);
      const int32_t e = __shfl_up_sync(kAll, item0, o);
      if (lane >= o) at += a, item0 += e;
    }
    const int64_t chunk = __shfl_sync(kAll, at, 31);
    const int32_t chunk_items = __shfl_sync(kAll, item0, 31);
    at += run - sum;
    item0 += run_items - n;
    int mine = -1;
    int64_t start = 0;
    int32_t first = 0;
#pragma unroll
    for (int j = 0; j < 4; ++j) {
      if (j >= per) break;
      if (at <= walk.from && walk.from < at + span[j]) mine = s0 + j, start = at, first = item0;
      at += span[j];
      item0 += g[j].items;
    }
    const unsigned hit = __ballot_sync(kAll, mine >= 0);
    if (hit) {
      const int from = __ffs(hit) - 1;
      walk.s = __shfl_sync(kAll, mine, from);
      walk.start = __shfl_sync(kAll, start, from);
      walk.item0 = __shfl_sync(kAll, first, from);
    }
    run += chunk;
    run_items += chunk_items;
  }
  if (walk.s >= b.groups) walk.item0 = (int64_t)(walk.s - b.groups) * p.ws.own_items;
  return walk;
}
// What the issuer's warp does in the last CTAs before its first tile has come: each
// looks at 128 segments for lengths that the tables do not hold, the last one also notes
// the prefixes' first items for the join.
__device__ __noinline__ void note_segments(const AttentionParams& p) {
  const BatchView& b = p.batch;
  const int lane = threadIdx.x & 31;
  const int segments = b.groups + b.sequences, place = (int)(gridDim.x - 1 - blockIdx.x);
  bool over = false;
  for (int s0 = place * 128; s0 < segments; s0 += p.ctas * 128)
    for (int s = s0 + lane; s < min(s0 + 128, segments); s += 32) {
      const Raw raw = raw_segment(b, s, true, false);
      over |= raw.len > 0 &&
              raw.len > capped(p, raw.len, s < b.groups ? b.prefix_width : b.table_width);
    }
  if (over) atomicOr(p.cache.err, kErrRange);
  if (place != 0) return;
  int32_t* items = reinterpret_cast<int32_t*>(p.workspace + p.ws.items);
  int32_t run = 0;
  __syncwarp();
  for (int s0 = 0; s0 < b.groups; s0 += 32) {
    const int s = s0 + lane;
    const int32_t n = s < b.groups ? segment_of(p, s, raw_segment(b, s, true, false)).items : 0;
    int32_t sum = n;
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
      const int32_t e = __shfl_up_sync(kAll, sum, o);
      if (lane >= o) sum += e;
    }
    if (s < b.groups) items[s] = run + sum - n;
    run += __shfl_sync(kAll, sum, 31);
  }
}

// Announces part after part and brings its tiles: K at place 2n of the ring's
// sequence, V at 2n + 1.
template <int DIM>
__device__ void produce_kv(const AttentionParams& p, const CUtensorMap* maps, uint8_t* smem,
                           Bars* bars, const Ctl& ctl) {
  using L = Layout<DIM>;
  constexpr int kHalves = DIM / 64;
  const int lane = threadIdx.x & 31;
  const int page = 1 << p.cache.page_shift;
  const int mine = lane / kHalves, half = lane % kHalves;   // this lane's box and half of it
  const BatchView& b = p.batch;
  // The way to the first part twice: a rehearsal, while the previous kernel ends, that
  // brings its instructions into the cache (cold, they took 10,000 cycles), then in
  // earnest.
  Walk walk;
  Part part;
  bool more = false;
#pragma unroll 1
  for (int pass = 0; pass < 2; ++pass) {
    if (pass == 1) wait_prerequisites();
    walk = share_out(p, pass == 0);
    part.n = 0;
    part.kind = kOne;
    more = walk.next(p, part);
  }
  uint32_t seq = 0;
  bool ok = true;
  for (uint32_t k = 0; ok; ++k) {
    const uint32_t e = k % kQueue, turn = k / kQueue;
    if (turn) ok = __all_sync(kAll, wait(&bars->heard[e], (turn - 1) & 1u, ctl));
    if (!ok) break;
    Announced& told = bars->queue[e];
    if (more && part.kind == kFew && lane < part.rows) {
      const Row row = row_of(p, part, lane);
      told.limit[lane] = row.limit;
      told.q[lane] = row.q;
    }
    if (lane == 0) told.part = part;
    __syncwarp();
    if (lane == 0) {
      mbar_arrive(&bars->told[e]);
      if (more && part.place < 0) {
        atomicOr(p.cache.err, kErrRange);
      } else if (more) {
        if (part.first) part.spans[0] = (int32_t)blockIdx.x;
        if (part.last) part.spans[1] = (int32_t)blockIdx.x;
      }
    }
    if (!more) break;
    const int32_t* row = part.far ? b.prefix_table + (int64_t)walk.s * b.prefix_stride
                                  : b.table + (int64_t)part.seq0 * b.table_stride;
    // A tile: kKvTile tokens of one head, rows of 128 bytes by halves of the head;
    // or few_tokens of few_heads, by boxes, halves, heads.
    const bool few = part.kind == kFew;
    const int tile = few ? p.few_tokens : kKvTile;
    const int box = min(page, tile);
    const uint32_t box_bytes = (uint32_t)(box * (few ? p.few_heads : 1)) * 128u;
    const uint32_t dst = few ? (uint32_t)lane * box_bytes
                             : (uint32_t)(half * kKvTile + mine * box) * 128u;
    const CUtensorMap* map = maps + (few ? 2 : 0);
    for (int t = 0; t < part.n; ++t) {
      const int t0 = (part.tile0 + t) * tile;
      const int boxes = (min(tile, part.len - t0) + box - 1) / box;
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
#pragma unroll 1
      for (int kv = 0; kv < 2; ++kv, ++seq) {
        const uint32_t slot = seq % L::kRing, again = seq / L::kRing;
        if (again) ok = wait(&bars->empty[slot], (again - 1) & 1u, ctl);
        ok = __all_sync(kAll, ok);
        if (!ok) break;
        if (lane == 0)
          mbar_expect_tx(&bars->full[slot], (uint32_t)(boxes * kHalves) * box_bytes);
        __syncwarp();
        if (on)
          tma_load_4d(smem_u32(smem + L::kRingOff + slot * L::kTile) + dst, map + kv, half * 64,
                      token & (page - 1), part.kvh, id, &bars->full[slot]);
      }
      if (!ok) break;
    }
    part.n = 0;
    part.kind = kOne;
    more = walk.next(p, part);
  }
  // No CTA leaves while its copies run.
  const WaitCtl dc = drain_ctl_default(p.cache.err);
  if (lane == 0)
    for (uint32_t k = seq > (uint32_t)L::kRing ? seq - L::kRing : 0u; k < seq; ++k)
      wait_bounded(&bars->full[k % L::kRing], (k / L::kRing) & 1u, dc);
}

// Reads the next announced part (a whole warp); false when a wait gave up.  What
// else the entry holds is read before `heard`.
__device__ __forceinline__ bool hear(Bars* bars, uint32_t k, Part* part, const Ctl& ctl) {
  const uint32_t e = k % kQueue;
  if (!__all_sync(kAll, wait(&bars->told[e], (k / kQueue) & 1u, ctl))) return false;
  *part = bars->queue[e].part;
  return true;
}
__device__ __forceinline__ void heard(Bars* bars, uint32_t k) {
  __syncwarp();
  if ((threadIdx.x & 31) == 0) mbar_arrive(&bars->heard[k % kQueue]);
}

// One team's use of one tile, in the order the products are issued: teams in turn.
struct Unit {
  uint32_t tile;   // of the CTA
  bool first;      // the team's first of a part
  bool last;       // the team's last of a part
  bool both;       // the other team uses the tile, too
};
struct Units {
  uint32_t tile = 0, team = 0, k = 0;
  int left = 0, begun = 0;  // uses left of the part, teams that have begun it (bits)
  bool both = false, end = false;
  // The next unit; false when there is none (end), or none yet while `pending` of
  // the issuer's units still lack their P V: the softmax warps may need those to
  // come to the part that follows, so the issuer must not wait for it.
  __device__ __forceinline__ bool next(Bars* bars, const Ctl& ctl, int pending, Unit& u,
                                       uint32_t& team_out) {
    while (left == 0 && !end) {
      const uint32_t e = k % kQueue;
      if (pending > 0 && (!__all_sync(kAll, mbar_test_wait(&bars->told[e], (k / kQueue) & 1u)) ||
                          bars->queue[e].part.kind == kFew))
        return false;
      Part part;
      if (!hear(bars, k, &part, ctl)) part.n = 0;
      heard(bars, k++);
      end = part.n == 0;
      if (part.kind == kFew) {   // the softmax warps multiply
        tile += (uint32_t)part.n;
      } else {
        both = part.kind == kBoth;
        left = both ? 2 * part.n : part.n;
        begun = 0;
      }
    }
    if (end) return false;
    team_out = team;
    u.tile = tile;
    u.first = !(begun >> team & 1);
    begun |= 1 << team;
    --left;
    u.last = left < 2;
    u.both = both;
    if (!both || (left & 1) == 0) ++tile;
    team ^= 1;
    return true;
  }
};

// Issues every product of the CTA (a whole warp, its first lane in effect).  A
// commit costs the issuer about as much as two products, so tiles that both teams use
// get one a unit: it follows a team's P V and the S of its next unit, and the teams
// pass the tiles they have then done with back to the producer.  Where a tile has one
// user memory is the bound, and V goes back by a commit of its own (so that two thirds
// of the ring are on their way instead of two fifths).
template <int DIM>
__device__ void issue_products(const AttentionParams& p, uint8_t* smem, Bars* bars,
                               const Ctl& ctl) {
  using L = Layout<DIM>;
  const uint32_t leader = (threadIdx.x & 31) == 0;
  const uint32_t tmem = bars->tmem;
  const uint32_t ring = smem_u32(smem + L::kRingOff), q = smem_u32(smem + L::kQOff);
  constexpr uint32_t id_s = umma_idesc_bf16(kTeamRows, kKvTile);
  constexpr uint32_t id_o = umma_idesc_bf16_bmn(kTeamRows, DIM);
  uint32_t q_turn[2] = {0, 0}, p_turn[2] = {0, 0};
  Units units;

  // A wait that gives up may do so for some lanes only: the warp goes by all of them,
  // as it meets again in votes and barriers of all lanes.
  auto issue_s = [&](const Unit& u, uint32_t w) -> bool {
    const uint32_t seq = 2 * u.tile, slot = seq % L::kRing;
    const bool ready = (!u.first || wait(&bars->qfull[w], q_turn[w]++ & 1u, ctl)) &&
                       wait(&bars->full[slot], (seq / L::kRing) & 1u, ctl);
    if (!__all_sync(kAll, ready)) return false;
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
    const uint32_t seq = 2 * u.tile + 1, slot = seq % L::kRing;
    const bool ready = wait(&bars->pfull[w], p_turn[w]++ & 1u, ctl) &&
                       wait(&bars->full[slot], (seq / L::kRing) & 1u, ctl);
    if (!__all_sync(kAll, ready)) return false;
    tc_fence_after();
    const uint64_t b = umma_desc_mn_sw128(ring + slot * L::kTile, kKvTile * 128u);
#pragma unroll
    for (int k = 0; k < kKvTile / 16; ++k)
      umma_bf16_ts_by(leader, tmem + 256u + w * 128u, tmem + w * 128u + 8u * k,
                      b + ((uint32_t)k * 2048u >> 4), id_o, !u.first || k > 0);
    if (u.last) umma_commit_by(leader, &bars->ofull[w]);
    if (!u.both) {   // alone with V: it goes back as soon as it has been read
      if (leader) mbar_arrive_n(&bars->empty[slot], 7);
      umma_commit_by(leader, &bars->empty[slot]);
    }
    return true;
  };

  // S runs up to two units ahead of P V, but does not wait for a part's Q while
  // there are P V to issue: the team that loads it may need those.
  Unit unit[2], u;
  uint32_t team[2], w;
  int pending = 0;
  bool has = false;
  for (;;) {
    if (!has && pending < 2) has = units.next(bars, ctl, pending, u, w);
    if (has && pending < 2 &&
        (pending == 0 || !u.first ||
         __all_sync(kAll, mbar_test_wait(&bars->qfull[w], q_turn[w] & 1u)))) {
      if (!issue_s(u, w)) break;
      if (pending == 0) unit[0] = u, team[0] = w;
      if (pending == 1) unit[1] = u, team[1] = w;
      ++pending;
      has = false;
      continue;
    }
    if (pending == 0) break;
    if (!issue_o(unit[0], team[0])) break;
    unit[0] = unit[1], team[0] = team[1];
    --pending;
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

// A part of a segment of at most kFewRows rows (what the registers of G = 2 hold).  128
// rows would keep the tensor cores and a team's chain busy with padding (3,800 cycles a
// tile of 64 KiB against 1,600 here; memory's share of one is 2,700), so each
// of the eight softmax warps takes one head's 16 tokens of every tile and
// multiplies them in registers (m16n8k16: S^T = K Q^T with the tokens as M, O^T +=
// V^T P^T with the elements as M, G groups of eight rows as N), on its own until
// the part ends.  A tile holds up to eight heads, so that a warp has a head to
// itself, a page comes in two copies and a short sequence is one part; where there
// are fewer heads, a team's warps of one head join their maxima, sums and values
// through its Q buffer.
template <int DIM, int G>
__device__ bool few_part(const AttentionParams& p, const Part& part, uint8_t* smem, Bars* bars,
                         const Ctl& ctl, uint32_t k, uint32_t tiles, uint32_t* meets, float c,
                         uint32_t flip) {
  using L = Layout<DIM>;
  // Floats between rows in the buffer: four more spread the banks, where it fits.
  constexpr int kStride = G == 1 ? DIM + 4 : DIM;
  static_assert(4 * 8 * G * kStride * 4 <= L::kTile, "room to join the warps");
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  const int g = lane >> 2, q2 = 2 * (lane & 3);   // row and column pair of fragments
  const uint32_t w = (uint32_t)warp >> 2;
  const int sharing = 8 / p.few_heads;            // warps of a head
  const int hd = warp / sharing, sub = warp - hd * sharing;
  // Fragments of Q^T: row g of each group; limits of rows q2 and q2 + 1.
  const Announced& told = bars->queue[k % kQueue];
  uint32_t qb[G][DIM / 16][2];
  int limit[G][2];
  const uint16_t* src[G];
#pragma unroll
  for (int n = 0; n < G; ++n) {
    src[n] = 8 * n + g < part.rows
                 ? static_cast<const uint16_t*>(p.q.data) + told.q[8 * n + g] +
                       (int64_t)(hd * p.gq) * p.q.head_stride
                 : nullptr;
#pragma unroll
    for (int j = 0; j < 2; ++j)
      limit[n][j] = 8 * n + q2 + j < part.rows ? told.limit[8 * n + q2 + j] : 0;
  }
  heard(bars, k);
#pragma unroll
  for (int n = 0; n < G; ++n)
#pragma unroll
    for (int d = 0; d < DIM / 16; ++d)
#pragma unroll
      for (int j = 0; j < 2; ++j)
        qb[n][d][j] =
            src[n] ? *reinterpret_cast<const uint32_t*>(src[n] + 16 * d + 8 * j + q2) ^ flip : 0u;
  float m[G][2], l[G][2], o[DIM / 16][G][4];
#pragma unroll
  for (int n = 0; n < G; ++n) {
    m[n][0] = m[n][1] = -INFINITY;
    l[n][0] = l[n][1] = 0.f;
#pragma unroll
    for (int d = 0; d < DIM / 16; ++d)
#pragma unroll
      for (int j = 0; j < 4; ++j) o[d][n][j] = 0.f;
  }
  // Where this lane points ldmatrix.  K's four matrices: tokens 0-7, 8-15, then
  // both with the next 8 elements; V's, transposed: elements 0-7, 8-15 of tokens
  // 0-7, then both of tokens 8-15.
  const int box = min(1 << p.cache.page_shift, p.few_tokens);
  const uint32_t half = (uint32_t)(box * p.few_heads) * 128u;   // bytes from half to half
  auto row_at = [&](int token) -> uint32_t {                    // of this warp's head
    const int n = token / box;
    return (uint32_t)n * (DIM / 64) * half + (uint32_t)(hd * box + token - n * box) * 128u;
  };
  const int kc = lane >> 4, vc = (lane >> 3) & 1, l7 = lane & 7;
  const uint32_t k_at = row_at(16 * sub + (lane & 15));
  const uint32_t v_at = row_at(16 * sub + l7 + (lane >> 4) * 8);
  bool ok = true;
  for (int t = 0; t < part.n; ++t) {
    const int t0 = (part.tile0 + t) * p.few_tokens + 16 * sub;  // this warp's first token
    const int there = part.len - t0;                            // of its tokens, how many are
    const uint32_t ks = 2 * (tiles + (uint32_t)t), kslot = ks % L::kRing;
    const uint32_t vs = ks + 1, vslot = vs % L::kRing;
    ok = __all_sync(kAll, wait(&bars->full[kslot], (ks / L::kRing) & 1u, ctl));
    if (!ok) break;
    uint32_t pb[G][2];
    if (there > 0) {
      const uint32_t kb = smem_u32(smem + L::kRingOff + kslot * L::kTile) + k_at;
      float s[G][2][4];
#pragma unroll
      for (int n = 0; n < G; ++n)
#pragma unroll
        for (int j = 0; j < 8; ++j) s[n][j >> 2][j & 3] = 0.f;
#pragma unroll
      for (int d = 0; d < DIM / 16; ++d) {
        uint32_t a[4];
        ldmatrix_x4(
            kb + (uint32_t)(d / 4) * half + (uint32_t)(((2 * d + kc) & 7) ^ l7) * 16u, a);
#pragma unroll
        for (int n = 0; n < G; ++n)
          mma_bf16_16816(s[n][d & 1], a[0], a[1], a[2], a[3], qb[n][d][0], qb[n][d][1]);
      }
#pragma unroll
      for (int n = 0; n < G; ++n) {
        float x[4], now[2];   // tokens g (rows q2, q2 + 1), then g + 8
#pragma unroll
        for (int j = 0; j < 4; ++j)
          x[j] = g + 8 * (j >> 1) < limit[n][j & 1] - t0 ? s[n][0][j] + s[n][1][j] : -INFINITY;
#pragma unroll
        for (int j = 0; j < 2; ++j) {
          now[j] = fmaxf(x[j], x[j + 2]);
#pragma unroll
          for (int d = 4; d < 32; d <<= 1) now[j] = fmaxf(now[j], __shfl_xor_sync(kAll, now[j], d));
          now[j] = fmaxf(now[j], m[n][j]);
        }
        const bool grow0 = now[0] > m[n][0] && !((now[0] - m[n][0]) * c <= kLazy);
        const bool grow1 = now[1] > m[n][1] && !((now[1] - m[n][1]) * c <= kLazy);
        if (__any_sync(kAll, grow0 || grow1)) {
          const float f0 =
              !grow0 ? 1.f : m[n][0] == -INFINITY ? 0.f : exp2_approx((m[n][0] - now[0]) * c);
          const float f1 =
              !grow1 ? 1.f : m[n][1] == -INFINITY ? 0.f : exp2_approx((m[n][1] - now[1]) * c);
#pragma unroll
          for (int d = 0; d < DIM / 16; ++d) {
            o[d][n][0] *= f0, o[d][n][2] *= f0;
            o[d][n][1] *= f1, o[d][n][3] *= f1;
          }
          l[n][0] *= f0, l[n][1] *= f1;
          if (grow0) m[n][0] = now[0];
          if (grow1) m[n][1] = now[1];
        }
#pragma unroll
        for (int j = 0; j < 4; ++j) {
          const float shift = m[n][j & 1] == -INFINITY ? 0.f : m[n][j & 1] * c;
          x[j] = exp2_approx(fmaf(x[j], c, -shift));
          l[n][j & 1] += x[j];
        }
        pb[n][0] = transpose_8x8(round_bf16x2(x[0], x[1]));
        pb[n][1] = transpose_8x8(round_bf16x2(x[2], x[3]));
      }
    }
    __syncwarp();
    if (lane == 0) mbar_arrive(&bars->empty[kslot]);
    ok = __all_sync(kAll, wait(&bars->full[vslot], (vs / L::kRing) & 1u, ctl));
    if (!ok) break;
    if (there > 0) {
      // Tokens behind the segment's last count as zeros, whatever the page holds.
      const int left = there - q2;
      const uint32_t keep0 = (left > 0 ? 0xFFFFu : 0u) | (left > 1 ? 0xFFFF0000u : 0u);
      const uint32_t keep1 = (left > 8 ? 0xFFFFu : 0u) | (left > 9 ? 0xFFFF0000u : 0u);
      const uint32_t vb = smem_u32(smem + L::kRingOff + vslot * L::kTile) + v_at;
#pragma unroll
      for (int d = 0; d < DIM / 16; ++d) {
        uint32_t a[4];
        ldmatrix_x4_trans(
            vb + (uint32_t)(d / 4) * half + (uint32_t)(((2 * d + vc) & 7) ^ l7) * 16u, a);
        a[0] &= keep0, a[1] &= keep0, a[2] &= keep1, a[3] &= keep1;
#pragma unroll
        for (int n = 0; n < G; ++n)
          mma_bf16_16816(o[d][n], a[0], a[1], a[2], a[3], pb[n][0], pb[n][1]);
      }
    }
    __syncwarp();
    if (lane == 0) mbar_arrive(&bars->empty[vslot]);
  }
  if (!ok) return false;
#pragma unroll
  for (int n = 0; n < G; ++n)
#pragma unroll
    for (int j = 0; j < 2; ++j)
#pragma unroll
      for (int d = 4; d < 32; d <<= 1) l[n][j] += __shfl_xor_sync(kAll, l[n][j], d);
  float2* ml_at = reinterpret_cast<float2*>(p.workspace + (part.far ? p.ws.far_ml : p.ws.own_ml));
  float* o_at = reinterpret_cast<float*>(p.workspace + (part.far ? p.ws.far_o : p.ws.own_o));
  // Results by heads, rows; of a single head by teams, rows.
  const int64_t place =
      part.place + (p.few_heads == 1 ? (int)w : hd) * (part.far ? kFewRows : p.ws.seq_rows);
  if (sharing == 1) {
#pragma unroll
    for (int n = 0; n < G; ++n)
#pragma unroll
      for (int j = 0; j < 2; ++j) {
        const int row = 8 * n + q2 + j;
        if (row < part.rows && part.place >= 0) {
          if (g == 0) ml_at[place + row] = make_float2(m[n][j] * c, l[n][j]);
          float* dst = o_at + (place + row) * DIM + g;
#pragma unroll
          for (int d = 0; d < DIM / 16; ++d) {
            dst[16 * d] = o[d][n][j];
            dst[16 * d + 8] = o[d][n][j + 2];
          }
        }
      }
    return true;
  }
  const int tw = warp & 3, mates = min(sharing, 4), tw0 = tw / mates * mates;
  float* buf = reinterpret_cast<float*>(smem + L::kQOff + w * L::kTile);
#pragma unroll
  for (int n = 0; n < G; ++n)
#pragma unroll
    for (int j = 0; j < 2; ++j) {
      const int row = 8 * n + q2 + j;
      if (row < part.rows) {
        if (g == 0) bars->ml[w][tw][row] = make_float2(m[n][j] * c, l[n][j]);
        float* dst = buf + (tw * 8 * G + row) * kStride + g;
#pragma unroll
        for (int d = 0; d < DIM / 16; ++d) {
          dst[16 * d] = o[d][n][j];
          dst[16 * d + 8] = o[d][n][j + 2];
        }
      }
    }
  __syncwarp();
  if (lane == 0) mbar_arrive(&bars->team[w]);
  if (!__all_sync(kAll, wait(&bars->team[w], (*meets)++ & 1u, ctl))) return false;
  for (int row = tw - tw0; part.place >= 0 && row < part.rows; row += mates) {
    float top = -INFINITY, sum = 0.f;
    for (int j = 0; j < mates; ++j) top = fmaxf(top, bars->ml[w][tw0 + j][row].x);
    const float zero = top == -INFINITY ? 0.f : top;
    float2 a[DIM / 64];
#pragma unroll
    for (int d = 0; d < DIM / 64; ++d) a[d] = make_float2(0.f, 0.f);
    for (int j = 0; j < mates; ++j) {
      const float2 ml = bars->ml[w][tw0 + j][row];
      const float f = exp2_approx(ml.x - zero);
      sum += f * ml.y;
#pragma unroll
      for (int d = 0; d < DIM / 64; ++d) {
        const float2 x = *reinterpret_cast<const float2*>(
            buf + ((tw0 + j) * 8 * G + row) * kStride + 64 * d + 2 * lane);
        a[d].x += f * x.x, a[d].y += f * x.y;
      }
    }
    if (lane == 0) ml_at[place + row] = make_float2(top, sum);
#pragma unroll
    for (int d = 0; d < DIM / 64; ++d)
      *reinterpret_cast<float2*>(o_at + (place + row) * DIM + 64 * d + 2 * lane) = a[d];
  }
  __syncwarp();
  if (lane == 0) mbar_arrive(&bars->team[w]);
  return __all_sync(kAll, wait(&bars->team[w], (*meets)++ & 1u, ctl));
}

// Scores are in units of log2; a scale of zero is replaced by the least FP32 number,
// which leaves every finite score below 2^-20 (so that masked scores of -inf stay what
// they are).
__device__ __forceinline__ float score_unit(float scale) {
  return fmaxf(fabsf(scale) * 1.4426950408889634f, 0x1p-149f);
}

// A softmax team: thread r has row r of the team's rows.
template <int DIM>
__device__ void softmax_team(const AttentionParams& p, uint8_t* smem, Bars* bars,
                             const Ctl& ctl, uint32_t w) {
  using L = Layout<DIM>;
  const int r = threadIdx.x % kTeamThreads;
  const uint32_t lane_base = (uint32_t)(r & ~31) << 16;
  const uint32_t ts = bars->tmem + w * 128u + lane_base;         // S and P
  const uint32_t to = bars->tmem + 256u + w * 128u + lane_base;  // O
  // (A negative scale turns Q's sign, which is exact.)
  const float c = score_unit(p.scale);
  const uint32_t flip = p.scale < 0.f ? 0x80008000u : 0u;
  uint32_t turn = 0;       // this team's uses of tiles so far
  uint32_t done = 0;       // and its parts with at least one
  uint32_t meets = 0;      // times the team's warps have met
  uint32_t uses = 0;       // both teams' uses so far
  uint32_t tiles = 0;      // tiles of the CTA so far
  for (uint32_t k = 0;; ++k) {
    Part part;
    if (!hear(bars, k, &part, ctl) || part.n == 0) return;
    if (part.kind == kFew) {
      const bool ok =
          part.rows <= 8
              ? few_part<DIM, 1>(p, part, smem, bars, ctl, k, tiles, &meets, c, flip)
              : few_part<DIM, 2>(p, part, smem, bars, ctl, k, tiles, &meets, c, flip);
      if (!ok) return;
      tiles += (uint32_t)part.n;
      continue;
    }
    heard(bars, k);
    const bool both = part.kind == kBoth;
    const int from = both ? (int)w * kTeamRows : 0;              // the team's first row
    const int team_rows = min(part.rows - from, kTeamRows);
    const int first = both ? 0 : (int)((uses ^ w) & 1u);         // the team's first tile
    const int step = both ? 1 : 2;
    const bool zeroes = !both || w == (uses & 1u);               // the tile's first user
    const bool begins = first < part.n;
    // This thread's row; a team without a tile only leaves word that it has nothing.
    Row mine;
    mine.q = mine.limit = 0;
    if (begins && r < team_rows) mine = row_of(p, part, from + r);
    const int limit = mine.limit;
    if (begins) {
      // Q's rows into the team's buffer: 16-byte pieces, 128-byte swizzle, each
      // warp its own 32.  Rows behind the last get the tensor's first: no row's
      // result meets another's.
      constexpr int kPieces = DIM / 8, kStep = 32 / kPieces;
      const int lane = r & 31, piece = lane % kPieces;
      const uint32_t dst = smem_u32(smem + L::kQOff + w * L::kTile) +
                           (uint32_t)(piece / 8) * (kTeamRows * 128u);
      uint4 v[kPieces];   // all loads before the first store, which the compiler keeps in order
#pragma unroll
      for (int j = 0; j < kPieces; ++j) {
        const int64_t at = __shfl_sync(kAll, mine.q, j * kStep + lane / kPieces);
        v[j] = reinterpret_cast<const uint4*>(static_cast<const uint16_t*>(p.q.data) + at)[piece];
      }
#pragma unroll
      for (int j = 0; j < kPieces; ++j) {
        const int in = (r & ~31) + j * kStep + lane / kPieces;
        sts128(dst + (uint32_t)in * 128u + (uint32_t)((piece % 8) ^ (in & 7)) * 16u, v[j].x ^ flip,
               v[j].y ^ flip, v[j].z ^ flip, v[j].w ^ flip);
      }
      fence_proxy_async_smem();
      tc_fence_before();
      mbar_arrive(&bars->qfull[w]);
    }
    float m = -INFINITY, l = 0.f;
    const bool warp_live = __any_sync(kAll, limit > 0);
    for (int t = first; t < part.n; t += step, ++turn) {
      const int t0 = (part.tile0 + t) * kKvTile;
      if (!__all_sync(kAll, wait(&bars->sfull[w], turn & 1u, ctl))) return;
      tc_fence_after();
      if (r == 0) {   // S is there: K has been read, and a shared V of the unit before
        mbar_arrive_n(&bars->empty[2 * (tiles + (uint32_t)t) % L::kRing], both ? 4 : 8);
        if (both && t != first)
          mbar_arrive_n(&bars->empty[(2 * (tiles + (uint32_t)(t - 1)) + 1) % L::kRing], 4);
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
      const int there = part.len - t0;
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
    const int64_t place = part.place + (int)w * (part.far ? kTeamRows : p.ws.own_rows / 2);
    float* o_at = reinterpret_cast<float*>(p.workspace + (part.far ? p.ws.far_o : p.ws.own_o));
    if (r < team_rows && part.place >= 0)
      reinterpret_cast<float2*>(p.workspace +
                                (part.far ? p.ws.far_ml : p.ws.own_ml))[place + r] =
          make_float2(m * c, l);
    if (begins) {
      if (!__all_sync(kAll, wait(&bars->ofull[w], done++ & 1u, ctl))) return;
      tc_fence_after();
      if (both && r == 0)
        mbar_arrive_n(&bars->empty[(2 * (tiles + (uint32_t)part.n) - 1) % L::kRing], 4);
      if (warp_live) {
        // Rows of a lane each become rows of a warp through the Q buffer (pieces of
        // 16 bytes, spread over the banks): a lane's own row of 512 bytes stored
        // piece by piece touched 32 lines a store, 8,000 cycles a part.
        constexpr int kCols = DIM / 2, kPieces = kCols / 4;
        const int lane = r & 31, wrow = r & ~31;
        const uint32_t buf = smem_u32(smem + L::kQOff + w * L::kTile) +
                             (uint32_t)(r >> 5) * (L::kTile / 4);
#pragma unroll 1
        for (int k = 0; k < DIM; k += kCols) {
          float o[kCols];
#pragma unroll
          for (int j = 0; j < kCols; j += 32) tmem_load32(to + (uint32_t)(k + j), o + j);
          tmem_wait_load();
          tmem_tie<kCols>(o);
          __syncwarp();
#pragma unroll
          for (int j = 0; j < kPieces; ++j)
            sts128(buf + (uint32_t)(lane * kPieces + (j ^ (lane & 7))) * 16u,
                   __float_as_uint(o[4 * j]), __float_as_uint(o[4 * j + 1]),
                   __float_as_uint(o[4 * j + 2]), __float_as_uint(o[4 * j + 3]));
          __syncwarp();
          const int piece = lane % kPieces;
#pragma unroll 8
          for (int row = lane / kPieces; row < 32; row += 32 / kPieces) {
            const uint4 v = lds128(buf + (uint32_t)(row * kPieces + (piece ^ (row & 7))) * 16u);
            if (wrow + row < team_rows && part.place >= 0)
              reinterpret_cast<uint4*>(o_at + (place + wrow + row) * DIM + k)[piece] = v;
          }
        }
      }
      tc_fence_before();
      // The buffer is the whole team's again.
      __syncwarp();
      if ((r & 31) == 0) mbar_arrive(&bars->team[w]);
      if (!__all_sync(kAll, wait(&bars->team[w], meets++ & 1u, ctl))) return;
    }
    uses += (uint32_t)(both ? 2 * part.n : part.n);
    tiles += (uint32_t)part.n;
  }
}

template <int DIM>
__global__ void __launch_bounds__(kThreads, 1)
    attention_kernel(const __grid_constant__ AttentionParams p,
                     const __grid_constant__ PageMaps maps) {
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
      mbar_init(&bars->empty[k], 8);
    }
    for (int k = 0; k < kQueue; ++k) {
      mbar_init(&bars->told[k], 1);
      mbar_init(&bars->heard[k], 9);
    }
    for (int w = 0; w < 2; ++w) {
      mbar_init(&bars->qfull[w], kTeamThreads);
      mbar_init(&bars->sfull[w], 1);
      mbar_init(&bars->pfull[w], kTeamThreads);
      mbar_init(&bars->ofull[w], 1);
      mbar_init(&bars->team[w], 4);
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
  if (warp != kProducerWarp) wait_prerequisites();
  const Ctl ctl{p.cache.err, p.wait_limit ? p.wait_limit : kDefaultWaitLimit,
                p.wait_limit != 0, &bars->abort};
  if (warp < 8) {
    softmax_team<DIM>(p, smem, bars, ctl, (uint32_t)(warp >> 2));
  } else if (warp == kProducerWarp) {
    produce_kv<DIM>(p, maps.map, smem, bars, ctl);
  } else {
    if ((gridDim.x - 1 - blockIdx.x) * 128u < (unsigned)(p.batch.groups + p.batch.sequences))
      note_segments(p);
    issue_products<DIM>(p, smem, bars, ctl);
  }
  __syncwarp();
  tc_fence_before();
  __syncthreads();
  if (warp == kIssuerWarp)
    asm volatile("tcgen05.dealloc.cta_group::1.sync.aligned.b32 %0, 512;" ::"r"(bars->tmem));
}

// ---- joining the parts ------------------------------------------------------------


// Where a row's results lie in a segment's parts: for k < n in row place + k / teams *
// part_rows + k % teams * team_rows (a part has the row once, or for each of the
// two teams that share it).
struct Side {
  int64_t place;
  int n, teams, team_rows, part_rows;
};
__device__ __forceinline__ Side side_of(const AttentionParams& p, bool far, int rows, int row,
                                        int kvh, int64_t first_item) {
  Side d;
  const bool few = rows <= kFewRows;
  const int block = row / kPairRows, in_block = row - block * kPairRows;
  const bool both = !few && min(rows - block * kPairRows, kPairRows) > kTeamRows;
  const int in_heads = few ? kvh % p.few_heads : 0;
  const int64_t item = first_item + (few ? kvh / p.few_heads : block * p.kv_heads + kvh);
  d.teams = few ? (p.few_heads == 1 ? 2 : 1) : both ? 1 : 2;
  d.team_rows = few ? (far ? kFewRows : p.ws.seq_rows) : far ? kTeamRows : p.ws.own_rows / 2;
  d.part_rows = far ? kPairRows : p.ws.own_rows;
  const int at = few    ? (p.few_heads == 1 ? 0 : in_heads) * d.team_rows + row
                 : both ? in_block / kTeamRows * d.team_rows + in_block % kTeamRows
                        : in_block;
  d.n = 0;
  d.place = 0;
  const int64_t slots = far ? p.ws.far_slots : p.ws.own_slots;
  if (0 <= item && item < slots - p.ctas) {
    const int2 span = *reinterpret_cast<const int2*>(
        p.workspace + (far ? p.ws.far_spans : p.ws.own_spans) + 8 * item);
    // (After a wait that gave up, what is there may be anything.)
    if (0 <= span.x && span.x <= span.y && span.y < p.ctas) {
      d.n = (span.y - span.x + 1) * d.teams;
      d.place = (item + span.x) * d.part_rows + at;
    }
  }
  return d;
}

// Whether V of a token in [from, to) of a sequence holds what is not finite in this head
// (a warp; pages that are not there count as zeros).
template <int DIM>
__device__ __noinline__ bool any_not_finite(const AttentionParams& p, const int32_t* table,
                                            int from, int to, int kvh) {
  const CacheView& cv = p.cache;
  const int lane = threadIdx.x & 31, mask = (1 << cv.page_shift) - 1;
  for (int j = from; j < to; ++j) {
    const int64_t page = table[j >> cv.page_shift];
    if (page < 0 || page >= cv.pages) continue;
    const uint16_t* v = cv.v + page * cv.v_page + (j & mask) * cv.v_token + kvh * cv.v_head;
    bool bad = false;
    for (int e = lane; e < DIM; e += 32) bad |= (v[e] & 0x7F80) == 0x7F80;
    if (__any_sync(kAll, bad)) return true;
  }
  return false;
}
// Weighted values of a segment's first `limit` tokens for one row, by a warp token by
// token, E elements a lane, with the row's maximum known: for rows where a V that they do
// not see spoilt the products (zero times infinity is not zero).
template <int DIM>
__device__ __noinline__ void add_seen(const AttentionParams& p, const int32_t* table, int limit,
                                      int kvh, const uint16_t (&q)[DIM / 32], float top,
                                      float* acc) {
  constexpr int E = DIM / 32;
  const CacheView& cv = p.cache;
  const int lane = threadIdx.x & 31, mask = (1 << cv.page_shift) - 1;
  const float c = copysignf(score_unit(p.scale), p.scale);
  float qe[E];
  for (int e = 0; e < E; ++e) qe[e] = __uint_as_float((uint32_t)q[e] << 16);
  for (int j = 0; j < limit; ++j) {
    const int64_t page = table[j >> cv.page_shift];
    if (page < 0 || page >= cv.pages) continue;   // its V counts as zeros
    const uint16_t* k = cv.k + page * cv.k_page + (j & mask) * cv.k_token + kvh * cv.k_head;
    const uint16_t* v = cv.v + page * cv.v_page + (j & mask) * cv.v_token + kvh * cv.v_head;
    float s = 0.f;
    for (int e = 0; e < E; ++e) s += qe[e] * __uint_as_float((uint32_t)k[lane * E + e] << 16);
    for (int d = 16; d > 0; d >>= 1) s += __shfl_xor_sync(kAll, s, d);
    const float f = exp2f(s * c - top);
    for (int e = 0; e < E; ++e) acc[e] += f * __uint_as_float((uint32_t)v[lane * E + e] << 16);
  }
}

// One CTA a row and query head: over the parts of its prefix and its own tokens,
// out = sum 2^(m_i - M) O_i / sum 2^(m_i - M) l_i, in a fixed order.  A thread a
// part for the weights, then a warp a part for the values, four parts in flight.
// CHUNK: more than one new token a sequence.
template <int DIM, int kJoinWarps, bool CHUNK>
__global__ void __launch_bounds__(kJoinWarps * 32)
    join_kernel(const __grid_constant__ AttentionParams p) {
  constexpr int E = DIM / 32, kJoinThreads = kJoinWarps * 32;
  __shared__ float weight[kJoinThreads];
  __shared__ const float* source[kJoinThreads];
  __shared__ float values[kJoinWarps][DIM];
  __shared__ float red[2][kJoinWarps];
  allow_dependents();
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  const BatchView& b = p.batch;
  const int token = (int)blockIdx.x, head = (int)blockIdx.y;
  const int seq = b.chunk == 1 ? token : token / b.chunk, i = token - seq * b.chunk;
  const int kvh = head / p.gq, h = head - kvh * p.gq, in_seq = i * p.gq + h;
  wait_prerequisites();
  Side far, own;
  far.n = own.n = 0;
  int group = -1;
  const int fresh = fresh_of(b, seq);
  uint16_t q[E] = {};   // read before any warp writes: out may be q itself
  if (CHUNK) {
    const uint16_t* src = static_cast<const uint16_t*>(p.q.data) +
                          (int64_t)token * p.q.token_stride + (int64_t)head * p.q.head_stride;
    if (E == 4) {
      const uint2 v = reinterpret_cast<const uint2*>(src)[lane];
      q[0] = (uint16_t)v.x, q[1] = (uint16_t)(v.x >> 16);
      q[2 % E] = (uint16_t)v.y, q[3 % E] = (uint16_t)(v.y >> 16);
    } else {
      const uint32_t v = reinterpret_cast<const uint32_t*>(src)[lane];
      q[0] = (uint16_t)v, q[1] = (uint16_t)(v >> 16);
    }
  }
  if (i < fresh) {
    // (Tokens that no table holds have no parts: what the workspace says is then old.)
    if (b.lens[seq] > 0 && b.table_width > 0)
      own = side_of(p, false, p.seq_rows, in_seq, kvh, (int64_t)seq * p.ws.own_items);
    for (int g0 = 0; g0 < b.groups; g0 += 32) {
      const int g = g0 + lane;
      int first = 0, end = 0, len = 0, item = 0;
      if (g < b.groups) {
        first = b.group_start[g];
        end = b.group_start[g + 1];
        len = b.prefix_lens[g];
        item = reinterpret_cast<const int32_t*>(p.workspace + p.ws.items)[g];
      }
      const unsigned hit = __ballot_sync(kAll, first <= seq && seq < end);
      if (hit) {
        const int from = __ffs(hit) - 1;
        first = max(__shfl_sync(kAll, first, from), 0);
        end = min(__shfl_sync(kAll, end, from), b.sequences);
        item = __shfl_sync(kAll, item, from);
        if (__shfl_sync(kAll, len, from) > 0 && b.prefix_width > 0)
          far = side_of(p, true, (end - first) * p.seq_rows, (seq - first) * p.seq_rows + in_seq,
                        kvh, item);
        group = g0 + from;
        break;
      }
    }
  }
  float top = -INFINITY, sum = 0.f, acc[E];
#pragma unroll
  for (int e = 0; e < E; ++e) acc[e] = 0.f;
  for (int k0 = 0; k0 < far.n + own.n; k0 += kJoinThreads) {
    const int count = min(far.n + own.n - k0, kJoinThreads);
    float2 v = make_float2(-INFINITY, 0.f);
    const float* src = nullptr;
    if ((int)threadIdx.x < count) {
      const bool in_far = k0 + (int)threadIdx.x < far.n;
      const int k = k0 + (int)threadIdx.x - (in_far ? 0 : far.n);
      const int part = (in_far ? far.teams : own.teams) == 2 ? k >> 1 : k;
      const int team = (in_far ? far.teams : own.teams) == 2 ? k & 1 : 0;
      const int64_t place = (in_far ? far.place : own.place) +
                            (int64_t)part * (in_far ? far.part_rows : own.part_rows) +
                            team * (in_far ? far.team_rows : own.team_rows);
      v = reinterpret_cast<const float2*>(p.workspace +
                                          (in_far ? p.ws.far_ml : p.ws.own_ml))[place];
      src = reinterpret_cast<const float*>(p.workspace + (in_far ? p.ws.far_o : p.ws.own_o)) +
            place * DIM;
    }
    float t = v.x;
#pragma unroll
    for (int d = 16; d > 0; d >>= 1) t = fmaxf(t, __shfl_xor_sync(kAll, t, d));
    if (lane == 0) red[0][warp] = t;
    __syncthreads();
    float now = top;
#pragma unroll
    for (int w = 0; w < kJoinWarps; ++w) now = fmaxf(now, red[0][w]);
    const float base = now == -INFINITY ? 0.f : now;
    const float keep = exp2f(top - base);
    // A part without weight is not read (its values were not written).
    const float f = v.y != 0.f ? exp2f(v.x - base) : 0.f;
    weight[threadIdx.x] = f;
    source[threadIdx.x] = f != 0.f ? src : nullptr;
    float part = f * v.y;
#pragma unroll
    for (int d = 16; d > 0; d >>= 1) part += __shfl_xor_sync(kAll, part, d);
    if (lane == 0) red[1][warp] = part;
    __syncthreads();
    sum *= keep;
#pragma unroll
    for (int w = 0; w < kJoinWarps; ++w) sum += red[1][w];
    top = now;
#pragma unroll
    for (int e = 0; e < E; ++e) acc[e] *= keep;
    for (int j = warp; j < count; j += 4 * kJoinWarps) {
      float x[4][E], fj[4];
#pragma unroll
      for (int u = 0; u < 4; ++u) {
        const int at = j + u * kJoinWarps;
        const float* from = at < count ? source[at] : nullptr;
        fj[u] = from ? weight[at] : 0.f;
#pragma unroll
        for (int e = 0; e < E; ++e) x[u][e] = 0.f;
        if (from) {
          if (E == 4) {
            const float4 y = reinterpret_cast<const float4*>(from)[lane];
            x[u][0] = y.x, x[u][1] = y.y, x[u][2 % E] = y.z, x[u][3 % E] = y.w;
          } else {
            const float2 y = reinterpret_cast<const float2*>(from)[lane];
            x[u][0] = y.x, x[u][1] = y.y;
          }
        }
      }
#pragma unroll
      for (int u = 0; u < 4; ++u)
#pragma unroll
        for (int e = 0; e < E; ++e) acc[e] += fj[u] * x[u][e];
    }
    __syncthreads();
  }
#pragma unroll
  for (int e = 0; e < E; ++e) values[warp][lane * E + e] = acc[e];
  __syncthreads();
  const float inv = sum != 0.f ? 1.f / sum : 0.f;
  uint16_t* out = static_cast<uint16_t*>(p.out.data) + (int64_t)token * p.out.token_stride +
                  (int64_t)head * p.out.head_stride;
  for (int e = 2 * (int)threadIdx.x; e < DIM; e += 2 * kJoinThreads) {
    float lo = 0.f, hi = 0.f;
#pragma unroll
    for (int w = 0; w < kJoinWarps; ++w) lo += values[w][e], hi += values[w][e + 1];
    *reinterpret_cast<uint32_t*>(out + e) = pack_bf16(lo * inv, hi * inv);
    // NaN with a sum that is none, and tokens of this call behind the row's own: where
    // their V is what is not finite, the warp works its 64 elements out again.  (A V that
    // the row sees needs no such pass, which takes milliseconds over 32768 tokens.)
    if (CHUNK && i + 1 < fresh && sum == sum && __any_sync(kAll, lo != lo || hi != hi)) {
      const int32_t* table = b.table + (int64_t)seq * b.table_stride;
      const int len = max(b.lens[seq], 0);
      const int seen = capped(p, len - fresh + i + 1, b.table_width);
      if (!any_not_finite<DIM>(p, table, seen, capped(p, len, b.table_width), kvh)) continue;
      float again[E];
      for (int j = 0; j < E; ++j) again[j] = 0.f;
      if (group >= 0)
        add_seen<DIM>(p, b.prefix_table + (int64_t)group * b.prefix_stride,
                      capped(p, b.prefix_lens[group], b.prefix_width), kvh, q, top, again);
      add_seen<DIM>(p, table, seen, kvh, q, top, again);
      if (lane * E / 64 == warp)
        for (int j = 0; j < E; j += 2)
          *reinterpret_cast<uint32_t*>(out + lane * E + j) =
              pack_bf16(again[j] * inv, again[j + 1] * inv);
    }
  }
  if (p.lse && threadIdx.x == 0)
    p.lse[(int64_t)token * p.heads + head] = sum != 0.f ? (top + log2f(sum)) * 0.69314718055994531f : -INFINITY;
}

template <int DIM>
cudaError_t launch_dim(const AttentionParams& p, const PageMaps& maps, cudaStream_t stream) {
  static std::atomic<bool> configured[64];   // calls may come from several threads
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
  e = cudaLaunchKernelEx(&cfg, attention_kernel<DIM>, p, maps);
  if (e != cudaSuccess) return e;
  // Eight warps a row and head while those are few and have many parts each; else
  // two, which all fit on the device at once (2048 rows and heads: 4.7 us a call
  // less than with four).
  const int64_t outputs = (int64_t)p.batch.sequences * p.batch.chunk * p.heads;
  const int warps = outputs <= 4 * p.ctas ? 8 : 2;
  cfg.gridDim =
      dim3((unsigned)(p.batch.sequences * p.batch.chunk), (unsigned)p.heads);  // <= 2^24, 2^12
  cfg.blockDim = dim3((unsigned)(32 * warps));
  cfg.dynamicSmemBytes = 0;
  if (p.batch.chunk == 1)
    return warps == 8 ? cudaLaunchKernelEx(&cfg, join_kernel<DIM, 8, false>, p)
                      : cudaLaunchKernelEx(&cfg, join_kernel<DIM, 2, false>, p);
  return warps == 8 ? cudaLaunchKernelEx(&cfg, join_kernel<DIM, 8, true>, p)
                    : cudaLaunchKernelEx(&cfg, join_kernel<DIM, 2, true>, p);
}

uint64_t up256(uint64_t x) { return (x + 255) & ~255ull; }

}  // namespace

AttentionWorkspace attention_workspace(int sequences, int chunk, int groups, int heads,
                                       int kv_heads, int dim, int ctas) {
  AttentionWorkspace w;
  const int64_t seq_rows = (int64_t)chunk * (heads / kv_heads);
  const int64_t far_items =
      groups ? ((seq_rows * sequences + kPairRows - 1) / kPairRows + groups) * kv_heads : 0;
  const int few_heads = few_heads_of(kv_heads);
  const bool few = seq_rows <= kFewRows;
  w.seq_rows = few ? (int32_t)seq_rows : 0;
  w.own_rows = (int32_t)(few ? seq_rows * (few_heads == 1 ? 2 : few_heads)
                             : 2 * (seq_rows < kTeamRows ? seq_rows : kTeamRows));
  w.own_items = (int32_t)(few ? kv_heads / few_heads
                              : (seq_rows + kPairRows - 1) / kPairRows * kv_heads);
  w.far_slots = groups ? far_items + ctas : 0;
  w.own_slots = (int64_t)sequences * w.own_items + ctas;
  uint64_t at = 0;
  auto take = [&](uint64_t bytes) {
    const uint64_t here = at;
    at += up256(bytes);
    return here;
  };
  w.far_spans = take(8ull * far_items);
  w.own_spans = take(8ull * sequences * w.own_items);
  w.items = take(4ull * ((uint64_t)groups + 1));
  w.far_ml = take(8ull * w.far_slots * kPairRows);
  w.far_o = take(4ull * w.far_slots * kPairRows * dim);
  w.own_ml = take(8ull * w.own_slots * w.own_rows);
  w.own_o = take(4ull * w.own_slots * w.own_rows * dim);
  w.bytes = at;
  return w;
}

cudaError_t launch_attention(const AttentionParams& p, const PageMaps& maps,
                             cudaStream_t stream) {
  return p.dim == 64 ? launch_dim<64>(p, maps, stream) : launch_dim<128>(p, maps, stream);
}

}  // namespace nwc
