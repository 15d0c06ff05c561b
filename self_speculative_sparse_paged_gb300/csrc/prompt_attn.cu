// Attention over whole prompts on the 5th-generation tensor cores, head_dim
// 128 or 64: every row of a packed batch of ragged sequences attends its own
// sequence's cache causally.
//
// For row t of sequence b (n_b rows behind a cached prefix of c_b positions),
// query head h, KV head g = h / G:
//   o_t^h = sum_{i <= c_b + t} softmax_i(scale * q_t^h . k_i) v_i.
//
// A work item is one pair of query tiles (A, B) of one (sequence, KV head):
// each tile holds TT = floor(128 / G) consecutive tokens times the G query
// heads of the group (row r = token * G + head), so a KV tile is read once for
// the whole group and for both query tiles.  Per KV tile of 128 positions (8
// pages) the tensor cores compute
//   S_X[128 x 128] = Q_X . K^T      (both operands in shared memory, K-major)
//   O_X[128 x D]  += P_X . V        (P_X in tensor memory, V MN-major)
// with S_A, S_B, O_A, O_B in tensor memory; P_X (bf16) overwrites the first 64
// columns of S_X at head_dim 128, which fills tensor memory, and has columns of
// its own at 64, where the next S follows as soon as this one is read.  The
// softmax is the running one: thread r of X's warpgroup owns row r
// (tensor-memory lane r) and keeps the row's reference m and sum l in registers.
// m is the row's maximum over the item's first tile; any other reference gives
// the same quotient, so later tiles take p = 2^(scale s - M), M = fl(scale m), in
// one fused multiply-add, without looking for their maximum, and only check the
// tile's sum: past 2^20 (or where nothing had been seen) m is raised to the tile's
// maximum, l and the row of O are rescaled, and the tile is taken again.  bf16 and
// fp32 hold numbers of that size as exactly as smaller ones.  Where M itself is
// past 2^20, what its rounding leaves would show: there the tile is always taken
// again, as 2^(scale (s - m)).
//
// The sum is checked once a tile: with a check in the middle (to hand P over in
// halves) the two halves' instructions could not overlap, which cost more than the
// earlier product gained (8192 rows of 64-wide heads 592 us with it, 539 without,
// 514 with the fused multiply-add too).
//
// Warps 0-3: softmax of A; 4-7: softmax of B; 8, 9: TMA of K and V tiles into
// one ring; 10: MMA issue; 11: walks the CTA's items, publishes them in a small
// shared ring and loads the Q tiles.
//
// Work division, found by every CTA from the lengths alone (no plan kernel):
// with enough items they are dealt out whole, longest first and back and forth
// over the CTAs.  Otherwise items carry the cost c0 + (positions up to the
// item's last row), whose prefix sums have a closed form, and CTA i of N takes
// the i-th of N equal ranges of the summed cost.  A range may begin and end
// inside an item; such an item's partial (m, l, O) go through the workspace and
// the CTA that arrives last joins them in range order.  So a single decode row
// with a long cache spreads over all SMs, with at most two partial items a CTA.
// Sequences of few rows (decode) and of many (prompts) in one batch get CTAs of
// their own, so that only items that are cheap to join are split: divide().
//
// What bounds it: at long lengths the tensor cores and the softmax together.  A
// pair of tiles needs 2048 tensor cycles a KV tile at head_dim 128; the softmax
// of one 128 x 128 tile takes a warp about 900 cycles alone and 750 when two
// share a scheduler (ex2 issues every 4 cycles, beside conversions; in the kernel
// 1100, where A and B, the fetches and the checks meet), and at
// head_dim 128 S(t + 1) needs tensor memory that P(t) occupies, so a tile's
// softmax and its two products follow one another and A and B overlap each
// other's: 2580 cycles a KV tile measured.  A prompt of 16384 rows (32 query
// heads of 128): 1190 us alone (1.85 PFLOP/s, 0.96 of the measured cuBLAS burst,
// tensor pipe 79 % active), 1280-1390 us back to back (power-capped, as cuBLAS
// is); 1000 rows behind 31768 cached: 332 us alone (1.59 PFLOP/s).  At head_dim 64
// the softmax sets the pace by its latency (7128 packed rows: 142 us, no pipe more
// than 47 % busy; among other things each tile waits for the last one's P.V before
// it reads its S).  One row each of eight sequences of 32000 positions: 162 us
// (6.5 TB/s, 0.96 of the measured copy).
#include "kernels.h"
#include "ticket.h"
#include "vegas_common.cuh"

namespace vegas {

namespace {

constexpr int kPThreads = 384;
constexpr int kTile = 128;            // KV positions per tile, query rows per tile
constexpr int kItemCost = 256;        // an item's fixed cost, in positions
constexpr int kMinShare = 256;        // a CTA's least share of the cost, in positions
constexpr int kFewRows = 32;          // an item of at most so many rows is shared by A and B (and joined by any thread)
constexpr int kSplitCost = 1024;      // what sharing items costs a CTA, in positions
constexpr int kSplitCostFew = 128;    // the same for items of few rows
// Time of a KV tile of an item of few rows, of a tile of two full query tiles (1850 / 2700 cycles).
constexpr float kFewWeight = 0.69f;
constexpr int kFew = 1, kMany = 2;    // sequences of at most kFewRows query rows a KV head, and others
constexpr float kNoMax = -3e38f;      // reference of a row that has seen nothing
constexpr float kSumLimit = 1048576.f;   // a tile's sum that makes a row raise its reference
constexpr float kBigRef = 1048576.f;     // a scaled reference whose rounding would show

// An item, or the part of it in one CTA's range, as published to all warps.
struct Piece {
  int seq, g, tok0;    // tok0: first token of tile A in its sequence; seq < 0: no more
  int row0, n, ctx;
  int k0, k1;          // KV tiles of this piece
  int na, nb;          // KV tiles that query tiles A and B need
  int first, last;     // CTAs that share the item
  int alt;             // 1: few rows, all in tile A: A and B take its KV tiles in turn
};
constexpr int kPieces = 4;   // depth of the ring of published items

// The items that a CTA shares with others, at most two: the end of one that an earlier CTA began
// (0), and the one that it leaves unfinished (1).
struct Owed {
  int first, arrivals, tiles;   // the item's ticket, its CTAs (0: no such item), its query tiles
  int arrived[2];               // query tile x's group has arrived on its ticket
};

template <int D>
struct PCfg {
  static constexpr int kHalves = D / 64;
  static constexpr int kQ = kHalves * 128 * 128;      // one query tile [half][128 rows][128 B]
  static constexpr int kSlot = kHalves * 128 * 128;   // one K or V tile
  static constexpr int kSlots = D == 128 ? 5 : 10;
  // At head_dim 64 tensor memory has room for P beside S, so the next S is computed as soon as
  // the softmax has read this one, and shared memory for the next item's query tiles.
  static constexpr bool kOwnP = D == 64;
  static constexpr int kQBufs = D == 64 ? 2 : 1;
  static constexpr int kOffRing = 2 * kQBufs * kQ;
  static constexpr int kOffBar = kOffRing + kSlots * kSlot;
  static constexpr int kNumBars = 2 * kSlots + 2 + 2 + 2 + 2 + 2 * kQBufs + 1 + 2 * kPieces + 2;
  static constexpr int kOffMisc = kOffBar + 8 * kNumBars;
  static constexpr int kOffPieces = kOffMisc + 96 + 2 * (int)sizeof(Owed);
  static constexpr int kOffAlt = kOffPieces + kPieces * (int)sizeof(Piece);   // (m, l) of 32 rows
  static constexpr size_t kSmem = kOffAlt + 32 * 8 + 1024;
  static_assert(kSmem <= 227 * 1024 && kOffAlt % 8 == 0 && kOffPieces % 8 == 0, "shared memory");
  static constexpr uint32_t kO = 256;                  // first tensor-memory column of O_A
  static constexpr uint32_t kP = kOwnP ? 384 : 0;      // ... of P_A, and the step to P_B
  static constexpr uint32_t kPStep = kOwnP ? 64 : 128;
};

// One point of the linear order of all (sequence, KV head, query-tile pair) items.
struct Point {
  int seq, g, p, k;    // k: KV tile inside the item
  long long us;        // cost before the item
};

// A sequence's rows and its geometry.
struct Seq {
  int row0, n, ctx, pairs;
  long long per_head;  // summed cost of one head's items
};


// n / pair_tokens for 0 <= n < 2^24 + 2 * pair_tokens: with M = ceil(2^32 / d) the product's
// excess n * (M * d - 2^32) < n * d stays below 2^32 (d <= 256; a power of two has none).
__device__ __forceinline__ int pairs_in(const PromptParams& q, int n) {
  return (int)__umulhi((uint32_t)n, q.pair_inverse);
}

// floor(a / b) for a quotient below 2^20: a fast fp32 division, put right (a 64-bit
// integer division takes several hundred cycles at the start of every call).
__device__ __forceinline__ int small_quotient(long long a, long long b) {
  long long q = (long long)__fdividef((float)a, (float)b);
  while (q * b > a) --q;
  while ((q + 1) * b <= a) ++q;
  return (int)q;
}

// floor(i * total / n) for i <= n <= 2^16.
__device__ __forceinline__ long long share_begin(int i, long long total, int n) {
  if (total >> 31) return i * total / n;
  const unsigned t = (unsigned)total, q = t / n, r = t - q * n;
  return (long long)i * q + (unsigned)i * r / n;
}

// A sequence that is not of one of the given classes counts as empty.  The cached length of one
// without rows may hold anything.
__device__ __forceinline__ Seq load_seq(const PromptParams& q, int s, int classes) {
  Seq r;
  r.row0 = q.row_start[s];
  const int end = q.row_start[s + 1];
  r.ctx = q.ctx_lens[s];
  r.n = end - r.row0;
  // (one test for ctx and its upper limit, and no branch before it: the loads stay together;
  // n <= total_rows < 2^24 and 16 max_pages < 2^24, so nothing wraps where the rows are sound)
  const bool rows = r.row0 >= 0 & end >= r.row0 & end <= q.total_rows;
  const bool fits = (unsigned)r.ctx <= (unsigned)(q.max_pages * 16 - r.n) & r.n <= q.max_pages * 16;
  const bool sound = rows & (end == r.row0 | fits);
  if (!sound) set_error(q.err, kErrDeviceFault);
  if (!sound | end == r.row0) r.n = r.ctx = 0;
  if (!(classes & (r.n * q.group <= kFewRows ? kFew : kMany))) r.n = 0;
  r.pairs = pairs_in(q, r.n + q.pair_tokens - 1);
  const long long P = r.pairs;
  r.per_head = P * (r.ctx + kItemCost) + q.pair_tokens * (P * (P + 1) / 2);
  return r;
}

// Summed cost of a head's items before item p.
__device__ __forceinline__ long long cost_before(const PromptParams& q, const Seq& s, long long p) {
  return p * (s.ctx + kItemCost) + q.pair_tokens * (p * (p + 1) / 2);
}

__device__ __forceinline__ int tiles_of(const PromptParams& q, const Seq& s, int p, int x) {
  const int first = p * q.pair_tokens + x * q.tile_tokens;
  if (first >= s.n) return 0;
  const int last = min(s.n, first + q.tile_tokens) - 1;
  return (s.ctx + last) / kTile + 1;
}

// What the division of the work goes by, the same in every CTA that works on the same classes.
struct Division {
  long long total;     // summed cost of the classes' items
  int items;
  int ncta;            // CTAs that take part: base .. base + ncta - 1
  int whole;           // 1: items are dealt out whole, longest first; 0: equal ranges of the cost
  int classes, base;
};

// Items by falling cost: positions up to the item's last row, as ctx + (p + 1) * pair_tokens.
// With at most 32 sequences each lane holds one, and an item's rank is found by bisection.
__device__ __forceinline__ int items_from(const PromptParams& q, const Seq& s, int cost) {
  // items of this lane's sequence whose cost is at least `cost`
  const int above = cost - s.ctx;   // (p + 1) * pair_tokens >= above
  const int skip = above <= 0 ? 0 : pairs_in(q, above + q.pair_tokens - 1) - 1;
  return max(0, s.pairs - max(skip, 0)) * q.hkv;
}

// The item of rank k (whole warp; sq: lane's sequence; hi: an upper bound of its cost, lowered to it).
__device__ __forceinline__ void ranked(const PromptParams& q, const Seq& sq, int k, int& hi, int& seq,
                                       int& g, int& p) {
  const unsigned active = __ballot_sync(0xffffffffu, sq.pairs > 0);
  if ((active & (active - 1)) == 0) {   // one sequence: its last pairs first, a pair's heads in order
    seq = __ffs(active) - 1;
    const int back = k / q.hkv;
    g = k - back * q.hkv;
    p = __shfl_sync(0xffffffffu, sq.pairs, seq & 31) - 1 - back;
    hi = __shfl_sync(0xffffffffu, sq.ctx, seq & 31) + (p + 1) * q.pair_tokens;
    return;
  }
  int lo = 0;                       // the largest cost c with more than k items of cost >= c
  while (lo < hi) {
    const int mid = lo + (hi - lo + 1) / 2;
    if (__reduce_add_sync(0xffffffffu, items_from(q, sq, mid)) > k)
      lo = mid;
    else
      hi = mid - 1;
  }
  const int before = __reduce_add_sync(0xffffffffu, items_from(q, sq, lo + 1));
  // at this cost each sequence has one item a head, or none
  const bool one = items_from(q, sq, lo) > items_from(q, sq, lo + 1);
  const unsigned who = __ballot_sync(0xffffffffu, one);
  const int nth = (k - before) / q.hkv;
  g = (k - before) - nth * q.hkv;
  seq = __fns(who, 0, nth + 1);
  const int mine = pairs_in(q, max(0, lo - sq.ctx)) - 1;
  p = __shfl_sync(0xffffffffu, mine, seq & 31);
}

// The work of one class, from all lanes' sequences.
struct Load {
  long long total;
  int items, longest;   // longest: positions of the longest sequence with rows
};

__device__ __forceinline__ Load sum_load(const PromptParams& q, long long w, int items, int longest) {
  // (24 bits at a time: reductions take a tenth of a 64-bit butterfly's time)
  const unsigned w0 = __reduce_add_sync(0xffffffffu, (unsigned)w & 0xffffffu);
  const unsigned w1 = __reduce_add_sync(0xffffffffu, (unsigned)(w >> 24) & 0xffffffu);
  const unsigned w2 = __reduce_add_sync(0xffffffffu, (unsigned)(w >> 48));
  Load r;
  r.total = (((long long)w2 << 48) + ((long long)w1 << 24) + w0) * q.hkv;
  r.items = __reduce_add_sync(0xffffffffu, items) * q.hkv;
  r.longest = __reduce_max_sync(0xffffffffu, longest);
  return r;
}

// Whole items keep every CTA busy when there are enough of them: the makespan is then about the
// mean plus the part of the last round's items that not every CTA gets, and at least the longest
// item.  Splitting costs a CTA the partial states it writes and joins (kSplitCost).
//
// Where some sequences have few rows (decode) and others many (prompts), a part of the CTAs takes
// the ones, the rest the others: prompts' items can then stay whole, and the split ones are those
// that are cheap to join.  Every number of CTAs is tried, against all CTAs taking both.
// (A 509-row chunk with decode rows of 8100 positions and fewer: 35.5 us without.)
__device__ __forceinline__ Division divide(const PromptParams& q) {
  const int lane = threadIdx.x & 31, grid = gridDim.x;
  long long wf = 0, wm = 0;
  int itf = 0, itm = 0, lf = 0, lm = 0;
  for (int s = lane; s < q.batch; s += 32) {
    const Seq sq = load_seq(q, s, kFew | kMany);
    const int len = sq.n > 0 ? sq.ctx + sq.n : 0;
    if (sq.n * q.group <= kFewRows) {
      wf += sq.per_head;
      itf += sq.pairs;
      lf = max(lf, len);
    } else {
      wm += sq.per_head;
      itm += sq.pairs;
      lm = max(lm, len);
    }
  }
  const Load few = sum_load(q, wf, itf, lf), many = sum_load(q, wm, itm, lm);
  Division d;
  d.classes = kFew | kMany;
  d.base = 0;
  d.total = few.total + many.total;
  d.items = few.items + many.items;
  d.whole = 0;
  const bool can_deal = q.batch <= 32;   // (ranked() holds a sequence a lane)
  int n = grid, longest = max(few.longest, many.longest);
  if (few.items > 0 && many.items > 0) {
    const float wmany = (float)many.total, wfew = (float)few.total * kFewWeight;
    float best = INFINITY;
    int at = 0;   // CTAs for the sequences of many rows; 0: all CTAs take both
    for (int c = lane; c < grid; c += 32) {
      // makespans on n CTAs: in equal ranges, and dealt out whole (the part of the last round's
      // items, at the mean cost, that not every CTA gets)
      const float n = c ? c : grid, items = c ? many.items : d.items, w = c ? wmany : wmany + wfew;
      const float each = __fdividef(1.f, n), mean = w * each;
      const float rest = items - floorf(items * each) * n;
      const float gap = rest > 0.5f ? (n - rest) * __fdividef(mean, items) : 0.f;
      float t = mean + kSplitCost;
      if (can_deal) t = fminf(t, fmaxf((c ? many.longest : longest) + kItemCost, mean + gap));
      if (c) t = fmaxf(t, __fdividef(wfew, grid - c) + kSplitCostFew);
      if (t < best) {
        best = t;
        at = c;
      }
    }
    const unsigned least = __reduce_min_sync(0xffffffffu, __float_as_uint(best));
    const unsigned who = __ballot_sync(0xffffffffu, __float_as_uint(best) == least);
    at = __shfl_sync(0xffffffffu, at, __ffs(who) - 1);
    if (at > 0) {
      const bool mine = (int)blockIdx.x < at;
      const Load& l = mine ? many : few;
      d.classes = mine ? kMany : kFew;
      d.base = mine ? 0 : at;
      d.total = l.total;
      d.items = l.items;
      longest = l.longest;
      n = mine ? at : grid - at;
    }
  }
  d.ncta = (int)min((long long)n, max(1ll, d.total / kMinShare));   // (a shift)
  const bool only_few = d.classes == kFew || many.items == 0;
  const long long limit = share_begin(1, d.total, d.ncta) + (only_few ? kSplitCostFew : kSplitCost);
  if (can_deal && longest + kItemCost <= limit) {
    long long span = 0;
    const int rounds = (d.items + n - 1) / n, rest = d.items - (rounds - 1) * n;
    if (rounds > 1 && rest < n) {
      Seq sq{};
      if (lane < q.batch) sq = load_seq(q, lane, d.classes);
      int cost = longest + q.pair_tokens, seq, g, p;
      ranked(q, sq, (rounds - 1) * n, cost, seq, g, p);
      span = share_begin(n - rest, cost + kItemCost, n);
    }
    d.whole = share_begin(1, d.total, n) + span <= limit;
  }
  if (d.whole) d.ncta = n;
  return d;
}

// The point at cost u, moved to an item boundary when it would leave fewer
// than two tiles on one side of it (whole warp; every lane gets the result).
__device__ __forceinline__ Point locate(const PromptParams& q, int classes, long long u) {
  const int lane = threadIdx.x & 31;
  Point r;
  r.seq = q.batch;
  r.g = r.p = r.k = 0;
  r.us = 0;
  long long base = 0;
  for (int s0 = 0; s0 < q.batch; s0 += 32) {
    const int s = s0 + lane;
    Seq sq{};
    if (s < q.batch) sq = load_seq(q, s, classes);
    const long long mine = sq.per_head * q.hkv;
    long long incl = mine;
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
      const long long v = __shfl_up_sync(0xffffffffu, incl, o);
      if (lane >= o) incl += v;
    }
    const bool hit = mine > 0 && u < base + incl;
    const unsigned who = __ballot_sync(0xffffffffu, hit);
    if (who) {
      const int src = __ffs(who) - 1;
      sq.row0 = __shfl_sync(0xffffffffu, sq.row0, src);
      sq.n = __shfl_sync(0xffffffffu, sq.n, src);
      sq.ctx = __shfl_sync(0xffffffffu, sq.ctx, src);
      sq.pairs = __shfl_sync(0xffffffffu, sq.pairs, src);
      sq.per_head = __shfl_sync(0xffffffffu, sq.per_head, src);
      const long long sbase = base + __shfl_sync(0xffffffffu, incl - mine, src);
      r.seq = s0 + src;
      r.g = small_quotient(u - sbase, sq.per_head);
      const long long hbase = sbase + r.g * sq.per_head;
      const long long rem = u - hbase;
      int lo = 0, hi = sq.pairs - 1;   // the last p with cost_before(p) <= rem
      while (lo < hi) {
        const int mid = (lo + hi + 1) >> 1;
        if (cost_before(q, sq, mid) <= rem)
          lo = mid;
        else
          hi = mid - 1;
      }
      r.p = lo;
      r.us = hbase + cost_before(q, sq, lo);
      const long long o = u - r.us;
      const int nt = max(tiles_of(q, sq, lo, 0), tiles_of(q, sq, lo, 1));
      const long long k = o < kItemCost ? 0 : (o - kItemCost + kTile / 2) / kTile;
      if (k < 2) {
        r.k = 0;
      } else if (k <= nt - 2) {
        r.k = (int)k;
      } else {   // the next item
        r.us = hbase + cost_before(q, sq, lo + 1);
        r.k = 0;
        if (++r.p == sq.pairs) {
          r.p = 0;
          if (++r.g == q.hkv) {
            r.g = 0;
            ++r.seq;   // may be an empty sequence: the walk skips those
          }
        }
      }
      return r;
    }
    base += __shfl_sync(0xffffffffu, incl, 31);
  }
  r.us = base;
  return r;
}

// Walks the items of a CTA's range.
struct Walk {
  Point at, end;
  Seq s;               // the sequence at `at`; whole items: the lane's sequence
  bool have;
  int round, cost;     // whole items: rounds dealt so far, the last item's cost

  __device__ __forceinline__ Walk(const Point& a, const Point& e)
      : at(a), end(e), have(false), round(0), cost(0) {}

  __device__ __forceinline__ void fill(const PromptParams& q, const Seq& sq, int seq, int g, int p,
                                       Piece& w) {
    w.seq = seq;
    w.g = g;
    w.tok0 = p * q.pair_tokens;
    w.row0 = sq.row0;
    w.n = sq.n;
    w.ctx = sq.ctx;
    w.na = tiles_of(q, sq, p, 0);
    w.nb = tiles_of(q, sq, p, 1);
    w.k0 = 0;
    w.k1 = max(w.na, w.nb);
    w.first = w.last = blockIdx.x;
    // (for the whole item, so that all its CTAs count the same partial states)
    w.alt = w.nb == 0 && w.na >= 4 && (sq.n - w.tok0) * q.group <= kFewRows;
  }

  // Items dealt out whole, longest first, back and forth over the CTAs.
  __device__ __forceinline__ bool next_whole(const PromptParams& q, const Division& d, Piece& w) {
    const int lane = threadIdx.x & 31;
    if (round == 0) {
      s = Seq{};
      if (lane < q.batch) s = load_seq(q, lane, d.classes);
      cost = __reduce_max_sync(0xffffffffu, s.pairs > 0 ? s.ctx + s.pairs * q.pair_tokens : 0);
    }
    const int N = d.ncta, me = (int)blockIdx.x - d.base;
    const int k = round * N + ((round & 1) ? N - 1 - me : me);
    ++round;
    if (k >= d.items) return false;
    int seq, g, p;
    ranked(q, s, k, cost, seq, g, p);
    Seq sq;
    sq.row0 = __shfl_sync(0xffffffffu, s.row0, seq & 31);
    sq.n = __shfl_sync(0xffffffffu, s.n, seq & 31);
    sq.ctx = __shfl_sync(0xffffffffu, s.ctx, seq & 31);
    fill(q, sq, seq, g, p, w);
    return true;
  }

  __device__ __forceinline__ bool next(const PromptParams& q, const Division& d, Piece& w) {
    if (d.whole) return next_whole(q, d, w);
    while (true) {
      if (at.seq >= q.batch || at.seq > end.seq) return false;
      if (!have) {
        s = load_seq(q, at.seq, d.classes);
        have = true;
      }
      if (s.pairs == 0) {
        ++at.seq;
        have = false;
        continue;
      }
      const bool stop = at.seq == end.seq && at.g == end.g && at.p == end.p;
      if (stop && end.k <= at.k) return false;
      fill(q, s, at.seq, at.g, at.p, w);
      const int nt = w.k1;
      w.k0 = at.k;
      w.k1 = stop ? end.k : nt;
      if (w.k0 > 0 || w.k1 < nt) {
        // Boundary i sits at floor(i * total / ncta), which is >= x exactly when
        // i >= ceil(x * ncta / total); those in [a, b) fall inside the item (locate()).
        const long long a = at.us + kItemCost + 2 * kTile - kTile / 2;
        const long long b = at.us + kItemCost + (long long)kTile * nt - 2 * kTile + kTile / 2;
        w.first = d.base + small_quotient(a * d.ncta + d.total - 1, d.total) - 1;
        w.last = d.base + small_quotient(b * d.ncta + d.total - 1, d.total) - 1;
      }
      if (stop) {
        at.seq = q.batch;   // done
      } else {
        at.us += s.ctx + kItemCost + (long long)q.pair_tokens * (at.p + 1);
        at.k = 0;
        if (++at.p == s.pairs) {
          at.p = 0;
          if (++at.g == q.hkv) {
            at.g = 0;
            ++at.seq;
            have = false;
          }
        }
      }
      return true;
    }
  }
};

}  // namespace

template <int D>
__global__ void __launch_bounds__(kPThreads, 1)
    prompt_attn_kernel(const __grid_constant__ CUtensorMap kmap,
                       const __grid_constant__ CUtensorMap vmap,
                       const __grid_constant__ CUtensorMap qmap, const PromptParams q) {
  using Cfg = PCfg<D>;
  constexpr int NS = Cfg::kSlots;
  griddep_launch_dependents();
  extern __shared__ uint8_t smem_raw[];
  uint8_t* smem = reinterpret_cast<uint8_t*>((reinterpret_cast<uintptr_t>(smem_raw) + 1023) &
                                             ~uintptr_t(1023));
  const uint32_t sbase = smem_u32(smem);
  const uint32_t bar0 = sbase + Cfg::kOffBar;
  auto full = [&](uint32_t s) { return bar0 + 8 * s; };
  auto freed = [&](uint32_t s) { return bar0 + 8 * (NS + s); };
  auto sfull = [&](int x) { return bar0 + 8 * (2 * NS + x); };
  constexpr int B1 = 2 * NS + 2, QB = Cfg::kQBufs, B2 = B1 + 6 + 2 * QB;
  auto pready = [&](int x) { return bar0 + 8 * (B1 + x); };
  auto odone = [&](int x) { return bar0 + 8 * (B1 + 2 + x); };
  auto sread = [&](int x) { return bar0 + 8 * (B1 + 4 + x); };
  auto qfull = [&](uint32_t i) { return bar0 + 8 * (B1 + 6 + i % QB); };
  auto qfree = [&](uint32_t i) { return bar0 + 8 * (B1 + 6 + QB + i % QB); };
  const uint32_t drain = bar0 + 8 * B2, altfull = drain + 8, alttaken = drain + 16;
  auto pcfull = [&](uint32_t i) { return bar0 + 8 * (B2 + 3 + i); };
  auto pcfree = [&](uint32_t i) { return bar0 + 8 * (B2 + 3 + kPieces + i); };
  uint32_t* tmem_slot = reinterpret_cast<uint32_t*>(smem + Cfg::kOffMisc);
  int* flags = reinterpret_cast<int*>(smem + Cfg::kOffMisc + 4);          // [2]
  int* ends = reinterpret_cast<int*>(smem + Cfg::kOffMisc + 16);          // [2][6]
  Division* division = reinterpret_cast<Division*>(smem + Cfg::kOffMisc + 64);
  Owed* owed = reinterpret_cast<Owed*>(smem + Cfg::kOffMisc + 96);        // [2]
  float2* alt_ml = reinterpret_cast<float2*>(smem + Cfg::kOffAlt);
  Piece* pieces = reinterpret_cast<Piece*>(smem + Cfg::kOffPieces);

  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
  if (tid == 0) {
    for (int s = 0; s < NS; ++s) {
      mbar_init(full(s), 1);
      mbar_init(freed(s), 1);
    }
    for (int x = 0; x < 2; ++x) {
      mbar_init(sfull(x), 1);
      mbar_init(pready(x), 4);   // a warp each
      mbar_init(odone(x), 1);
      mbar_init(sread(x), 4);
    }
    for (int i = 0; i < QB; ++i) {
      mbar_init(qfull(i), 1);
      mbar_init(qfree(i), 1);
    }
    mbar_init(drain, 1);
    mbar_init(altfull, 32);
    mbar_init(alttaken, 32);
    for (int i = 0; i < kPieces; ++i) {
      mbar_init(pcfull(i), 1);
      mbar_init(pcfree(i), 11);   // one arrival per reading warp
    }
    fence_mbar_init();
  }
  if (warp == 4 && lane < 2) owed[lane] = Owed{};
  if (tid == 32) prefetch_tensormap(&kmap);
  if (tid == 64) prefetch_tensormap(&vmap);
  if (tid == 96) prefetch_tensormap(&qmap);
  if (warp == 10) {
    tmem_alloc(smem_u32(tmem_slot), 512);
    tmem_relinquish();
  }
  griddep_wait();

  // The CTA's range of the summed cost: warp 8 finds its begin, warp 9 its end.
  if (warp >= 8 && warp < 10) {
    const Division d = divide(q);
    const int i = (int)blockIdx.x - d.base + (warp - 8);
    Point pt;
    if (i >= d.ncta || d.total == 0 || d.whole) {
      pt.seq = q.batch;
      pt.g = pt.p = pt.k = 0;
      pt.us = d.total;
    } else {
      pt = locate(q, d.classes, share_begin(i, d.total, d.ncta));
    }
    if (lane == 0) {
      int* e = ends + 6 * (warp - 8);
      e[0] = pt.seq;
      e[1] = pt.g;
      e[2] = pt.p;
      e[3] = pt.k;
      e[4] = (int)(pt.us & 0xffffffffll);
      e[5] = (int)(pt.us >> 32);
      if (warp == 8) *division = d;
    }
  }
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  const uint32_t tmem = *tmem_slot;
  uint32_t pc = 0;   // items read so far
  // The next published item (whole warp); false when there is none.
  auto next_piece = [&](Piece& w, bool& ok) {
    const uint32_t i = pc % kPieces;
    if (!__all_sync(0xffffffffu, mbar_wait_bounded(pcfull(i), (pc / kPieces) & 1))) {
      ok = false;
      return false;
    }
    w = pieces[i];
    __syncwarp();
    if (lane == 0) mbar_arrive(pcfree(i));
    ++pc;
    return w.seq >= 0;
  };
  Piece w;
  bool ok = true;
  // 384 threads launch with 168 registers each: 2 x 128 x 216 + 128 x 72 are that.  Each
  // warpgroup's instruction stands inside its branch (where the branches join the smaller count
  // would rule) and is one for all its warps, whatever their roles.
  if (warp >= 8) {
    leave_registers<72>();
    if (warp < 10) {
      // ------------------------------------------------------------ K (8) and V (9) tiles
      // Lane j < 8 * D/64 issues box (page j % 8, half j / 8): 16 positions x 64 dims.
      const bool is_v = warp == 9;
      const CUtensorMap* map = is_v ? &vmap : &kmap;
      const int page = lane & 7, half = lane >> 3;
      uint32_t c = 0;       // tiles so far
      uint32_t issued = 0;  // of them, issued
      while (ok && next_piece(w, ok)) {
        const int32_t* row = q.block_table + size_t(w.seq) * q.max_pages;
        const int npages = (w.ctx + w.n + 15) / 16;
        int phys = __ldg(&row[min(8 * w.k0 + page, npages - 1)]);
        for (int t = w.k0; t < w.k1; ++t, ++c) {
          // a tile's pages past the sequence's end are loaded as its last page (their
          // positions are masked)
          const int now = phys;
          if (t + 1 < w.k1) phys = __ldg(&row[min(8 * (t + 1) + page, npages - 1)]);
          int pg = now;
          if (pg < 0 || pg >= q.num_pages) {
            set_error(q.err, kErrDeviceFault);
            pg = 0;
          }
          const uint32_t j = 2 * c + (is_v ? 1 : 0), s = j % NS, use = j / NS;
          if (use > 0 &&
              !__all_sync(0xffffffffu, mbar_wait_bounded(freed(s), (use - 1) & 1))) {
            ok = false;
            break;
          }
          if (lane == 0) mbar_arrive_expect_tx(full(s), Cfg::kSlot);
          __syncwarp();
          if (half < Cfg::kHalves)
            tma_load_2d(sbase + Cfg::kOffRing + s * Cfg::kSlot + half * 16384 + page * 2048, map,
                        64 * half, (pg * q.hkv + w.g) * 16, full(s));
          __syncwarp();
          issued = c + 1;
        }
      }
      // every copy in flight lands before the CTA ends (the ring's last NS tiles)
      for (uint32_t t = issued > NS ? issued - NS : 0; t < issued; ++t) {
        const uint32_t j = 2 * t + (is_v ? 1 : 0);
        if (j + NS >= 2 * issued) (void)mbar_wait_bounded(full(j % NS), (j / NS) & 1);
      }
      if (!ok && lane == 0) set_error(q.err, kErrDeviceTimeout);
    } else if (warp == 11) {
      // ------------------------------------------------------------ items, Q tiles
      auto point = [&](int e0) {
        const int* e = ends + 6 * e0;
        Point r;
        r.seq = e[0];
        r.g = e[1];
        r.p = e[2];
        r.k = e[3];
        r.us = ((long long)e[5] << 32) | (uint32_t)e[4];
        return r;
      };
      Walk walk(point(0), point(1));
      const Division d = *division;
      uint32_t c = 0;
      auto owe = [&]() {   // (read once every warp is done)
        if (lane == 0 && w.first != w.last) {
          Owed& o = owed[w.last == (int)blockIdx.x ? 0 : 1];
          o.first = w.first;
          o.arrivals = w.last - w.first + 1;
          o.tiles = w.nb > 0 ? 2 : 1;
        }
      };
      while (ok) {
        const bool more = walk.next(q, d, w);
        if (more) owe();
        if (!more) w.seq = -1;
        const uint32_t i = c % kPieces;
        if (c >= kPieces &&
            !__all_sync(0xffffffffu, mbar_wait_bounded(pcfree(i), (c / kPieces - 1) & 1))) {
          ok = false;
          break;
        }
        if (lane == 0) {
          pieces[i] = w;
          mbar_arrive(pcfull(i));
        }
        __syncwarp();
        if (!more) break;
        const int tiles = w.nb > 0 ? 2 : 1;
        const int qrow = w.row0 + w.tok0;
        if (c >= QB && lane < tiles * Cfg::kHalves)   // on their way while the last item still uses the buffer
          tma_prefetch_3d(&qmap, 64 * (lane % Cfg::kHalves), w.g * q.group,
                          qrow + lane / Cfg::kHalves * q.tile_tokens);
        if (c >= QB && !__all_sync(0xffffffffu, mbar_wait_bounded(qfree(c), (c / QB - 1) & 1))) {
          ok = false;
          break;
        }
        const uint32_t bytes = uint32_t(q.tile_tokens * q.group) * 128;   // one box
        if (lane == 0) {
          mbar_arrive_expect_tx(qfull(c), bytes * tiles * Cfg::kHalves);
          for (int x = 0; x < tiles; ++x)
            for (int h = 0; h < Cfg::kHalves; ++h)
              tma_load_3d(sbase + (2 * (c % QB) + x) * Cfg::kQ + h * 16384, &qmap, 64 * h, w.g * q.group,
                          qrow + x * q.tile_tokens, qfull(c));
        }
        __syncwarp();
        ++c;
      }
      for (uint32_t i = c > QB ? c - QB : 0; i < c; ++i)   // landed before the CTA ends
        (void)mbar_wait_bounded(qfull(i), (i / QB) & 1);
      if (!ok && lane == 0) set_error(q.err, kErrDeviceTimeout);
      if (!ok)
        while (walk.next(q, d, w)) owe();
    } else if (warp == 10) {
      // ------------------------------------------------------------ MMA issue
      // One thread waits, issues and commits: its instructions lie on the path from a tile's P
      // to its next S, so ring positions and phases are kept as running values and a step's
      // descriptors differ from its first one by constants.
      if (elect_one()) {
        constexpr uint32_t idS = idesc_bf16(128, 128, 0, 0);
        constexpr uint32_t idPV = idesc_bf16(128, D, 0, 1);
        // K-major operands with the 128-byte swizzle; V MN-major, 64-dim halves 16 KB apart.
        // Addresses are below 2^18, so the descriptor's address field takes plain sums.
        constexpr uint64_t dSw = smem_desc_const(16, 1024, 2), dVmn = smem_desc_const(16384, 1024, 2);
        const uint32_t q16 = sbase >> 4, ring16 = (sbase + Cfg::kOffRing) >> 4;
        struct Ring {          // a position in the ring: slot and phase
          uint32_t s, ph;
          __device__ __forceinline__ void next() {   // (K and V take turns)
            s += 2;
            if (s >= NS) {
              s -= NS;
              ph ^= 1;
            }
          }
        };
        Ring kr{0, 0}, vr{1, 0};   // the next K to multiply, the next V
        uint32_t pa = 0, pb = 0;   // phases of A's and B's P
        uint32_t ra = 0, rb = 0;   // and of their S being read (kOwnP)
        uint32_t items = 0;
        auto wait_k = [&]() { return mbar_wait_bounded(full(kr.s), kr.ph); };
        auto wait_v = [&]() { return mbar_wait_bounded(full(vr.s), vr.ph); };
        auto free_k = [&]() {
          tc_commit(freed(kr.s));
          kr.next();
        };
        auto free_v = [&]() {
          tc_commit(freed(vr.s));
          vr.next();
        };
        auto issue_s = [&](int x, int qtile) {
          const uint64_t a = dSw + (q16 + (2 * (items % QB) + qtile) * (Cfg::kQ / 16));
          const uint64_t bk = dSw + (ring16 + kr.s * (Cfg::kSlot / 16));
          tc_fence_after();
  #pragma unroll
          for (int ks = 0; ks < D / 16; ++ks)
            tc_mma(tmem + 128 * x, a + ((ks >> 2) * 1024 + (ks & 3) * 2),
                   bk + ((ks >> 2) * 1024 + (ks & 3) * 2), idS, ks > 0);
          tc_commit(sfull(x));
        };
        // where P has its own place, S may be overwritten once the softmax has read it
        auto wait_read = [&](int x) {
          if constexpr (!Cfg::kOwnP) return true;
          uint32_t& ph = x ? rb : ra;
          const bool read = mbar_wait_bounded(sread(x), ph);
          ph ^= 1;
          return read;
        };
        // O_X += P_X . V, once the softmax has left P_X; last: X's last tile here
        auto issue_pv = [&](int x, bool accumulate, bool last) {
          uint32_t& ph = x ? pb : pa;
          const uint64_t bv = dVmn + (ring16 + vr.s * (Cfg::kSlot / 16));
          if (!mbar_wait_bounded(pready(x), ph)) return false;
          tc_fence_after();
  #pragma unroll
          for (int kp = 0; kp < kTile / 16; ++kp)
            tc_mma_ts(tmem + Cfg::kO + D * x, tmem + Cfg::kP + Cfg::kPStep * x + 8 * kp, bv + kp * 128,
                      idPV, accumulate || kp > 0);
          ph ^= 1;
          if (Cfg::kOwnP || last) tc_commit(odone(x));
          return true;
        };
        // false: a wait ran out
        auto run_pair = [&](int k0, int k1, int ea, int eb) {
          if (!wait_k()) return false;
          if (k0 < ea) issue_s(0, 0);
          if (k0 < eb) issue_s(1, 1);
          free_k();
          if (k0 + 1 == k1) tc_commit(qfree(items));
          for (int t = k0; t < k1; ++t) {
            bool have_k = false, have_v = false;
  #pragma unroll
            for (int x = 0; x < 2; ++x) {
              const int ex = x ? eb : ea;
              if (t >= ex) continue;
              auto next_s = [&]() {
                if (!wait_read(x)) return false;
                if (t + 1 >= ex) return true;
                if (!have_k && !wait_k()) return false;
                have_k = true;
                issue_s(x, x);
                return true;
              };
              if (Cfg::kOwnP && !next_s()) return false;
              if (!have_v && !wait_v()) return false;
              have_v = true;
              if (!issue_pv(x, t > k0, t + 1 == ex)) return false;
              if (!Cfg::kOwnP) {
                if (x == 1 || t >= eb) free_v();
                if (!next_s()) return false;
              }
            }
            if (Cfg::kOwnP) free_v();
            if (t + 1 < k1) {
              free_k();
              if (t + 2 == k1) tc_commit(qfree(items));
            }
          }
          return true;
        };
        // tile i to A or B in turn, each with its own S, P and O, both from query tile A
        auto run_alternating = [&](int tiles) {
          for (int i = 0; i < min(2, tiles); ++i) {
            if (!wait_k()) return false;
            issue_s(i, 0);
            free_k();
          }
          if (tiles <= 2) tc_commit(qfree(items));
          for (int i = 0; i < tiles; ++i) {
            const int x = i & 1;
            auto next_s = [&]() {
              if (!wait_read(x)) return false;
              if (i + 2 >= tiles) return true;
              if (!wait_k()) return false;
              issue_s(x, 0);
              free_k();
              if (i + 3 == tiles) tc_commit(qfree(items));
              return true;
            };
            if (Cfg::kOwnP && !next_s()) return false;
            if (!wait_v() || !issue_pv(x, i >= 2, i + 2 >= tiles)) return false;
            free_v();
            if (!Cfg::kOwnP && !next_s()) return false;
          }
          return true;
        };
        while (true) {
          const uint32_t i = pc % kPieces;
          if (!mbar_wait_bounded(pcfull(i), (pc / kPieces) & 1)) {
            ok = false;
            break;
          }
          const int seq = pieces[i].seq, k0 = pieces[i].k0, k1 = pieces[i].k1;
          const int ea = min(k1, pieces[i].na), eb = min(k1, pieces[i].nb), alt = pieces[i].alt;
          mbar_arrive(pcfree(i));
          ++pc;
          if (seq < 0) break;
          if (!mbar_wait_bounded(qfull(items), (items / QB) & 1) ||
              !(alt ? run_alternating(k1 - k0) : run_pair(k0, k1, ea, eb))) {
            ok = false;
            break;
          }
          ++items;
        }
        if (!ok) set_error(q.err, kErrDeviceTimeout);
        tc_commit(drain);
      }
      __syncwarp();
      // every MMA issued has completed before tensor memory is released
      (void)mbar_wait_bounded(drain, 0);
    }
  } else {
    take_registers<216>();
    // ------------------------------------------------------------ softmax of tile X
    const int x = warp >> 2;
    const int r = tid & 127;
    const uint32_t tl = tmem + (uint32_t(32 * (warp & 3)) << 16);
    const uint32_t scol = 128 * x, ocol = Cfg::kO + D * x, pcol = Cfg::kP + Cfg::kPStep * x;
    uint32_t c = 0, ns = 0, no = 0;   // ring tiles, S tiles, finished items of X
    uint32_t nalt = 0;                // items that A and B shared
    // A row's exponents are scale * logit - M with M = m * scale rounded once, which any other
    // reference could replace; residue() is what the rounding left, for states of another m.
    // Where M is so large that its rounding would show, the difference is taken before scaling.
    auto residue = [&](float of) {
      const float M = of * q.scale_log2;
      return fabsf(M) < kBigRef ? fmaf(of, q.scale_log2, -M) : 0.f;
    };
    // the factor that takes a state of reference `from` to the reference `to`
    auto moved = [&](float from, float to) {
      return ex2(fmaf(from - to, q.scale_log2, residue(to) - residue(from)));
    };
    // The item's fields stay in shared memory until its end: the tile loop needs the registers.
    auto release = [&]() {
      __syncwarp();
      if (lane == 0) mbar_arrive(pcfree(pc % kPieces));
      ++pc;
    };
    // The group's four warps leave this loop together, by a vote that all of them see: here, or
    // at the end of an item.  A warp that left by itself after a wait that ran out would be
    // missed, for good, at the group's next barrier by warps whose wait just ended in time.
    while (true) {
      const Piece& w = pieces[pc % kPieces];
      const bool got =
          __all_sync(0xffffffffu, mbar_wait_bounded(pcfull(pc % kPieces), (pc / kPieces) & 1));
      if (!got || w.seq < 0) {
        ok = !named_bar_any(1 + x, 128, !got);
        break;
      }
      const int kbeg = w.k0 + (w.alt ? x : 0), kstep = w.alt ? 2 : 1;
      const int kend = w.alt ? w.k1 : min(w.k1, (x ? w.nb : w.na));
      // lim: the last position this row may see (rows behind the sequence: its last);
      // seen: the last one that all rows of the tile may; vzero: the tile whose V this group mends
      int lim, seen, vzero;
      bool live;   // rows 0 .. rows - 1 of the tile exist
      {
        const int first_tok = w.tok0 + (w.alt ? 0 : x * q.tile_tokens);
        lim = w.ctx + min(first_tok + r / q.group, w.n - 1);
        seen = w.ctx + first_tok;
        live = r < min(q.tile_tokens, w.n - first_tok) * q.group;
        vzero = (w.ctx + w.n) % kTile ? (w.ctx + w.n) / kTile : -1;
        if (!w.alt && x == 1 && vzero < w.na) vzero = -1;
      }
      float m = kNoMax, l = 0.f;
      for (int t = kbeg; t < kend; t += kstep) {
        if (!__all_sync(0xffffffffu, mbar_wait_bounded(sfull(x), ns & 1))) {
          ok = false;
          break;
        }
        ++ns;
        tc_fence_after();
        float s[128];
        const int pos0 = t * kTile;
        const bool diagonal = pos0 + kTile - 1 > seen;
        const int cut = lim - pos0;   // the row's last visible position in the tile
#pragma unroll
        for (int i = 0; i < 4; ++i) tmem_ld32(tl + scol + 32 * i, s + 32 * i);
        if constexpr (Cfg::kOwnP) {
          if (t > kbeg) {   // the last tile's P has been used (and its O is complete)
            ok = __all_sync(0xffffffffu, mbar_wait_bounded(odone(x), no & 1)) && ok;
            ++no;
            tc_fence_after();
          }
        }
        tmem_ld_wait();
        if constexpr (Cfg::kOwnP) {
          tc_fence_before();
          __syncwarp();
          if (lane == 0) mbar_arrive(sread(x));
        }
        if (diagonal) {   // whatever the logits hold
#pragma unroll
          for (int i = 0; i < 128; ++i)
            if (i > cut) s[i] = -INFINITY;
        }
        if (t == kbeg) {
          float mx = s[0];
#pragma unroll
          for (int i = 1; i < 128; ++i) mx = fmaxf(mx, s[i]);
          m = fmaxf(mx, kNoMax);
        }
        if (t == vzero) {
          // slots past the sequence may hold anything: zero their V rows, as 0 * NaN is NaN
          const uint32_t j = 2 * (c + (t - w.k0)) + 1;
          const int kv_len = w.ctx + w.n;
          ok = __all_sync(0xffffffffu, mbar_wait_bounded(full(j % NS), (j / NS) & 1)) && ok;
          if (ok && pos0 + r >= kv_len) {
            uint8_t* row = smem + Cfg::kOffRing + (j % NS) * Cfg::kSlot + r * 128;
#pragma unroll
            for (int h = 0; h < Cfg::kHalves; ++h)
#pragma unroll
              for (int e = 0; e < 8; ++e)
                *reinterpret_cast<uint4*>(row + h * 16384 + 16 * ((e + r) & 7)) =
                    make_uint4(0, 0, 0, 0);   // (8 lanes, 8 banks)
          }
          fence_proxy_async_smem();
        }
        const uint64_t sc2 = pair_f32(q.scale_log2, q.scale_log2);
        uint32_t pk[kTile / 2];   // P to 8 bits of mantissa: the tensor cores' operand type
        float ts;
        auto take = [&](auto exponents) {
          uint64_t sum[2] = {0ull, 0ull};
#pragma unroll
          for (int e = 0; e < kTile / 2; ++e) {
            float a, b;
            unpair_f32(exponents(pair_f32(s[2 * e], s[2 * e + 1])), a, b);
            a = ex2(a);
            b = ex2(b);
            sum[e & 1] = add_f32x2(sum[e & 1], pair_f32(a, b));
            pk[e] = pack_bf16x2(a, b);
            // (nothing reads it before this tile's arrival)
            if ((e & 15) == 15) tmem_st16(tl + pcol + (e - 15), pk + (e - 15));
          }
          float la, lb;
          unpair_f32(add_f32x2(sum[0], sum[1]), la, lb);
          ts = la + lb;
        };
        {
          const float M = m * q.scale_log2, nm = fabsf(M) < kBigRef ? -M : NAN;
          const uint64_t nm2 = pair_f32(nm, nm);
          take([&](uint64_t v) { return fma_f32x2(v, sc2, nm2); });
        }
        if (__any_sync(0xffffffffu, !(ts < kSumLimit) && live)) {
          tmem_st_wait();   // stores are asynchronous: this P lies before the next goes over it
          float mx = s[0];
#pragma unroll
          for (int i = 1; i < 128; ++i) mx = fmaxf(mx, s[i]);
          const float m2 = fmaxf(m, mx);
          const float f = moved(m, m2);
          m = m2;
          l *= f;
          if (t > kbeg) {   // O holds the row's earlier tiles, complete (S came after them, or waited for)
#pragma unroll
            for (int i = 0; i < D / 16; ++i) {
              float o[16];
              tmem_ld16(tl + ocol + 16 * i, o);
              tmem_ld_wait();
              uint32_t ob[16];
#pragma unroll
              for (int e = 0; e < 16; ++e) ob[e] = __float_as_uint(o[e] * f);
              tmem_st16(tl + ocol + 16 * i, ob);
            }
          }
          const float rest = residue(m);
          const uint64_t nm2 = pair_f32(-m, -m), rest2 = pair_f32(rest, rest);
          take([&](uint64_t v) { return fma_f32x2(add_f32x2(v, nm2), sc2, rest2); });
        }
        l += ts;
        tmem_st_wait();
        tc_fence_before();
        __syncwarp();
        if (lane == 0) mbar_arrive(pready(x));
        if (!ok) break;
      }
      c += w.k1 - w.k0;
      const bool any = kend > kbeg;
      if (any) {
        if (ok && !__all_sync(0xffffffffu, mbar_wait_bounded(odone(x), no & 1))) ok = false;
        ++no;
        tc_fence_after();
      }
      if (w.alt && (warp & 3) == 0) {
        // The item's rows lie in tensor-memory lanes 0-31, which both groups' first warps
        // reach: B's tells its (m, l), A's joins O_B to O_A and says when it has read it.
        if (x == 1) {
          alt_ml[lane] = make_float2(m, l);
          tc_fence_before();
          mbar_arrive(altfull);
          if (ok && !__all_sync(0xffffffffu, mbar_wait_bounded(alttaken, nalt & 1))) ok = false;
        } else {
          if (ok && !__all_sync(0xffffffffu, mbar_wait_bounded(altfull, nalt & 1))) ok = false;
          tc_fence_after();
          if (ok && w.k1 - w.k0 > 1) {
            const float2 b = alt_ml[lane];
            const float m2 = fmaxf(m, b.x);
            const float fa = moved(m, m2), fb = moved(b.x, m2);
            m = m2;
            l = fa * l + fb * b.y;
#pragma unroll 1
            for (int i = 0; i < D / 16; ++i) {
              float oa[16], ob[16];
              tmem_ld16(tl + Cfg::kO + 16 * i, oa);
              tmem_ld16(tl + Cfg::kO + D + 16 * i, ob);
              tmem_ld_wait();
              uint32_t o[16];
#pragma unroll
              for (int e = 0; e < 16; ++e) o[e] = __float_as_uint(fa * oa[e] + fb * ob[e]);
              tmem_st16(tl + Cfg::kO + 16 * i, o);
            }
            tmem_st_wait();
          }
          tc_fence_before();
          mbar_arrive(alttaken);
        }
      }
      if (w.alt) ++nalt;
      ok = !named_bar_any(1 + x, 128, !ok);
      if (!ok) break;
      if ((x ? w.nb : w.na) == 0) {   // no such rows, or joined to A's
        release();
        continue;
      }
      const int first_tok = w.tok0 + (w.alt ? 0 : x * q.tile_tokens);
      const int rows = min(q.tile_tokens, w.n - first_tok) * q.group;
      __nv_bfloat16* out0 = reinterpret_cast<__nv_bfloat16*>(q.out) +
                            ((size_t(w.row0) + first_tok) * q.hq + size_t(w.g) * q.group) * D;
      auto out_row = [&](int rr) {
        const int tk = rr / q.group;
        return out0 + (size_t(tk) * q.hq + (rr - tk * q.group)) * D;
      };
      if (w.first == w.last) {
        const float inv = 1.f / l;
        __nv_bfloat16* o_row = out_row(r);
#pragma unroll
        for (int i = 0; i < D / 32; ++i) {
          float o[32];
          tmem_ld32(tl + ocol + 32 * i, o);
          tmem_ld_wait();
          if (live) {
#pragma unroll
            for (int e = 0; e < 2; ++e) {   // whole 32-byte sectors
              uint32_t v[8];
#pragma unroll
              for (int u = 0; u < 8; ++u)
                v[u] = pack_bf16x2(o[16 * e + 2 * u] * inv, o[16 * e + 2 * u + 1] * inv);
              store_32_bytes(o_row + 32 * i + 16 * e, v);
            }
          }
        }
        tc_fence_before();
        release();
        continue;
      }
      // A partial item.  Slot 2 * CTA + 1 holds the piece that the CTA leaves
      // unfinished, slot 2 * CTA the end of an item begun by an earlier CTA;
      // O as [D / 4][128 rows] float4.  Whoever arrives last joins the states,
      // in their fixed order.
      const int first = w.first, last = w.last, me = blockIdx.x;
      auto slot_of = [&](int cta, int tile) { return (2 * cta + (cta == last ? 0 : 1)) * 2 + tile; };
      int* ticket = &q.tickets[2 * first + x];
      int* arrived = &owed[me == last ? 0 : 1].arrived[x];
      const int arrivals = last - first + 1;
      const float2* ml = reinterpret_cast<const float2*>(q.part_ml);
      const float4* po = reinterpret_cast<const float4*>(q.part_o);
      auto leave = [&]() {   // this state, for whoever joins them
        float4* dst = reinterpret_cast<float4*>(q.part_o) + size_t(slot_of(me, x)) * (D / 4) * 128;
#pragma unroll
        for (int i = 0; i < D / 32; ++i) {
          float o[32];
          if (any) {
            tmem_ld32(tl + ocol + 32 * i, o);
            tmem_ld_wait();
          } else {
#pragma unroll
            for (int e = 0; e < 32; ++e) o[e] = 0.f;
          }
          if (live) {
#pragma unroll
            for (int e = 0; e < 8; ++e)
              dst[(8 * i + e) * 128 + r] =
                  make_float4(o[4 * e], o[4 * e + 1], o[4 * e + 2], o[4 * e + 3]);
          }
        }
        if (live)
          reinterpret_cast<float2*>(q.part_ml)[size_t(slot_of(me, x)) * 128 + r] =
              make_float2(m, l);
        __threadfence();
        named_bar(1 + x, 128);
        if (r == 0) {
          const TicketTurn turn = ticket_turn(atomicAdd(ticket, kTicketLeft), arrivals, false);
          if (turn.last && !turn.join) *ticket = 0;
          flags[x] = turn.join;
          *arrived = 1;
        }
        named_bar(1 + x, 128);
      };
      if (rows <= kFewRows) {
        leave();
        if (flags[x]) {
          __threadfence();
          // thread r: row r % rows, every sub-th float4 of it, kJoin states in flight (those past
          // the last are read again and count nothing: a remainder loop would take a state a round)
          constexpr int kJoin = 8;
          const int subs = 128 / rows, rr = r % rows, sub = r / rows;
          if (sub < subs) {
            float mm = kNoMax;
#pragma unroll 1
            for (int c0 = first; c0 <= last; c0 += kJoin) {
              float v[kJoin];
#pragma unroll
              for (int i = 0; i < kJoin; ++i)
                v[i] = __ldcg(&ml[size_t(slot_of(min(c0 + i, last), x)) * 128 + rr]).x;
#pragma unroll
              for (int i = 0; i < kJoin; ++i) mm = fmaxf(mm, v[i]);
            }
            __nv_bfloat16* o_row = out_row(rr);
#pragma unroll 1
            for (int d0 = sub; d0 < D / 4; d0 += 2 * subs) {
              const int d1 = min(d0 + subs, D / 4 - 1);   // (twice the last one at the end)
              float4 acc[2] = {make_float4(0.f, 0.f, 0.f, 0.f), make_float4(0.f, 0.f, 0.f, 0.f)};
              float lsum = 0.f;
#pragma unroll 1
              for (int c0 = first; c0 <= last; c0 += kJoin) {
                float2 v[kJoin];
                float4 o[kJoin][2];
#pragma unroll
                for (int i = 0; i < kJoin; ++i) {
                  const size_t sl = slot_of(min(c0 + i, last), x);
                  v[i] = __ldcg(&ml[sl * 128 + rr]);
                  o[i][0] = __ldcg(&po[(sl * (D / 4) + d0) * 128 + rr]);
                  o[i][1] = __ldcg(&po[(sl * (D / 4) + d1) * 128 + rr]);
                }
#pragma unroll
                for (int i = 0; i < kJoin; ++i) {
                  const float f = c0 + i <= last ? moved(v[i].x, mm) : 0.f;
                  lsum = fmaf(f, v[i].y, lsum);
#pragma unroll
                  for (int j = 0; j < 2; ++j) {
                    acc[j].x = fmaf(f, o[i][j].x, acc[j].x);
                    acc[j].y = fmaf(f, o[i][j].y, acc[j].y);
                    acc[j].z = fmaf(f, o[i][j].z, acc[j].z);
                    acc[j].w = fmaf(f, o[i][j].w, acc[j].w);
                  }
                }
              }
              const float inv = 1.f / lsum;
#pragma unroll
              for (int j = 0; j < 2; ++j)
                *reinterpret_cast<uint2*>(o_row + 4 * (j ? d1 : d0)) =
                    make_uint2(pack_bf16x2(acc[j].x * inv, acc[j].y * inv),
                               pack_bf16x2(acc[j].z * inv, acc[j].w * inv));
            }
          }
          if (r == 0) *ticket = 0;
        }
      } else {
        // Many rows, a thread each: the last one to arrive takes its own state from
        // tensor memory, and need not leave it at all where the others are done.
        if (r == 0) flags[x] = *reinterpret_cast<volatile int*>(ticket) == arrivals - 1;
        named_bar(1 + x, 128);
        const bool done = flags[x];
        if (done && r == 0) *arrived = 1;
        named_bar(1 + x, 128);
        if (!done) leave();
        if (done || flags[x]) {
          __threadfence();
          const int rr = live ? r : 0;
          float mm = m, lsum = 0.f;
          for (int cc = first; cc <= last; ++cc)
            if (cc != me) mm = fmaxf(mm, __ldcg(&ml[size_t(slot_of(cc, x)) * 128 + rr]).x);
          for (int cc = first; cc <= last; ++cc) {
            const float2 v = cc == me ? make_float2(m, l) : __ldcg(&ml[size_t(slot_of(cc, x)) * 128 + rr]);
            lsum = fmaf(moved(v.x, mm), v.y, lsum);
          }
          const float inv = 1.f / lsum;
          __nv_bfloat16* o_row = out_row(rr);
          const int others = last - first;
          auto other = [&](int j) { return first + j + (first + j >= me ? 1 : 0); };
          float fj[3];   // the first other states' factors
#pragma unroll
          for (int j = 0; j < 3; ++j)
            fj[j] = j < others
                        ? moved(__ldcg(&ml[size_t(slot_of(other(j), x)) * 128 + rr]).x, mm)
                        : 0.f;
          auto factor = [&](int j) {
            return j == 0   ? fj[0]
                   : j == 1 ? fj[1]
                   : j == 2
                       ? fj[2]
                       : moved(__ldcg(&ml[size_t(slot_of(other(j), x)) * 128 + rr]).x, mm);
          };
          float4 next[8];
          auto fetch = [&](int i, int j) {   // columns 32 i .. of the j-th other state
            const float4* src = po + size_t(slot_of(other(j), x)) * (D / 4) * 128 + rr;
#pragma unroll
            for (int e = 0; e < 8; ++e) next[e] = __ldcg(&src[(8 * i + e) * 128]);
          };
          fetch(0, 0);
          const float fo = any ? moved(m, mm) : 0.f;
#pragma unroll 1
          for (int i = 0; i < D / 32; ++i) {
            float o[32], acc[32];
            if (any) {
              tmem_ld32(tl + ocol + 32 * i, o);
              tmem_ld_wait();
            }
#pragma unroll
            for (int e = 0; e < 32; ++e) {
              if (!any) o[e] = 0.f;
              acc[e] = me == first ? fmaf(fo, o[e], 0.f) : 0.f;
            }
#pragma unroll 1
            for (int j = 0; j < others; ++j) {
              float4 v[8];
#pragma unroll
              for (int e = 0; e < 8; ++e) v[e] = next[e];
              if (j + 1 < others)
                fetch(i, j + 1);
              else if (i + 1 < D / 32)
                fetch(i + 1, 0);
              const float f = factor(j);
#pragma unroll
              for (int e = 0; e < 8; ++e) {
                acc[4 * e] = fmaf(f, v[e].x, acc[4 * e]);
                acc[4 * e + 1] = fmaf(f, v[e].y, acc[4 * e + 1]);
                acc[4 * e + 2] = fmaf(f, v[e].z, acc[4 * e + 2]);
                acc[4 * e + 3] = fmaf(f, v[e].w, acc[4 * e + 3]);
              }
              if (other(j) + 1 == me) {
#pragma unroll
                for (int e = 0; e < 32; ++e) acc[e] = fmaf(fo, o[e], acc[e]);
              }
            }
            if (live) {
#pragma unroll
              for (int e = 0; e < 2; ++e) {
                uint32_t v[8];
#pragma unroll
                for (int u = 0; u < 8; ++u)
                  v[u] = pack_bf16x2(acc[16 * e + 2 * u] * inv, acc[16 * e + 2 * u + 1] * inv);
                store_32_bytes(o_row + 32 * i + 16 * e, v);
              }
            }
          }
          if (r == 0) *ticket = 0;
        }
      }
      tc_fence_before();
      named_bar(1 + x, 128);   // flags[x] is rewritten by the next partial item
      release();
    }
    if (!ok && lane == 0) set_error(q.err, kErrDeviceTimeout);
  }
  tc_fence_before();
  __syncthreads();
  // after a wait that ran out: the shared items that this CTA leaves no state of
  if (tid < 4) {
    const int x = tid & 1;
    const Owed& o = owed[tid >> 1];
    if (x < o.tiles && !o.arrived[x]) {
      int* ticket = &q.tickets[2 * o.first + x];
      if (ticket_turn(atomicAdd(ticket, kTicketGivenUp), o.arrivals, true).last) *ticket = 0;
    }
  }
  if (warp == 10) {
    tc_fence_after();
    tmem_dealloc(tmem, 512);
  }
}

template <int D>
static cudaError_t launch_prompt_t(const CUtensorMap& kmap, const CUtensorMap& vmap,
                                   const CUtensorMap& qmap, const PromptParams& p, int grid,
                                   cudaStream_t stream) {
  static std::atomic<uint32_t> configured{0};
  cudaError_t e = once_per_device(configured, [] {
    return cudaFuncSetAttribute(prompt_attn_kernel<D>, cudaFuncAttributeMaxDynamicSharedMemorySize,
                                (int)PCfg<D>::kSmem);
  });
  if (e != cudaSuccess) return e;
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3(grid, 1, 1);
  cfg.blockDim = dim3(kPThreads, 1, 1);
  cfg.dynamicSmemBytes = PCfg<D>::kSmem;
  cfg.stream = stream;
  cudaLaunchAttribute attr[1];
  attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[0].val.programmaticStreamSerializationAllowed = 1;
  cfg.attrs = attr;
  cfg.numAttrs = 1;
  return cudaLaunchKernelEx(&cfg, prompt_attn_kernel<D>, kmap, vmap, qmap, p);
}

cudaError_t launch_prompt(const CUtensorMap& kmap, const CUtensorMap& vmap,
                          const CUtensorMap& qmap, const PromptParams& p, int head_dim, int grid,
                          cudaStream_t stream) {
  return head_dim == 64 ? launch_prompt_t<64>(kmap, vmap, qmap, p, grid, stream)
                        : launch_prompt_t<128>(kmap, vmap, qmap, p, grid, stream);
}

}  // namespace vegas
