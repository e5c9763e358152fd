// mk_tree_attn.cu -- attention of new tokens (a drafted tree, or a run) over
// the paged pools, on the tcgen05 tensor cores.
//
// The work is cut into tiles: 128 slots of K and V of one (sequence, K/V head)
// against one group of up to 256 query rows.  A query row is a (token, query
// head) pair of the K/V head, in the order token * group + head, so that the
// rows of a tree share each K/V tile that is read.  All tiles, in the order
// (sequence, head, query group, tile), are dealt to the SMs in runs of equal
// cost: a unit for each tile, and three for the opening of each item (all tiles
// of one query group): the fill and the drain of the pipeline and the output
// cost about as much.  So a long context is split over many SMs, a short one
// costs no more than it holds, and nothing about the lengths is known to the
// host.  Where an item is cut by the
// border between two SMs, each leaves its part (row maxima, sums, unnormalised
// outputs, fp32) in the workspace and a second kernel joins the parts in order.
//
// Sequences that share their first slots (kShared, mk_prefix_attn) are planned as
// two kinds of items: a group's rows, all of its sequences' tokens, against the
// shared slots, and each sequence's rows against its own.  A row's items leave
// their results in the workspace as parts do, and the second kernel joins both.
//
// One CTA per SM, 12 warps:
//   warp 0      producer: page ids from the block table, K and V tiles by TMA
//               (one box per page and 64 dims, 128-byte swizzle) into a ring
//   warps 1, 2  issue the MMAs, one warp for each group of query rows: S = Q K^T
//               (both from shared memory) and O += P V (P from tensor memory,
//               V as it lies in the pages: the MMA takes its B operand with N
//               contiguous)
//   warp 3      rows of V that lie behind the sequence, or that only some rows
//               see and that hold an infinity or NaN, are zeroed before the
//               MMA reads them (0 * NaN would reach every row)
//   warps 4-11  two groups of 128 threads, a thread per query row: S from
//               tensor memory, the running maximum and sum, P back as bf16
// The two groups take the two halves of 256 query rows, or, where an item has
// at most 128 rows, the two halves of every tile's slots.  S comes in pieces of
// 64 slots, two buffers a group: while a group works on one piece the MMAs
// make its next one and the other group's.
//
// Measured on a GB300 (heads of 128, 8 query heads to a K/V head, BF16): 32
// trees of up to 16 tokens over 512 to 32K slots 182 us, 1.09 GB of K and V at
// 6.0 TB/s (a copy: 6.7), bound by memory; 2048 tokens of a run over 8K slots
// 217 us, 1.42 PFLOP/s (cuBLAS: 1.9), the tensor pipe active 65% of the
// kernel's cycles, bound by the hand-overs between exponentials and MMAs (a
// step of 64 slots takes a group some 1570 cycles, its share of plan and
// openings among them, of which its own and the other group's MMAs run 1024); eight tokens over 8K slots 17 us: 2.6 the
// plan, 6 two tiles and the output, 2 to end and begin a kernel, 4 the join.
// Shared prefixes: 64 sequences of one token over 32K shared and 50 to 2000 own
// slots 73 us (7 to the plan, 46 of tiles and openings on average, 54 at most, 8
// for the join): a tile against 256 rows takes 1.6 us, where its MMAs run 1.07,
// one against 8 rows 1.1, and the opening of one of the 256 own items 4; 32
// trees of up to 8 tokens over prefixes of 3K to 16K slots 66 us; 8 sequences
// over 8K 20 us, latency throughout.
#include <cmath>

#include "mk_ops_mma.cuh"
#include "mk_ops_parts.h"
#include "mk_ops_tmem.cuh"

namespace mk {
namespace ops {
namespace {

using namespace mk::dev;

struct AttnArgs {
  Pools pools;
  Batch b;
  const uint16_t* q;
  uint16_t* out;
  float* lse;
  const uint64_t* mask;
  int64_t q_stride, out_stride;
  int32_t n_q, group, mask_words, window, layer;
  float scale_log2;  // scale * log2(e)
  float4* part_o;    // [2 * grid][D / 4][kRows]
  float2* part_ml;   // [2 * grid][kRows]: maximum (log2 units), sum
  struct Border* borders;  // [grid + 1]
  // sequences that share their first slots (kShared)
  const int32_t *group_seqs, *prefix_lens;
  int32_t n_groups;
  int32_t op;              // what records name
  float4* seg_o;           // [2][D / 4][n_kv * n_tokens * group]: whole items that are joined with others
  float2* seg_ml;          // [2][n_kv * n_tokens * group]
  struct Placed* placed;   // [2][n_kv][item_rows]: where each item's tiles are
  struct Token* tokens;    // [n_tokens]
  int64_t item_rows;
  uint32_t* status;
  CUtensorMap tm_k, tm_v;
};

constexpr int kTile = 128;               // slots of a K/V tile, rows of an MMA
constexpr int kPiece = kTile / 2;        // slots of a piece of S
constexpr int kRows = 2 * kTile;         // query rows of an item
constexpr int kThreads = 384;
constexpr int kOpening = 3;              // units before an item's first tile
constexpr int kMaxItems = 8;             // items planned at a time
constexpr float kSlack = 8.0f;           // log2: how far the maximum in use may lag
constexpr int64_t kWaitNs = 2000000000;  // a wait that takes longer is given up

template <int D>
struct Geo {
  static constexpr int kHalves = D / 64;           // 128-byte columns of a row
  static constexpr int kHalfBytes = kTile * 128;   // a tile's 64 dims
  static constexpr int kTileBytes = kHalves * kHalfBytes;
  static constexpr int kStages = D == 128 ? 5 : 8;  // K and V tiles in flight
  static constexpr int kQ = 0, kRing = 2 * kTileBytes, kCtl = kRing + kStages * kTileBytes;
};

// One item as far as this CTA has to compute it.
struct Item {
  int b, h, t0, n, ctx;        // sequence, K/V head, its first token row, new tokens, cached
  int row0, rows;              // query rows of the K/V head: first, count (1 .. kRows)
  int lo, hi;                  // tiles of this part
  int masked_from, window_to;  // slots >= the one or < the other may be masked for some rows
  int slot;                    // workspace slot of the part, -1: the item is whole
  int from;                    // kShared: a sequence's slots from here on; kPrefix: the slots below ctx, for a whole group
};

// Where a CTA's units begin: its first unit, and the first whole item that it
// has tiles of (its first tile at unit `at`; at = first where there is none).
struct Border {
  int64_t first, at;
  Item item;
};

// A token as the joining kernel sees it: its sequence's first row and the sequence (-1: left
// out), its group's (-1: it has no prefix).
struct Token {
  int32_t t0, b, group_t0, group_b;
};

struct Ctl {
  uint64_t full[8], empty[8], s_full[2][2], p_ready[2][2], o_full[2], v_go, v_ok, q_ready, rows_done, drain;
  uint32_t tmem, abort;
  int n_items;
  int64_t first, end;  // this CTA's units
  int64_t next;
  int bad_v[kMaxItems];  // an infinity or NaN was zeroed in one of the item's tiles
  Item items[kMaxItems];
  float2 ml[2][kTile];   // the groups' maxima and sums
};

// ------------------------------------------------------------- the plan

// What the plan takes for a sequence: new tokens [t0, t0 + n) against the slots
// [from, ctx + n) of sequence b.  kShared: the batch is taken as n_groups
// groups, whose tokens (all of a group's sequences') go against the slots below
// ctx of their first sequence (from = kPrefix), and then the sequences, each
// from its group's prefix on.
struct Part : Seq {
  int from, b;
};
constexpr int kPrefix = -1;

__device__ __forceinline__ Seq attn_seq(const AttnArgs& a, int b) {
  Seq s = seq_of(a.b, b, a.pools.page_shift, a.status, a.op);
  if (a.mask && s.n > 64 * (int64_t)a.mask_words) {
    record(a.status, ERR_RANGE, a.op, b, 2, s.n, 64 * a.mask_words);
    s.n = 0;
  }
  return s;
}

// Group g's tokens against its prefix; n = 0 where there is nothing to do, and
// ctx < 0 where its numbers cannot be (its sequences are left out).
__device__ __forceinline__ Part group_part(const AttnArgs& a, int g) {
  Part p;
  const int b0 = a.group_seqs[g], b1 = a.group_seqs[g + 1];
  p.ctx = a.prefix_lens[g];
  p.from = kPrefix, p.b = b0, p.t0 = 0, p.n = 0;
  if (b0 < 0 || b0 > b1 || b1 > a.b.batch) {
    record(a.status, ERR_INDEX, a.op, g, 6, b1, a.b.batch);
    p.ctx = -1;
  } else if (b0 == b1) {
    p.ctx = 0;
  } else if (p.ctx < 0 || p.ctx > ((int64_t)a.b.max_pages << a.pools.page_shift)) {
    record(a.status, ERR_RANGE, a.op, g, 7, p.ctx, a.b.max_pages << a.pools.page_shift);
    p.ctx = -1;
  } else {
    p.t0 = a.b.cu[b0];
    const int t1 = a.b.cu[b1];
    if (p.t0 < 0 || t1 < p.t0 || t1 > a.b.n_tokens) {
      record(a.status, ERR_INDEX, a.op, g, 8, t1, a.b.n_tokens);
      p.ctx = -1;
    } else if (p.ctx > 0) {
      p.n = t1 - p.t0;
    }
  }
  return p;
}
// The group of sequence b, -1: none.
__device__ __forceinline__ int group_at(const AttnArgs& a, int b) {
  int lo = 0, hi = a.n_groups;  // the last group that begins at or before b
  while (lo < hi) {
    const int mid = (lo + hi) >> 1;
    if (a.group_seqs[mid] <= b)
      lo = mid + 1;
    else
      hi = mid;
  }
  return lo > 0 && b < a.group_seqs[lo] ? lo - 1 : -1;
}
// Sequence b from its group's prefix on.
__device__ __forceinline__ Part own_part(const AttnArgs& a, int b) {
  Part p;
  static_cast<Seq&>(p) = attn_seq(a, b);
  p.from = 0, p.b = b;
  const int g = p.n > 0 ? group_at(a, b) : -1;
  if (g >= 0) {
    const Part all = group_part(a, g);
    if (all.ctx < 0) {
      p.n = 0;
    } else if (p.ctx < all.ctx || (all.ctx > 0 && (p.t0 < all.t0 || p.t0 + p.n > all.t0 + all.n))) {
      record(a.status, ERR_RANGE, a.op, b, 5, p.ctx, all.ctx);
      p.n = 0;
    } else {
      p.from = all.ctx;
    }
  }
  return p;
}
// The same for a whole warp that has the groups in its lanes (32 of them at
// most): the search goes by shuffles, so that the numbers of all its sequences
// are one round trip to memory (with the search in memory the plan of 64
// sequences took 7 us).
struct Group {
  Part all;
  int end;  // the sequence behind its last
};
__device__ __forceinline__ Part own_part(const AttnArgs& a, const Group& mine, int b) {
  Part p;
  p.t0 = p.n = p.ctx = p.from = 0, p.b = b;
  if (b < a.b.batch) static_cast<Seq&>(p) = attn_seq(a, b);
  int lo = 0, hi = a.n_groups;  // as group_at, step by step (they differ on no input)
#pragma unroll
  for (int i = 0; i < 6; ++i) {
    const int mid = (lo + hi) >> 1, start = __shfl_sync(FULL, mine.all.b, mid & 31);
    if (lo < hi) {
      if (start <= b)
        lo = mid + 1;
      else
        hi = mid;
    }
  }
  const int g = lo - 1, src = g & 31, end = __shfl_sync(FULL, mine.end, src), ctx = __shfl_sync(FULL, mine.all.ctx, src),
            t0 = __shfl_sync(FULL, mine.all.t0, src), n = __shfl_sync(FULL, mine.all.n, src);
  if (p.n > 0 && g >= 0 && b < end) {
    if (ctx < 0) {
      p.n = 0;
    } else if (p.ctx < ctx || (ctx > 0 && (p.t0 < t0 || p.t0 + p.n > t0 + n))) {
      record(a.status, ERR_RANGE, a.op, b, 5, p.ctx, ctx);
      p.n = 0;
    } else {
      p.from = ctx;
    }
  }
  return p;
}

// Rounds of 32 of the plan's sequences (kShared: of the groups, then of the sequences).
template <bool kShared>
__device__ __forceinline__ int rounds_of(const AttnArgs& a) {
  return (a.b.batch + 31) / 32 + (kShared ? (a.n_groups + 31) / 32 : 0);
}
// The lane's part in a round.
template <bool kShared>
__device__ __forceinline__ Part part_at(const AttnArgs& a, const Group& mine, int round) {
  const int lane = threadIdx.x % 32;
  Part p;
  p.t0 = p.n = p.ctx = p.from = p.b = 0;
  if (kShared) {
    const int before = (a.n_groups + 31) / 32;
    if (round < before) {
      if (a.n_groups <= 32) return mine.all;
      if (round * 32 + lane < a.n_groups) p = group_part(a, round * 32 + lane);
      return p;
    }
    const int b = (round - before) * 32 + lane;
    if (a.n_groups <= 32) return own_part(a, mine, b);
    if (b < a.b.batch) p = own_part(a, b);
    return p;
  }
  p.b = round * 32 + lane;
  if (p.b < a.b.batch) static_cast<Seq&>(p) = attn_seq(a, p.b);
  return p;
}

// The token of a query row of a sequence.  kFew: the first and the last, which
// plans of single tokens ask for, without a division (1024 of them over 1K slots
// 505 us, 513 with it); not where the lanes of a warp ask for rows of different
// kinds and would go through all the branches (200 prompts of 40 tokens over up
// to 300 slots 169 us, 156 without).
template <bool kFew>
__device__ __forceinline__ int token_of(const AttnArgs& a, const Part& s, int row) {
  if (kFew && row == 0) return 0;
  if (kFew && row == s.n * a.group - 1) return s.n - 1;
  return (int)((uint32_t)row / (uint32_t)a.group);
}

// Tiles [lo, hi) of query group m of a sequence.
template <bool kShared, bool kFew = true>
__device__ __forceinline__ void tiles_of(const AttnArgs& a, const Part& s, int m, int& lo, int& hi) {
  if (kShared && s.from == kPrefix) {  // no token's position is below the prefix
    hi = (s.ctx + kTile - 1) / kTile;
    const int first = a.window ? s.ctx - a.window + 1 : 0;
    lo = first > 0 ? first / kTile : 0;
    if (lo == hi) --lo;
    return;
  }
  const int all = s.n * a.group, r0 = m * kRows, r1 = all - r0 < kRows ? all : r0 + kRows;  // below 2^31
  const int i0 = a.mask ? 0 : token_of<kFew>(a, s, r0), i1 = a.mask ? 0 : token_of<kFew>(a, s, r1 - 1);
  const int end = s.ctx + (a.mask ? s.n : i1 + 1);
  hi = (end + kTile - 1) / kTile;
  lo = kShared ? s.from / kTile : 0;
  if (a.window) {
    const int first = s.ctx + (a.b.positions ? 0 : i0) - a.window + 1;  // the lowest slot that a row sees
    if (first > 0 && first / kTile > lo) lo = first / kTile;
  }
}

__device__ __forceinline__ int groups_of(const AttnArgs& a, const Seq& s) {
  return (s.n * a.group - 1) / kRows + (s.n > 0 ? 1 : 0);
}

// A lane's sequence of a round of 32, and the tiles of one of its heads.
struct Load {
  Part s;
  int64_t tiles, big;  // big: those against more than kTile query rows (kShared)
};
// What a tile costs, and an item before its first one.
struct Costs {
  int opening, big, small;
};
// Lane src's part.
template <bool kShared>
__device__ __forceinline__ Part part_from(const Part& s, int src) {
  Part q;
  q.t0 = __shfl_sync(FULL, s.t0, src), q.n = __shfl_sync(FULL, s.n, src), q.ctx = __shfl_sync(FULL, s.ctx, src);
  q.from = kShared ? __shfl_sync(FULL, s.from, src) : 0;
  q.b = __shfl_sync(FULL, s.b, src);
  return q;
}
// Whether query group m of a sequence has more than kTile rows.
__device__ __forceinline__ bool is_big(const AttnArgs& a, const Part& s, int m) { return s.n * a.group - m * kRows > kTile; }
template <bool kShared>
__device__ __forceinline__ int weight(const AttnArgs& a, const Costs& c, const Part& s, int m) {
  return !kShared ? 1 : is_big(a, s, m) ? c.big : c.small;
}
template <bool kShared>
__device__ __forceinline__ int64_t cost_of(const AttnArgs& a, const Costs& c, const Load& x) {
  return (kShared ? x.big * c.big + (x.tiles - x.big) * c.small : x.tiles) + (int64_t)groups_of(a, x.s) * c.opening;
}
// (By all lanes of a warp: a prompt's many query groups are counted by all of
// them, which took the plan of 2048 tokens from 15 to 5 us.)
template <bool kShared>
__device__ __forceinline__ Load load_of(const AttnArgs& a, const Group& mine, int round) {
  const int lane = threadIdx.x % 32;
  Load x;
  x.s = part_at<kShared>(a, mine, round);
  x.tiles = x.big = 0;
  const int M = groups_of(a, x.s);
  int lo, hi;
  if (M == 1) {
    tiles_of<kShared>(a, x.s, 0, lo, hi);
    x.tiles = hi - lo;
    if (kShared && is_big(a, x.s, 0)) x.big = x.tiles;
  }
  for (uint32_t many = __ballot_sync(FULL, M > 1); many; many &= many - 1) {
    const int src = __ffs(many) - 1;
    const Part q = part_from<kShared>(x.s, src);
    int64_t u = 0, big = 0;
    for (int m = lane, n = groups_of(a, q); m < n; m += 32) {
      tiles_of<kShared, false>(a, q, m, lo, hi);
      u += hi - lo;
      if (kShared && is_big(a, q, m)) big += hi - lo;
    }
    for (int o = 16; o > 0; o >>= 1) {
      u += __shfl_xor_sync(FULL, u, o);
      if (kShared) big += __shfl_xor_sync(FULL, big, o);
    }
    if (lane == src) x.tiles = u, x.big = big;
  }
  return x;
}

// All units (by one warp), what counts how many, and the lane's sequence of
// the first round.  Openings cost nothing where every SM has a tile at most:
// an item is then the first of its SMs.  With more, counting 3 for one took
// 30 ragged prompts of up to 273 tokens (each over up to 785 slots) from 195
// to 121 us, 32 trees of 16 tokens over up to 32K slots from 197 to 191 us; 1,
// 2 and 4 were slower.
// With shared prefixes tiles against 256 rows stand beside tiles against few:
// they took 1.75 us against 1.1, an item's opening 5.5.  (Openings of 4 to 12 units of a
// small tile's 3, and other weights of a big one, were slower by 1 to 6 us of 73.)
template <bool kShared>
__device__ __forceinline__ int64_t total_units(const AttnArgs& a, int grid, Group& mine, Load& first, Costs& c) {
  const int lane = threadIdx.x % 32;
  if (kShared) {
    mine.all.t0 = mine.all.n = mine.all.ctx = mine.all.from = mine.all.b = mine.end = 0;
    if (a.n_groups <= 32 && lane < a.n_groups) {
      mine.all = group_part(a, lane);
      mine.end = a.group_seqs[lane + 1];
    }
  }
  int64_t u = 0, big = 0, items = 0;
#pragma unroll 1
  for (int r = 0; r < rounds_of<kShared>(a); ++r) {  // (one copy of the code: see copy_q)
    const Load x = load_of<kShared>(a, mine, r);
    if (r == 0) first = x;
    u += x.tiles;
    big += x.big;
    items += groups_of(a, x.s);
  }
  for (int o = 16; o > 0; o >>= 1) {
    u += __shfl_xor_sync(FULL, u, o);
    items += __shfl_xor_sync(FULL, items, o);
    if (kShared) big += __shfl_xor_sync(FULL, big, o);
  }
  c = {u * a.pools.n_kv > grid ? kOpening : 0, 1, 1};
  if (kShared) {
    // every SM has a tile's cost at least, so that none between two parts of an item is without one
    const Costs fine = {18, 5, 3};
    const int64_t all = (big * fine.big + (u - big) * fine.small + items * fine.opening) * a.pools.n_kv;
    if (all >= (int64_t)grid * fine.big) {
      c = fine;
      return all;
    }
  }
  return (u + items * c.opening) * a.pools.n_kv;
}

// The first unit of CTA c: even runs, the longer ones first.
__device__ __forceinline__ int64_t border(int64_t total, int c, int grid) {
  const int64_t base = divide(total, grid), rest = total - base * grid;
  return base * c + (c < rest ? c : rest);
}

// a / w for the costs of a tile, rounded up.
__device__ __forceinline__ int64_t tiles_in(int64_t units, int w) {
  if (w == 1) return units;
  if (units >> 31) return (units + w - 1) / w;
  const uint32_t u = (uint32_t)units + w - 1;
  return w == 3 ? u / 3u : w == 5 ? u / 5u : u / (uint32_t)w;
}

// Item m of K/V head h of a sequence, whole.
template <bool kShared>
__device__ __forceinline__ Item make_item(const AttnArgs& a, const Part& s, int h, int m) {
  Item it;
  it.b = s.b, it.h = h, it.t0 = s.t0, it.n = s.n, it.ctx = s.ctx, it.from = s.from;
  it.row0 = m * kRows;
  it.rows = s.n * a.group - it.row0 < kRows ? s.n * a.group - it.row0 : kRows;
  tiles_of<kShared>(a, s, m, it.lo, it.hi);
  it.slot = -1;
  if (kShared && s.from == kPrefix) {
    it.masked_from = s.ctx;
    it.window_to = a.window ? s.ctx : 0;  // the sequences' own lengths say which
    return it;
  }
  const int i0 = token_of<false>(a, s, it.row0), i1 = token_of<false>(a, s, it.row0 + it.rows - 1);
  // without a mask every row sees the new tokens up to the first row's own,
  // unless positions set them a window or more apart
  const bool apart = a.window && a.b.positions && s.n > a.window;
  it.masked_from = s.ctx + (a.mask || apart ? 0 : i0 + 1);
  it.window_to = 0;
  if (a.window) it.window_to = s.ctx + (a.b.positions ? s.n - 1 : i1) - a.window + 1;  // the highest row's lowest slot
  if (kShared && s.from > it.window_to) it.window_to = s.from;
  return it;
}

// Calls f(item, unit of the item's first tile) for the items whose tiles lie in
// units [u, end), in order, while it returns true.  By one warp, whose lanes
// hold the first round's sequences; f runs on every lane.
template <bool kShared, typename F>
__device__ __forceinline__ void each_item(const AttnArgs& a, const Group& mine, const Load& first, const Costs& c, int64_t u, int64_t end, F f) {
  const int lane = threadIdx.x % 32;
  int64_t base = 0;  // units before this round of sequences
  for (int r = 0; r < rounds_of<kShared>(a) && base < end; ++r) {
    const Load x = r == 0 ? first : load_of<kShared>(a, mine, r);
    const Part s = x.s;
    const int64_t per_head = cost_of<kShared>(a, c, x);
    const int64_t incl = warp_scan(per_head * a.pools.n_kv);
    uint32_t hit = __ballot_sync(FULL, per_head > 0 && base + incl > u && base + incl - per_head * a.pools.n_kv < end);
    while (hit) {
      const int src = __ffs(hit) - 1;
      hit &= hit - 1;
      const Part q = part_from<kShared>(s, src);
      const int64_t ph = __shfl_sync(FULL, per_head, src), begin = base + __shfl_sync(FULL, incl, src) - ph * a.pools.n_kv;
      const int M = groups_of(a, q);
      int h = u > begin ? (int)divide(u - begin, ph) : 0;
      for (; h < a.pools.n_kv; ++h) {
        int64_t at = begin + h * ph;
        if (at >= end) return;
        int m = 0;
        if (at < u && M > 1) {  // the first group whose tiles end behind u
          int64_t skipped = 0;
          bool found = false;
          for (m = 0; m < M && !found; m += 32) {
            int lo = 0, hi = 0;
            if (m + lane < M) tiles_of<kShared, false>(a, q, m + lane, lo, hi);
            const int64_t n = m + lane < M ? (hi - lo) * weight<kShared>(a, c, q, m + lane) + c.opening : 0, sum = warp_scan(n);
            const uint32_t past = __ballot_sync(FULL, m + lane < M && at + skipped + sum > u);
            found = past != 0;
            const int j = found ? __ffs(past) - 1 : 31;
            skipped += __shfl_sync(FULL, found ? sum - n : sum, j);
            if (found) m += j - 32;
          }
          at += skipped;
        }
        for (; m < M; ++m) {
          int lo, hi;
          tiles_of<kShared>(a, q, m, lo, hi);
          const int w = weight<kShared>(a, c, q, m);
          at += c.opening;
          if (at + (hi - lo) * w > u) {
            if (at >= end) return;
            if (!f(make_item<kShared>(a, q, h, m), at, w)) return;
          }
          at += (hi - lo) * w;
        }
      }
    }
    base += __shfl_sync(FULL, incl, 31);
  }
}

// ------------------------------------------------------------- waits

// Waits for a phase; false when this wait, or another one of the CTA, has
// taken too long.  (Inlined like all the roles use: a function that is called
// would have to keep to the smaller of their two register budgets.)
__device__ __forceinline__ bool wait_slow(Ctl& c, uint64_t* bar, uint32_t parity, const AttnArgs& a) {
  const int64_t until = gtimer() + kWaitNs;
  for (;;) {
    if (mbar_try_wait(bar, parity)) return true;
    if (ld_volatile(&c.abort)) return false;
    if (gtimer() > until) {
      *reinterpret_cast<volatile uint32_t*>(&c.abort) = 1;
      record(a.status, ERR_TIMEOUT, a.op, blockIdx.x, threadIdx.x, 0, 0);
      return false;
    }
  }
}
__device__ __forceinline__ bool wait(Ctl& c, uint64_t* bar, uint32_t parity, const AttnArgs& a) {
  return mbar_try_wait(bar, parity) || wait_slow(c, bar, parity, a);
}

__device__ __forceinline__ bool both_in(const Item& it) { return it.rows > kTile; }
// Whether tile j holds slots behind the sequence or masked for some rows.
__device__ __forceinline__ bool in_part(int masked_from, int window_to, int j) {
  return (j + 1) * kTile > masked_from || j * kTile < window_to;
}
__device__ __forceinline__ bool in_part(const Item& it, int j) { return in_part(it.masked_from, it.window_to, j); }

// ------------------------------------------------------------- visibility

// Bits of the new tokens j0 .. j0 + 31 in a token's mask row (j0 > -32; bits
// below token 0 are clear), whose first word is at hand.
__device__ __forceinline__ uint32_t mask_bits(const uint64_t* row, uint64_t word0, int words, int j0) {
  if (j0 < 0) return (uint32_t)(word0 << -j0);
  const int w = j0 >> 6, sh = j0 & 63;
  uint64_t v = w == 0 ? word0 >> sh : w < words ? row[w] >> sh : 0;
  if (sh > 32 && w + 1 < words) v |= row[w + 1] << (64 - sh);
  return (uint32_t)v;
}

// Position of new token j (a position out of range is moved into it).
__device__ __forceinline__ int position_of(const AttnArgs& a, const Item& it, int j) {
  if (!a.b.positions) return it.ctx + j;
  const int p = a.b.positions[it.t0 + j];
  if (p < it.ctx || p >= it.ctx + it.n) {
    record(a.status, ERR_RANGE, a.op, it.b, 3, p, it.ctx + it.n);
    return p < it.ctx ? it.ctx : it.ctx + it.n - 1;
  }
  return p;
}

// kShared: the position of token i of a group, whichever its sequence.
__device__ __forceinline__ int position_in_group(const AttnArgs& a, const Item& it, int i) {
  const int t = it.t0 + i;
  int lo = it.b + 1, hi = a.b.batch;  // the last sequence that begins at or before the token
  while (lo < hi) {
    const int mid = (lo + hi) >> 1;
    if (a.b.cu[mid] <= t)
      lo = mid + 1;
    else
      hi = mid;
  }
  const int ctx = a.b.ctx[lo - 1], t0 = a.b.cu[lo - 1], n = a.b.cu[lo] - t0;
  const int p = a.b.positions ? a.b.positions[t] : ctx + t - t0;
  return p < ctx ? ctx : p >= ctx + n ? ctx + n - 1 : p;  // what is out of range is recorded with the sequence
}

// The first slot behind an item's.
template <bool kShared>
__device__ __forceinline__ int end_of(const Item& it) {
  return it.ctx + (kShared && it.from == kPrefix ? 0 : it.n);
}

// Which of the slots s0 .. s0 + 31 token i sees.
template <bool kShared>
__device__ __forceinline__ uint32_t seen(const AttnArgs& a, const Item& it, int i, int pos, uint64_t word0, int s0) {
  const int len = end_of<kShared>(it);
  if (s0 >= len) return 0;
  uint32_t v = FULL;
  if (len - s0 < 32) v = FULL >> (32 - (len - s0));
  if (kShared) {
    if (it.from == kPrefix) {
      const int first = a.window ? pos - a.window + 1 - s0 : 0;
      return first <= 0 ? v : first >= 32 ? 0 : v & (FULL << first);
    }
    if (it.from >= s0 + 32) return 0;
    if (it.from > s0) v &= FULL << (it.from - s0);
  }
  const int j0 = s0 - it.ctx;
  if (j0 > -32) {
    uint32_t d;
    if (a.mask) {
      d = mask_bits(a.mask + (int64_t)(it.t0 + i) * a.mask_words, word0, a.mask_words, j0);
      if (j0 < 0) d |= (1u << -j0) - 1;
    } else {
      const int k = i + 1 - j0;  // tokens from j0 up to i
      d = k <= 0 ? 0 : k >= 32 ? FULL : (1u << k) - 1;
    }
    v &= d;
  }
  if (a.window) {
    const int first = pos - a.window + 1 - s0;  // cached slots (and a run's tokens) below it are out
    uint32_t in = first <= 0 ? FULL : first >= 32 ? 0 : FULL << first;
    if (a.b.positions && j0 > -32) {
      const uint32_t fresh = j0 >= 0 ? FULL : FULL << -j0;
      uint32_t near = fresh;
      if (it.n > a.window)  // else no two new tokens are a window apart
        for (uint32_t w = v & fresh; w; w &= w - 1) {
          const int k = __ffs(w) - 1;
          if (pos - position_of(a, it, j0 + k) >= a.window) near &= ~(1u << k);
        }
      in = (in & ~fresh) | near;
    }
    v &= in;
  }
  return v;
}

__device__ __forceinline__ int64_t pool_row(const AttnArgs& a, const Item& it, int slot) {
  int64_t page = a.b.tables[(int64_t)it.b * a.b.max_pages + (slot >> a.pools.page_shift)];
  if (page < 0 || page >= a.pools.num_pages) page = 0;
  return ((page * a.pools.n_kv + it.h) << a.pools.page_shift) + (slot & ((1 << a.pools.page_shift) - 1));
}

// ------------------------------------------------------------- roles

template <int D, bool kShared>
__device__ bool produce(const AttnArgs& a, uint8_t* smem, Ctl& c, Ring& r, uint32_t& filled) {
  using G = Geo<D>;
  const int lane = threadIdx.x % 32;
  const int P = 1 << a.pools.page_shift, box = P < kTile ? P : kTile;  // slots of a box
  const int slice = lane / G::kHalves, half = lane % G::kHalves;       // this lane's box of a tile
  for (int k = 0; k < c.n_items; ++k) {
    const Item it = c.items[k];
    const int len = end_of<kShared>(it);
    const int32_t* table = a.b.tables + (int64_t)it.b * a.b.max_pages;
    auto page_at = [&](int j) {  // the page of this lane's box in tile j, -1: no slot of it is in use
      const int s = j * kTile + slice * box;
      if (slice * box >= kTile || s >= len || (kShared && s + box <= it.from)) return -1;
      int page = table[s >> a.pools.page_shift];
      if (page < 0 || page >= a.pools.num_pages) {
        record(a.status, ERR_PAGE, a.op, it.b, s, page, (uint32_t)a.pools.num_pages);
        page = 0;
      }
      return page;
    };
    int page = page_at(it.lo);
    for (int j = it.lo; j < it.hi; ++j) {
      const int next = j + 1 < it.hi ? page_at(j + 1) : -1;
      const uint32_t bytes = __popc(__ballot_sync(FULL, page >= 0)) * box * 128;
      const int y = ((page * a.pools.n_kv + it.h) << a.pools.page_shift) + ((j * kTile + slice * box) & (P - 1));
#pragma unroll
      for (int kv = 0; kv < 2; ++kv) {
        // the tile before last in this stage has been read
        const bool ok = filled < (uint32_t)G::kStages || wait(c, &c.empty[r.stage], r.phase ^ 1, a);
        if (!__all_sync(FULL, ok)) return false;
        if (lane == 0) mbar_expect_tx(&c.full[r.stage], bytes);
        __syncwarp();
        if (page >= 0) {
          uint8_t* dst = smem + G::kRing + r.stage * G::kTileBytes + half * G::kHalfBytes + slice * box * 128;
          asm volatile(
              "cp.async.bulk.tensor.3d.shared::cluster.global.tile.mbarrier::complete_tx::bytes"
              " [%0], [%1, {%2, %3, %4}], [%5];" ::"r"(smem_u32(dst)),
              "l"(reinterpret_cast<uint64_t>(kv ? &a.tm_v : &a.tm_k)), "r"(half * 64), "r"(y), "r"(a.layer),
              "r"(smem_u32(&c.full[r.stage]))
              : "memory");
        }
        ++filled;
        r.advance<G::kStages>();
      }
      page = next;
    }
  }
  return true;
}

// TMEM columns: four pieces of S (P takes the first half of its piece), then
// the two groups' outputs.
__device__ __forceinline__ uint32_t s_cols(int w, int buf) { return (w * 2 + buf) * kPiece; }
__device__ __forceinline__ uint32_t o_cols(int w) { return 4 * kPiece + w * 128; }

struct MmaState {
  Ring k;                        // the next K or V tile of the ring
  uint32_t p_phase = 0;          // of p_ready, a bit per buffer
  uint32_t q_phase = 0, v_phase = 0;  // of q_ready, of v_ok
};

// The MMAs of group w.  Its step t is a piece of 64 slots: with 256 rows half
// t % 2 of tile t / 2, with 128 rows half w of tile t.  S of step t + 2 is made
// right after O takes step t, whose buffer it reuses; the MMAs of a thread run
// in the order of their issue.  s_full[w][t % 2] then says that step t + 2 of S
// is there and P V of step t is done.
//
// By one whole warp without branches on the lane: an MMA takes its operands
// from uniform registers, and only code that all lanes run together keeps its
// addresses there (issued by a lone thread an MMA costs 80 cycles, behind a
// branch of one lane 45, where it runs 32 or 64).  One elected lane issues.
// One warp for both groups would spend on barriers and issue what the MMAs of
// a step take; for the same reason the steps are written out two by two.
template <int D>
__device__ __forceinline__ bool issue_mmas(const AttnArgs& a, uint8_t* smem, Ctl& c, MmaState& st, const int w) {
  using G = Geo<D>;
  constexpr uint32_t idesc_s = tc_idesc_bf16(kTile, kPiece);
  constexpr uint32_t idesc_o = tc_idesc_bf16(kTile, D) | (1u << 16);  // B with N contiguous
  const uint32_t base = smem_u32(smem) >> 4, tmem = uniform(c.tmem), vlo = (G::kHalfBytes >> 4) << 16, klo = 1u << 16;
  const uint32_t empty = smem_u32(c.empty), s_full = smem_u32(c.s_full[w]), v_go = smem_u32(&c.v_go);
  const uint32_t ts = tmem + s_cols(w, 0), to = tmem + o_cols(w);
  const uint32_t lead = elected();
  // The warp's lanes leave every wait together: one that fell behind could
  // miss a phase of a barrier and wait for its parity for good.  Every tile of
  // the ring is waited for, in order, for the same reason.
  auto ready = [&](uint64_t* bar, uint32_t parity) { return __all_sync(FULL, wait(c, bar, parity, a)) != 0; };
  const int n_items = uniform(c.n_items);
  for (int k = 0; k < n_items; ++k) {
    const Item& it = c.items[k];
    const bool both = uniform(both_in(it));
    const int lo = uniform(it.lo), tiles = uniform(it.hi) - lo;
    const int masked_from = uniform(it.masked_from) - lo * kTile, window_to = uniform(it.window_to) - lo * kTile;
    // tile x of the item: K at ring position 2x, V at 2x + 1 from here on
    Ring kpos = st.k, vpos = st.k;
    vpos.advance<G::kStages>();
    if (!ready(&c.q_ready, st.q_phase)) return false;
    st.q_phase ^= 1;
    tc_fence_after();
    const uint32_t qd = (base + (G::kQ + (both ? w * G::kTileBytes : 0)) / 16) | klo;
    auto qk = [&](int half, int buf) {  // S of a piece of K's tile
      const uint32_t kd = (base + (G::kRing + kpos.stage * G::kTileBytes + half * kPiece * 128) / 16) | klo;
#pragma unroll
      for (int e = 0; e < D / 16; ++e) {
        const uint32_t off = (e / 4 * G::kHalfBytes + e % 4 * 32) / 16;
        mma_ss_if(lead, ts + buf * kPiece, desc(qd + off), desc(kd + off), idesc_s, e > 0);
      }
    };
    auto pv = [&](int half, int buf, bool more) {  // O (+)= P V of a piece of V's tile
      const uint32_t vd = (base + (G::kRing + vpos.stage * G::kTileBytes + half * kPiece * 128) / 16) | vlo;
#pragma unroll
      for (int e = 0; e < kPiece / 16; ++e)  // 16 slots: 8 columns of P, two 1024-byte groups of V
        mma_ts_if(lead, to, ts + buf * kPiece + e * 8, desc(vd + e * (2048 / 16)), idesc_o, more || e > 0);
    };
    auto p_ready = [&](int buf) {
      if (!ready(&c.p_ready[w][buf], st.p_phase >> buf & 1)) return false;
      st.p_phase ^= 1u << buf;
      return true;
    };
    auto v_there = [&](int x) {  // tile x of V, and clean_v's go on it
      if (!ready(&c.full[vpos.stage], vpos.phase)) return false;
      if (in_part(masked_from, window_to, x)) {
        arrive_if(lead, v_go);
        if (!ready(&c.v_ok, st.v_phase)) return false;
        st.v_phase ^= 1;
      }
      return true;
    };
    auto free_k = [&]() {
      commit_if(lead, empty + kpos.stage * 8);
      kpos.advance<G::kStages>();
      kpos.advance<G::kStages>();
    };
    auto free_v = [&]() {
      commit_if(lead, empty + vpos.stage * 8);
      vpos.advance<G::kStages>();
      vpos.advance<G::kStages>();
    };
    if (both) {
      if (!ready(&c.full[kpos.stage], kpos.phase)) return false;
      qk(0, 0);
      commit_if(lead, s_full);
      qk(1, 1);
      commit_if(lead, s_full + 8);
      free_k();
      for (int x = 0; x < tiles; ++x) {
        const bool next = x + 1 < tiles;
        if (!v_there(x) || !p_ready(0)) return false;
        tc_fence_after();
        pv(0, 0, x > 0);
        if (next) {
          if (!ready(&c.full[kpos.stage], kpos.phase)) return false;
          qk(0, 0);
        }
        commit_if(lead, s_full);
        if (!p_ready(1)) return false;
        tc_fence_after();
        pv(1, 1, true);
        if (next) qk(1, 1);
        commit_if(lead, s_full + 8);
        free_v();
        if (next) free_k();
      }
    } else {
      for (int x = 0; x < 2 && x < tiles; ++x) {
        if (!ready(&c.full[kpos.stage], kpos.phase)) return false;
        qk(w, x);
        commit_if(lead, s_full + x * 8);
        free_k();
      }
      for (int x = 0; x < tiles; ++x) {
        const int buf = x & 1;
        if (!v_there(x) || !p_ready(buf)) return false;
        tc_fence_after();
        pv(w, buf, x > 0);
        free_v();
        if (x + 2 < tiles) {
          if (!ready(&c.full[kpos.stage], kpos.phase)) return false;
          qk(w, buf);
          commit_if(lead, s_full + buf * 8);
          free_k();
        } else {
          commit_if(lead, s_full + buf * 8);
        }
      }
    }
    // what this warp has seen (clean_v's word on the item), to the group
    arrive_if(lead, smem_u32(&c.o_full[w]));
    st.k = kpos;  // two positions per tile: behind the item's last V
  }
  return true;
}

// Whether one of two bf16 is an infinity or NaN (its exponent all ones).
__device__ __forceinline__ uint32_t any_odd(uint32_t w) { return ((w & 0x7f80u) == 0x7f80u) | ((w & 0x7f800000u) == 0x7f800000u); }

// Rows of a partly masked tile's V that must not reach the MMA.
struct CleanState {
  Ring k;
  uint32_t phase = 0;  // of v_go
};

template <int D, bool kShared>
__device__ bool clean_v(const AttnArgs& a, uint8_t* smem, Ctl& c, CleanState& st) {
  using G = Geo<D>;
  const int lane = threadIdx.x % 32;
  for (int k = 0; k < c.n_items; ++k) {
    const Item it = c.items[k];
    for (int j = it.lo; j < it.hi; ++j) {
      st.k.advance<G::kStages>();  // K
      if (in_part(it, j)) {
        if (!__all_sync(FULL, wait(c, &c.v_go, st.phase, a))) return false;
        st.phase ^= 1;
        const uint32_t tile = smem_u32(smem + G::kRing + st.k.stage * G::kTileBytes);
        const int len = end_of<kShared>(it), s0 = j * kTile;
        for (int row = lane; row < kTile; row += 32) {
          bool drop = s0 + row >= len || (kShared && s0 + row < it.from);
          if (!drop && (s0 + row >= it.masked_from || s0 + row < it.window_to)) {
            uint32_t odd = 0;
#pragma unroll
            for (int ch = 0; ch < D / 8; ++ch) {
              const uint4 u = lds128(tile + ch / 8 * G::kHalfBytes + row * 128 + ((ch % 8) ^ (row & 7)) * 16);
              odd |= any_odd(u.x) | any_odd(u.y) | any_odd(u.z) | any_odd(u.w);
            }
            if (odd) {
              drop = true;
              *reinterpret_cast<volatile int*>(&c.bad_v[k]) = 1;
            }
          }
          if (drop)
#pragma unroll
            for (int ch = 0; ch < D / 8; ++ch)
              asm volatile("st.shared.v4.u32 [%0], {%1, %1, %1, %1};" ::"r"(tile + ch / 8 * G::kHalfBytes + row * 128 + ((ch % 8) ^ (row & 7)) * 16),
                           "r"(0u)
                           : "memory");
        }
        fence_proxy_async_smem();
        __syncwarp();
        if (lane == 0) mbar_arrive(&c.v_ok);
      }
      st.k.advance<G::kStages>();  // V
    }
  }
  return true;
}

struct RowState {
  uint32_t s_phase = 0;  // of s_full, a bit per buffer
  uint32_t o_phase = 0, done_phase = 0;
};

__device__ __forceinline__ float max3(float a, uint32_t b, uint32_t c) {
  float r;
  asm("max.f32 %0, %1, %2, %3;" : "=f"(r) : "f"(a), "f"(__uint_as_float(b)), "f"(__uint_as_float(c)));
  return r;
}
// What clean_v zeroed, for the rows that see it: its products with the row's
// probabilities, added to 32 columns of the row's output.
template <int D, bool kShared>
__device__ __forceinline__ void add_odd_v(const AttnArgs& a, const Item& it, int i, int g, int pos, uint64_t word0, float m, int col, float (&o)[32]) {
  const uint16_t* q = a.q + (int64_t)(it.t0 + i) * a.q_stride + (int64_t)(it.h * a.group + g) * D;
  for (int j = it.lo; j < it.hi; ++j) {
    if (!in_part(it, j)) continue;
    for (int s = j * kTile; s < min((j + 1) * kTile, end_of<kShared>(it)); ++s) {
      if (s < it.masked_from && s >= it.window_to) continue;
      const int64_t row = pool_row(a, it, s) * D;
      uint32_t odd = 0;  // the same for all rows, and quickly known
#pragma unroll
      for (int e = 0; e < D; e += 8) {
        const uint4 u = *reinterpret_cast<const uint4*>(a.pools.v + row + e);
        odd |= any_odd(u.x) | any_odd(u.y) | any_odd(u.z) | any_odd(u.w);
      }
      if (!odd || !(seen<kShared>(a, it, i, pos, word0, s) & 1)) continue;
      float dot = 0;
      for (int e = 0; e < D; ++e)
        dot += __uint_as_float((uint32_t)q[e] << 16) * __uint_as_float((uint32_t)a.pools.k[row + e] << 16);
      const float p = ex2(dot * a.scale_log2 - (m == -INFINITY ? 0.0f : m));
      for (int e = 0; e < 32; ++e) o[e] += p * __uint_as_float((uint32_t)a.pools.v[row + col + e] << 16);
    }
  }
}

// Q of an item: 16-byte chunks of its rows, first into registers, then into the
// MMA's K-major layout.  By ordinary loads: the kernel before this one may have
// written Q while this one was resident already, and read-only loads hold for
// data that no one writes as long as a kernel lives.
template <int D>
struct QTile {
  static constexpr int kChunks = kRows * (D / 8) / 256;  // of a thread
  uint4 u[kChunks];
};
template <int D>
__device__ __forceinline__ void load_q(const AttnArgs& a, const Item& it, QTile<D>& q) {
  constexpr uint32_t kStep = 256 / (D / 8);  // rows from chunk to chunk
  const int tid = threadIdx.x - 128, ch = tid % (D / 8), n = both_in(it) ? QTile<D>::kChunks : QTile<D>::kChunks / 2;
  // token and head of the first chunk's row, and the step to the next one's
  const uint32_t group = a.group, f = it.row0 + tid / (D / 8), by_i = kStep / group, by_g = kStep - by_i * group;
  uint32_t i = f / group, g = f - i * group;
#pragma unroll
  for (int x = 0; x < QTile<D>::kChunks; ++x) {
    const int row = tid / (D / 8) + x * kStep;
    if (x * kStep >= (uint32_t)it.rows) break;  // few rows: little code
    q.u[x] = make_uint4(0, 0, 0, 0);
    if (x < n && row < it.rows)
      q.u[x] = reinterpret_cast<const uint4*>(a.q + (int64_t)(it.t0 + (int)i) * a.q_stride + (int64_t)(it.h * a.group + (int)g) * D)[ch];
    i += by_i, g += by_g;
    if (g >= group) g -= group, ++i;
  }
}
// Q of a batch's first item, straight into its place, which nothing else uses
// yet: a short loop, for the code that a CTA runs once at its start comes from
// memory, and all SMs ask for it at the same time.
template <int D>
__device__ __forceinline__ void copy_q(const AttnArgs& a, uint8_t* smem, const Item& it) {
  using G = Geo<D>;
  constexpr uint32_t kStep = 256 / (D / 8);
  const int tid = threadIdx.x - 128, ch = tid % (D / 8), rows = both_in(it) ? kRows : kTile;
  const uint32_t group = a.group, f = it.row0 + tid / (D / 8), by_i = kStep / group, by_g = kStep - by_i * group;
  uint32_t i = f / group, g = f - i * group;
#pragma unroll 1
  for (int row = tid / (D / 8); row < rows; row += kStep) {
    const int rr = row % kTile;
    const uint16_t* src = a.q + (int64_t)(it.t0 + (int)i) * a.q_stride + (int64_t)(it.h * a.group + (int)g) * D + ch * 8;
    asm volatile("cp.async.cg.shared.global [%0], [%1], 16, %2;" ::"r"(
                     smem_u32(smem + G::kQ + row / kTile * G::kTileBytes + ch / 8 * G::kHalfBytes + rr * 128 + ((ch % 8) ^ (rr & 7)) * 16)),
                 "l"(row < it.rows ? src : a.q), "r"(row < it.rows ? 16 : 0)
                 : "memory");
    i += by_i, g += by_g;
    if (g >= group) g -= group, ++i;
  }
}
// (Rows behind the item's, up to a whole chunk of all threads, are zeros, others
// what was there: their scores stay with them.)
template <int D>
__device__ __forceinline__ void store_q(uint8_t* smem, int rows, const QTile<D>& q) {
  using G = Geo<D>;
  const int tid = threadIdx.x - 128, ch = tid % (D / 8);
#pragma unroll
  for (int x = 0; x < QTile<D>::kChunks; ++x) {
    const int row = tid / (D / 8) + x * (256 / (D / 8)), rr = row % kTile;
    if (x * (256 / (D / 8)) >= rows) break;
    *reinterpret_cast<uint4*>(smem + G::kQ + row / kTile * G::kTileBytes + ch / 8 * G::kHalfBytes + rr * 128 + ((ch % 8) ^ (rr & 7)) * 16) = q.u[x];
  }
}

template <int D, bool kShared>
__device__ __forceinline__ bool softmax_rows(const AttnArgs& a, uint8_t* smem, Ctl& c, RowState& st) {
  using G = Geo<D>;
  const int tid = threadIdx.x - 128, w = tid / 128, r = tid % 128;
  const uint32_t lane_base = c.tmem + ((uint32_t)(r / 32 * 32) << 16);
  const uint32_t t_o = lane_base + o_cols(w);
  const int n_items = c.n_items;
  QTile<D> q = {};
  if (n_items > 0) copy_q<D>(a, smem, c.items[0]);
  for (int k = 0; k < n_items; ++k) {
    const Item& it = c.items[k];
    const bool both = both_in(it);
    if (k > 0)
      store_q<D>(smem, it.rows, q);
    else
      asm volatile("cp.async.wait_all;" ::: "memory");
    fence_proxy_async_smem();
    mbar_arrive(&c.q_ready);

    const int local = both ? w * kTile + r : r;  // row of the item
    const bool mine = local < it.rows;
    const bool warp_mine = (both ? w * kTile : 0) + r / 32 * 32 < it.rows;
    const uint32_t f = it.row0 + (mine ? local : 0);
    const int i = f / (uint32_t)a.group, g = f % (uint32_t)a.group;
    const int pos = !a.window ? 0 : kShared && it.from == kPrefix ? position_in_group(a, it, i) : position_of(a, it, i);
    const uint64_t word0 = a.mask ? a.mask[(int64_t)(it.t0 + i) * a.mask_words] : 0;
    float m = -INFINITY, l = 0.0f;
    const int lo = it.lo, steps = both ? 2 * (it.hi - lo) : it.hi - lo, masked_from = it.masked_from, window_to = it.window_to;
    for (int t = 0; t < steps; ++t) {
      const int buf = t & 1, j = lo + (both ? t >> 1 : t);
      if (!__all_sync(FULL, wait(c, &c.s_full[w][buf], st.s_phase >> buf & 1, a))) return false;
      st.s_phase ^= 1u << buf;
      if (!warp_mine) {  // no row of this warp: P's lanes are never used
        mbar_arrive(&c.p_ready[w][buf]);
        continue;
      }
      tc_fence_after();
      const uint32_t t_s = lane_base + s_cols(w, buf);
      uint32_t s[kPiece];
      tmem_load(t_s, s);
      if (in_part(masked_from, window_to, j)) {
#pragma unroll
        for (int x = 0; x < 2; ++x) {
          const uint32_t v = seen<kShared>(a, it, i, pos, word0, j * kTile + (both ? buf : w) * kPiece + x * 32);
#pragma unroll
          for (int e = 0; e < 32; ++e)
            if (!((v >> e) & 1)) s[x * 32 + e] = 0xff800000u;
        }
      }
      float t0 = -INFINITY, t1 = -INFINITY, t2 = -INFINITY, t3 = -INFINITY;
#pragma unroll
      for (int e = 0; e < kPiece; e += 8) {
        t0 = max3(t0, s[e], s[e + 1]);
        t1 = max3(t1, s[e + 2], s[e + 3]);
        t2 = max3(t2, s[e + 4], s[e + 5]);
        t3 = max3(t3, s[e + 6], s[e + 7]);
      }
      const float top = fmaxf(fmaxf(t0, t1), fmaxf(t2, t3)) * a.scale_log2;
      // The maximum in use may lag by kSlack (p <= 2^8, exact enough in bf16
      // and fp32): the output is rescaled only where it lags further.
      const bool up = top > m + kSlack;
      if (__any_sync(FULL, up)) {
        const float to = up ? top : m, by = up ? ex2(m - to) : 1.0f;
        if (t > 0) {
          // P V of the step before is done once the next one's barrier says so
          if (!__all_sync(FULL, wait(c, &c.s_full[w][buf ^ 1], st.s_phase >> (buf ^ 1) & 1, a))) return false;
          tc_fence_after();
#pragma unroll 1
          for (int x = 0; x < D; x += 32) {
            uint32_t o[32];
            tmem_load(t_o + x, o);
#pragma unroll
            for (int e = 0; e < 32; ++e) o[e] = __float_as_uint(__uint_as_float(o[e]) * by);
            tmem_store(t_o + x, o);
          }
        }
        l *= by;
        m = to;
      }
      // P as one BF16, the MMA's operand: 2^-8 of a probability, averaged over the
      // slots.  Two terms would keep fp32's accuracy for twice the MMAs of P V.
      // (Beside 64 bits an output's error is 0.0023 of it, 0.0017 with P in fp32:
      // the output's own rounding is most of either.)  The sum is of P in fp32.
      const float z = m == -INFINITY ? 0.0f : m;
      const uint32_t zb = __float_as_uint(-z), sb = __float_as_uint(a.scale_log2);
      const uint64_t z2 = pair(zb, zb), scale2 = pair(sb, sb);
      uint64_t l0 = 0, l1 = 0;
      uint32_t p[kPiece / 2];
#pragma unroll
      for (int e = 0; e < kPiece; e += 4) {
        float2 u = halves(fma2(pair(s[e], s[e + 1]), scale2, z2)), v = halves(fma2(pair(s[e + 2], s[e + 3]), scale2, z2));
        u.x = ex2(u.x), u.y = ex2(u.y), v.x = ex2(v.x), v.y = ex2(v.y);
        l0 = add2(l0, pair(__float_as_uint(u.x), __float_as_uint(u.y)));
        l1 = add2(l1, pair(__float_as_uint(v.x), __float_as_uint(v.y)));
        p[e / 2] = pack_bf16(u.x, u.y);
        p[e / 2 + 1] = pack_bf16(v.x, v.y);
      }
      tmem_store(t_s, p);
      const float2 ls = halves(add2(l0, l1));
      l += ls.x + ls.y;
      tmem_store_wait();
      tc_fence_before();
      mbar_arrive(&c.p_ready[w][buf]);
    }

    // the output: every P V is done with the barriers of the two steps behind
    // the last one (the first of them is not there if there was only one step)
    q = QTile<D>{};  // what it held is not kept through the tiles
    if (k + 1 < n_items) load_q<D>(a, c.items[k + 1], q);
#pragma unroll
    for (int x = 0; x < 2; ++x) {
      const int buf = (steps + x) & 1;
      if (steps + x < 2) continue;
      if (!__all_sync(FULL, wait(c, &c.s_full[w][buf], st.s_phase >> buf & 1, a))) return false;
      st.s_phase ^= 1u << buf;
    }
    if (!__all_sync(FULL, wait(c, &c.o_full[w], st.o_phase, a))) return false;
    st.o_phase ^= 1;
    tc_fence_after();
    auto groups_meet = [&]() {
      mbar_arrive(&c.rows_done);
      const bool ok = __all_sync(FULL, wait(c, &c.rows_done, st.done_phase, a));
      st.done_phase ^= 1;
      return ok;
    };
    // 128 rows: the groups' sums over their halves of the slots are joined, each
    // group writing half of the columns; the other half goes through Q's place
    const bool join = !both;
    const int col0 = join ? w * (D / 2) : 0, cols = join ? D / 2 : D;
    float4* mail = reinterpret_cast<float4*>(smem + G::kQ);  // [D / 4][kTile]: four columns of a row
    float f0 = 1.0f, f1 = 0.0f;
    if (join) {
      if (!groups_meet()) return false;  // no MMA reads Q any more
      if (warp_mine) {
#pragma unroll 1
        for (int x = 0; x < D / 2; x += 32) {
          uint32_t o[32];
          tmem_load(t_o + (w ^ 1) * (D / 2) + x, o);
#pragma unroll
          for (int e = 0; e < 32; e += 4)
            mail[((w ^ 1) * (D / 2) + x + e) / 4 * kTile + r] =
                make_float4(__uint_as_float(o[e]), __uint_as_float(o[e + 1]), __uint_as_float(o[e + 2]), __uint_as_float(o[e + 3]));
        }
      }
      c.ml[w][r] = make_float2(m, l);
      if (!groups_meet()) return false;
      const float2 ml = c.ml[w ^ 1][r];
      const float top = fmaxf(m, ml.x), z = top == -INFINITY ? 0.0f : top;
      f0 = ex2(m - z), f1 = ex2(ml.x - z);
      m = top;
      l = l * f0 + ml.y * f1;
    }
    const bool odd = *reinterpret_cast<volatile int*>(&c.bad_v[k]) != 0;
    if (warp_mine) {
      const bool joined = kShared && it.slot < 0 && it.from != 0;  // whole, but its rows have another item
      const float inv = it.slot >= 0 || joined ? 1.0f : l == 0.0f ? 0.0f : 1.0f / l;
      const int64_t rows = (int64_t)a.b.n_tokens * a.group, at = it.h * rows + (int64_t)it.t0 * a.group + it.row0 + local;
      const int kind = kShared && it.from == kPrefix ? 0 : 1;
      uint16_t* dst = a.out + (int64_t)(it.t0 + i) * a.out_stride + (int64_t)(it.h * a.group + g) * D;
#pragma unroll 1
      for (int x = col0; x < col0 + cols; x += 32) {
        uint32_t u[32];
        tmem_load(t_o + x, u);
        float o[32];
        const uint64_t by0 = pair(__float_as_uint(f0), __float_as_uint(f0)), by1 = pair(__float_as_uint(f1), __float_as_uint(f1));
#pragma unroll
        for (int e = 0; e < 32; e += 4) {
          uint64_t y0 = mul2(pair(u[e], u[e + 1]), by0), y1 = mul2(pair(u[e + 2], u[e + 3]), by0);
          if (join) {
            const float4 v = mail[(x + e) / 4 * kTile + r];
            y0 = fma2(pair(__float_as_uint(v.x), __float_as_uint(v.y)), by1, y0);
            y1 = fma2(pair(__float_as_uint(v.z), __float_as_uint(v.w)), by1, y1);
          }
          const float2 h0 = halves(y0), h1 = halves(y1);
          o[e] = h0.x, o[e + 1] = h0.y, o[e + 2] = h1.x, o[e + 3] = h1.y;
        }
        if (odd && mine) add_odd_v<D, kShared>(a, it, i, g, pos, word0, m, x, o);
        if (mine && (joined || it.slot >= 0)) {
          float4* to = kShared && joined ? a.seg_o + (kind * (D / 4) + x / 4) * rows * a.pools.n_kv + at
                                         : a.part_o + ((int64_t)it.slot * (D / 4) + x / 4) * kRows + local;
          const int64_t step = kShared && joined ? rows * a.pools.n_kv : kRows;
#pragma unroll
          for (int e = 0; e < 32; e += 4) to[e / 4 * step] = make_float4(o[e], o[e + 1], o[e + 2], o[e + 3]);
        } else if (mine) {
#pragma unroll
          for (int e = 0; e < 32; e += 8) {
            uint4 v;
            v.x = pack_bf16(o[e] * inv, o[e + 1] * inv), v.y = pack_bf16(o[e + 2] * inv, o[e + 3] * inv);
            v.z = pack_bf16(o[e + 4] * inv, o[e + 5] * inv), v.w = pack_bf16(o[e + 6] * inv, o[e + 7] * inv);
            *reinterpret_cast<uint4*>(dst + x + e) = v;
          }
        }
      }
      if (mine && col0 == 0) {
        if (it.slot >= 0)
          a.part_ml[(int64_t)it.slot * kRows + local] = make_float2(m, l);
        else if (joined)
          a.seg_ml[kind * rows * a.pools.n_kv + at] = make_float2(m, l);
        else if (a.lse)
          a.lse[(int64_t)(it.t0 + i) * a.n_q + it.h * a.group + g] = (m + log2f(l)) * 0.693147180559945309f;
      }
    }
    tc_fence_before();
    if (!groups_meet()) return false;  // Q and the outputs may be overwritten
  }
  return true;
}

// Where the joining kernel finds an item (kind 0 a group's, 1 a sequence's own):
// token rows ascend with the sequences, so no two items of a kind and head share a place.
__device__ __forceinline__ int64_t placed_at(const AttnArgs& a, int kind, int h, int b, int t0, int row0) {
  return ((int64_t)kind * a.pools.n_kv + h) * a.item_rows + (int64_t)t0 * a.group / kRows + row0 / kRows + b;
}

// The next items of a CTA's units [u, end), which began at `begin` (by one warp).
template <bool kShared>
__device__ __forceinline__ void plan_items(const AttnArgs& a, Ctl& c, const Group& mine, const Load& first, const Costs& costs, int64_t begin, int64_t u, int64_t end) {
  const bool one = threadIdx.x % 32 == 0;
  int n = 0;
  int64_t next = end;
  each_item<kShared>(a, mine, first, costs, u, end, [&](Item it, int64_t at, int w) {
    if (!kShared && one && u == begin && n == 0) {
      a.borders[blockIdx.x].at = at;
      a.borders[blockIdx.x].item = it;
    }
    if (n == kMaxItems) {
      next = at;
      return false;
    }
    if (kShared) {  // the tiles whose first unit is in [begin, end)
      const int tiles = it.hi - it.lo;
      const int64_t k0 = at < begin ? tiles_in(begin - at, w) : 0, k1 = tiles_in(end - at, w);
      if (k0 >= tiles) return true;  // its last tile begins in front
      if (one) {
        Placed& p = a.placed[placed_at(a, it.from == kPrefix ? 0 : 1, it.h, it.b, it.t0, it.row0)];
        if (k0 == 0) p.first = blockIdx.x;
        if (k1 >= tiles) p.last = blockIdx.x;
      }
      if (k0 > 0)
        it.slot = 2 * blockIdx.x;
      else if (k1 < tiles)
        it.slot = 2 * blockIdx.x + 1;
      it.hi = it.lo + (int)(k1 < tiles ? k1 : tiles);
      it.lo += (int)k0;
    } else {
      const int64_t stop = at + (it.hi - it.lo);
      const int64_t from = at < begin ? begin : at, to = stop < end ? stop : end;
      // a part that begins its item is the run's last, any other its first
      if (from > at)
        it.slot = 2 * blockIdx.x;
      else if (to < stop)
        it.slot = 2 * blockIdx.x + 1;
      it.hi = it.lo + (int)(to - at);
      it.lo += (int)(from - at);
    }
    if (one) {
      c.items[n] = it;
      c.bad_v[n] = 0;
    }
    ++n;
    return true;
  });
  if (one) {
    c.n_items = n;
    c.next = next;
  }
}

template <int D, bool kShared>
__global__ void __launch_bounds__(kThreads, 1) attn_kernel(const __grid_constant__ AttnArgs a) {
  using G = Geo<D>;
  extern __shared__ __align__(1024) uint8_t smem[];
  Ctl& c = *reinterpret_cast<Ctl*>(smem + G::kCtl);
  const int tid = threadIdx.x, warp = uniform(tid / 32);
  wait_before();
  let_next_in();
  if ((smem_u32(smem) & 1023) != 0) {  // the MMAs' layouts count on it
    if (tid == 0) {
      record(a.status, ERR_SMEM_ALIGN, a.op, 0, 0, smem_u32(smem), 1024);
      if (!kShared) {
        a.borders[blockIdx.x].first = a.borders[blockIdx.x].at = 0;
        if (blockIdx.x == 0) a.borders[gridDim.x].first = 0;
      }
    }
    if (kShared)
      for (int64_t t = blockIdx.x * kThreads + tid; t < a.b.n_tokens; t += gridDim.x * kThreads) a.tokens[t].b = -1;
    return;
  }
  Group mine;
  Load load;
  Costs costs;
  int64_t u = 0, end = 0;
  if (warp == 0) {  // this CTA's units, and its first items
    const int64_t total = total_units<kShared>(a, gridDim.x, mine, load, costs);
    u = border(total, blockIdx.x, gridDim.x);
    end = border(total, blockIdx.x + 1, gridDim.x);
    if (tid == 0) {
      c.first = u;
      c.end = end;
      if (!kShared) {
        a.borders[blockIdx.x].first = u;
        a.borders[blockIdx.x].at = u;  // until the plan says more
        if (blockIdx.x == 0) a.borders[gridDim.x].first = total;
      }
    }
    plan_items<kShared>(a, c, mine, load, costs, u, u, end);
  } else if (warp == 1) {
    if (tid == 32) {
      c.abort = 0;
      for (int i = 0; i < G::kStages; ++i) {
        mbar_init(&c.full[i], 1);
        mbar_init(&c.empty[i], 2);
      }
      for (int i = 0; i < 2; ++i) {
        for (int b = 0; b < 2; ++b) {
          mbar_init(&c.s_full[i][b], 1);
          mbar_init(&c.p_ready[i][b], 128);
        }
        mbar_init(&c.o_full[i], 1);
      }
      mbar_init(&c.v_go, 2);
      mbar_init(&c.v_ok, 1);
      mbar_init(&c.q_ready, 256);
      mbar_init(&c.rows_done, 256);
      mbar_init(&c.drain, 2);
      asm volatile("fence.mbarrier_init.release.cluster;" ::: "memory");
    }
    __syncwarp();
    tmem_alloc(&c.tmem, 512);
  } else if (kShared) {  // what the joining kernel asks of a token, by the warps that have nothing to do yet
    for (int64_t i = blockIdx.x + (warp - 2) * gridDim.x; i < a.b.n_tokens; i += (kThreads / 32 - 2) * gridDim.x) {
      const int t = (int)i;
      Seq s;
      const int b = sequence_at(a.b, t, a.pools.page_shift, a.status, a.op, s);
      Token x = {0, -1, 0, -1};
      if (b >= 0) {
        const Part own = own_part(a, b);
        if (own.n > 0) x.b = b, x.t0 = own.t0;
        if (own.n > 0 && own.from > 0) {
          const Part all = group_part(a, group_at(a, b));
          x.group_b = all.b, x.group_t0 = all.t0;
        }
      }
      if (tid % 32 == 0) a.tokens[t] = x;
    }
  }
  __syncthreads();
  const int64_t begin = c.first;
  u = begin, end = c.end;

  // The softmax warps keep a row of S in registers: the other warps hand them
  // theirs (128 x 80 + 256 x 208 of the launch's 384 x 168).
  bool ok = true;
  Ring fill;
  uint32_t filled = 0;
  if (warp < 4) {
    asm volatile("setmaxnreg.dec.sync.aligned.u32 80;");
    CleanState check;
    MmaState mma;
    while (u < end && ok) {
      if (u > begin) {
        if (warp == 0) plan_items<kShared>(a, c, mine, load, costs, begin, u, end);
        __syncthreads();
      }
      if (warp == 0)
        ok = produce<D, kShared>(a, smem, c, fill, filled);
      else if (warp < 3)
        ok = issue_mmas<D>(a, smem, c, mma, warp - 1);
      else
        ok = clean_v<D, kShared>(a, smem, c, check);
      ok = __syncthreads_and(ok);
      u = c.next;
      __syncthreads();
    }
  } else {
    asm volatile("setmaxnreg.inc.sync.aligned.u32 208;");
    RowState rows;
    while (u < end && ok) {
      if (u > begin) __syncthreads();
      ok = softmax_rows<D, kShared>(a, smem, c, rows);
      ok = __syncthreads_and(ok);
      u = c.next;
      __syncthreads();
    }
  }
  if (!ok) {
    // a wait was given up: the copies and MMAs in flight first (bounded)
    if (tid == 0) {
      Ring r = fill;
      for (uint32_t i = 0; i < (uint32_t)G::kStages && i < filled; ++i) {  // the last fill of every stage
        r.stage = r.stage == 0 ? G::kStages - 1 : r.stage - 1;
        if (r.stage == G::kStages - 1) r.phase ^= 1;
        for (int64_t until = gtimer() + kWaitNs; !mbar_try_wait(&c.full[r.stage], r.phase) && gtimer() < until;) {
        }
      }
    }
    if ((warp == 1 || warp == 2) && elected()) {  // the lanes that issued the MMAs
      tc_commit(&c.drain);
      for (int64_t until = gtimer() + kWaitNs; !mbar_try_wait(&c.drain, 0) && gtimer() < until;) {
      }
    }
    __syncthreads();
  }
  __syncwarp();
  if (warp == 1) tmem_dealloc(c.tmem, 512);
}

// ------------------------------------------------------------- the join

constexpr int kJoinRows = 32, kJoinThreads = 256, kJoinCols = kJoinThreads / 32 * 4, kMaxGrid = 160;

// A block joins 32 rows of an item that is cut (the border between CTAs c - 1
// and c of the first kernel is the first one inside it): the parts of CTAs c -
// 1, c, ..., four columns to a warp, a row to a lane.  It is bound by the
// latency of its loads (a part's rows lie side by side: 512 bytes per warp and
// load).  kShare 1: block (c - 1, y), if that border is such a one, for all
// columns, two parts under way: most items have no more, and few blocks are
// few rounds of latency (a 2048-token run 232 us as a whole; 241 with eight
// parts under way in blocks of 32 columns, 234 with two; items of 38 parts
// among others take 2 us longer).  kShare 4, for few items, whose parts are
// many: block (k, y, z) takes the k-th cut and 32 columns, four warps share its
// parts and meet in shared memory (38 parts of one sequence's four heads: 7.7
// us with eight parts under way and kShare 1).
template <int D, int kShare>
__global__ void __launch_bounds__(kJoinThreads* kShare) join_kernel(const __grid_constant__ AttnArgs a, int grid) {
  constexpr int kWarps = kJoinThreads / 32, kHeld = kShare == 1 ? 2 : 4;  // parts under way
  constexpr int kQuads = kShare == 1 ? D / kJoinCols : 1;  // fours of columns of a thread
  __shared__ float2 meet_ml[kShare == 1 ? 1 : kWarps * kShare][32];
  __shared__ float4 meet_o[kShare == 1 ? 1 : kWarps * kShare][32];
  __shared__ int cuts[kShare == 1 ? 1 : 32];
  __shared__ int which;
  const int tid = threadIdx.x, lane = tid % 32, warp = tid / 32;
  wait_before();
  let_next_in();
  int c = blockIdx.x + 1;
  if (kShare > 1) {
    const bool cut = tid > 0 && tid < grid && a.borders[tid].at < a.borders[tid].first && a.borders[tid - 1].first <= a.borders[tid].at;
    const uint32_t in = __ballot_sync(FULL, cut);
    if (lane == 0) cuts[warp] = __popc(in);
    if (tid == 0) which = 0;
    __syncthreads();
    int rank = __popc(in & ((1u << lane) - 1));
    for (int w = 0; w < warp; ++w) rank += cuts[w];
    if (cut && rank == (int)blockIdx.x) which = tid;
    __syncthreads();
    c = which;
    if (c == 0) return;
  }
  const Border& here = a.borders[c];
  const int64_t first = here.first, at = here.at;
  if (at >= first || a.borders[c - 1].first > at || (int)blockIdx.y * kJoinRows >= here.item.rows) return;
  const Item& item = here.item;
  const int64_t to = at + (item.hi - item.lo);
  const int parts = __syncthreads_count(tid < grid - (c - 1) && a.borders[c - 1 + tid].first < to);
  const int row = blockIdx.y * kJoinRows + lane, col = blockIdx.z * kWarps * kQuads + warp % kWarps;  // columns in fours
  float4 o[kQuads];
#pragma unroll
  for (int y = 0; y < kQuads; ++y) o[y] = make_float4(0, 0, 0, 0);
  float top = -INFINITY, sum = 0.0f;
  for (int k0 = warp / kWarps; k0 < parts; k0 += kHeld * kShare) {
    float2 ml[kHeld];
    float4 p[kHeld][kQuads];
#pragma unroll
    for (int x = 0; x < kHeld; ++x) {
      const int k = k0 + x * kShare;
      ml[x] = make_float2(-INFINITY, 0.0f);
      if (k < parts) {
        // a part that begins its item is its CTA's last, the others their CTA's first
        const int64_t s = 2 * (c - 1 + k) + (k == 0 ? 1 : 0);
        ml[x] = a.part_ml[s * kRows + row];
#pragma unroll
        for (int y = 0; y < kQuads; ++y) p[x][y] = a.part_o[(s * (D / 4) + col + y * kWarps) * kRows + row];
      }
    }
    float up = top;
#pragma unroll
    for (int x = 0; x < kHeld; ++x) up = fmaxf(up, ml[x].x);
    const float z = up == -INFINITY ? 0.0f : up, by = ex2(top - z);
#pragma unroll
    for (int y = 0; y < kQuads; ++y) o[y].x *= by, o[y].y *= by, o[y].z *= by, o[y].w *= by;
    sum *= by;
    top = up;
#pragma unroll
    for (int x = 0; x < kHeld; ++x) {
      if (k0 + x * kShare >= parts) break;
      const float f = ex2(ml[x].x - z);
#pragma unroll
      for (int y = 0; y < kQuads; ++y)
        o[y].x += p[x][y].x * f, o[y].y += p[x][y].y * f, o[y].z += p[x][y].z * f, o[y].w += p[x][y].w * f;
      sum += ml[x].y * f;
    }
  }
  if (kShare > 1) {
    meet_ml[warp][lane] = make_float2(top, sum);
    meet_o[warp][lane] = o[0];
    __syncthreads();
    if (warp >= kWarps) return;
    float up = top;
    for (int x = 1; x < kShare; ++x) up = fmaxf(up, meet_ml[warp + x * kWarps][lane].x);
    const float z = up == -INFINITY ? 0.0f : up, by = ex2(top - z);
    o[0].x *= by, o[0].y *= by, o[0].z *= by, o[0].w *= by;
    sum *= by;
    top = up;
    for (int x = 1; x < kShare; ++x) {
      const float2 ml = meet_ml[warp + x * kWarps][lane];
      const float4 p = meet_o[warp + x * kWarps][lane];
      const float f = ex2(ml.x - z);
      o[0].x += p.x * f, o[0].y += p.y * f, o[0].z += p.z * f, o[0].w += p.w * f;
      sum += ml.y * f;
    }
  }
  if (row >= item.rows) return;
  const uint32_t f = item.row0 + row;
  const int i = f / (uint32_t)a.group, g = f % (uint32_t)a.group;
  const float inv = sum == 0.0f ? 0.0f : 1.0f / sum;
  uint16_t* dst = a.out + (int64_t)(item.t0 + i) * a.out_stride + (int64_t)(item.h * a.group + g) * D;
#pragma unroll
  for (int y = 0; y < kQuads; ++y)
    *reinterpret_cast<uint2*>(dst + (col + y * kWarps) * 4) = make_uint2(pack_bf16(o[y].x * inv, o[y].y * inv), pack_bf16(o[y].z * inv, o[y].w * inv));
  if (col == 0 && a.lse) a.lse[(int64_t)(item.t0 + i) * a.n_q + item.h * a.group + g] = (top + log2f(sum)) * 0.693147180559945309f;
}

// kShared: a lane joins a query head's row of token blockIdx.x, four columns to
// a warp, from its group's item and its sequence's own; each of them lies as a
// whole in seg_o, or in the parts of the CTAs that its tiles were dealt to.  A
// row that has neither another item nor another part was written by the first
// kernel; one whose items are nowhere (parts_of: a wait was given up, which is
// recorded) stays as it is.  Bound by latency: two round trips for the token and
// its items, one for the first part of both, one for each kUnderWay further
// parts.  kShare 4, for few tokens, whose parts are many: four warps share a
// quad's further parts and meet in shared memory.
template <int D, int kShare>
__global__ void __launch_bounds__(kJoinThreads) merge_kernel(const __grid_constant__ AttnArgs a, int grid) {
  constexpr int kWarps = kJoinThreads / 32 / kShare, kUnderWay = kShare == 1 ? 6 : 4;
  __shared__ float2 meet_ml[kShare == 1 ? 1 : kWarps * kShare][32];
  __shared__ float4 meet_o[kShare == 1 ? 1 : kWarps * kShare][32];
  const int tid = threadIdx.x, lane = tid % 32, warp = tid / 32, t = blockIdx.x;
  wait_before();
  let_next_in();
  const Token tok = a.tokens[t];
  if (tok.b < 0) return;
  const int head = blockIdx.y * 32 + lane, at = min(head, a.n_q - 1), h = at / a.group, g = at - h * a.group;
  const int64_t all_rows = (int64_t)a.b.n_tokens * a.group * a.pools.n_kv, row = (h * (int64_t)a.b.n_tokens + t) * a.group + g;
  const int r1 = (t - tok.t0) * a.group + g, r0 = (t - tok.group_t0) * a.group + g;
  const Placed own = a.placed[placed_at(a, 1, h, tok.b, tok.t0, r1)];
  Placed all = {0, -1};
  if (tok.group_b >= 0) all = a.placed[placed_at(a, 0, h, tok.group_b, tok.group_t0, r0)];
  const int n0 = parts_of(all, grid), n1 = parts_of(own, grid);
  const bool mine = head < a.n_q && (n0 > 0 ? n1 > 0 : n1 > 1 && tok.group_b < 0);
  if (kShare == 1 ? !__any_sync(FULL, mine) : !__syncthreads_or(mine)) return;
  const int share = warp / kWarps, col = blockIdx.z * kWarps + warp % kWarps;  // columns in fours
  float4 o = make_float4(0, 0, 0, 0);
  float top = -INFINITY, sum = 0.0f;
  auto add = [&](float2 ml, const float4& p) {
    const float up = fmaxf(top, ml.x), z = up == -INFINITY ? 0.0f : up, by = ex2(top - z), f = ex2(ml.x - z);
    o.x = o.x * by + p.x * f, o.y = o.y * by + p.y * f, o.z = o.z * by + p.z * f, o.w = o.w * by + p.w * f;
    sum = sum * by + ml.y * f;
    top = up;
  };
  // the first parts: a whole item, or its first CTA's last part
  if (mine && share == 0) {
    float2 ml[2];
    float4 p[2];
#pragma unroll
    for (int x = 0; x < 2; ++x) {
      const int n = x ? n1 : n0;
      ml[x] = make_float2(-INFINITY, 0.0f);
      p[x] = make_float4(0, 0, 0, 0);
      if (n == 1) {
        ml[x] = a.seg_ml[x * all_rows + row];
        p[x] = a.seg_o[(x * (D / 4) + col) * all_rows + row];
      } else if (n > 1) {
        const int64_t slot = part_slot(x ? own : all, 0);
        ml[x] = a.part_ml[slot * kRows + (x ? r1 : r0) % kRows];
        p[x] = a.part_o[(slot * (D / 4) + col) * kRows + (x ? r1 : r0) % kRows];
      }
    }
    add(ml[0], p[0]);
    add(ml[1], p[1]);
  }
  // the others: their CTAs' first parts, one slot in two
#pragma unroll
  for (int x = 0; x < 2; ++x) {
    const int n = mine ? x ? n1 : n0 : 0, r = (x ? r1 : r0) % kRows;
    const int64_t slot = part_slot(x ? own : all, 1 + share);
    const float2* pml = a.part_ml + slot * kRows + r;
    const float4* po = a.part_o + (slot * (D / 4) + col) * kRows + r;
    constexpr int kStep = 2 * kShare;  // slots from part to part
#pragma unroll 1
    for (int k = 1 + share; k < n; k += kUnderWay * kShare, pml += kUnderWay * kStep * kRows, po += (int64_t)kUnderWay * kStep * (D / 4) * kRows) {
      float2 ml[kUnderWay];
      float4 p[kUnderWay];
#pragma unroll
      for (int y = 0; y < kUnderWay; ++y) {
        ml[y] = make_float2(-INFINITY, 0.0f);
        p[y] = make_float4(0, 0, 0, 0);
        if (k + y * kShare < n) ml[y] = pml[y * kStep * kRows], p[y] = po[y * kStep * (D / 4) * kRows];
      }
      float up = top;
#pragma unroll
      for (int y = 0; y < kUnderWay; ++y) up = fmaxf(up, ml[y].x);
      const float z = up == -INFINITY ? 0.0f : up, by = ex2(top - z);
      o.x *= by, o.y *= by, o.z *= by, o.w *= by;
      sum *= by;
      top = up;
#pragma unroll
      for (int y = 0; y < kUnderWay; ++y) {
        const float f = ex2(ml[y].x - z);
        o.x += p[y].x * f, o.y += p[y].y * f, o.z += p[y].z * f, o.w += p[y].w * f;
        sum += ml[y].y * f;
      }
    }
  }
  if (kShare > 1) {
    meet_ml[warp][lane] = make_float2(top, sum);
    meet_o[warp][lane] = o;
    __syncthreads();
    if (share > 0) return;
    for (int x = 1; x < kShare; ++x) add(meet_ml[warp + x * kWarps][lane], meet_o[warp + x * kWarps][lane]);
  }
  if (!mine) return;
  const float inv = sum == 0.0f ? 0.0f : 1.0f / sum;
  *reinterpret_cast<uint2*>(a.out + (int64_t)t * a.out_stride + (int64_t)head * D + col * 4) =
      make_uint2(pack_bf16(o.x * inv, o.y * inv), pack_bf16(o.z * inv, o.w * inv));
  if (col == 0 && a.lse) a.lse[(int64_t)t * a.n_q + head] = (top + log2f(sum)) * 0.693147180559945309f;
}

size_t part_bytes(int grid, int head_dim) {
  return (size_t)2 * grid * kRows * (head_dim * 4 + 8) + (grid + 1) * sizeof(Border);
}

int64_t item_rows(int64_t n_tokens, int64_t group, int64_t batch) { return n_tokens * group / kRows + batch + 1; }

// The shared form's workspace: the parts, whole items, the tokens, where items are.
size_t shared_bytes(int grid, int head_dim, int n_kv, int64_t n_tokens, int64_t group, int64_t batch) {
  return (size_t)2 * grid * kRows * (head_dim * 4 + 8) + (size_t)2 * n_kv * n_tokens * group * (head_dim * 4 + 8) +
         (size_t)2 * n_kv * item_rows(n_tokens, group, batch) * sizeof(Placed) + (size_t)n_tokens * sizeof(Token);
}

constexpr int kFew = 32;
template <int D>
int launch_shared(const AttnArgs& a, int grid, cudaStream_t st) {
  constexpr int smem = Geo<D>::kCtl + (int)sizeof(Ctl);
  static std::atomic<uint64_t> ready{0};
  int rc = allow_smem(ready, reinterpret_cast<const void*>(&attn_kernel<D, true>), smem, "prefix_attn");
  if (rc != MK_OK) return rc;
  rc = launch("prefix_attn", attn_kernel<D, true>, dim3(grid), kThreads, smem, st, a);
  if (rc != MK_OK) return rc;
  const unsigned T = (unsigned)a.b.n_tokens, heads = (unsigned)(a.n_q + 31) / 32;
  if ((int64_t)T * heads <= kFew) return launch("prefix_attn", merge_kernel<D, 4>, dim3(T, heads, D / 8), kJoinThreads, 0, st, a, grid);
  return launch("prefix_attn", merge_kernel<D, 1>, dim3(T, heads, D / 32), kJoinThreads, 0, st, a, grid);
}

template <int D>
int launch_both(const AttnArgs& a, int grid, cudaStream_t st) {
  constexpr int smem = Geo<D>::kCtl + (int)sizeof(Ctl);
  static_assert(smem <= 232448, "shared memory of a block");
  static std::atomic<uint64_t> ready{0};
  int rc = allow_smem(ready, reinterpret_cast<const void*>(&attn_kernel<D, false>), smem, "tree_attn");
  if (rc != MK_OK) return rc;
  rc = launch("tree_attn", attn_kernel<D, false>, dim3(grid), kThreads, smem, st, a);
  if (rc != MK_OK || grid == 1) return rc;
  const int64_t rows = (int64_t)a.b.n_tokens * a.group;
  const unsigned y = rows < kRows ? (unsigned)((rows + kJoinRows - 1) / kJoinRows) : kRows / kJoinRows;
  // items at most: one for each K/V head of a sequence, and one more for every
  // kRows query rows
  const int64_t items = ((int64_t)a.b.batch + rows / kRows) * a.pools.n_kv;
  if (items * 8 <= grid)  // eight parts or more to an item
    return launch("tree_attn", join_kernel<D, 4>, dim3((unsigned)items, y, D / kJoinCols), kJoinThreads * 4, 0, st, a, grid);
  return launch("tree_attn", join_kernel<D, 1>, dim3(grid - 1, y), kJoinThreads, 0, st, a, grid);
}

int grid_size() {
  const int n = mk::query_num_sms();
  return n > kMaxGrid ? kMaxGrid : n;
}

}  // namespace
}  // namespace ops
}  // namespace mk

using mk::fail;
using namespace mk::ops;

extern "C" {

size_t mk_tree_attn_workspace_bytes(const mk_kv* kv) {
  const int grid = kv ? grid_size() : 0;
  return grid < 1 ? 0 : part_bytes(grid, kv->cfg.head_dim);
}

static int attend(mk_kv* kv, int32_t layer, const mk_tokens* tok, const mk_attn_io* io, const mk_prefix* prefix,
                  void* workspace, size_t workspace_bytes, uint32_t* status, void* stream) {
  int rc = check_tokens(kv, layer, tok);
  if (rc != MK_OK) return rc;
  const mk_kv_config& c = kv->cfg;
  if (!io) return fail(MK_ERR_ARG, "null argument");
  if (tok->batch == 0 || tok->n_tokens == 0) return MK_OK;
  if (!io->q || !io->out) return fail(MK_ERR_ARG, "null q or out");
  if (io->n_q < c.n_kv || io->n_q % c.n_kv != 0 || io->n_q > (1 << 16)) return fail(MK_ERR_ARG, "n_q must be a multiple of n_kv");
  if ((int64_t)tok->n_tokens * (io->n_q / c.n_kv) > INT32_MAX) return fail(MK_ERR_ARG, "more than 2^31 - 1 query rows per K/V head");
  const int64_t row = (int64_t)io->n_q * c.head_dim;
  if (misaligned(io->q) || misaligned(io->out) || io->q_stride < row || io->out_stride < row || io->q_stride % 8 ||
      io->out_stride % 8 || endless(tok->n_tokens, io->q_stride, 2) || endless(tok->n_tokens, io->out_stride, 2))
    return fail(MK_ERR_ARG, "misaligned q or out, or a stride that is too small, too large or no multiple of 16 bytes");
  if (overlap(io->out, span(tok->n_tokens, io->out_stride, row, 2), io->q, span(tok->n_tokens, io->q_stride, row, 2)))
    return fail(MK_ERR_ARG, "out overlaps q");
  if (misplaced(io->tree_mask, io->lse, status)) return fail(MK_ERR_ARG, "misaligned tree_mask, lse or status");
  if (io->tree_mask ? io->mask_words < 1 : io->mask_words != 0)
    return fail(MK_ERR_ARG, "mask_words must be positive with a tree_mask and 0 without");
  if (io->window < 0) return fail(MK_ERR_ARG, "negative window");
  if (!(io->scale >= 0) || !std::isfinite(io->scale * 1.5f)) return fail(MK_ERR_ARG, "scale must be positive (0: 1 / sqrt(head_dim))");
  if (!workspace || misaligned(workspace)) return fail(MK_ERR_ARG, "workspace null or misaligned");
  const size_t lse_bytes = io->lse ? (size_t)tok->n_tokens * io->n_q * 4 : 0;
  const size_t out_bytes = span(tok->n_tokens, io->out_stride, row, 2), q_bytes = span(tok->n_tokens, io->q_stride, row, 2);
  if (overlap(workspace, workspace_bytes, io->out, out_bytes) || overlap(workspace, workspace_bytes, io->q, q_bytes) ||
      overlap(workspace, workspace_bytes, io->lse, lse_bytes) || overlap(io->lse, lse_bytes, io->out, out_bytes) ||
      overlap(io->lse, lse_bytes, io->q, q_bytes))
    return fail(MK_ERR_ARG, "workspace or lse overlaps another argument");
  const size_t mask_bytes = (size_t)tok->n_tokens * io->mask_words * 8;
  auto over_inputs = [&](const void* p, size_t bytes) {
    return over_batch(tok, p, bytes) || over_pools(kv, status, p, bytes) || overlap(p, bytes, io->tree_mask, mask_bytes);
  };
  if (over_inputs(io->out, out_bytes) || over_inputs(io->lse, lse_bytes) || over_inputs(workspace, workspace_bytes))
    return fail(MK_ERR_ARG, "out, lse or workspace overlaps the batch's arrays, the mask, the status or the pools");
  if (prefix) {
    const size_t groups = (size_t)prefix->n_groups * 4;
    auto over_groups = [&](const void* p, size_t bytes) {
      return overlap(p, bytes, prefix->group_seqs, groups + 4) || overlap(p, bytes, prefix->prefix_lens, groups);
    };
    if (over_groups(io->out, out_bytes) || over_groups(io->lse, lse_bytes) || over_groups(workspace, workspace_bytes))
      return fail(MK_ERR_ARG, "out, lse or workspace overlaps the groups");
  }
  const int grid = grid_size();
  if (grid < 1) return fail(MK_ERR_CUDA, "no device");
  const int32_t group = io->n_q / c.n_kv;
  if (workspace_bytes < (prefix ? shared_bytes(grid, c.head_dim, c.n_kv, tok->n_tokens, group, tok->batch) : part_bytes(grid, c.head_dim)))
    return fail(MK_ERR_ARG, prefix ? "workspace smaller than mk_prefix_attn_workspace_bytes" : "workspace smaller than mk_tree_attn_workspace_bytes");
  rc = encode_pools(kv);
  if (rc != MK_OK) return rc;
  AttnArgs a = {};
  a.pools = pools_of(kv, layer);
  a.b = batch_of(tok);
  a.q = static_cast<const uint16_t*>(io->q), a.out = static_cast<uint16_t*>(io->out), a.lse = io->lse;
  a.mask = io->tree_mask;
  a.q_stride = io->q_stride, a.out_stride = io->out_stride;
  a.n_q = io->n_q, a.group = group, a.mask_words = io->mask_words;
  a.window = io->window < kMaxSlots ? io->window : kMaxSlots;  // a longer one leaves nothing out, and differences stay in 32 bits
  a.layer = layer;
  a.scale_log2 = (float)((io->scale > 0 ? (double)io->scale : 1.0 / std::sqrt((double)c.head_dim)) * 1.4426950408889634);
  a.part_o = static_cast<float4*>(workspace);
  a.part_ml = reinterpret_cast<float2*>(a.part_o + (size_t)2 * grid * kRows * (c.head_dim / 4));
  a.op = prefix ? OP_PREFIX : OP_ATTN;
  a.status = status;
  a.tm_k = kv->tm_k, a.tm_v = kv->tm_v;
  cudaStream_t st = static_cast<cudaStream_t>(stream);
  if (prefix) {
    const size_t rows = (size_t)c.n_kv * tok->n_tokens * group;
    a.group_seqs = prefix->group_seqs, a.prefix_lens = prefix->prefix_lens, a.n_groups = prefix->n_groups;
    a.item_rows = item_rows(tok->n_tokens, group, tok->batch);
    a.seg_o = reinterpret_cast<float4*>(a.part_ml + (size_t)2 * grid * kRows);
    a.seg_ml = reinterpret_cast<float2*>(a.seg_o + 2 * rows * (c.head_dim / 4));
    a.tokens = reinterpret_cast<Token*>(a.seg_ml + 2 * rows);
    a.placed = reinterpret_cast<Placed*>(a.tokens + tok->n_tokens);
    return c.head_dim == 128 ? launch_shared<128>(a, grid, st) : launch_shared<64>(a, grid, st);
  }
  a.borders = reinterpret_cast<Border*>(a.part_ml + (size_t)2 * grid * kRows);
  return c.head_dim == 128 ? launch_both<128>(a, grid, st) : launch_both<64>(a, grid, st);
}

int mk_tree_attn(mk_kv* kv, int32_t layer, const mk_tokens* tok, const mk_attn_io* io, void* workspace,
                 size_t workspace_bytes, uint32_t* status, void* stream) {
  return attend(kv, layer, tok, io, nullptr, workspace, workspace_bytes, status, stream);
}

size_t mk_prefix_attn_workspace_bytes(const mk_kv* kv, int32_t n_tokens, int32_t n_q, int32_t batch) {
  const int grid = kv ? grid_size() : 0;
  if (grid < 1 || n_tokens < 0 || batch < 0 || n_q < kv->cfg.n_kv || n_q % kv->cfg.n_kv != 0 || n_q > (1 << 16)) return 0;
  return shared_bytes(grid, kv->cfg.head_dim, kv->cfg.n_kv, n_tokens, n_q / kv->cfg.n_kv, batch);
}

int mk_prefix_attn(mk_kv* kv, int32_t layer, const mk_tokens* tok, const mk_attn_io* io, const mk_prefix* prefix,
                   void* workspace, size_t workspace_bytes, uint32_t* status, void* stream) {
  if (!prefix || !tok) return fail(MK_ERR_ARG, "null argument");
  if (prefix->n_groups < 0 || prefix->n_groups > tok->batch) return fail(MK_ERR_ARG, "n_groups is 0 to batch");
  if (prefix->n_groups > 0 && (!prefix->group_seqs || !prefix->prefix_lens)) return fail(MK_ERR_ARG, "null groups");
  if (misplaced(prefix->group_seqs, prefix->prefix_lens)) return fail(MK_ERR_ARG, "misaligned groups");
  return attend(kv, layer, tok, io, prefix, workspace, workspace_bytes, status, stream);
}

}  // extern "C"
