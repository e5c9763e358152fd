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
// trees of up to 16 tokens over 512 to 32K slots 181 us, 1.09 GB of K and V at
// 6.0 TB/s (a copy: 6.8), bound by memory; 2048 tokens of a run over 8K slots
// 232 us, 1.33 PFLOP/s (cuBLAS: 1.9), the tensor pipe active 64% of the
// kernel's cycles, bound by the hand-overs between exponentials and MMAs (a
// step of 64 slots takes a group some 1730 cycles, of which its own and the
// other group's MMAs run 1024); eight tokens over 8K slots 19 us: 2.6 the
// plan, 8 two tiles and the output, 2 to end and begin a kernel, 4 the join.
#include <cmath>

#include "mk_ops_common.cuh"
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
};

// Where a CTA's units begin: its first unit, and the first whole item that it
// has tiles of (its first tile at unit `at`; at = first where there is none).
struct Border {
  int64_t first, at;
  Item item;
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

__device__ __forceinline__ Seq attn_seq(const AttnArgs& a, int b) {
  Seq s = seq_of(a.b, b, a.pools.page_shift, a.status, OP_ATTN);
  if (a.mask && s.n > 64 * (int64_t)a.mask_words) {
    record(a.status, ERR_RANGE, OP_ATTN, b, 2, s.n, 64 * a.mask_words);
    s.n = 0;
  }
  return s;
}

// Tiles [lo, hi) of query group m of a sequence.
__device__ __forceinline__ void tiles_of(const AttnArgs& a, const Seq& s, int m, int& lo, int& hi) {
  const int all = s.n * a.group, r0 = m * kRows, r1 = all - r0 < kRows ? all : r0 + kRows;  // below 2^31
  const int i0 = a.mask ? 0 : (uint32_t)r0 / (uint32_t)a.group, i1 = a.mask ? 0 : (uint32_t)(r1 - 1) / (uint32_t)a.group;
  const int end = s.ctx + (a.mask ? s.n : i1 + 1);
  hi = (end + kTile - 1) / kTile;
  lo = 0;
  if (a.window) {
    const int first = s.ctx + (a.b.positions ? 0 : i0) - a.window + 1;  // the lowest slot that a row sees
    if (first > 0) lo = first / kTile;
  }
}

__device__ __forceinline__ int groups_of(const AttnArgs& a, const Seq& s) {
  return (s.n * a.group - 1) / kRows + (s.n > 0 ? 1 : 0);
}

__device__ __forceinline__ int64_t warp_scan(int64_t v) {  // inclusive
  for (int o = 1; o < 32; o <<= 1) {
    const int64_t w = __shfl_up_sync(FULL, v, o);
    if ((int)(threadIdx.x % 32) >= o) v += w;
  }
  return v;
}

__device__ __forceinline__ int64_t divide(int64_t a, int64_t b) {  // of numbers that are not negative
  return (a | b) >> 32 ? a / b : (int64_t)((uint32_t)a / (uint32_t)b);
}

// A lane's sequence of a round of 32, and the tiles of one of its heads.
struct Load {
  Seq s;
  int64_t tiles;
};
// (By all lanes of a warp: a prompt's many query groups are counted by all of
// them, which took the plan of 2048 tokens from 15 to 5 us.)
__device__ __forceinline__ Load load_of(const AttnArgs& a, int b) {
  const int lane = threadIdx.x % 32;
  Load x = {{0, 0, 0}, 0};
  if (b < a.b.batch) x.s = attn_seq(a, b);
  const int M = groups_of(a, x.s);
  int lo, hi;
  if (M == 1) {
    tiles_of(a, x.s, 0, lo, hi);
    x.tiles = hi - lo;
  }
  for (uint32_t many = __ballot_sync(FULL, M > 1); many; many &= many - 1) {
    const int src = __ffs(many) - 1;
    const Seq q = {__shfl_sync(FULL, x.s.t0, src), __shfl_sync(FULL, x.s.n, src), __shfl_sync(FULL, x.s.ctx, src)};
    int64_t u = 0;
    for (int m = lane, n = groups_of(a, q); m < n; m += 32) {
      tiles_of(a, q, m, lo, hi);
      u += hi - lo;
    }
    for (int o = 16; o > 0; o >>= 1) u += __shfl_xor_sync(FULL, u, o);
    if (lane == src) x.tiles = u;
  }
  return x;
}

// All units (by one warp), the units of an opening, and the lane's sequence of
// the first round.  Openings cost nothing where every SM has a tile at most:
// an item is then the first of its SMs.  With more, counting 3 for one took
// 30 ragged prompts of up to 273 tokens (each over up to 785 slots) from 195
// to 121 us, 32 trees of 16 tokens over up to 32K slots from 197 to 191 us; 1,
// 2 and 4 were slower.
__device__ __forceinline__ int64_t total_units(const AttnArgs& a, int grid, Load& first, int& opening) {
  const int lane = threadIdx.x % 32;
  first = load_of(a, lane);
  int64_t u = first.tiles, items = groups_of(a, first.s);
  for (int b0 = 32; b0 < a.b.batch; b0 += 32) {
    const Load x = load_of(a, b0 + lane);
    u += x.tiles;
    items += groups_of(a, x.s);
  }
  for (int o = 16; o > 0; o >>= 1) {
    u += __shfl_xor_sync(FULL, u, o);
    items += __shfl_xor_sync(FULL, items, o);
  }
  opening = u * a.pools.n_kv > grid ? kOpening : 0;
  return (u + items * opening) * a.pools.n_kv;
}

// The first unit of CTA c: even runs, the longer ones first.
__device__ __forceinline__ int64_t border(int64_t total, int c, int grid) {
  const int64_t base = divide(total, grid), rest = total - base * grid;
  return base * c + (c < rest ? c : rest);
}

// Item m of K/V head h of sequence b, whole.
__device__ __forceinline__ Item make_item(const AttnArgs& a, const Seq& s, int b, int h, int m) {
  Item it;
  it.b = b, it.h = h, it.t0 = s.t0, it.n = s.n, it.ctx = s.ctx;
  it.row0 = m * kRows;
  it.rows = s.n * a.group - it.row0 < kRows ? s.n * a.group - it.row0 : kRows;
  tiles_of(a, s, m, it.lo, it.hi);
  const int i0 = (uint32_t)it.row0 / (uint32_t)a.group, i1 = (uint32_t)(it.row0 + it.rows - 1) / (uint32_t)a.group;
  // without a mask every row sees the new tokens up to the first row's own,
  // unless positions set them a window or more apart
  const bool apart = a.window && a.b.positions && s.n > a.window;
  it.masked_from = s.ctx + (a.mask || apart ? 0 : i0 + 1);
  it.window_to = 0;
  if (a.window) it.window_to = s.ctx + (a.b.positions ? s.n - 1 : i1) - a.window + 1;  // the highest row's lowest slot
  it.slot = -1;
  return it;
}

// Calls f(item, unit of the item's first tile) for the items whose tiles lie in
// units [u, end), in order, while it returns true.  By one warp, whose lanes
// hold the first round's sequences; f runs on every lane.
template <typename F>
__device__ __forceinline__ void each_item(const AttnArgs& a, const Load& first, int opening, int64_t u, int64_t end, F f) {
  const int lane = threadIdx.x % 32;
  int64_t base = 0;  // units before this round of sequences
  for (int b0 = 0; b0 < a.b.batch && base < end; b0 += 32) {
    const Load x = b0 == 0 ? first : load_of(a, b0 + lane);
    const Seq s = x.s;
    const int64_t per_head = x.tiles + groups_of(a, s) * opening;
    const int64_t incl = warp_scan(per_head * a.pools.n_kv);
    uint32_t hit = __ballot_sync(FULL, per_head > 0 && base + incl > u && base + incl - per_head * a.pools.n_kv < end);
    while (hit) {
      const int src = __ffs(hit) - 1;
      hit &= hit - 1;
      const Seq q = {__shfl_sync(FULL, s.t0, src), __shfl_sync(FULL, s.n, src), __shfl_sync(FULL, s.ctx, src)};
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
            if (m + lane < M) tiles_of(a, q, m + lane, lo, hi);
            const int64_t n = m + lane < M ? hi - lo + opening : 0, sum = warp_scan(n);
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
          tiles_of(a, q, m, lo, hi);
          at += opening;
          if (at + (hi - lo) > u) {
            if (at >= end) return;
            if (!f(make_item(a, q, b0 + src, h, m), at)) return;
          }
          at += hi - lo;
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
__device__ __forceinline__ bool wait_slow(Ctl& c, uint64_t* bar, uint32_t parity, uint32_t* status) {
  const int64_t until = gtimer() + kWaitNs;
  for (;;) {
    if (mbar_try_wait(bar, parity)) return true;
    if (ld_volatile(&c.abort)) return false;
    if (gtimer() > until) {
      *reinterpret_cast<volatile uint32_t*>(&c.abort) = 1;
      record(status, ERR_TIMEOUT, OP_ATTN, blockIdx.x, threadIdx.x, 0, 0);
      return false;
    }
  }
}
__device__ __forceinline__ bool wait(Ctl& c, uint64_t* bar, uint32_t parity, uint32_t* status) {
  return mbar_try_wait(bar, parity) || wait_slow(c, bar, parity, status);
}

// A ring position: stage and phase of the k-th tile.
struct Ring {
  int stage = 0;
  uint32_t phase = 0;
  template <int N>
  __device__ __forceinline__ void advance() {
    if (++stage == N) {
      stage = 0;
      phase ^= 1;
    }
  }
};

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
    record(a.status, ERR_RANGE, OP_ATTN, it.b, 3, p, it.ctx + it.n);
    return p < it.ctx ? it.ctx : it.ctx + it.n - 1;
  }
  return p;
}

// Which of the slots s0 .. s0 + 31 token i sees.
__device__ __forceinline__ uint32_t seen(const AttnArgs& a, const Item& it, int i, int pos, uint64_t word0, int s0) {
  const int len = it.ctx + it.n;
  if (s0 >= len) return 0;
  uint32_t v = FULL;
  if (len - s0 < 32) v = FULL >> (32 - (len - s0));
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

template <int D>
__device__ bool produce(const AttnArgs& a, uint8_t* smem, Ctl& c, Ring& r, uint32_t& filled) {
  using G = Geo<D>;
  const int lane = threadIdx.x % 32;
  const int P = 1 << a.pools.page_shift, box = P < kTile ? P : kTile;  // slots of a box
  const int slice = lane / G::kHalves, half = lane % G::kHalves;       // this lane's box of a tile
  for (int k = 0; k < c.n_items; ++k) {
    const Item it = c.items[k];
    const int len = it.ctx + it.n;
    const int32_t* table = a.b.tables + (int64_t)it.b * a.b.max_pages;
    auto page_at = [&](int j) {  // the page of this lane's box in tile j, -1: no slot of it is in use
      const int s = j * kTile + slice * box;
      if (slice * box >= kTile || s >= len) return -1;
      int page = table[s >> a.pools.page_shift];
      if (page < 0 || page >= a.pools.num_pages) {
        record(a.status, ERR_PAGE, OP_ATTN, it.b, s, page, (uint32_t)a.pools.num_pages);
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
        const bool ok = filled < (uint32_t)G::kStages || wait(c, &c.empty[r.stage], r.phase ^ 1, a.status);
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

// Shared-memory operands of the MMAs, as their descriptors' lower words (the
// address in 16-byte units; adding an offset's sixteenth moves the operand)
// and a common upper word: 128-byte rows with the 128-byte swizzle, groups of
// 8 rows every 1024 bytes.  K-major for Q and K; V as the pages hold it, N
// contiguous, the next 64 dims a half tile further (the lower word's upper
// half, which K-major operands ignore).
constexpr uint32_t kDescHi = (1024 >> 4) | (1u << 14) | (2u << 29);
__device__ __forceinline__ uint64_t desc(uint32_t lo) { return (uint64_t)kDescHi << 32 | lo; }

__device__ __forceinline__ uint32_t elected() {
  uint32_t r;
  asm volatile("{\n .reg .pred p;\n elect.sync _|p, 0xffffffff;\n selp.u32 %0, 1, 0, p;\n}" : "=r"(r));
  return r;
}
// The lane for which `on` is not zero issues.
__device__ __forceinline__ void mma_ss_if(uint32_t on, uint32_t d, uint64_t adesc, uint64_t bdesc, uint32_t idesc, uint32_t accumulate) {
  asm volatile(
      "{\n .reg .pred p, q;\n setp.ne.b32 p, %4, 0;\n setp.ne.b32 q, %5, 0;\n"
      " @q tcgen05.mma.cta_group::1.kind::f16 [%0], %1, %2, %3, p;\n}" ::"r"(d),
      "l"(adesc), "l"(bdesc), "r"(idesc), "r"(accumulate), "r"(on)
      : "memory");
}
// A from tensor memory: a lane holds a row, two elements of K per column.
__device__ __forceinline__ void mma_ts_if(uint32_t on, uint32_t d, uint32_t a, uint64_t bdesc, uint32_t idesc, uint32_t accumulate) {
  asm volatile(
      "{\n .reg .pred p, q;\n setp.ne.b32 p, %4, 0;\n setp.ne.b32 q, %5, 0;\n"
      " @q tcgen05.mma.cta_group::1.kind::f16 [%0], [%1], %2, %3, p;\n}" ::"r"(d),
      "r"(a), "l"(bdesc), "r"(idesc), "r"(accumulate), "r"(on)
      : "memory");
}
__device__ __forceinline__ void commit_if(uint32_t on, uint32_t bar) {
  asm volatile(
      "{\n .reg .pred q;\n setp.ne.b32 q, %1, 0;\n"
      " @q tcgen05.commit.cta_group::1.mbarrier::arrive::one.shared::cluster.b64 [%0];\n}" ::"r"(bar),
      "r"(on)
      : "memory");
}
__device__ __forceinline__ void arrive_if(uint32_t on, uint32_t bar) {
  asm volatile(
      "{\n .reg .pred q;\n setp.ne.b32 q, %1, 0;\n @q mbarrier.arrive.release.cta.shared::cta.b64 _, [%0];\n}" ::"r"(bar),
      "r"(on)
      : "memory");
}
__device__ __forceinline__ int uniform(int v) { return __shfl_sync(FULL, v, 0); }

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
  auto ready = [&](uint64_t* bar, uint32_t parity) { return __all_sync(FULL, wait(c, bar, parity, a.status)) != 0; };
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

template <int D>
__device__ bool clean_v(const AttnArgs& a, uint8_t* smem, Ctl& c, CleanState& st) {
  using G = Geo<D>;
  const int lane = threadIdx.x % 32;
  for (int k = 0; k < c.n_items; ++k) {
    const Item it = c.items[k];
    for (int j = it.lo; j < it.hi; ++j) {
      st.k.advance<G::kStages>();  // K
      if (in_part(it, j)) {
        if (!__all_sync(FULL, wait(c, &c.v_go, st.phase, a.status))) return false;
        st.phase ^= 1;
        const uint32_t tile = smem_u32(smem + G::kRing + st.k.stage * G::kTileBytes);
        const int len = it.ctx + it.n, s0 = j * kTile;
        for (int row = lane; row < kTile; row += 32) {
          bool drop = s0 + row >= len;
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
template <int D>
__device__ __forceinline__ void add_odd_v(const AttnArgs& a, const Item& it, int i, int g, int pos, uint64_t word0, float m, int col, float (&o)[32]) {
  const uint16_t* q = a.q + (int64_t)(it.t0 + i) * a.q_stride + (int64_t)(it.h * a.group + g) * D;
  for (int j = it.lo; j < it.hi; ++j) {
    if (!in_part(it, j)) continue;
    for (int s = j * kTile; s < min((j + 1) * kTile, it.ctx + it.n); ++s) {
      if (s < it.masked_from && s >= it.window_to) continue;
      const int64_t row = pool_row(a, it, s) * D;
      uint32_t odd = 0;  // the same for all rows, and quickly known
#pragma unroll
      for (int e = 0; e < D; e += 8) {
        const uint4 u = *reinterpret_cast<const uint4*>(a.pools.v + row + e);
        odd |= any_odd(u.x) | any_odd(u.y) | any_odd(u.z) | any_odd(u.w);
      }
      if (!odd || !(seen(a, it, i, pos, word0, s) & 1)) continue;
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
  const int tid = threadIdx.x - 128, ch = tid % (D / 8), n = both_in(it) ? QTile<D>::kChunks : QTile<D>::kChunks / 2;
#pragma unroll
  for (int x = 0; x < QTile<D>::kChunks; ++x) {
    const int row = tid / (D / 8) + x * (256 / (D / 8));
    q.u[x] = make_uint4(0, 0, 0, 0);
    if (x < n && row < it.rows) {
      const uint32_t f = it.row0 + row, i = f / (uint32_t)a.group, g = f % (uint32_t)a.group;
      q.u[x] = reinterpret_cast<const uint4*>(a.q + (int64_t)(it.t0 + i) * a.q_stride + (int64_t)(it.h * a.group + g) * D)[ch];
    }
  }
}
template <int D>
__device__ __forceinline__ void store_q(uint8_t* smem, bool both, const QTile<D>& q) {
  using G = Geo<D>;
  const int tid = threadIdx.x - 128, ch = tid % (D / 8);
#pragma unroll
  for (int x = 0; x < QTile<D>::kChunks; ++x) {
    const int row = tid / (D / 8) + x * (256 / (D / 8)), rr = row % kTile;
    if (x < (both ? QTile<D>::kChunks : QTile<D>::kChunks / 2))
      *reinterpret_cast<uint4*>(smem + G::kQ + row / kTile * G::kTileBytes + ch / 8 * G::kHalfBytes + rr * 128 + ((ch % 8) ^ (rr & 7)) * 16) = q.u[x];
  }
}

template <int D>
__device__ __forceinline__ bool softmax_rows(const AttnArgs& a, uint8_t* smem, Ctl& c, RowState& st) {
  using G = Geo<D>;
  const int tid = threadIdx.x - 128, w = tid / 128, r = tid % 128;
  const uint32_t lane_base = c.tmem + ((uint32_t)(r / 32 * 32) << 16);
  const uint32_t t_o = lane_base + o_cols(w);
  const int n_items = c.n_items;
  QTile<D> q = {};
  if (n_items > 0) load_q<D>(a, c.items[0], q);
  for (int k = 0; k < n_items; ++k) {
    const Item& it = c.items[k];
    const bool both = both_in(it);
    store_q<D>(smem, both, q);
    fence_proxy_async_smem();
    mbar_arrive(&c.q_ready);

    const int local = both ? w * kTile + r : r;  // row of the item
    const bool mine = local < it.rows;
    const bool warp_mine = (both ? w * kTile : 0) + r / 32 * 32 < it.rows;
    const uint32_t f = it.row0 + (mine ? local : 0);
    const int i = f / (uint32_t)a.group, g = f % (uint32_t)a.group;
    const int pos = a.window ? position_of(a, it, i) : 0;
    const uint64_t word0 = a.mask ? a.mask[(int64_t)(it.t0 + i) * a.mask_words] : 0;
    float m = -INFINITY, l = 0.0f;
    const int lo = it.lo, steps = both ? 2 * (it.hi - lo) : it.hi - lo, masked_from = it.masked_from, window_to = it.window_to;
    for (int t = 0; t < steps; ++t) {
      const int buf = t & 1, j = lo + (both ? t >> 1 : t);
      if (!__all_sync(FULL, wait(c, &c.s_full[w][buf], st.s_phase >> buf & 1, a.status))) return false;
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
          const uint32_t v = seen(a, it, i, pos, word0, j * kTile + (both ? buf : w) * kPiece + x * 32);
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
          if (!__all_sync(FULL, wait(c, &c.s_full[w][buf ^ 1], st.s_phase >> (buf ^ 1) & 1, a.status))) return false;
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
      if (!__all_sync(FULL, wait(c, &c.s_full[w][buf], st.s_phase >> buf & 1, a.status))) return false;
      st.s_phase ^= 1u << buf;
    }
    if (!__all_sync(FULL, wait(c, &c.o_full[w], st.o_phase, a.status))) return false;
    st.o_phase ^= 1;
    tc_fence_after();
    auto groups_meet = [&]() {
      mbar_arrive(&c.rows_done);
      const bool ok = __all_sync(FULL, wait(c, &c.rows_done, st.done_phase, a.status));
      st.done_phase ^= 1;
      return ok;
    };
    // 128 rows: the groups' sums over their halves of the slots are joined, each
    // group writing half of the columns; the other half goes through Q's place
    const bool join = !both;
    const int col0 = join ? w * (D / 2) : 0, cols = join ? D / 2 : D;
    float* mail = reinterpret_cast<float*>(smem + G::kQ);  // [2][D / 2][kTile]
    float f0 = 1.0f, f1 = 0.0f;
    if (join) {
      if (!groups_meet()) return false;  // no MMA reads Q any more
      if (warp_mine) {
#pragma unroll 1
        for (int x = 0; x < D / 2; x += 32) {
          uint32_t o[32];
          tmem_load(t_o + (w ^ 1) * (D / 2) + x, o);
#pragma unroll
          for (int e = 0; e < 32; ++e) mail[((w ^ 1) * (D / 2) + x + e) * kTile + r] = __uint_as_float(o[e]);
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
      const float inv = it.slot >= 0 ? 1.0f : l == 0.0f ? 0.0f : 1.0f / l;
      uint16_t* dst = a.out + (int64_t)(it.t0 + i) * a.out_stride + (int64_t)(it.h * a.group + g) * D;
#pragma unroll 1
      for (int x = col0; x < col0 + cols; x += 32) {
        uint32_t u[32];
        tmem_load(t_o + x, u);
        float o[32];
#pragma unroll
        for (int e = 0; e < 32; ++e) o[e] = __uint_as_float(u[e]) * f0;
        if (join) {
#pragma unroll
          for (int e = 0; e < 32; ++e) o[e] += mail[(x + e) * kTile + r] * f1;
        }
        if (odd && mine) add_odd_v<D>(a, it, i, g, pos, word0, m, x, o);
        if (mine && it.slot >= 0) {
#pragma unroll
          for (int e = 0; e < 32; e += 4)
            a.part_o[((int64_t)it.slot * (D / 4) + (x + e) / 4) * kRows + local] = make_float4(o[e], o[e + 1], o[e + 2], o[e + 3]);
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
        else if (a.lse)
          a.lse[(int64_t)(it.t0 + i) * a.n_q + it.h * a.group + g] = (m + log2f(l)) * 0.693147180559945309f;
      }
    }
    tc_fence_before();
    if (!groups_meet()) return false;  // Q and the outputs may be overwritten
  }
  return true;
}

// The next items of a CTA's units [u, end), which began at `begin` (by one warp).
__device__ __forceinline__ void plan_items(const AttnArgs& a, Ctl& c, const Load& first, int opening, int64_t begin, int64_t u, int64_t end) {
  const bool one = threadIdx.x % 32 == 0;
  int n = 0;
  int64_t next = end;
  each_item(a, first, opening, u, end, [&](Item it, int64_t at) {
    if (one && u == begin && n == 0) {
      a.borders[blockIdx.x].at = at;
      a.borders[blockIdx.x].item = it;
    }
    if (n == kMaxItems) {
      next = at;
      return false;
    }
    const int64_t stop = at + (it.hi - it.lo);
    const int64_t from = at < begin ? begin : at, to = stop < end ? stop : end;
    // a part that begins its item is the run's last, any other its first
    if (from > at)
      it.slot = 2 * blockIdx.x;
    else if (to < stop)
      it.slot = 2 * blockIdx.x + 1;
    it.hi = it.lo + (int)(to - at);
    it.lo += (int)(from - at);
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

template <int D>
__global__ void __launch_bounds__(kThreads, 1) attn_kernel(const __grid_constant__ AttnArgs a) {
  using G = Geo<D>;
  extern __shared__ __align__(1024) uint8_t smem[];
  Ctl& c = *reinterpret_cast<Ctl*>(smem + G::kCtl);
  const int tid = threadIdx.x, warp = uniform(tid / 32);
  wait_before();
  let_next_in();
  if ((smem_u32(smem) & 1023) != 0) {  // the MMAs' layouts count on it
    if (tid == 0) {
      record(a.status, ERR_SMEM_ALIGN, OP_ATTN, 0, 0, smem_u32(smem), 1024);
      a.borders[blockIdx.x].first = a.borders[blockIdx.x].at = 0;
      if (blockIdx.x == 0) a.borders[gridDim.x].first = 0;
    }
    return;
  }
  Load load;
  int opening = 0;
  int64_t u = 0, end = 0;
  if (warp == 0) {  // this CTA's units, and its first items
    const int64_t total = total_units(a, gridDim.x, load, opening);
    u = border(total, blockIdx.x, gridDim.x);
    end = border(total, blockIdx.x + 1, gridDim.x);
    if (tid == 0) {
      c.first = u;
      c.end = end;
      a.borders[blockIdx.x].first = u;
      a.borders[blockIdx.x].at = u;  // until the plan says more
      if (blockIdx.x == 0) a.borders[gridDim.x].first = total;
    }
    plan_items(a, c, load, opening, u, u, end);
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
        if (warp == 0) plan_items(a, c, load, opening, begin, u, end);
        __syncthreads();
      }
      if (warp == 0)
        ok = produce<D>(a, smem, c, fill, filled);
      else if (warp < 3)
        ok = issue_mmas<D>(a, smem, c, mma, warp - 1);
      else
        ok = clean_v<D>(a, smem, c, check);
      ok = __syncthreads_and(ok);
      u = c.next;
      __syncthreads();
    }
  } else {
    asm volatile("setmaxnreg.inc.sync.aligned.u32 208;");
    RowState rows;
    while (u < end && ok) {
      if (u > begin) __syncthreads();
      ok = softmax_rows<D>(a, smem, c, rows);
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

size_t part_bytes(int grid, int head_dim) {
  return (size_t)2 * grid * kRows * (head_dim * 4 + 8) + (grid + 1) * sizeof(Border);
}

template <int D>
int launch_both(const AttnArgs& a, int grid, cudaStream_t st) {
  constexpr int smem = Geo<D>::kCtl + (int)sizeof(Ctl);
  static_assert(smem <= 232448, "shared memory of a block");
  static std::atomic<uint64_t> ready{0};
  int rc = allow_smem(ready, reinterpret_cast<const void*>(&attn_kernel<D>), smem, "tree_attn");
  if (rc != MK_OK) return rc;
  rc = launch("tree_attn", attn_kernel<D>, dim3(grid), kThreads, smem, st, a);
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

int mk_tree_attn(mk_kv* kv, int32_t layer, const mk_tokens* tok, const mk_attn_io* io, void* workspace,
                 size_t workspace_bytes, uint32_t* status, void* stream) {
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
  const int grid = grid_size();
  if (grid < 1) return fail(MK_ERR_CUDA, "no device");
  if (workspace_bytes < part_bytes(grid, c.head_dim)) return fail(MK_ERR_ARG, "workspace smaller than mk_tree_attn_workspace_bytes");
  rc = encode_pools(kv);
  if (rc != MK_OK) return rc;
  AttnArgs a;
  a.pools = pools_of(kv, layer);
  a.b = batch_of(tok);
  a.q = static_cast<const uint16_t*>(io->q), a.out = static_cast<uint16_t*>(io->out), a.lse = io->lse;
  a.mask = io->tree_mask;
  a.q_stride = io->q_stride, a.out_stride = io->out_stride;
  a.n_q = io->n_q, a.group = io->n_q / c.n_kv, a.mask_words = io->mask_words;
  a.window = io->window < kMaxSlots ? io->window : kMaxSlots;  // a longer one leaves nothing out, and differences stay in 32 bits
  a.layer = layer;
  a.scale_log2 = (float)((io->scale > 0 ? (double)io->scale : 1.0 / std::sqrt((double)c.head_dim)) * 1.4426950408889634);
  a.part_o = static_cast<float4*>(workspace);
  a.part_ml = reinterpret_cast<float2*>(a.part_o + (size_t)2 * grid * kRows * (c.head_dim / 4));
  a.borders = reinterpret_cast<Border*>(a.part_ml + (size_t)2 * grid * kRows);
  a.status = status;
  a.tm_k = kv->tm_k, a.tm_v = kv->tm_v;
  cudaStream_t st = static_cast<cudaStream_t>(stream);
  return c.head_dim == 128 ? launch_both<128>(a, grid, st) : launch_both<64>(a, grid, st);
}

}  // extern "C"
