// mk_attn_mass.cu -- how much attention each cached slot receives: the
// probabilities of mk_tree_attn, summed over the new tokens and the query heads
// of a K/V head, on the tcgen05 tensor cores.
//
//   mass[b][h][s] = decay * mass[b][h][s] + sum_{t, g} exp(scale q_tg . K_s - lse_tg)
//
// The product is formed as S^T = K Q^T: a tile of 128 slots is the MMA's M, so a
// slot is a lane of tensor memory and its sum stays in one thread's register;
// the query rows are the MMA's N, in blocks of up to 128 rows (whole tokens of
// the K/V head's query heads).  A tile belongs to one SM, which adds its
// blocks in order: no atomics, the same call gives the same bits.
//
// The tiles of all (sequence, K/V head) are dealt to the SMs in runs of equal
// cost.  Up to kQ blocks of Q stay in shared memory while the run's tiles of K
// stream past them; more rows are taken in passes over the run.
//
// One CTA per SM, 12 warps:
//   warp 0     Q blocks and K tiles by TMA (one box per page and 64 dims)
//   warps 1, 2 issue the MMAs of the even and of the odd tiles, block by block
//   warp 3     plans the runs
//   warps 4-11 two groups of 128 threads, one for the even tiles and one for the
//              odd, a thread per slot: S from tensor memory (two buffers of 128
//              columns a group), the exponentials, the sums
//
// Measured on a GB300 (heads of 128, 8 query heads to a K/V head): one token of
// each of 32 sequences over 512 to 32K slots 96 us, 0.6 GB of K at 6.2 TB/s (a copy:
// 6.7), bound by memory; the last 42 to 64 tokens of four prompts of 18K to 32K
// slots 53 us, of which 8 before the first sum: a block of 128 x 128 takes an SM
// 950 cycles, its MMAs 512, its exponentials as much of the special-function
// units and its K, at the memory's rate, 480; without the exponentials a call
// took 9 us less, without the MMAs or the loads 2; one token over 8K slots 6.9
// us, latency.  Steps on the way for the four prompts: 125 us with
// visibility asked column by column, 76 with it in closed form and S read ahead, 72
// with a warp of MMAs for each group, 58 with whole blocks summed without votes, 53
// with one warp planning and openings counted; 16 summing warps with half a block
// each took 8 more, S of the next block asked for before the last columns 5, a
// rolled loop over columns 8.
#include <cuda.h>

#include <cmath>

#include "mk_ops_mma.cuh"
#include "mk_ops_tmem.cuh"

namespace mk {
namespace ops {
namespace {

struct MassArgs {
  Pools pools;
  Batch b;
  const float* lse;
  float* mass;
  const uint64_t* mask;
  int64_t mass_stride;
  int32_t n_q, group, mask_words, window, layer;
  int32_t heads, tokens, head_blocks;  // query heads and tokens of a block, blocks that share a token
  float scale_log2, decay;             // scale * log2(e)
  uint32_t* status;
  CUtensorMap tm_k, tm_q;
};

constexpr int kTile = 128;               // slots of a tile, rows of a block at most
constexpr int kThreads = 384;
constexpr int kOpening = 15;             // units of a tile's cost
constexpr int kItems = 4;                // runs planned ahead
constexpr int64_t kWaitNs = 2000000000;  // a wait that takes longer is given up
// The planning warp's, which lasts as long as a run does (a prompt of 2^19 tokens
// over 2^20 slots takes seconds); where a role is stuck its own wait, of a tile or
// a block, ends all of them.
constexpr int64_t kPlanNs = 60 * kWaitNs;

template <int D, int kQ>
struct Geo {
  static constexpr int kHalves = D / 64;          // 128-byte columns of a row
  static constexpr int kHalfBytes = kTile * 128;  // a tile's 64 dims
  static constexpr int kTileBytes = kHalves * kHalfBytes;
  static constexpr int kSlots = D == 128 ? 7 : 13;  // tiles that fit
  static constexpr int kStages = kSlots - kQ < 8 ? kSlots - kQ : 8;
  static constexpr int kRing = kQ * kTileBytes, kLse = kRing + kStages * kTileBytes, kCtl = kLse + kQ * kTile * 4;
};

// ------------------------------------------------------------- the plan

// A run of tiles [lo, hi) of K/V head h of sequence b.
struct Item {
  int b, h, t0, n, ctx, lo, hi;
};

struct Ctl {
  alignas(16) uint32_t live[16];  // the rows of each block of the pass that count, a bit each
  int rows[4];                    // and how many it has
  uint64_t full[8], empty[8], q_full, q_empty, s_full[2][2], s_empty[2][2], meet, drain;
  uint64_t planned[kItems], taken[kItems];
  uint32_t tmem, abort;
  Item items[kItems];
};

__device__ __forceinline__ Seq mass_seq(const MassArgs& a, int b) {
  Seq s = seq_of(a.b, b, a.pools.page_shift, a.status, OP_MASS);
  if (s.n > 0 && a.mask && s.n > 64 * (int64_t)a.mask_words) {
    record(a.status, ERR_RANGE, OP_MASS, b, 2, s.n, 64 * a.mask_words);
    s.n = 0;
  }
  if (s.n > 0 && (int64_t)s.ctx + s.n > a.mass_stride) {
    record(a.status, ERR_RANGE, OP_MASS, b, 4, s.ctx + s.n, (uint32_t)a.mass_stride);
    s.n = 0;
  }
  return s;
}

__device__ __forceinline__ int blocks_of(const MassArgs& a, int n) { return (n + a.tokens - 1) / a.tokens * a.head_blocks; }
// What a tile costs, in quarters of a load of K: the load, or the steps of its
// blocks (blocks that do not stay together load the tile again, which hides
// behind their steps, but where there are few of them).
__device__ __forceinline__ int64_t cost_of_tile(int blocks) { return blocks <= 2 ? 5 : 2 * (int64_t)blocks + 1; }
// What a run costs before its first tile (Q, the start of its sums), where loads do not hide it.
// (0, 12 and 18 units took 55.6, 53.1 and 52.9 us for four prompts.)
__device__ __forceinline__ int opening(int blocks) { return blocks <= 2 ? 0 : kOpening; }
// The first tile that a token of the sequence may see.
__device__ __forceinline__ int first_tile(const MassArgs& a, int ctx) {
  const int first = a.window ? ctx - a.window + 1 : 0;
  return first > 0 ? first / kTile : 0;
}

// Calls f(item) for the runs of this CTA, in order, while it returns true.  By
// a whole warp: a lane holds one sequence of a round of 32.
template <typename F>
__device__ __forceinline__ bool each_item(const MassArgs& a, F f) {
  const int lane = threadIdx.x % 32;
  auto load = [&](int b) {
    Seq s = {0, 0, 0};
    if (b < a.b.batch) s = mass_seq(a, b);
    return s;
  };
  auto cost_of = [&](const Seq& s, int& tiles, int& lo, int64_t& each, int& open) {
    const int blocks = blocks_of(a, s.n);
    lo = first_tile(a, s.ctx);
    tiles = s.n > 0 ? (s.ctx + s.n + kTile - 1) / kTile - lo : 0;
    each = cost_of_tile(blocks);
    open = s.n > 0 ? opening(blocks) : 0;
    return (tiles * each + open) * a.pools.n_kv;
  };
  const Seq first = load(lane);
  int tiles, lo, open;
  int64_t each, total = cost_of(first, tiles, lo, each, open);
  for (int b0 = 32; b0 < a.b.batch; b0 += 32) total += cost_of(load(b0 + lane), tiles, lo, each, open);
  for (int o = 16; o > 0; o >>= 1) total += __shfl_xor_sync(FULL, total, o);
  const int64_t grid = gridDim.x, q = divide(total, grid), rest = total - q * grid;
  const int64_t u = q * blockIdx.x + ((int)blockIdx.x < rest ? (int)blockIdx.x : rest);
  const int64_t end = u + q + ((int)blockIdx.x < rest ? 1 : 0);
  int64_t base = 0;
  for (int b0 = 0; b0 < a.b.batch && base < end; b0 += 32) {
    const Seq s = b0 == 0 ? first : load(b0 + lane);
    const int64_t mine = cost_of(s, tiles, lo, each, open), incl = warp_scan(mine);
    uint32_t hit = __ballot_sync(FULL, mine > 0 && base + incl > u && base + incl - mine < end);
    while (hit) {
      const int src = __ffs(hit) - 1;
      hit &= hit - 1;
      Item it;
      it.b = b0 + src;
      it.t0 = __shfl_sync(FULL, s.t0, src), it.n = __shfl_sync(FULL, s.n, src), it.ctx = __shfl_sync(FULL, s.ctx, src);
      const int n = __shfl_sync(FULL, tiles, src), from = __shfl_sync(FULL, lo, src), before = __shfl_sync(FULL, open, src);
      const int64_t cost = __shfl_sync(FULL, each, src), head = n * cost + before;
      int64_t at = base + __shfl_sync(FULL, incl - mine, src);
      int h = u > at ? (int)divide(u - at, head) : 0;
      for (at += h * head; h < a.pools.n_kv && at < end; ++h, at += head) {
        // the tiles that begin in [u, end)
        const int64_t t0 = at + before;
        const int64_t k0 = u > t0 ? divide(u - t0 + cost - 1, cost) : 0, k1 = end > t0 ? divide(end - t0 + cost - 1, cost) : 0;
        it.h = h;
        it.lo = from + (int)(k0 < n ? k0 : n), it.hi = from + (int)(k1 < n ? k1 : n);
        if (it.lo < it.hi && !f(it)) return false;
      }
    }
    base += __shfl_sync(FULL, incl, 31);
  }
  return true;
}

// A pass over a run: the blocks [q0, q0 + nq) of its rows against the tiles [lo, hi).
struct Pass {
  int q0, nq, lo, hi;
};
// Pass p; the first one takes all tiles of the run, later ones those that their tokens may see.
template <int kQ>
__device__ __forceinline__ Pass pass_of(const MassArgs& a, const Item& it, int p) {
  const int all = blocks_of(a, it.n);
  Pass x = {p * kQ, all - p * kQ < kQ ? all - p * kQ : kQ, it.lo, it.hi};
  if (p > 0) {
    const int i0 = x.q0 / a.head_blocks * a.tokens, i1 = ((x.q0 + x.nq - 1) / a.head_blocks + 1) * a.tokens;
    if (!a.mask && !(a.window && a.b.positions)) {
      const int end = (it.ctx + (i1 < it.n ? i1 : it.n) + kTile - 1) / kTile;
      if (end < x.hi) x.hi = end;
      if (a.window) {
        const int first = it.ctx + i0 - a.window + 1;
        if (first > 0 && first / kTile > x.lo) x.lo = first / kTile;
      }
    }
  }
  return x;
}
// The rows of block q of a sequence: its first token, tokens, rows, first head.
struct Rows {
  int i0, tokens, rows, g0;
};
__device__ __forceinline__ Rows rows_of(const MassArgs& a, const Item& it, int q) {
  Rows r;
  const int i = a.head_blocks == 1 ? q : q / a.head_blocks;
  r.i0 = i * a.tokens;
  r.g0 = (q - i * a.head_blocks) * a.heads;
  r.tokens = it.n - r.i0 < a.tokens ? it.n - r.i0 : a.tokens;
  r.rows = (r.tokens - 1) * a.heads + (a.group - r.g0 < a.heads ? a.group - r.g0 : a.heads);
  return r;
}

// ------------------------------------------------------------- waits

// Waits for a phase; false when this wait, or another one of the CTA, has
// taken too long.
__device__ __forceinline__ bool wait_slow(Ctl& c, uint64_t* bar, uint32_t parity, uint32_t* status, int64_t limit) {
  const int64_t until = gtimer() + limit;
  for (;;) {
    if (mbar_try_wait(bar, parity)) return true;
    if (ld_volatile(&c.abort)) return false;
    if (gtimer() > until) {
      *reinterpret_cast<volatile uint32_t*>(&c.abort) = 1;
      record(status, ERR_TIMEOUT, OP_MASS, blockIdx.x, threadIdx.x, 0, 0);
      return false;
    }
  }
}
// By a whole warp, whose lanes leave every wait together.
__device__ __forceinline__ bool wait(Ctl& c, uint64_t* bar, uint32_t parity, uint32_t* status, int64_t limit = kWaitNs) {
  return __all_sync(FULL, mbar_try_wait(bar, parity) || wait_slow(c, bar, parity, status, limit)) != 0;
}

// The plan is made by one warp and handed to the others through shared memory,
// kItems runs ahead.  Made by every warp for itself it was three copies of code
// that comes from memory once, and its state cost the roles registers: one
// token over 8K slots took 8.5 us, not 7.6, four prompts' last tokens 55.5, not
// 53.  A run of no tokens is the end.
__device__ __forceinline__ bool plan(const MassArgs& a, Ctl& c) {
  uint32_t n = 0;
  auto give = [&](const Item& it) {
    const int s = n % kItems;
    if (n >= kItems && !wait(c, &c.taken[s], (n / kItems - 1) & 1, a.status, kPlanNs)) return false;
    if (threadIdx.x % 32 == 0) {
      c.items[s] = it;
      mbar_arrive(&c.planned[s]);
    }
    __syncwarp();
    ++n;
    return true;
  };
  return each_item(a, give) && give(Item{});
}
constexpr int kTakers = 11;  // warps
template <typename F>
__device__ __forceinline__ bool each_planned(const MassArgs& a, Ctl& c, F f) {
  for (uint32_t n = 0;; ++n) {
    const int s = n % kItems;
    if (!wait(c, &c.planned[s], n / kItems & 1, a.status)) return false;
    const Item it = c.items[s];
    __syncwarp();
    if (threadIdx.x % 32 == 0) mbar_arrive(&c.taken[s]);
    if (it.n == 0) return true;
    if (!f(it)) return false;
  }
}

// ------------------------------------------------------------- visibility

// Position of new token j (a position out of range is moved into it).
__device__ __forceinline__ int position_of(const MassArgs& a, const Item& it, int j) {
  if (!a.b.positions) return it.ctx + j;
  const int p = a.b.positions[it.t0 + j];
  if (p < it.ctx || p >= it.ctx + it.n) {
    record(a.status, ERR_RANGE, OP_MASS, it.b, 3, p, it.ctx + it.n);
    return p < it.ctx ? it.ctx : it.ctx + it.n - 1;
  }
  return p;
}
// Whether new token i sees a slot.
__device__ __forceinline__ bool sees(const MassArgs& a, const Item& it, int i, int slot) {
  const int j = slot - it.ctx;
  if (j >= it.n) return false;
  if (j >= 0) {
    if (a.mask ? !(a.mask[(int64_t)(it.t0 + i) * a.mask_words + (j >> 6)] >> (j & 63) & 1) : j > i) return false;
  }
  if (a.window && position_of(a, it, i) - (j >= 0 ? position_of(a, it, j) : slot) >= a.window) return false;
  return true;
}
// Which of the block's rows x0 .. x0 + 31 are of tokens that see a slot.
__device__ __forceinline__ uint32_t seen(const MassArgs& a, const Item& it, const Rows& r, int slot, int x0) {
  if (slot >= it.ctx + it.n) return 0;
  if (!a.mask && !a.window) {  // the rows from the slot's own token on
    const int first = slot - it.ctx - r.i0;
    const int64_t x = first > 0 ? (int64_t)first * a.heads - x0 : 0;
    return x <= 0 ? FULL : x >= 32 ? 0 : FULL << x;
  }
  uint32_t v = 0;
  for (int i = x0 / a.heads; i < r.tokens && i * a.heads < x0 + 32; ++i) {
    const int from = i * a.heads - x0, to = from + a.heads;  // the token's rows
    if (sees(a, it, r.i0 + i, slot)) v |= (from <= 0 ? FULL : FULL << from) & (to >= 32 ? FULL : (1u << to) - 1);
  }
  return v;
}
// Whether a token of the block may not see a slot of tile j.
__device__ __forceinline__ bool in_part(const MassArgs& a, const Item& it, const Rows& r, int j) {
  const bool apart = a.window && a.b.positions && it.n > a.window;  // new tokens a window apart
  if ((j + 1) * kTile > it.ctx + (a.mask || apart ? 0 : r.i0 + 1)) return true;
  return a.window && j * kTile < it.ctx + (a.b.positions ? it.n : r.i0 + r.tokens) - a.window;
}

// ------------------------------------------------------------- roles

struct Filled {
  Ring k;
  uint32_t tiles = 0, passes = 0;
};

template <int D, int kQ>
__device__ __forceinline__ bool produce(const MassArgs& a, uint8_t* smem, Ctl& c, Filled& f) {
  using G = Geo<D, kQ>;
  const int lane = threadIdx.x % 32;
  const int P = 1 << a.pools.page_shift, box = P < kTile ? P : kTile;  // slots of a box
  const int slice = lane / G::kHalves, half = lane % G::kHalves;       // this lane's box of a tile
  asm volatile("fence.proxy.async.global;" ::: "memory");
  return each_planned(a, c, [&](const Item& it) {
    const int len = it.ctx + it.n;
    const int32_t* table = a.b.tables + (int64_t)it.b * a.b.max_pages;
    auto page_at = [&](int j) {  // the page of this lane's box in tile j, -1: no slot of it is in use
      const int s = j * kTile + slice * box;
      if (slice * box >= kTile || s >= len) return -1;
      int page = table[s >> a.pools.page_shift];
      if (page < 0 || page >= a.pools.num_pages) {
        record(a.status, ERR_PAGE, OP_MASS, it.b, s, page, (uint32_t)a.pools.num_pages);
        page = 0;
      }
      return page;
    };
    const int passes = (blocks_of(a, it.n) + kQ - 1) / kQ;
    for (int p = 0; p < passes; ++p) {
      const Pass x = pass_of<kQ>(a, it, p);
      if (x.lo >= x.hi) continue;
      int page = page_at(x.lo);
      if (f.passes > 0 && !wait(c, &c.q_empty, (f.passes - 1) & 1, a.status)) return false;
      if (lane == 0) mbar_expect_tx(&c.q_full, x.nq * G::kHalves * a.heads * a.tokens * 128);
      __syncwarp();
      if (slice < x.nq) {
        const Rows r = rows_of(a, it, x.q0 + slice);
        asm volatile(
            "cp.async.bulk.tensor.3d.shared::cluster.global.tile.mbarrier::complete_tx::bytes"
            " [%0], [%1, {%2, %3, %4}], [%5];" ::"r"(smem_u32(smem + slice * G::kTileBytes + half * G::kHalfBytes)),
            "l"(reinterpret_cast<uint64_t>(&a.tm_q)), "r"(half * 64), "r"(it.h * a.group + r.g0), "r"(it.t0 + r.i0),
            "r"(smem_u32(&c.q_full))
            : "memory");
      }
      ++f.passes;
      for (int j = x.lo; j < x.hi; ++j) {
        const int next = j + 1 < x.hi ? page_at(j + 1) : -1;
        const uint32_t bytes = __popc(__ballot_sync(FULL, page >= 0)) * box * 128;
        const int y = ((page * a.pools.n_kv + it.h) << a.pools.page_shift) + ((j * kTile + slice * box) & (P - 1));
        if (f.tiles >= (uint32_t)G::kStages && !wait(c, &c.empty[f.k.stage], f.k.phase ^ 1, a.status)) return false;
        if (lane == 0) mbar_expect_tx(&c.full[f.k.stage], bytes);
        __syncwarp();
        if (page >= 0)
          asm volatile(
              "cp.async.bulk.tensor.3d.shared::cluster.global.tile.mbarrier::complete_tx::bytes"
              " [%0], [%1, {%2, %3, %4}], [%5];" ::"r"(
                  smem_u32(smem + G::kRing + f.k.stage * G::kTileBytes + half * G::kHalfBytes + slice * box * 128)),
              "l"(reinterpret_cast<uint64_t>(&a.tm_k)), "r"(half * 64), "r"(y), "r"(a.layer), "r"(smem_u32(&c.full[f.k.stage]))
              : "memory");
        ++f.tiles;
        f.k.template advance<G::kStages>();
        page = next;
      }
    }
    return true;
  });
}

// TMEM columns of a group's buffer.
__device__ __forceinline__ uint32_t s_cols(int w, int buf) { return (w * 2 + buf) * kTile; }

// The MMAs of group w's tiles (those of its parity), block by block, its buffers
// in turn.  By a warp for each group: the waits and the issue of a step take
// about as long as its MMAs, one warp for both left the tensor cores idle half
// of the time.  The lanes leave every wait together, and every tile of the ring
// is waited for in order, the other group's too, and handed back by both warps:
// one that skipped phases of a barrier, or that a refilled stage overtook, could
// wait for its parity for good.
template <int D, int kQ>
__device__ __forceinline__ bool issue_mmas(const MassArgs& a, uint8_t* smem, Ctl& c, const int w) {
  using G = Geo<D, kQ>;
  const uint32_t base = smem_u32(smem) >> 4, klo = 1u << 16, ts = uniform(c.tmem) + s_cols(w, 0);
  const uint32_t empty = smem_u32(c.empty), s_full = smem_u32(c.s_full[w]), q_empty = smem_u32(&c.q_empty);
  const uint32_t lead = elected();
  Ring k;
  uint32_t passes_done = 0, step = 0;
  return each_planned(a, c, [&](const Item& it) {
    const int passes = (blocks_of(a, it.n) + kQ - 1) / kQ;
    for (int p = 0; p < passes; ++p) {
      const Pass x = pass_of<kQ>(a, it, p);
      const int lo = uniform(x.lo), hi = uniform(x.hi), nq = uniform(x.nq);
      if (lo >= hi) continue;
      // full blocks but for the last token's: columns of the last block, the others have a.heads * a.tokens rows
      const int most = a.heads * a.tokens, last = uniform(rows_of(a, it, x.q0 + nq - 1).rows);
      const bool even = a.head_blocks == 1;  // else blocks of one token differ
      const uint32_t idesc_all = tc_idesc_bf16(kTile, (even ? most + 15 : kTile) & ~15);
      const uint32_t idesc_last = tc_idesc_bf16(kTile, (even ? last + 15 : kTile) & ~15);
      if (!wait(c, &c.q_full, passes_done & 1, a.status)) return false;
      ++passes_done;
      for (int j = lo; j < hi; ++j) {
        if (!wait(c, &c.full[k.stage], k.phase, a.status)) return false;
        if ((j & 1) == w) {
          const uint32_t kd = (base + (G::kRing + k.stage * G::kTileBytes) / 16) | klo;
#pragma unroll
          for (int q = 0; q < kQ; ++q) {
            if (q >= nq) break;
            const uint32_t buf = step & 1;
            if (step >= 2 && !wait(c, &c.s_empty[w][buf], ((step >> 1) - 1) & 1, a.status)) return false;
            tc_fence_after();
            const uint32_t idesc = q == nq - 1 ? idesc_last : idesc_all, qd = (base + q * (G::kTileBytes / 16)) | klo;
#pragma unroll
            for (int i = 0; i < D / 16; ++i) {
              const uint32_t off = (i / 4 * G::kHalfBytes + i % 4 * 32) / 16;
              mma_ss_if(lead, ts + buf * kTile, desc(kd + off), desc(qd + off), idesc, i > 0);
            }
            commit_if(lead, s_full + buf * 8);
            ++step;
          }
          commit_if(lead, empty + k.stage * 8);
        } else {
          arrive_if(lead, empty + k.stage * 8);
        }
        k.advance<G::kStages>();
      }
      commit_if(lead, q_empty);
    }
    return true;
  });
}

template <int D, int kQ>
__device__ __forceinline__ bool sum_slots(const MassArgs& a, uint8_t* smem, Ctl& c) {
  using G = Geo<D, kQ>;
  const int tid = threadIdx.x - 128, w = tid / 128, row = tid % 128, lane = tid % 32;  // row: this thread's slot of a tile
  const uint32_t lanes = c.tmem + ((uint32_t)(row & ~31) << 16);
  float* lse = reinterpret_cast<float*>(smem + G::kLse);  // -lse * log2(e) of the pass's rows
  uint32_t step = 0, met = 0;
  auto meet = [&]() {
    mbar_arrive(&c.meet);
    return wait(c, &c.meet, met++ & 1, a.status);
  };
  auto release = [&](int w, int buf) {  // the buffer has been read
    tc_fence_before();
    __syncwarp();
    if (lane == 0) mbar_arrive(&c.s_empty[w][buf]);
  };
  // Slots that no token's window reaches only fade.  (In front of the sums, row
  // by row, each row's from the first CTA on: 32 sequences of one token over 512
  // to 32K slots with a window of 4096 take 87 us with a decay of 0.5, 28 with 1.)
  if (a.window && a.decay != 1.0f)
    for (int b = 0; b < a.b.batch; ++b) {
      const Seq s = mass_seq(a, b);
      const int n = s.n > 0 ? first_tile(a, s.ctx) * kTile : 0;
      for (int h = 0; h < a.pools.n_kv; ++h) {
        float* m = a.mass + ((int64_t)b * a.pools.n_kv + h) * a.mass_stride;
        for (int i = blockIdx.x * 256 + tid; i < n; i += gridDim.x * 256) m[i] = a.decay == 0.0f ? 0.0f : m[i] * a.decay;
      }
    }
  const uint32_t sb = __float_as_uint(a.scale_log2);
  const uint64_t scale2 = pair(sb, sb);
  return each_planned(a, c, [&](const Item& it) {
    float* mass = a.mass + ((int64_t)it.b * a.pools.n_kv + it.h) * a.mass_stride;
    const int passes = (blocks_of(a, it.n) + kQ - 1) / kQ;
    for (int p = 0; p < passes; ++p) {
      const Pass x = pass_of<kQ>(a, it, p);
      if (x.lo >= x.hi) continue;
      float mine[(kQ * kTile + 255) / 256];
      uint32_t live[(kQ * kTile + 255) / 256];
      int rows[(kQ * kTile + 255) / 256] = {};
#pragma unroll
      for (int e = 0; e < (kQ * kTile + 255) / 256; ++e) {
        const int at = e * 256 + tid, q = at / kTile, f = at % kTile;
        bool counts = false;
        mine[e] = -INFINITY;
        if (q < x.nq) {
          const Rows r = rows_of(a, it, x.q0 + q);
          if (f < r.rows) {
            const float v = a.lse[(int64_t)(it.t0 + r.i0 + f / a.heads) * a.n_q + it.h * a.group + r.g0 + f % a.heads];
            counts = v != -INFINITY;  // a row that saw nothing gives nothing, whatever its scores
            mine[e] = v * -1.44269504088896341f;
          }
          rows[e] = r.rows;
        }
        live[e] = __ballot_sync(FULL, counts);
      }
      if (!meet()) return false;  // the pass before has been summed
#pragma unroll
      for (int e = 0; e < (kQ * kTile + 255) / 256; ++e)
        if (e * 256 + tid < kQ * kTile) {
          lse[e * 256 + tid] = mine[e];
          if (lane == 0) c.live[(e * 256 + tid) / 32] = live[e];
          if (row == 0) c.rows[(e * 256 + tid) / kTile] = rows[e];
        }
      if (!meet()) return false;
      uint32_t full = 0;  // blocks all of whose rows count, a bit each
#pragma unroll
      for (int q = 0; q < kQ; ++q) {
        const uint4 v = lds128(smem_u32(c.live + q * 4));
        full |= (uint32_t)(__popc(v.x) + __popc(v.y) + __popc(v.z) + __popc(v.w) == c.rows[q]) << q;
      }
      for (int j = x.lo + ((x.lo ^ w) & 1); j < x.hi; j += 2) {
        const int slot = j * kTile + row;
        const bool inside = slot < it.ctx + it.n;
        float old = 0.0f;
        if (inside && (p > 0 || (slot < it.ctx && a.decay != 0.0f))) old = mass[slot];
        uint64_t s0 = 0, s1 = 0;
        // of them those for which the tile lies in front of the new tokens and inside every window
        const bool clear = (j + 1) * kTile <= it.ctx && !(a.window && j * kTile < it.ctx + it.n - a.window);
        const uint32_t whole = clear ? full : 0;
        for (int q = 0; q < x.nq; ++q) {
          const uint32_t buf = step & 1, from = lanes + s_cols(w, buf);
          const float* neg = lse + q * kTile;
          auto add = [&](const uint32_t (&s)[32], int x0) {
#pragma unroll
            for (int e = 0; e < 32; e += 4) {
              const uint4 n = lds128(smem_u32(neg + x0 + e));
              float2 u = halves(fma2(pair(s[e], s[e + 1]), scale2, pair(n.x, n.y)));
              float2 v = halves(fma2(pair(s[e + 2], s[e + 3]), scale2, pair(n.z, n.w)));
              u.x = ex2(u.x), u.y = ex2(u.y), v.x = ex2(v.x), v.y = ex2(v.y);
              s0 = add2(s0, pair(__float_as_uint(u.x), __float_as_uint(u.y)));
              s1 = add2(s1, pair(__float_as_uint(v.x), __float_as_uint(v.y)));
            }
          };
          const int rows = c.rows[q];
          bool part = false;
          if (!(whole >> q & 1)) part = in_part(a, it, rows_of(a, it, x.q0 + q), j);
          const bool clean = (full >> q & 1) && !part;
          if (!wait(c, &c.s_full[w][buf], step >> 1 & 1, a.status)) return false;
          ++step;
          tc_fence_after();
          if (clean && rows == kTile) {
            // a whole block: the next 32 columns are on their way while these are summed
            uint32_t even[32], odd[32];
            tmem_load_begin(from, even);
            tmem_load_end(even);
            tmem_load_begin(from + 32, odd);
            add(even, 0);
            tmem_load_end(odd);
            tmem_load_begin(from + 64, even);
            add(odd, 32);
            tmem_load_end(even);
            tmem_load_begin(from + 96, odd);
            add(even, 64);
            tmem_load_end(odd);
            release(w, buf);
            add(odd, 96);
            continue;
          }
#pragma unroll 1
          for (int x0 = 0; x0 < rows; x0 += 32) {
            uint32_t s[32];
            tmem_load(from + x0, s);
            if (x0 + 32 >= rows) release(w, buf);
            uint32_t on = c.live[q * 4 + x0 / 32];
            if (part) on &= seen(a, it, rows_of(a, it, x.q0 + q), slot, x0);
#pragma unroll
            for (int z = 0; z < 32; z += 16) {
              if (!__any_sync(FULL, (on >> z & 0xffff) != 0)) continue;
              // masked scores, and columns behind the rows, whatever they hold
#pragma unroll
              for (int e = z; e < z + 16; e += 4) {
                const uint4 n = lds128(smem_u32(neg + x0 + e));
                float2 u = halves(fma2(pair(s[e], s[e + 1]), scale2, pair(n.x, n.y)));
                float2 v = halves(fma2(pair(s[e + 2], s[e + 3]), scale2, pair(n.z, n.w)));
                u.x = ex2(on >> e & 1 ? u.x : -INFINITY), u.y = ex2(on >> (e + 1) & 1 ? u.y : -INFINITY);
                v.x = ex2(on >> (e + 2) & 1 ? v.x : -INFINITY), v.y = ex2(on >> (e + 3) & 1 ? v.y : -INFINITY);
                s0 = add2(s0, pair(__float_as_uint(u.x), __float_as_uint(u.y)));
                s1 = add2(s1, pair(__float_as_uint(v.x), __float_as_uint(v.y)));
              }
            }
          }
        }
        const float2 sum = halves(add2(s0, s1));
        if (inside) mass[slot] = p > 0 ? old + (sum.x + sum.y) : fmaf(old, a.decay, sum.x + sum.y);
      }
    }
    return true;
  });
}

template <int D, int kQ>
__global__ void __launch_bounds__(kThreads, 1) mass_kernel(const __grid_constant__ MassArgs a) {
  using G = Geo<D, kQ>;
  extern __shared__ __align__(1024) uint8_t smem[];
  Ctl& c = *reinterpret_cast<Ctl*>(smem + G::kCtl);
  const int tid = threadIdx.x, warp = uniform(tid / 32);
  if (warp == 3) {  // it goes on to the plan at once
    if (tid == 96) {
      c.abort = 0;
      for (int i = 0; i < G::kStages; ++i) {
        mbar_init(&c.full[i], 1);
        mbar_init(&c.empty[i], 2);
      }
      for (int i = 0; i < 4; ++i) {
        mbar_init(&c.s_full[i / 2][i % 2], 1);
        mbar_init(&c.s_empty[i / 2][i % 2], 4);
      }
      for (int i = 0; i < kItems; ++i) {
        mbar_init(&c.planned[i], 1);
        mbar_init(&c.taken[i], kTakers);
      }
      mbar_init(&c.q_full, 1);
      mbar_init(&c.q_empty, 2);
      mbar_init(&c.meet, 256);
      mbar_init(&c.drain, 2);
      asm volatile("fence.mbarrier_init.release.cluster;" ::: "memory");
    }
    __syncwarp();
    asm volatile("bar.arrive 1, 384;" ::: "memory");
  } else {
    if (warp == 1) tmem_alloc(&c.tmem, 512);
    asm volatile("bar.sync 1, 384;" ::: "memory");
    tc_fence_after();
  }
  wait_before();
  let_next_in();
  const bool placed = (smem_u32(smem) & 1023) == 0;  // the MMAs' layouts count on it
  if (!placed && tid == 0) record(a.status, ERR_SMEM_ALIGN, OP_MASS, 0, 0, smem_u32(smem), 1024);
  // The summing warps keep two buffers of S in registers: the other warps hand
  // them theirs (128 x 104 + 256 x 200 of the launch's 384 x 168).
  bool ok = true;
  Filled f;
  if (!placed) {
  } else if (warp < 4) {
    asm volatile("setmaxnreg.dec.sync.aligned.u32 104;");
    if (warp == 0) {
      ok = produce<D, kQ>(a, smem, c, f);
    } else if (warp == 3) {
      ok = plan(a, c);
    } else {
      ok = issue_mmas<D, kQ>(a, smem, c, warp - 1);
      // every MMA, and every arrival that one of them owes, before the block ends
      commit_if(elected(), smem_u32(&c.drain));
      for (const int64_t until = gtimer() + kWaitNs; !mbar_try_wait(&c.drain, 0) && gtimer() < until;) {
      }
      __syncwarp();
    }
  } else {
    asm volatile("setmaxnreg.inc.sync.aligned.u32 200;");
    ok = sum_slots<D, kQ>(a, smem, c);
  }
  tc_fence_before();
  if (__syncthreads_or(!ok) && tid == 0) {  // a wait was given up: the copies in flight (bounded)
    const int64_t until = gtimer() + kWaitNs;
    Ring r = f.k;
    for (uint32_t i = 0; i < (uint32_t)G::kStages && i < f.tiles; ++i) {  // the last fill of every stage
      r.stage = r.stage == 0 ? G::kStages - 1 : r.stage - 1;
      if (r.stage == G::kStages - 1) r.phase ^= 1;
      while (!mbar_try_wait(&c.full[r.stage], r.phase) && gtimer() < until) {
      }
    }
    while (f.passes > 0 && !mbar_try_wait(&c.q_full, (f.passes - 1) & 1) && gtimer() < until) {
    }
  }
  __syncthreads();
  if (warp == 1) tmem_dealloc(c.tmem, 512);
}

template <int D, int kQ>
int launch_mass(const MassArgs& a, int grid, cudaStream_t st) {
  constexpr int smem = Geo<D, kQ>::kCtl + (int)sizeof(Ctl);
  static_assert(smem <= 232448, "shared memory of a block");
  static std::atomic<uint64_t> ready{0};
  const int rc = allow_smem(ready, reinterpret_cast<const void*>(&mass_kernel<D, kQ>), smem, "attn_mass");
  if (rc != MK_OK) return rc;
  return launch("attn_mass", mass_kernel<D, kQ>, dim3(grid), kThreads, smem, st, a);
}

// Q [n_tokens][n_q][head_dim] in boxes of a block's heads and tokens.
int encode_q(const mk_kv_config& c, const mk_mass_io* io, int n_tokens, MassArgs& a) {
  const EncodeTiledFn f = encode_tiled();
  if (!f) return fail(MK_ERR_CUDA, "cuTensorMapEncodeTiled is not available");
  const cuuint64_t dims[3] = {(cuuint64_t)c.head_dim, (cuuint64_t)io->n_q, (cuuint64_t)n_tokens};
  const int64_t row = (int64_t)io->n_q * c.head_dim;
  const cuuint64_t strides[2] = {(cuuint64_t)c.head_dim * 2, (cuuint64_t)(n_tokens > 1 ? io->q_stride : row) * 2};
  const cuuint32_t box[3] = {64, (cuuint32_t)a.heads, (cuuint32_t)a.tokens}, step[3] = {1, 1, 1};
  const CUresult r = f(&a.tm_q, CU_TENSOR_MAP_DATA_TYPE_BFLOAT16, 3, const_cast<void*>(io->q), dims, strides, box, step,
                       CU_TENSOR_MAP_INTERLEAVE_NONE, CU_TENSOR_MAP_SWIZZLE_128B, CU_TENSOR_MAP_L2_PROMOTION_L2_256B,
                       CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE);
  if (r != CUDA_SUCCESS) return fail(MK_ERR_CUDA, "cuTensorMapEncodeTiled failed (" + std::to_string((int)r) + ")");
  return MK_OK;
}

}  // namespace
}  // namespace ops
}  // namespace mk

using mk::fail;
using namespace mk::ops;

extern "C" int mk_attn_mass(mk_kv* kv, int32_t layer, const mk_tokens* tok, const mk_mass_io* io, uint32_t* status,
                            void* stream) {
  int rc = check_tokens(kv, layer, tok);
  if (rc != MK_OK) return rc;
  const mk_kv_config& c = kv->cfg;
  if (!io) return fail(MK_ERR_ARG, "null argument");
  if (tok->batch == 0 || tok->n_tokens == 0) return MK_OK;
  if (!io->q || !io->lse || !io->mass) return fail(MK_ERR_ARG, "null q, lse or mass");
  if (io->n_q < c.n_kv || io->n_q % c.n_kv != 0 || io->n_q > (1 << 16)) return fail(MK_ERR_ARG, "n_q must be a multiple of n_kv");
  if ((int64_t)tok->n_tokens * (io->n_q / c.n_kv) > INT32_MAX) return fail(MK_ERR_ARG, "more than 2^31 - 1 query rows per K/V head");
  const int64_t row = (int64_t)io->n_q * c.head_dim;
  if (misaligned(io->q) || io->q_stride < row || io->q_stride % 8 ||
      (tok->n_tokens > 1 && io->q_stride >= (int64_t)1 << 39) || endless(tok->n_tokens, io->q_stride, 2))
    return fail(MK_ERR_ARG, "misaligned q, or a stride that is too small, too large or no multiple of 16 bytes");
  if (misplaced(io->tree_mask, status) || misplaced(io->lse, io->mass)) return fail(MK_ERR_ARG, "misaligned tree_mask, lse, mass or status");
  if (io->tree_mask ? io->mask_words < 1 : io->mask_words != 0)
    return fail(MK_ERR_ARG, "mask_words must be positive with a tree_mask and 0 without");
  if (io->window < 0) return fail(MK_ERR_ARG, "negative window");
  if (!(io->scale >= 0) || !std::isfinite(io->scale * 1.5f)) return fail(MK_ERR_ARG, "scale must be positive (0: 1 / sqrt(head_dim))");
  if (!(io->decay >= 0 && io->decay <= 1)) return fail(MK_ERR_ARG, "decay must be from 0 to 1");
  const int64_t rows = (int64_t)tok->batch * c.n_kv;
  if (io->mass_stride < 1 || endless(rows, io->mass_stride, 4)) return fail(MK_ERR_ARG, "mass_stride too small or too large");
  const size_t mass = span(rows, io->mass_stride, io->mass_stride, 4);
  if (overlap(io->mass, mass, io->q, span(tok->n_tokens, io->q_stride, row, 2)) ||
      overlap(io->mass, mass, io->lse, (size_t)tok->n_tokens * io->n_q * 4) ||
      overlap(io->mass, mass, io->tree_mask, (size_t)tok->n_tokens * io->mask_words * 8) || over_batch(tok, io->mass, mass) ||
      over_pools(kv, status, io->mass, mass))
    return fail(MK_ERR_ARG, "mass overlaps another argument or the pools");
  const int grid = mk::query_num_sms();
  if (grid < 1) return fail(MK_ERR_CUDA, "no device");
  rc = encode_pools(kv);
  if (rc != MK_OK) return rc;
  MassArgs a;
  a.pools = pools_of(kv, layer);
  a.b = batch_of(tok);
  a.lse = io->lse, a.mass = io->mass, a.mask = io->tree_mask;
  a.mass_stride = io->mass_stride;
  a.n_q = io->n_q, a.group = io->n_q / c.n_kv, a.mask_words = io->mask_words;
  a.window = io->window < kMaxSlots ? io->window : kMaxSlots;  // a longer one leaves nothing out, and differences stay in 32 bits
  a.layer = layer;
  a.heads = a.group < kTile ? a.group : kTile;
  a.tokens = kTile / a.heads;
  a.head_blocks = (a.group + a.heads - 1) / a.heads;
  a.scale_log2 = (float)((io->scale > 0 ? (double)io->scale : 1.0 / std::sqrt((double)c.head_dim)) * 1.4426950408889634);
  a.decay = io->decay;
  a.status = status;
  a.tm_k = kv->tm_k;
  rc = encode_q(c, io, tok->n_tokens, a);
  if (rc != MK_OK) return rc;
  cudaStream_t st = static_cast<cudaStream_t>(stream);
  // Blocks of Q that stay: as many as an average sequence has, up to 4.  Fewer
  // leave more of the ring to K, more save passes over it: with 1, 2 and 4 one
  // token of each of 32 sequences over 512 to 32K slots takes 94.8, 94.4 and 96.9
  // us (heads of 64 with 1 and 4 32.7 and 32.9), the last 17 tokens of four
  // prompts of up to 32K 29, 24 and 24, 2048 tokens over 8K slots 354, 281 and 254.
  // The mean does not tell sequences of unlike lengths: 64 tokens of one among 31
  // single ones, over up to 8K slots, take 56 us with the 1 that it gives, 43 with
  // 4; 512 tokens among them 119 with its 2, 110 with 4.
  const int64_t each = ((int64_t)tok->n_tokens + tok->batch - 1) / tok->batch;
  const int64_t blocks = (each + a.tokens - 1) / a.tokens * a.head_blocks;
  if (c.head_dim == 128)
    return blocks <= 1 ? launch_mass<128, 1>(a, grid, st) : blocks == 2 ? launch_mass<128, 2>(a, grid, st) : launch_mass<128, 4>(a, grid, st);
  return blocks <= 1 ? launch_mass<64, 1>(a, grid, st) : launch_mass<64, 4>(a, grid, st);
}
