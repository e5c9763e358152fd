// mk_beam.cu -- one step of beam search: the n_out best continuations of
// each request over beams x vocabulary.
//
// Two kernels.  The first reads the logits once: blocks (row, part) keep the
// running maximum and sum of exponentials of their part of a row beside its
// n_out largest logits (within a beam no score is above that of a larger logit,
// so nothing else of the part can be better).  The second, a block per request,
// joins the parts' sums in 64 bits, forms the scores of what is left and takes
// the best n_out.  Different logits can round to one score, where the lower
// index comes first: if that may concern the last place, the request's logits
// are gone through once more (lowest_ties).
//
// Measured on a GB300: 64 requests of 8 beams over 65536 tokens (134 MB), the
// best 16, 34 us: the first kernel 27 (4.9 TB/s) and the second 7 (latency:
// 64-bit logarithms and the ranks); 4 beams over 32768 tokens 12 us, 8 requests
// of 8 beams over 65536 25.  The first kernel issues in half of its cycles: of
// the 12 that a warp takes to an instruction it waits 3 for loads, 3 for earlier
// results and 2 at the barriers of the bounds, and with 512 blocks on 152 SMs
// (four on some, three on most) an SM is busy 77 % of the time.
#include <cmath>

#include "mk_ops_common.cuh"

namespace mk {
namespace ops {
namespace {

using dev::FULL;

constexpr int kThreads = 256, kWarps = kThreads / 32;
constexpr int kMaxOut = 128;
constexpr int kMaxParts = 16;
constexpr int kPer = 16;                 // logits of a tile per thread
constexpr int kTile = kThreads * kPer;
constexpr int kWarpTile = 32 * kPer;

// Candidates in one order: the larger value first, then the lower index.  Key
// 0 stands for "none".
__device__ __forceinline__ uint32_t ordered(float x) {
  const uint32_t u = __float_as_uint(x + 0.0f);  // -0 counts as 0
  return x != x ? 1u : (u & 0x80000000u) ? ~u : u | 0x80000000u;  // NaN below -inf
}
__device__ __forceinline__ float unordered(uint32_t o) {
  return o == 1u ? __uint_as_float(0x7fffffffu) : __uint_as_float((o & 0x80000000u) ? o & 0x7fffffffu : ~o);
}
// The next numbers below and above the one ordered as o (-0 has no code of its own).
__device__ __forceinline__ float just_below(uint32_t o) { return unordered(o - (o == 0x80000000u ? 2 : 1)); }
__device__ __forceinline__ float just_above(uint32_t o) { return unordered(o + 1); }
__device__ __forceinline__ uint64_t key_of(float x, uint32_t index) { return (uint64_t)ordered(x) << 32 | (uint32_t)~index; }

struct Key2 {  // a score in 64 bits and the candidate's index
  uint64_t score;
  uint32_t index;  // complement: larger is earlier
};
__device__ __forceinline__ bool above(const Key2& a, const Key2& b) {
  return a.score > b.score || (a.score == b.score && a.index > b.index);
}
__device__ __forceinline__ uint64_t ordered64(double x) {
  const uint64_t u = (uint64_t)__double_as_longlong(x + 0.0);
  return (u >> 63) ? ~u : u | 0x8000000000000000ull;
}
__device__ __forceinline__ double unordered64(uint64_t o) {
  return __longlong_as_double((long long)((o >> 63) ? o & 0x7fffffffffffffffull : ~o));
}

struct SelectArgs {
  const float* logits;
  int64_t stride;
  const float* scores;
  const uint8_t* finished;
  int32_t eos, beams, vocab, n_out, parts, part_len;
  float* out_scores;
  int32_t *out_parents, *out_tokens;
  uint64_t* keys;   // [rows][parts][n_out]
  double2* sums;    // [rows][parts]: maximum, sum of exp(x - maximum)
  bool vec;
};

// e^d for d <= 0: the error is |d| 2^-23 + 2^-22, least where the term counts most.
constexpr float kLog2e = 1.44269504089f;
__device__ __forceinline__ float e_to(float d) { return ex2(d * kLog2e); }

// A warp's candidates: at least the n best of its logits so far.  A tile's
// logits are compared with a bound as numbers; only lanes that beat it look
// further, so the stream costs the maximum and the exponentials.
template <int N>  // n_out is at most N
struct alignas(16) Best {
  static constexpr int kFull = 2 * N;   // kept before they are sorted out
  uint64_t buf[kFull + kWarpTile + 8];  // eight zeros behind the last
  uint64_t next[N];
  int count;
};
template <int N>
struct Parts {
  Best<N> best[kWarps];
  uint64_t list[kWarps * Best<N>::kFull + 8];
  float top[kThreads];  // the groups' maxima
  int count;
  uint32_t least[2];  // the n-th largest of them, ordered, by turns
  uint32_t bound;  // the best bound of any warp, ordered
};

// How many of keys[0 .. count) are above `mine`; eight zeros follow the last.
__device__ __forceinline__ int rank_in(const uint64_t* keys, int count, uint64_t mine) {
  int rank = 0;
  for (int j = 0; j < count; j += 8) {
#pragma unroll
    for (int x = 0; x < 8; ++x) rank += keys[j + x] > mine;
  }
  return rank;
}

// Leaves the n best of buf[0 .. count), count >= n, in no order, and returns
// the least of them: the largest K, found bit by bit, that n keys reach.
template <int N>
__device__ __forceinline__ uint64_t keep_best(Best<N>& k, int count, int n) {
  const int lane = threadIdx.x % 32;
  uint64_t least = 0;
  __syncwarp();
  for (int bit = 63; bit >= 0; --bit) {
    const uint64_t t = least | (uint64_t)1 << bit;
    int reach = 0;
    for (int i = lane; i < count; i += 32) reach += k.buf[i] >= t;
    reach = __reduce_add_sync(FULL, reach);
    if (reach >= n) least = t;
    if (reach == n) break;
  }
  int kept = 0;
  for (int i0 = 0; i0 < count; i0 += 32) {
    const uint64_t mine = i0 + lane < count ? k.buf[i0 + lane] : 0;
    const uint32_t in = __ballot_sync(FULL, mine >= least);
    if (mine >= least) k.next[kept + __popc(in & ((1u << lane) - 1))] = mine;
    kept += __popc(in);
  }
  __syncwarp();
  for (int i = lane; i < n; i += 32) k.buf[i] = k.next[i];
  if (lane == 0) k.count = n;
  __syncwarp();
  return least;
}

// The n-th largest of the maxima of the block's groups of threads, ordered: at
// least n of the logits seen so far reach it.  64 groups for n_out up to 32,
// 256 beyond: of 4096 random logits few more than n reach it (the n-th best of
// a warp's 512 would let eight times as many pass).  The calls take turns (0, 1,
// 0, ...): a warp may still read one call's result while another begins the next.
template <int N>
__device__ __forceinline__ uint32_t bound_of(Parts<N>& sh, float t, int n, int turn) {
  constexpr int kLanes = N == 32 ? 4 : 1, kGroups = kThreads / kLanes;
  const int tid = threadIdx.x;
#pragma unroll
  for (int o = 1; o < kLanes; o <<= 1) t = fmaxf(t, __shfl_xor_sync(FULL, t, o));
  if (tid % kLanes == 0) sh.top[tid / kLanes] = t;
  if (tid == 0) sh.least[turn] = 0xffffffffu;
  __syncthreads();
  if (tid < kGroups) {
    const float mine = sh.top[tid];
    int above = 0;
#pragma unroll 8
    for (int j = 0; j < kGroups / 4; ++j) {
      const float4 o = reinterpret_cast<const float4*>(sh.top)[j];
      above += (o.x > mine) + (o.y > mine) + (o.z > mine) + (o.w > mine);
    }
    const uint32_t least = __reduce_min_sync(FULL, above < n ? ordered(mine) : 0xffffffffu);
    if (tid % 32 == 0) atomicMin(&sh.least[turn], least);
  }
  __syncthreads();
  return sh.least[turn];
}

template <int N>
__global__ void __launch_bounds__(kThreads, N == 32 ? 4 : 3) select_parts(const __grid_constant__ SelectArgs a) {
  extern __shared__ uint4 raw[];
  Parts<N>& sh = *reinterpret_cast<Parts<N>*>(raw);
  __shared__ float wm[kWarps];
  __shared__ double ws[kWarps];
  wait_before();
  let_next_in();
  const int row = blockIdx.y, part = blockIdx.x, tid = threadIdx.x, lane = tid % 32, warp = tid / 32, n = a.n_out;
  const int lo = part * a.part_len, hi = min(a.vocab, lo + a.part_len);
  const float* x = a.logits + row * a.stride;
  // four runs of four per thread
  float next[kPer];
  auto load = [&](int base) {
    const bool whole = a.vec && base + kTile <= hi;
#pragma unroll
    for (int q = 0; q < kPer / 4; ++q) {
      const int at = base + (q * kThreads + tid) * 4;
      if (whole) {
        const float4 f = __ldcs(reinterpret_cast<const float4*>(x + at));
        next[4 * q] = f.x, next[4 * q + 1] = f.y, next[4 * q + 2] = f.z, next[4 * q + 3] = f.w;
      } else {
#pragma unroll
        for (int j = 0; j < 4; ++j) next[4 * q + j] = at + j < hi ? x[at + j] : -INFINITY;
      }
    }
  };
  if (a.finished && a.finished[row]) return;
  load(lo);
  Best<N>& k = sh.best[warp];
  if (lane == 0) k.count = 0;
  if (tid == 0) sh.bound = 0, sh.count = 0;
  __syncthreads();
  int count = 0;
  bool bounded = false;
  float tau = -INFINITY;  // at least n logits of this and earlier tiles reach it, once bounded
  float m = -INFINITY, s = 0.0f;
  for (int base = lo; base < hi; base += kTile) {
    float v[kPer];
#pragma unroll
    for (int i = 0; i < kPer; ++i) v[i] = next[i];
    if (base + kTile < hi) load(base + kTile);
    float t = v[0];
#pragma unroll
    for (int i = 1; i < kPer; ++i) t = fmaxf(t, v[i]);
    if (t > m) {
      s *= e_to(m - t);  // m = -inf: 0 * 0
      m = t;
    }
    const float z = m == -INFINITY ? 0.0f : m;
    const uint32_t zb = __float_as_uint(-z), eb = __float_as_uint(kLog2e);
    uint64_t sums = 0;
#pragma unroll
    for (int i = 0; i < kPer; i += 2) {
      float2 e = halves(mul2(add2(pair(__float_as_uint(v[i]), __float_as_uint(v[i + 1])), pair(zb, zb)), pair(eb, eb)));
      e.x = ex2(e.x), e.y = ex2(e.y);
      sums = add2(sums, pair(__float_as_uint(e.x), __float_as_uint(e.y)));
    }
    s += halves(sums).x + halves(sums).y;
    // A bound of the whole block after 1, 2, 4, 8 ... tiles (of the running
    // maxima), and each warp's own once its buffer was full.  Equal logits of
    // later tiles have higher indices: only a larger one passes a bound of
    // earlier tiles.  This tile's bound, or one of another warp that may be
    // further on, lets an equal one pass.
    float least = tau;
    const int tile = (base - lo) / kTile;
    bool all = false;
    if ((tile & (tile + 1)) == 0 && (tile == 0 || base + kTile < hi)) {
      const uint32_t o = bound_of(sh, m, n, __popc(tile) & 1);
      if (o > ordered(-INFINITY)) {
        if (tid == 0) atomicMax(&sh.bound, o);
        least = fmaxf(least, just_below(o));
        tau = fmaxf(tau, unordered(o));
        bounded = true;
      }
    }
    if (bounded) {
      const uint32_t shared = *reinterpret_cast<volatile uint32_t*>(&sh.bound);
      if (shared > ordered(-INFINITY)) least = fmaxf(least, just_below(shared));
      if (!__any_sync(FULL, t > least)) continue;
    }
    all = !bounded;  // too few numbers so far: every logit in the range
    if (all || t > least) {
#pragma unroll
      for (int i = 0; i < kPer; ++i) {
        const int at = base + (i / 4 * kThreads + tid) * 4 + i % 4;
        if (all ? at < hi : v[i] > least) k.buf[atomicAdd(&k.count, 1)] = key_of(v[i], at);
      }
    }
    __syncwarp();
    // one lane's reading for all: one that came late could see the next tile's candidates
    count = __shfl_sync(FULL, *reinterpret_cast<volatile int*>(&k.count), 0);
    if (count > Best<N>::kFull || (!bounded && count >= n)) {
      const uint32_t o = (uint32_t)(keep_best(k, count, n) >> 32);
      count = n;
      if (o >= ordered(-INFINITY)) {  // n numbers among them
        tau = fmaxf(tau, unordered(o));
        bounded = true;
        if (lane == 0) atomicMax(&sh.bound, o);
      }
    }
  }
  // the sums of the threads, joined in 64 bits
  float bm = m;
  for (int o = 16; o > 0; o >>= 1) bm = fmaxf(bm, __shfl_xor_sync(FULL, bm, o));
  if (lane == 0) wm[warp] = bm;
  __syncthreads();
  bm = wm[0];
  for (int w = 1; w < kWarps; ++w) bm = fmaxf(bm, wm[w]);
  // s times e^(m - bm): the factor's error, an fp32 exponential's, is that of the terms themselves
  double d = m == -INFINITY ? (double)s : (double)(s * e_to(m - bm));
  for (int o = 16; o > 0; o >>= 1) d += __shfl_xor_sync(FULL, d, o);
  if (lane == 0) ws[warp] = d;
  // the n best of the warps' candidates; none below the bound is among them
  for (int i = lane; i < count; i += 32) {
    const uint64_t mine = k.buf[i];
    if ((uint32_t)(mine >> 32) >= sh.bound) sh.list[atomicAdd(&sh.count, 1)] = mine;
  }
  __syncthreads();
  const int c = sh.count;
  if (tid < 8) sh.list[c + tid] = 0;
  __syncthreads();
  uint64_t* out = a.keys + ((int64_t)row * a.parts + part) * n;
  for (int i = tid; i < c; i += kThreads) {
    const uint64_t mine = sh.list[i];
    const int rank = rank_in(sh.list, c, mine);
    if (rank < n) out[rank] = mine;
  }
  for (int i = tid; i < n; i += kThreads)
    if (i >= c) out[i] = 0;
  if (tid == 0) {
    d = 0;
    for (int w = 0; w < kWarps; ++w) d += ws[w];
    a.sums[(int64_t)row * a.parts + part] = make_double2(bm, d);
  }
}

constexpr int kMaxBeams = 64;
constexpr int kDirect = 384;  // candidates that are ranked against each other at once

// The request's candidates, and its best so far; scores and indices apart, so
// that a comparison is two plain loads.
struct Joined {
  static constexpr int kRoom = kMaxOut * kPer + kMaxOut;
  uint64_t score[kRoom + 8];
  uint32_t index[kRoom + 8];
  Key2 next[kMaxOut];
  Key2 best[kThreads];
  Key2 tau, bound;
  int count;
};

// Leaves the n best of the candidates, best first, and sets tau.
__device__ __forceinline__ void sort_out(Joined& k, int n) {
  __syncthreads();
  const int c = k.count, tid = threadIdx.x;
  if (tid < 8) k.score[c + tid] = 0;
  __syncthreads();
  for (int i = tid; i < c; i += kThreads) {
    const Key2 mine = {k.score[i], k.index[i]};
    int rank = 0;
    for (int j = 0; j < c; j += 8) {
#pragma unroll
      for (int x = 0; x < 8; ++x) {
        const uint64_t s = k.score[j + x];
        rank += (s > mine.score) | ((s == mine.score) & (k.index[j + x] > mine.index));
      }
    }
    if (rank < n) k.next[rank] = mine;
  }
  __syncthreads();
  const int m = min(c, n);
  for (int i = tid; i < m; i += kThreads) k.score[i] = k.next[i].score, k.index[i] = k.next[i].index;
  if (tid == 0) {
    k.count = m;
    if (m == n) k.tau = k.next[n - 1];
  }
  __syncthreads();
}

// Gives the places of the last one's score to the lowest indices of all
// continuations that score the same (by the whole block; all that score higher
// are among the n, so the scores stay).  score(w, x): of logit x in beam w, top:
// the beams' largest logits.  Only for scores above -inf, so beams without a
// log-sum-exp have none.  The parts' keys tell first whether there is anything
// to do: of a part of more than n logits no other one scores above its last kept
// one, and one that scores the same is of no account unless that is the last
// place's score and either of them has another logit.  It takes logits that
// differ by less than the last bit of their score: not made fast.
template <typename F>
__device__ __noinline__ void settle_ties(const SelectArgs& a, Joined& k, const bool* done, const float* scores,
                                         const double* lse, const float* top, F score) {
  __shared__ int found[kWarps];
  const int tid = threadIdx.x, lane = tid % 32, warp = tid / 32, n = a.n_out;
  const uint64_t last = k.score[n - 1];
  bool other = false;
  for (int i = tid; i < a.beams * a.parts; i += kThreads) {
    const int w = i / a.parts;
    if (done[w] || lse[w] != lse[w]) continue;
    const uint32_t o = (uint32_t)(a.keys[((int64_t)blockIdx.x * a.beams * a.parts + i) * n + n - 1] >> 32);
    if (o > ordered(-INFINITY) && ordered64(score(w, unordered(o))) == last)
      other |= ordered64(score(w, just_below(o))) == last || ordered64(score(w, just_above(o))) == last;
  }
  if (!__syncthreads_or(other)) return;
  int at = 0;
  while (k.score[at] > last) ++at;
  for (int w = 0; w < a.beams && at < n; ++w) {
    if (done[w]) {
      if (ordered64(scores[w]) == last) {
        if (tid == 0) k.index[at] = ~(uint32_t)(w * a.vocab + a.eos);
        ++at;
      }
      continue;
    }
    if (lse[w] != lse[w] || ordered64(score(w, top[w])) < last) continue;
    const float* x = a.logits + ((int64_t)blockIdx.x * a.beams + w) * a.stride;
    for (int v0 = 0; v0 < a.vocab && at < n; v0 += kTile) {
      uint32_t hit = 0;
#pragma unroll
      for (int i = 0; i < kPer; ++i) {
        const int v = v0 + i * kThreads + tid;
        if (v < a.vocab && ordered64(score(w, x[v])) == last) hit |= 1u << i;
      }
      if (!__syncthreads_or(hit)) continue;
      for (int i = 0; i < kPer && at < n; ++i) {
        const uint32_t in = __ballot_sync(FULL, hit >> i & 1);
        if (lane == 0) found[warp] = __popc(in);
        __syncthreads();
        int mine = at + __popc(in & ((1u << lane) - 1));
        for (int x = 0; x < warp; ++x) mine += found[x];
        if ((hit >> i & 1) && mine < n) k.index[mine] = ~(uint32_t)(w * a.vocab + v0 + i * kThreads + tid);
        for (int x = 0; x < kWarps; ++x) at += found[x];
        __syncthreads();
      }
    }
  }
  __syncthreads();
}

__global__ void __launch_bounds__(kThreads) select_join(const __grid_constant__ SelectArgs a) {
  extern __shared__ uint4 raw[];
  Joined& k = *reinterpret_cast<Joined*>(raw);
  __shared__ double lse[kMaxBeams];  // NaN: every score of the beam is -inf
  __shared__ double share[kMaxBeams * kMaxParts];
  __shared__ float top[kMaxBeams], scores[kMaxBeams];
  __shared__ bool done[kMaxBeams];
  const int r = blockIdx.x, tid = threadIdx.x, W = a.beams, n = a.n_out, parts = a.parts;
  const int per_row = parts * n, N = W * per_row;
  if (tid == 0) {
    k.count = 0;
    k.tau = {0, 0};
  }
  wait_before();
  let_next_in();
  for (int w = tid; w < W; w += kThreads) {
    done[w] = a.finished && a.finished[r * W + w];
    scores[w] = a.scores[r * W + w];
  }
  // the first candidates on their way beside the parts' sums
  const uint64_t* keys = a.keys + (int64_t)r * N;
  const uint64_t early = tid < N ? keys[tid] : 0;
  // the parts' sums, joined in 64 bits: a thread per part, then per beam (the
  // logarithm's hundred or so 64-bit operations are most of this kernel's time)
  const double2* sums = a.sums + (int64_t)r * W * parts;
  for (int i0 = 0; i0 < W * parts; i0 += kThreads) {
    const int i = i0 + tid, w = i / parts;
    const bool in = i < W * parts;
    double2 p = make_double2(0, 0);
    if (in) p = sums[i];
    __syncthreads();  // done[] of this block, and top[] of the round before
    if (in && done[w]) p = make_double2(0, 0);
    if (in && i % parts == 0) {
      float t = (float)p.x;  // an fp32 number
      for (int x = 1; x < parts; ++x) t = fmaxf(t, done[w] ? 0.0f : (float)sums[i + x].x);
      top[w] = t;
    }
    __syncthreads();
    if (in) share[i] = (float)p.x == top[w] || p.y == 0.0 ? p.y : p.y * exp(p.x - (double)top[w]);
  }
  __syncthreads();
  for (int w = tid; w < W; w += kThreads) {
    if (done[w]) continue;
    double sum = 0;
    for (int i = 0; i < parts; ++i) sum += share[w * parts + i];
    const double l = (double)top[w] + log(sum);
    lse[w] = isfinite(l) && scores[w] > -INFINITY ? l : NAN;
  }
  __syncthreads();
  auto score_of = [&](int w, float x) {
    const double s = (double)scores[w] + ((double)x - lse[w]);
    return s != s ? -INFINITY : s;
  };
  for (int base = 0; base < N; base += kTile) {
    Key2 key[kPer], b = {0, 0};
#pragma unroll
    for (int i = 0; i < kPer; ++i) {
      const int c = base + i * kThreads + tid;
      key[i] = {0, 0};
      if (c >= N) continue;
      const int w = c / per_row, j = c % per_row;
      double score = -INFINITY;
      int token;
      if (done[w] && scores[w] > -INFINITY) {
        // its one continuation, then the rest of the vocabulary at -inf
        token = j == 0 ? a.eos : j - 1 + (j - 1 >= a.eos);
        if (j >= n || token >= a.vocab) continue;
        if (j == 0) score = scores[w];
      } else if (done[w] || lse[w] != lse[w]) {  // all at -inf
        token = j;
        if (j >= n || token >= a.vocab) continue;
      } else {
        const uint64_t q = base == 0 && i == 0 ? early : keys[c];
        if (q == 0) continue;
        token = (int)~(uint32_t)q;
        score = score_of(w, unordered((uint32_t)(q >> 32)));
      }
      key[i] = {ordered64(score), ~(uint32_t)(w * a.vocab + token)};
      if (above(key[i], b)) b = key[i];
    }
    // Many candidates: at least n of them reach the n-th best of the threads'
    // best ones, and only n threads hold such, so that n * kPer enter at most.
    Key2 bound = k.tau;
    if (N > kDirect) {
      k.best[tid] = b;
      if (tid == 0) k.bound = bound;
      __syncthreads();
      int rank = 0;
#pragma unroll 8
      for (int j = 0; j < kThreads; ++j) {
        const Key2 o = k.best[j];
        rank += (o.score > b.score) | ((o.score == b.score) & (o.index > b.index));
      }
      if (rank == n - 1 && b.score != 0 && above(b, bound)) k.bound = b;
      __syncthreads();
      bound = k.bound;
    }
    const bool raised = above(bound, k.tau);
#pragma unroll
    for (int i = 0; i < kPer; ++i)
      if (raised ? !above(bound, key[i]) : above(key[i], bound)) {
        const int at = atomicAdd(&k.count, 1);
        k.score[at] = key[i].score;
        k.index[at] = key[i].index;
      }
    sort_out(k, n);
  }
  // Two logits of one score differ by less than the roundings on its way: from
  // the last place's score back to a logit, whose neighbours are 2^-24 of its
  // power of two away, nearly always the exponents tell that there are none (24:
  // 2^-50 of the larger result for both roundings, a step of either exponent).
  const uint64_t last = k.count == n ? k.score[n - 1] : 0;
  bool near = false;
  if (tid < W && last > ordered64(-INFINITY) && !done[tid] && lse[tid] == lse[tid]) {
    const double t = unordered64(last), off = t - (double)scores[tid], x = off + lse[tid];
    const auto power = [](double y) { return __double2hiint(y) >> 20 & 0x7ff; };
    near = t == INFINITY || max(power(off), power(t)) - power(x) >= 24;
  }
  if (__syncthreads_or(near)) settle_ties(a, k, done, scores, lse, top, score_of);
  for (int i = tid; i < n; i += kThreads) {
    const bool there = i < k.count;  // it is, unless an input changed between the kernels
    const uint32_t c = there ? ~k.index[i] : 0;
    const int64_t o = (int64_t)r * n + i;
    a.out_scores[o] = there ? (float)unordered64(k.score[i]) : -INFINITY;
    a.out_parents[o] = (int32_t)(c / (uint32_t)a.vocab);
    a.out_tokens[o] = (int32_t)(c % (uint32_t)a.vocab);
  }
}

// Parts of a row, whole tiles each: as many blocks as the GPU holds at once (four
// per SM; three where n_out is above 32, so that some come second there).  A
// longer part is cheaper per logit, its bound being nearer: 512 rows of 65536 logits took 38 us whole and 48, 63 and 56 us
// in 2, 3 and 4 parts; 4 rows of 32768 fill 32 SMs in 8 parts.
int parts_of(int64_t rows, int vocab) {
  const int64_t tiles = (vocab + kTile - 1) / kTile;
  int64_t want = rows > 0 ? 152 * 4 / rows : 1;
  if (want < 1) want = 1;
  if (want > kMaxParts) want = kMaxParts;
  if (want > tiles) want = tiles;
  const int64_t per = (tiles + want - 1) / want;
  return (int)((tiles + per - 1) / per);
}

// The kernels count a row's logits in 32 bits, up to two tiles behind its end;
// the rows are a grid's second dimension.
bool shape_ok(int32_t requests, int32_t beams, int32_t vocab, int32_t n_out) {
  return requests >= 0 && beams >= 1 && beams <= kMaxBeams && vocab >= 1 && n_out >= 1 && n_out <= kMaxOut &&
         n_out <= (int64_t)beams * vocab && (int64_t)beams * vocab <= 1 << 30 && (int64_t)requests * beams <= 65535;
}

size_t sums_bytes(int64_t rows, int parts) { return (size_t)rows * parts * sizeof(double2); }

}  // namespace
}  // namespace ops
}  // namespace mk

using mk::fail;
using namespace mk::ops;

extern "C" {

size_t mk_beam_select_workspace_bytes(int32_t requests, int32_t beams, int32_t vocab, int32_t n_out) {
  if (!shape_ok(requests, beams, vocab, n_out)) return 0;
  const int64_t rows = (int64_t)requests * beams;
  const int parts = parts_of(rows, vocab);
  return 16 + sums_bytes(rows, parts) + (size_t)rows * parts * n_out * sizeof(uint64_t);
}

int mk_beam_select(const float* logits, int64_t logits_stride, const float* scores, const uint8_t* finished,
                   int32_t eos, int32_t requests, int32_t beams, int32_t vocab, int32_t n_out, float* out_scores,
                   int32_t* out_parents, int32_t* out_tokens, void* workspace, size_t workspace_bytes, void* stream) {
  if (!shape_ok(requests, beams, vocab, n_out))
    return fail(MK_ERR_ARG, "beams 1 to 64, n_out 1 to 128 and at most beams * vocab (up to 2^30), requests * beams up to 65535");
  if (requests == 0) return MK_OK;
  if (!logits || !scores || !out_scores || !out_parents || !out_tokens) return fail(MK_ERR_ARG, "null argument");
  if (misplaced(logits, scores, finished, out_scores, out_parents, out_tokens)) return fail(MK_ERR_ARG, "misaligned argument");
  if (logits_stride < vocab || endless((int64_t)requests * beams, logits_stride, 4))
    return fail(MK_ERR_ARG, "logits_stride below vocab, or rows beyond 2^48 bytes");
  if (finished && (eos < 0 || eos >= vocab)) return fail(MK_ERR_ARG, "eos outside the vocabulary");
  if (misaligned(workspace) || !workspace ||
      workspace_bytes < mk_beam_select_workspace_bytes(requests, beams, vocab, n_out))
    return fail(MK_ERR_ARG, "workspace null, misaligned or too small");
  const int64_t rows = (int64_t)requests * beams;
  const size_t in = span(rows, logits_stride, vocab, 4), out = (size_t)requests * n_out * 4, row_bytes = (size_t)rows * 4;
  void* const outs[] = {out_scores, out_parents, out_tokens};
  for (int i = 0; i < 3; ++i)
    if (overlap(outs[i], out, logits, in) || overlap(outs[i], out, scores, row_bytes) ||
        overlap(outs[i], out, finished, (size_t)rows) || overlap(outs[i], out, outs[(i + 1) % 3], out) ||
        overlap(outs[i], out, workspace, workspace_bytes))
      return fail(MK_ERR_ARG, "an output overlaps another argument");
  if (overlap(workspace, workspace_bytes, logits, in) || overlap(workspace, workspace_bytes, scores, row_bytes) ||
      overlap(workspace, workspace_bytes, finished, (size_t)rows))
    return fail(MK_ERR_ARG, "the workspace overlaps an input");
  SelectArgs a;
  a.logits = logits, a.stride = logits_stride, a.scores = scores, a.finished = finished, a.eos = eos;
  a.beams = beams, a.vocab = vocab, a.n_out = n_out;
  a.parts = parts_of(rows, vocab);
  const int tiles = (vocab + kTile - 1) / kTile;
  a.part_len = (tiles + a.parts - 1) / a.parts * kTile;
  a.out_scores = out_scores, a.out_parents = out_parents, a.out_tokens = out_tokens;
  a.sums = static_cast<double2*>(workspace);
  a.keys = reinterpret_cast<uint64_t*>(static_cast<uint8_t*>(workspace) + sums_bytes(rows, a.parts));
  a.vec = !misaligned(logits) && logits_stride % 4 == 0;
  cudaStream_t st = static_cast<cudaStream_t>(stream);
  constexpr int smem = (int)sizeof(Joined);
  static std::atomic<uint64_t> join_ready{0}, wide_ready{0};
  int rc = allow_smem(join_ready, reinterpret_cast<const void*>(&select_join), smem, "select");
  if (rc != MK_OK) return rc;
  const dim3 grid((unsigned)a.parts, (unsigned)rows);
  if (n_out <= 32) {
    rc = launch("select", select_parts<32>, grid, kThreads, sizeof(Parts<32>), st, a);
  } else {
    constexpr int wide = (int)sizeof(Parts<kMaxOut>);
    rc = allow_smem(wide_ready, reinterpret_cast<const void*>(&select_parts<kMaxOut>), wide, "select");
    if (rc == MK_OK) rc = launch("select", select_parts<kMaxOut>, grid, kThreads, wide, st, a);
  }
  if (rc != MK_OK) return rc;
  return launch("select", select_join, dim3((unsigned)requests), kThreads, smem, st, a);
}

}  // extern "C"
