// mk_beam.cu -- one step of beam search: the n_out best continuations of
// each request over beams x vocabulary.
//
// Two kernels.  The first reads the logits once: blocks (row, part) keep the
// running maximum and sum of exponentials of their part of a row beside its
// n_out largest logits (within a beam the order of the scores is that of the
// logits, so nothing else of the part can be chosen).  The second, a block per
// request, joins the parts' sums in 64 bits, forms the scores of what is left
// and takes the best n_out.
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

__device__ __forceinline__ float ex2(float x) {
  float r;
  asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(r) : "f"(x));
  return r;
}
// e^d for d <= 0: the error is |d| 2^-23 + 2^-22, least where the term counts most.
__device__ __forceinline__ float e_to(float d) { return ex2(d * 1.44269504089f); }

// A warp's best candidates so far.  A tile's logits are compared with the n-th
// best as numbers; only a tile that beats it looks further, so the stream
// costs the maximum and the exponentials.
template <int N>  // n_out is at most N
struct Best {
  static constexpr int kGroups = N / 32;               // of a lane's logits in a tile
  static constexpr int kFull = 2 * N;                  // kept before they are sorted out
  uint64_t buf[kFull + kWarpTile];
  uint64_t next[N];
};

// The n best of buf[0 .. count), best first; returns how many there are.
template <int N>
__device__ __forceinline__ int sort_out(Best<N>& k, int count, int n) {
  const int lane = threadIdx.x % 32;
  __syncwarp();
  for (int i = lane; i < count; i += 32) {
    const uint64_t mine = k.buf[i];
    int rank = 0;
    for (int j = 0; j < count; ++j) rank += k.buf[j] > mine;
    if (rank < n) k.next[rank] = mine;
  }
  __syncwarp();
  const int m = min(count, n);
  for (int i = lane; i < m; i += 32) k.buf[i] = k.next[i];
  __syncwarp();
  return m;
}

// The n-th best of the maxima of the tile's 32 kGroups groups, 0 if fewer hold
// a logit: at least n of the tile's keys reach it.
template <int N>
__device__ __forceinline__ uint64_t bound_of(Best<N>& k, const uint64_t (&key)[kPer], int n) {
  constexpr int G = Best<N>::kGroups;
  const int lane = threadIdx.x % 32;
  uint64_t top[G], found = 0;
  int rank[G];
  __syncwarp();
#pragma unroll
  for (int g = 0; g < G; ++g) {
    top[g] = 0;
#pragma unroll
    for (int i = 0; i < kPer / G; ++i) top[g] = max(top[g], key[g * (kPer / G) + i]);
    k.next[g * 32 + lane] = top[g];
  }
  __syncwarp();
#pragma unroll
  for (int g = 0; g < G; ++g) rank[g] = 0;
#pragma unroll 4
  for (int j = 0; j < 32 * G; ++j) {
    const uint64_t other = k.next[j];
#pragma unroll
    for (int g = 0; g < G; ++g) rank[g] += other > top[g];
  }
#pragma unroll
  for (int g = 0; g < G; ++g)
    if (rank[g] == n - 1) found = top[g];
  const uint32_t who = __ballot_sync(FULL, found != 0);
  return who ? __shfl_sync(FULL, found, __ffs(who) - 1) : 0;
}

template <int N>
__global__ void __launch_bounds__(kThreads, 4) select_parts(const __grid_constant__ SelectArgs a) {
  extern __shared__ uint4 raw[];
  Best<N>* best = reinterpret_cast<Best<N>*>(raw);
  __shared__ int counts[kWarps];
  __shared__ float wm[kWarps];
  __shared__ double ws[kWarps];
  asm volatile("griddepcontrol.launch_dependents;" ::: "memory");
  const int row = blockIdx.y, part = blockIdx.x, tid = threadIdx.x, lane = tid % 32, warp = tid / 32, n = a.n_out;
  if (a.finished && a.finished[row]) return;
  const int lo = part * a.part_len, hi = min(a.vocab, lo + a.part_len);
  const float* x = a.logits + row * a.stride;
  Best<N>& k = best[warp];
  int count = 0;
  uint64_t tau = 0;  // the n-th best key, 0 until there are n
  float tau_f = 0.0f;
  float m = -INFINITY, s = 0.0f;
  for (int base = lo; base < hi; base += kTile) {
    // four runs of four per thread
    float v[kPer];
    const bool whole = a.vec && base + kTile <= hi;
#pragma unroll
    for (int q = 0; q < kPer / 4; ++q) {
      const int at = base + (q * kThreads + tid) * 4;
      if (whole) {
        const float4 f = __ldcs(reinterpret_cast<const float4*>(x + at));
        v[4 * q] = f.x, v[4 * q + 1] = f.y, v[4 * q + 2] = f.z, v[4 * q + 3] = f.w;
      } else {
#pragma unroll
        for (int j = 0; j < 4; ++j) v[4 * q + j] = at + j < hi ? x[at + j] : -INFINITY;
      }
    }
    float t = v[0];
#pragma unroll
    for (int i = 1; i < kPer; ++i) t = fmaxf(t, v[i]);
    if (t > m) {
      s *= e_to(m - t);  // m = -inf: 0 * 0
      m = t;
    }
    const float z = m == -INFINITY ? 0.0f : m;
    float s0 = 0.0f, s1 = 0.0f;
#pragma unroll
    for (int i = 0; i < kPer; i += 2) s0 += e_to(v[i] - z), s1 += e_to(v[i + 1] - z);
    s += s0 + s1;
    // Equal logits of later tiles have higher indices: only a larger one passes.
    if (!__any_sync(FULL, tau == 0 || t > tau_f)) continue;
    uint64_t key[kPer];
    int pass = 0;
#pragma unroll
    for (int i = 0; i < kPer; ++i) {
      const int at = base + (i / 4 * kThreads + tid) * 4 + i % 4;
      key[i] = at < hi ? key_of(v[i], at) : 0;
      pass += key[i] > tau;
    }
    uint64_t above = tau;
    if (__reduce_add_sync(FULL, pass) > N) {  // many: the tile's own n-th best may be nearer
      const uint64_t bound = bound_of(k, key, n);
      if (bound > above) above = bound - 1;
    }
#pragma unroll
    for (int i = 0; i < kPer; ++i) {
      const uint32_t in = __ballot_sync(FULL, key[i] > above);
      if (key[i] > above) k.buf[count + __popc(in & ((1u << lane) - 1))] = key[i];
      count += __popc(in);
    }
    if (count > Best<N>::kFull || (tau == 0 && count >= n)) {
      count = sort_out(k, count, n);
      if (count == n) {
        tau = k.buf[n - 1];
        tau_f = unordered((uint32_t)(tau >> 32));
      }
    }
  }
  count = sort_out(k, count, n);
  // the sums of the threads, joined in 64 bits
  float bm = m;
  for (int o = 16; o > 0; o >>= 1) bm = fmaxf(bm, __shfl_xor_sync(FULL, bm, o));
  if (lane == 0) wm[warp] = bm, counts[warp] = count;
  __syncthreads();
  bm = wm[0];
  for (int w = 1; w < kWarps; ++w) bm = fmaxf(bm, wm[w]);
  // s times e^(m - bm): the factor's error, an fp32 exponential's, is that of the terms themselves
  double d = m == -INFINITY ? (double)s : (double)s * (double)e_to(m - bm);
  for (int o = 16; o > 0; o >>= 1) d += __shfl_xor_sync(FULL, d, o);
  if (lane == 0) ws[warp] = d;
  // the n best of the warps' candidates
  uint64_t* out = a.keys + ((int64_t)row * a.parts + part) * n;
  int all = 0;
  for (int w = 0; w < kWarps; ++w) all += counts[w];
  for (int i = lane; i < count; i += 32) {
    const uint64_t mine = k.buf[i];
    int rank = 0;
    for (int w = 0; w < kWarps; ++w)
      for (int j = 0; j < counts[w]; ++j) rank += best[w].buf[j] > mine;
    if (rank < n) out[rank] = mine;
  }
  for (int i = tid; i < n; i += kThreads)
    if (i >= all) out[i] = 0;
  __syncthreads();
  if (tid == 0) {
    d = 0;
    for (int w = 0; w < kWarps; ++w) d += ws[w];
    a.sums[(int64_t)row * a.parts + part] = make_double2(bm, d);
  }
}

constexpr int kMaxBeams = 64;
constexpr int kDirect = 384;  // candidates that are ranked against each other at once

// The request's candidates, and its best so far.
struct Joined {
  Key2 buf[kMaxOut * kPer + kMaxOut];
  Key2 next[kMaxOut];
  Key2 best[kThreads];
  Key2 tau, bound;
  int count;
};

// Leaves the n best of buf[0 .. count), best first, in buf and sets tau.
__device__ __forceinline__ void sort_out(Joined& k, int n) {
  __syncthreads();
  const int c = k.count;
  for (int i = threadIdx.x; i < c; i += kThreads) {
    const Key2 mine = k.buf[i];
    int rank = 0;
    for (int j = 0; j < c; ++j) rank += above(k.buf[j], mine);
    if (rank < n) k.next[rank] = mine;
  }
  __syncthreads();
  const int m = min(c, n);
  for (int i = threadIdx.x; i < m; i += kThreads) k.buf[i] = k.next[i];
  if (threadIdx.x == 0) {
    k.count = m;
    if (m == n) k.tau = k.next[n - 1];
  }
  __syncthreads();
}

__global__ void __launch_bounds__(kThreads) select_join(const __grid_constant__ SelectArgs a) {
  extern __shared__ uint4 raw[];
  Joined& k = *reinterpret_cast<Joined*>(raw);
  __shared__ double top[kMaxBeams];
  __shared__ double lse[kMaxBeams];  // NaN: every score of the beam is -inf
  __shared__ double share[kMaxBeams * kMaxParts];
  __shared__ bool done[kMaxBeams];
  const int r = blockIdx.x, tid = threadIdx.x, W = a.beams, n = a.n_out;
  if (tid == 0) {
    k.count = 0;
    k.tau = {0, 0};
  }
  asm volatile("griddepcontrol.wait;" ::: "memory");
  // the parts' sums, joined in 64 bits: a thread per part, then per beam
  const double2* sums = a.sums + (int64_t)r * W * a.parts;
  for (int w = tid; w < W; w += kThreads) {
    done[w] = a.finished && a.finished[r * W + w];
    top[w] = -INFINITY;
    if (!done[w])
      for (int i = 0; i < a.parts; ++i) top[w] = fmax(top[w], sums[w * a.parts + i].x);
  }
  __syncthreads();
  for (int i = tid; i < W * a.parts; i += kThreads) {
    const int w = i / a.parts;
    if (done[w]) continue;
    const double2 p = sums[i];
    share[i] = p.x == top[w] || p.y == 0.0 ? p.y : p.y * exp(p.x - top[w]);
  }
  __syncthreads();
  for (int w = tid; w < W; w += kThreads) {
    if (done[w]) continue;
    double sum = 0;
    for (int i = 0; i < a.parts; ++i) sum += share[w * a.parts + i];
    const double l = top[w] + log(sum);
    lse[w] = isfinite(l) && a.scores[r * W + w] > -INFINITY ? l : NAN;
  }
  __syncthreads();
  const int per_row = a.parts * n, N = W * per_row;
  for (int base = 0; base < N; base += kTile) {
    Key2 key[kPer], b = {0, 0};
#pragma unroll
    for (int i = 0; i < kPer; ++i) {
      const int c = base + i * kThreads + tid;
      key[i] = {0, 0};
      if (c >= N) continue;
      const int w = c / per_row, j = c % per_row, row = r * W + w;
      const double cum = a.scores[row];
      double score = -INFINITY;
      int token;
      if (done[w]) {
        // its one continuation, then the rest of the vocabulary at -inf
        token = j == 0 ? a.eos : j - 1 + (j - 1 >= a.eos);
        if (j >= n || token >= a.vocab) continue;
        if (j == 0) score = cum;
      } else if (lse[w] != lse[w]) {
        token = j;
        if (j >= n || token >= a.vocab) continue;
      } else {
        const uint64_t q = a.keys[(int64_t)row * per_row + j];
        if (q == 0) continue;
        token = (int)~(uint32_t)q;
        score = cum + ((double)unordered((uint32_t)(q >> 32)) - lse[w]);
      }
      if (score != score) score = -INFINITY;
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
      for (int j = 0; j < kThreads; ++j) rank += above(k.best[j], b);
      if (rank == n - 1 && b.score != 0 && above(b, bound)) k.bound = b;
      __syncthreads();
      bound = k.bound;
    }
    const bool raised = above(bound, k.tau);
#pragma unroll
    for (int i = 0; i < kPer; ++i)
      if (raised ? !above(bound, key[i]) : above(key[i], bound)) k.buf[atomicAdd(&k.count, 1)] = key[i];
    sort_out(k, n);
  }
  for (int i = tid; i < n; i += kThreads) {
    const uint32_t c = ~k.buf[i].index;
    const int64_t o = (int64_t)r * n + i;
    a.out_scores[o] = (float)unordered64(k.buf[i].score);
    a.out_parents[o] = (int32_t)(c / (uint32_t)a.vocab);
    a.out_tokens[o] = (int32_t)(c % (uint32_t)a.vocab);
  }
}

// Parts of a row: enough blocks to fill the GPU, whole tiles each.
int parts_of(int64_t rows, int vocab) {
  const int64_t tiles = (vocab + kTile - 1) / kTile;
  int64_t want = rows > 0 ? (152 * 4 + rows - 1) / rows : 1;
  if (want > kMaxParts) want = kMaxParts;
  if (want > tiles) want = tiles;
  const int64_t per = (tiles + want - 1) / want;
  return (int)((tiles + per - 1) / per);
}

bool shape_ok(int32_t requests, int32_t beams, int32_t vocab, int32_t n_out) {
  return requests >= 0 && beams >= 1 && beams <= kMaxBeams && vocab >= 1 && n_out >= 1 && n_out <= kMaxOut &&
         n_out <= (int64_t)beams * vocab && (int64_t)beams * vocab <= INT32_MAX && requests <= 1 << 20;
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
    return fail(MK_ERR_ARG, "beams 1 to 64, n_out 1 to 128 and at most beams * vocab (below 2^31)");
  if (requests == 0) return MK_OK;
  if (!logits || !scores || !out_scores || !out_parents || !out_tokens) return fail(MK_ERR_ARG, "null argument");
  if (logits_stride < vocab) return fail(MK_ERR_ARG, "logits_stride below vocab");
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
  if (rows > 65535) return fail(MK_ERR_ARG, "more than 65535 rows of logits");
  constexpr int smem = (int)sizeof(Joined);
  static std::atomic<uint64_t> join_ready{0}, wide_ready{0};
  int rc = allow_smem(join_ready, reinterpret_cast<const void*>(&select_join), smem, "select");
  if (rc != MK_OK) return rc;
  const dim3 grid((unsigned)a.parts, (unsigned)rows);
  if (n_out <= 32) {
    select_parts<32><<<grid, kThreads, kWarps * sizeof(Best<32>), st>>>(a);
  } else {
    constexpr int wide = (int)(kWarps * sizeof(Best<kMaxOut>));
    rc = allow_smem(wide_ready, reinterpret_cast<const void*>(&select_parts<kMaxOut>), wide, "select");
    if (rc != MK_OK) return rc;
    select_parts<kMaxOut><<<grid, kThreads, wide, st>>>(a);
  }
  rc = launched("select");
  if (rc != MK_OK) return rc;
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3((unsigned)requests);
  cfg.blockDim = dim3(kThreads);
  cfg.dynamicSmemBytes = smem;
  cfg.stream = st;
  cudaLaunchAttribute early;  // resident (waiting) before the last part is written
  early.id = cudaLaunchAttributeProgrammaticStreamSerialization;
  early.val.programmaticStreamSerializationAllowed = 1;
  cfg.attrs = &early;
  cfg.numAttrs = 1;
  cudaLaunchKernelEx(&cfg, select_join, a);
  return launched("select");
}

}  // extern "C"
