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

constexpr int kThreads = 256;
constexpr int kMaxOut = 128;
constexpr int kMaxParts = 16;
constexpr int kPer = 16;                 // logits of a tile per thread
constexpr int kTile = kThreads * kPer;
constexpr int kBuf = kMaxOut * kPer + kMaxOut;  // what one tile can add to the kept candidates, and those

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
__device__ __forceinline__ bool above(uint64_t a, uint64_t b) { return a > b; }
__device__ __forceinline__ uint64_t ordered64(double x) {
  const uint64_t u = (uint64_t)__double_as_longlong(x + 0.0);
  return (u >> 63) ? ~u : u | 0x8000000000000000ull;
}
__device__ __forceinline__ double unordered64(uint64_t o) {
  return __longlong_as_double((long long)((o >> 63) ? o & 0x7fffffffffffffffull : ~o));
}

// The best n of the block's candidates so far, in no order, and what a new
// one has to beat once n are kept.
template <typename Key>
struct Kept {
  Key buf[kBuf];
  Key next[kMaxOut];
  Key best[kThreads];
  Key tau;
  int count;
};

// Leaves the n best of buf[0 .. count), best first, in buf and sets tau.
template <typename Key>
__device__ void prune(Kept<Key>& k, int n) {
  __syncthreads();
  const int c = k.count;
  for (int i = threadIdx.x; i < c; i += kThreads) {
    const Key mine = k.buf[i];
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

// A tile that would overflow the buffer, or the first: at least n of its keys
// lie at or above the n-th best of the threads' best keys, and only n
// threads hold such keys, so at most n * kPer enter.
template <typename Key>
__device__ void raise_tau(Kept<Key>& k, const Key (&mine)[kPer], const Key& none, int n) {
  Key b = none;
#pragma unroll
  for (int i = 0; i < kPer; ++i)
    if (above(mine[i], b)) b = mine[i];
  k.best[threadIdx.x] = b;
  __syncthreads();
  int rank = 0;
  for (int j = 0; j < kThreads; ++j) rank += above(k.best[j], b) || (j < (int)threadIdx.x && !above(b, k.best[j]) && !above(k.best[j], b));
  __syncthreads();
  if (rank == n - 1 && above(b, k.tau)) k.best[0] = b, k.count |= 1 << 30;
  __syncthreads();
  const bool up = k.count >> 30;
  const Key t = k.best[0];
  __syncthreads();
  // strictly above the new bound, or the bound itself: keep tau just below it
  if (up && threadIdx.x == 0) {
    k.count &= ~(1 << 30);
    k.tau = t;
  }
  __syncthreads();
  if (up) {
#pragma unroll
    for (int i = 0; i < kPer; ++i)
      if (!above(t, mine[i])) k.buf[atomicAdd(&k.count, 1)] = mine[i];
  } else {
#pragma unroll
    for (int i = 0; i < kPer; ++i)
      if (above(mine[i], k.tau)) k.buf[atomicAdd(&k.count, 1)] = mine[i];
  }
  prune(k, n);
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

__global__ void __launch_bounds__(kThreads) select_parts(const __grid_constant__ SelectArgs a) {
  __shared__ Kept<uint64_t> k;
  __shared__ float wm[kThreads / 32];
  __shared__ double ws[kThreads / 32];
  const int row = blockIdx.y, part = blockIdx.x, tid = threadIdx.x, n = a.n_out;
  if (a.finished && a.finished[row]) return;
  const int lo = part * a.part_len, hi = min(a.vocab, lo + a.part_len);
  const float* x = a.logits + row * a.stride;
  if (tid == 0) {
    k.count = 0;
    k.tau = 0;
  }
  float m = -INFINITY, s = 0.0f;
  bool nan = false;
  for (int base = lo; base < hi; base += kTile) {
    // four runs of four per thread
    float v[kPer];
    const bool whole = base + kTile <= hi;
#pragma unroll
    for (int q = 0; q < kPer / 4; ++q) {
      const int at = base + (q * kThreads + tid) * 4;
      if (a.vec && whole) {
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
      s *= expf(m - t);  // m = -inf: 0 * 0
      m = t;
    }
    const float z = m == -INFINITY ? 0.0f : m;
    float part_sum = 0.0f;
#pragma unroll
    for (int i = 0; i < kPer; ++i) {
      part_sum += expf(v[i] - z);
      nan |= v[i] != v[i];
    }
    s += part_sum;
    uint64_t key[kPer];
#pragma unroll
    for (int i = 0; i < kPer; ++i) {
      const int at = base + (i / 4 * kThreads + tid) * 4 + i % 4;
      key[i] = at < hi ? key_of(v[i], at) : 0;
    }
    __syncthreads();
    int pass = 0;
#pragma unroll
    for (int i = 0; i < kPer; ++i) pass += key[i] > k.tau;
    const int total = __syncthreads_count(pass > 0) ? 1 : 0;
    if (!total) continue;
    raise_tau<uint64_t>(k, key, 0, n);
  }
  // the sums of the threads, joined in 64 bits
  float bm = m;
  for (int o = 16; o > 0; o >>= 1) bm = fmaxf(bm, __shfl_xor_sync(0xffffffffu, bm, o));
  if (tid % 32 == 0) wm[tid / 32] = bm;
  nan = __syncthreads_or(nan);
  bm = wm[0];
  for (int w = 1; w < kThreads / 32; ++w) bm = fmaxf(bm, wm[w]);
  double d = m == -INFINITY ? 0.0 : (double)s * exp((double)m - (double)bm);
  if (m == INFINITY) d = NAN;
  for (int o = 16; o > 0; o >>= 1) d += __shfl_xor_sync(0xffffffffu, d, o);
  if (tid % 32 == 0) ws[tid / 32] = d;
  __syncthreads();
  if (tid == 0) {
    d = 0;
    for (int w = 0; w < kThreads / 32; ++w) d += ws[w];
    a.sums[(int64_t)row * a.parts + part] = make_double2(bm, nan ? NAN : d);
  }
  for (int i = tid; i < n; i += kThreads) a.keys[((int64_t)row * a.parts + part) * n + i] = i < k.count ? k.buf[i] : 0;
}

constexpr int kMaxBeams = 64;

__global__ void __launch_bounds__(kThreads) select_join(const __grid_constant__ SelectArgs a) {
  extern __shared__ uint4 raw[];
  Kept<Key2>& k = *reinterpret_cast<Kept<Key2>*>(raw);
  __shared__ double lse[kMaxBeams];  // NaN: every score of the beam is -inf
  __shared__ bool done[kMaxBeams];
  const int r = blockIdx.x, tid = threadIdx.x, W = a.beams, n = a.n_out;
  if (tid == 0) {
    k.count = 0;
    k.tau = {0, 0};
  }
  for (int w = tid; w < W; w += kThreads) {
    const int row = r * W + w;
    done[w] = a.finished && a.finished[row];
    double top = -INFINITY, sum = 0;
    if (!done[w]) {
      const double2* p = a.sums + (int64_t)row * a.parts;
      for (int i = 0; i < a.parts; ++i) top = fmax(top, p[i].x);
      for (int i = 0; i < a.parts; ++i) sum += p[i].x == -INFINITY ? (p[i].y != p[i].y ? p[i].y : 0.0) : p[i].y * exp(p[i].x - top);
      const double l = top + log(sum);
      lse[w] = isfinite(l) && a.scores[row] > -INFINITY ? l : NAN;
    }
  }
  __syncthreads();
  const int per_row = a.parts * n, N = W * per_row;
  for (int base = 0; base < N; base += kTile) {
    Key2 key[kPer];
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
    }
    raise_tau<Key2>(k, key, {0, 0}, n);
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
  constexpr int smem = (int)sizeof(Kept<Key2>);
  if (cudaFuncSetAttribute(select_join, cudaFuncAttributeMaxDynamicSharedMemorySize, smem) != cudaSuccess)
    return launched("select");
  select_parts<<<dim3((unsigned)a.parts, (unsigned)rows), kThreads, 0, st>>>(a);
  const int rc = launched("select");
  if (rc != MK_OK) return rc;
  select_join<<<(unsigned)requests, kThreads, smem, st>>>(a);
  return launched("select");
}

}  // extern "C"
