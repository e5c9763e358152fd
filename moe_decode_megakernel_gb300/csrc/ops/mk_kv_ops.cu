// mk_kv_ops.cu -- the operators that move K and V rows of the paged pools:
// append (with the rotation), commit, beam reorder; the handle and the status
// record.
#include <cuda.h>

#include <cmath>
#include <new>

#include "mk_ops_common.cuh"

namespace mk {
namespace ops {
namespace {

constexpr int kThreads = 256;

// -------------------------------------------------------------------- append

struct AppendArgs {
  Pools pools;
  Batch b;
  const void *q, *k, *v;
  uint16_t* q_out;
  int64_t q_stride, k_stride, v_stride, q_out_stride;
  int32_t n_q;
  uint32_t* status;
  uint64_t freq[64];
};

// (cos, sin) of 2 pi pos f / 2^64.  The product wraps modulo 2^64, that is
// modulo whole turns, so no position loses low bits to a large angle: the
// error is pos * 2^-53 of the pair's frequency (its rounding on the host) plus
// 2^-25 of the turn left over.
__device__ __forceinline__ float2 turn(uint64_t f, int pos) {
  const int64_t a = (int64_t)(f * (uint64_t)(int64_t)pos);
  float s, c;
  sincospif((float)(int32_t)(a >> 32) * 0x1p-31f, &s, &c);
  return make_float2(c, s);
}

// Eight elements (a 16-byte chunk of bf16 output) of a head, as they lie.
template <bool F32>
struct Chunk {
  uint4 u[F32 ? 2 : 1];
};
template <bool F32>
__device__ __forceinline__ Chunk<F32> load8(const void* p, int64_t elem) {
  Chunk<F32> c;
  const uint4* s = reinterpret_cast<const uint4*>(static_cast<const uint8_t*>(p) + elem * (F32 ? 4 : 2));
#pragma unroll
  for (int i = 0; i < (F32 ? 2 : 1); ++i) c.u[i] = s[i];
  return c;
}
__device__ __forceinline__ void values(const Chunk<true>& c, float (&x)[8]) {
#pragma unroll
  for (int i = 0; i < 2; ++i) {
    x[4 * i] = __uint_as_float(c.u[i].x), x[4 * i + 1] = __uint_as_float(c.u[i].y);
    x[4 * i + 2] = __uint_as_float(c.u[i].z), x[4 * i + 3] = __uint_as_float(c.u[i].w);
  }
}
__device__ __forceinline__ void values(const Chunk<false>& c, float (&x)[8]) {
  const uint32_t w[4] = {c.u[0].x, c.u[0].y, c.u[0].z, c.u[0].w};
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    x[2 * i] = __uint_as_float(w[i] << 16);
    x[2 * i + 1] = __uint_as_float(w[i] & 0xffff0000u);
  }
}

// One block per token (and one for the batch), its heads in 16-byte chunks of
// output.  The first chunks of every thread are on their way before the token's
// slot is known (its sequence, then its page: two round trips to memory); the
// thread whose sequence holds the token looks the slot up, half a head of
// threads turns the position into sines.  12.6K tokens of 40 heads of 128 (258 MB moved) take 42
// us, 6.2 TB/s where a copy of that size reaches 6.8: bound by memory.  Small
// blocks with many chunks of a thread under way: 256 threads with three took 48
// us, 128 with three 44; 64 with ten were no faster.
// Eight tokens are a chain of four round trips, 3 us behind another kernel.  The
// batch's own block costs nothing beside them; with its check in the first
// token's block they took 3.3 us, with it in every block the 12.6K tokens 43.
constexpr int kAppend = 128;
template <int D, bool F32>
__global__ void __launch_bounds__(kAppend) append_kernel(const __grid_constant__ AppendArgs a) {
  constexpr int CPH = D / 8;  // chunks per head
  constexpr int kHeld = 5;    // chunks of a thread under way
  __shared__ float2 cs[D / 2];
  __shared__ int64_t row;  // row of head 0 in the pool, -1: not written
  __shared__ int pos, found;
  const int t = blockIdx.x, tid = threadIdx.x;
  wait_before();
  let_next_in();
  if (t == a.b.n_tokens) {  // the batch's block: sequences that may have no token whose block would see what is wrong
    for (int b = tid; b < a.b.batch; b += kAppend) {
      const int t0 = a.b.cu[b], t1 = a.b.cu[b + 1];
      if (t0 < 0 || t1 < t0 || t1 > a.b.n_tokens) record(a.status, dev::ERR_INDEX, OP_APPEND, b, 0, t1, a.b.n_tokens);
    }
    return;
  }
  const int n_kv = a.pools.n_kv, heads = a.n_q + 2 * n_kv, chunks = heads * CPH;
  Chunk<F32> held[kHeld];
  auto load = [&](int base) {
#pragma unroll
    for (int x = 0; x < kHeld; ++x) {
      const int i = base + x * kAppend + tid, h = i / CPH, c = i % CPH;
      if (i >= chunks) break;
      if (h < a.n_q)
        held[x] = load8<F32>(a.q, t * a.q_stride + h * D + c * 8);
      else if (h < a.n_q + n_kv)
        held[x] = load8<F32>(a.k, t * a.k_stride + (h - a.n_q) * D + c * 8);
      else
        held[x] = load8<F32>(a.v, t * a.v_stride + (h - a.n_q - n_kv) * D + c * 8);
    }
  };
  load(0);
  if (tid == 0) found = 0;
  __syncthreads();
  for (int b = tid; b < a.b.batch; b += kAppend) {
    if (a.b.cu[b] > t || t >= a.b.cu[b + 1]) continue;
    const Seq s = seq_of(a.b, b, a.pools.page_shift, a.status, OP_APPEND);
    if (s.n == 0) continue;
    const int slot = s.ctx + t - s.t0, P = 1 << a.pools.page_shift;
    const int page = a.b.tables[(int64_t)b * a.b.max_pages + (slot >> a.pools.page_shift)];
    pos = a.b.positions ? a.b.positions[t] : slot;
    row = (int64_t)page * n_kv * P + (slot & (P - 1));
    if (page < 0 || page >= a.pools.num_pages) {
      record(a.status, dev::ERR_PAGE, OP_APPEND, b, slot, page, (uint32_t)a.pools.num_pages);
      row = -1;
    }
    found = 1;
  }
  __syncthreads();
  if (!found) return;
  if (tid < D / 2) cs[tid] = turn(a.freq[tid], pos);
  __syncthreads();
  for (int base = 0; base < chunks; base += kHeld * kAppend) {
    if (base) load(base);
#pragma unroll
    for (int x = 0; x < kHeld; ++x) {
      const int i = base + x * kAppend + tid, h = i / CPH, c = i % CPH;
      if (i >= chunks || (h >= a.n_q && row < 0)) break;
      float v[8];
      values(held[x], v);
      if (h < a.n_q + n_kv) {
#pragma unroll
        for (int j = 0; j < 4; ++j) {
          const float2 w = cs[c * 4 + j];
          const float e = v[2 * j], o = v[2 * j + 1];
          v[2 * j] = e * w.x - o * w.y;
          v[2 * j + 1] = e * w.y + o * w.x;
        }
      }
      const bool is_k = h < a.n_q + n_kv;
      const int g = h - a.n_q - (is_k ? 0 : n_kv);
      uint16_t* dst = h < a.n_q ? a.q_out + t * a.q_out_stride + h * D + c * 8
                                : (is_k ? a.pools.k : a.pools.v) + ((row + ((int64_t)g << a.pools.page_shift)) * D + c * 8);
      *reinterpret_cast<uint4*>(dst) =
          make_uint4(pack_bf16(v[0], v[1]), pack_bf16(v[2], v[3]), pack_bf16(v[4], v[5]), pack_bf16(v[6], v[7]));
    }
  }
}

// -------------------------------------------------------------------- commit

struct CommitArgs {
  Pools pools;
  const int32_t *ctx, *path, *path_lens, *tables;
  int32_t* new_lens;
  int32_t max_path, max_pages, row_chunks;
  uint32_t* status;
};

constexpr int kRound = 32;  // path entries located at a time
constexpr int kHeld = 8;    // rows a thread holds between their loads and stores

// A thread owns one 16-byte chunk of (layer, K or V, head) and walks the path:
// an entry's source lies at or behind its place, and behind every place before
// it (the path ascends), so rows loaded before later places are written are
// still the drafted ones.  No two threads touch the same bytes.  Bound by
// latency at any real size (path, table and rows are three round trips to
// memory): behind another call, 32 sequences of up to five accepted tokens in 48
// layers (11 MB) take 5.2 us and one sequence in eight layers 2.4.  A thread has eight rows
// under way, so a path of eight costs what one of one does.
__global__ void __launch_bounds__(kThreads) commit_kernel(const __grid_constant__ CommitArgs a) {
  __shared__ int64_t from[kRound], to[kRound];  // rows of head 0, -1: nothing to do
  const int b = blockIdx.y, tid = threadIdx.x;
  wait_before();
  let_next_in();
  const int ctx = a.ctx[b], m = a.path_lens[b];
  const int32_t* path = a.path + (int64_t)b * a.max_path;
  const int32_t* table = a.tables + (int64_t)b * a.max_pages;
  const int64_t slots = (int64_t)a.max_pages << a.pools.page_shift;
  bool bad = ctx < 0 || m < 0 || m > a.max_path;
  const int P1 = (1 << a.pools.page_shift) - 1;
  auto row_of = [&](int page, int slot) {
    return (((int64_t)page * a.pools.n_kv) << a.pools.page_shift) + (slot & P1);
  };
  if (!bad)
    for (int k = tid; k < m; k += kThreads) {
      const int s = path[k];
      if (s < k || (k > 0 && s <= path[k - 1]) || (int64_t)ctx + s >= slots) {  // s < k: it cannot ascend from 0
        bad = true;
        record(a.status, dev::ERR_INDEX, OP_COMMIT, b, k, s, (uint32_t)slots);
      } else {
        const int page = table[(ctx + s) >> a.pools.page_shift], dst = table[(ctx + k) >> a.pools.page_shift];
        const bool from_bad = page < 0 || page >= a.pools.num_pages;
        if (from_bad || dst < 0 || dst >= a.pools.num_pages) {
          bad = true;
          record(a.status, dev::ERR_PAGE, OP_COMMIT, b, k, from_bad ? page : dst, (uint32_t)a.pools.num_pages);
        }
        if (k < kRound) {
          from[k] = s == k ? -1 : row_of(page, ctx + s);
          to[k] = row_of(dst, ctx + k);
        }
      }
    }
  else if (tid == 0)
    record(a.status, dev::ERR_RANGE, OP_COMMIT, b, m, ctx, a.max_path);
  bad = __syncthreads_or(bad);
  if (blockIdx.x == 0 && tid == 0 && a.new_lens) a.new_lens[b] = bad ? ctx : ctx + m;
  if (bad) return;
  // chunk i of a layer's rows: K or V, head, 16 bytes of the head
  const int i = blockIdx.x * kThreads + tid;
  const int per_layer = 2 * a.pools.n_kv * a.row_chunks;
  const bool mine = i < per_layer * a.pools.n_layers;
  const int layer = i / per_layer, rest = i % per_layer;
  const int h = rest / a.row_chunks % a.pools.n_kv, c = rest % a.row_chunks;
  uint16_t* pool = rest < per_layer / 2 ? a.pools.k : a.pools.v;
  uint4* base = reinterpret_cast<uint4*>(pool + (mine ? layer * a.pools.layer_elems : 0));
  const int64_t head = (int64_t)h << a.pools.page_shift;
  for (int k0 = 0; k0 < m; k0 += kRound) {
    if (k0) {
      __syncthreads();
      if (tid < kRound) {
        const int k = k0 + tid;
        from[tid] = -1;
        if (k < m && path[k] != k) {
          const int s = ctx + path[k], d = ctx + k;
          from[tid] = row_of(table[s >> a.pools.page_shift], s);
          to[tid] = row_of(table[d >> a.pools.page_shift], d);
        }
      }
    }
    __syncthreads();
    if (!mine) continue;
    for (int k = 0; k < kRound && k0 + k < m; k += kHeld) {
      uint4 x[kHeld];
#pragma unroll
      for (int j = 0; j < kHeld; ++j)
        if (k0 + k + j < m && from[k + j] >= 0) x[j] = base[(from[k + j] + head) * a.row_chunks + c];
#pragma unroll
      for (int j = 0; j < kHeld; ++j)
        if (k0 + k + j < m && from[k + j] >= 0) base[(to[k + j] + head) * a.row_chunks + c] = x[j];
    }
  }
}

// -------------------------------------------------------------- beam reorder

struct ReorderArgs {
  Pools pools;
  const int32_t *lens, *parents, *tables_in;
  int32_t* tables_out;
  int32_t beams, max_pages, row_chunks;
  uint32_t* status;
};

constexpr int kMaxBeams = 64;

// Blocks (r, y) share request r's copies: its extra children times (layer, K
// or V, head), each a run of (len % page_size) rows.  Sources are open pages
// of beams with children, destinations those of beams without: no copy reads
// what another writes.  Bound by memory: 16 requests of 8 beams, half of them
// replaced, 48 layers (325 MB) take 50 us, 6.5 TB/s.  (In 64 blocks of a
// request 56 us with four loads per thread under way, 67 with eight, 108 with one.)
__global__ void __launch_bounds__(kThreads) reorder_kernel(const __grid_constant__ ReorderArgs a) {
  __shared__ int par[kMaxBeams], open[kMaxBeams], kids[kMaxBeams], spare[kMaxBeams];
  __shared__ int src[kMaxBeams], dst[kMaxBeams], mine[kMaxBeams];
  __shared__ int n_copy;
  const int r = blockIdx.x, tid = threadIdx.x, W = a.beams, P = 1 << a.pools.page_shift;
  wait_before();
  let_next_in();
  const int len = a.lens[r];
  const int32_t* tin = a.tables_in + (int64_t)r * W * a.max_pages;
  int32_t* tout = a.tables_out + (int64_t)r * W * a.max_pages;
  bool bad = len < 0 || len > ((int64_t)a.max_pages << a.pools.page_shift);
  if (bad && tid == 0 && blockIdx.y == 0) record(a.status, dev::ERR_RANGE, OP_REORDER, r, 0, len, a.max_pages * P);
  const int full = bad ? 0 : len >> a.pools.page_shift, used = bad ? 0 : len & (P - 1);
  if (tid < W) {
    par[tid] = a.parents[(int64_t)r * W + tid];
    kids[tid] = 0;
    if (par[tid] < 0 || par[tid] >= W) {
      if (blockIdx.y == 0) record(a.status, dev::ERR_INDEX, OP_REORDER, r, tid, par[tid], W);
      bad = true;
    }
    open[tid] = used ? tin[(int64_t)tid * a.max_pages + full] : 0;
  }
  bad = __syncthreads_or(bad);
  if (!bad && tid == 0) {
    for (int i = 0; i < W; ++i) ++kids[par[i]];
    int n_spare = 0, n = 0;
    for (int i = 0; i < W; ++i)
      if (kids[i] == 0) spare[n_spare++] = open[i];
    for (int i = 0; i < W; ++i) {
      const int p = par[i];
      if (kids[p] > 0) {  // its first child
        kids[p] = -1;
        mine[i] = open[p];
      } else {
        mine[i] = spare[n];
        src[n] = open[p];
        dst[n] = spare[n];
        ++n;
      }
    }
    n_copy = used ? n : 0;
  }
  __syncthreads();
  // the tables
  for (int64_t i = (int64_t)blockIdx.y * kThreads + tid; i < (int64_t)W * a.max_pages; i += (int64_t)gridDim.y * kThreads) {
    const int w = (int)(i / a.max_pages), j = (int)(i % a.max_pages);
    int v = tin[i];
    if (!bad) {
      if (j < full) v = tin[(int64_t)par[w] * a.max_pages + j];
      if (j == full && used) v = mine[w];
    }
    tout[i] = v;
  }
  if (bad) return;
  // the open pages
  const int units = 2 * a.pools.n_kv * a.pools.n_layers, run = used * a.row_chunks;
  for (int u = blockIdx.y; u < units * n_copy; u += gridDim.y) {
    const int e = u / units, w = u % units;
    const int layer = w / (2 * a.pools.n_kv), h = w % a.pools.n_kv;
    const bool from_bad = src[e] < 0 || src[e] >= a.pools.num_pages;
    if (from_bad || dst[e] < 0 || dst[e] >= a.pools.num_pages) {
      if (tid == 0) record(a.status, dev::ERR_PAGE, OP_REORDER, r, e, from_bad ? src[e] : dst[e], (uint32_t)a.pools.num_pages);
      continue;
    }
    uint4* pool = reinterpret_cast<uint4*>((w / a.pools.n_kv % 2 ? a.pools.v : a.pools.k) + layer * a.pools.layer_elems);
    const uint4* from = pool + (((int64_t)src[e] * a.pools.n_kv + h) << a.pools.page_shift) * a.row_chunks;
    uint4* to = pool + (((int64_t)dst[e] * a.pools.n_kv + h) << a.pools.page_shift) * a.row_chunks;
    for (int i = tid; i < run; i += 4 * kThreads) {
      uint4 x[4];
#pragma unroll
      for (int j = 0; j < 4; ++j)
        if (i + j * kThreads < run) x[j] = from[i + j * kThreads];
#pragma unroll
      for (int j = 0; j < 4; ++j)
        if (i + j * kThreads < run) to[i + j * kThreads] = x[j];
    }
  }
}

// Blocks of a request: its copies' (layer, K or V, head) units dealt evenly, so
// that every child's copy keeps all of them equally busy, up to 4096 blocks in
// all (three times what the GPU holds; above 512 requests eight each).  16
// requests of 384 units: 192 blocks each 50 us, 384 the same, 64, 128 and 256
// took 56, 53 and 53; with nothing to copy a call takes 7 us behind another.
// One request: 11 us, 21 in 64.
unsigned reorder_blocks(int64_t requests, int64_t units) {
  int64_t most = 4096 / requests;
  most = most < 8 ? 8 : most > 384 ? 384 : most;
  if (units <= most) return (unsigned)(units > 64 ? units : most < 64 ? most : 64);
  const int64_t per = (units + most - 1) / most;
  return (unsigned)((units + per - 1) / per);
}

}  // namespace

int encode_pools(mk_kv* kv) {
  typedef CUresult (*EncodeTiledFn)(CUtensorMap*, CUtensorMapDataType, cuuint32_t, void*, const cuuint64_t*,
                                    const cuuint64_t*, const cuuint32_t*, const cuuint32_t*, CUtensorMapInterleave,
                                    CUtensorMapSwizzle, CUtensorMapL2promotion, CUtensorMapFloatOOBfill);
  if (kv->tm_ready) return MK_OK;
  std::lock_guard<std::mutex> hold(kv->tm_lock);
  if (kv->tm_ready) return MK_OK;
  void* f = nullptr;
  cudaDriverEntryPointQueryResult q;
  if (cudaGetDriverEntryPointByVersion("cuTensorMapEncodeTiled", &f, 12000, cudaEnableDefault, &q) != cudaSuccess ||
      q != cudaDriverEntryPointSuccess) {
    cudaGetLastError();
    return fail(MK_ERR_CUDA, "cuTensorMapEncodeTiled is not available");
  }
  const mk_kv_config& c = kv->cfg;
  // [layer][page][head][row] rows of head_dim, boxes of 64 elements (128
  // bytes, the swizzle's width) x one page (at most a tile of 128 rows)
  const cuuint64_t rows = (cuuint64_t)c.num_pages * c.n_kv * c.page_size;
  const cuuint64_t dims[3] = {(cuuint64_t)c.head_dim, rows, (cuuint64_t)c.n_layers};
  const cuuint64_t strides[2] = {(cuuint64_t)c.head_dim * 2, rows * c.head_dim * 2};
  const cuuint32_t box[3] = {64, (cuuint32_t)(c.page_size < 128 ? c.page_size : 128), 1};
  const cuuint32_t step[3] = {1, 1, 1};
  for (int i = 0; i < 2; ++i) {
    const CUresult r = reinterpret_cast<EncodeTiledFn>(f)(
        i ? &kv->tm_v : &kv->tm_k, CU_TENSOR_MAP_DATA_TYPE_BFLOAT16, 3, i ? c.v_pool : c.k_pool, dims, strides, box,
        step, CU_TENSOR_MAP_INTERLEAVE_NONE, CU_TENSOR_MAP_SWIZZLE_128B, CU_TENSOR_MAP_L2_PROMOTION_L2_256B,
        CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE);
    if (r != CUDA_SUCCESS) return fail(MK_ERR_CUDA, "cuTensorMapEncodeTiled failed (" + std::to_string((int)r) + ")");
  }
  kv->tm_ready = true;
  return MK_OK;
}

}  // namespace ops
}  // namespace mk

using mk::fail;
using namespace mk::ops;

extern "C" {

int mk_kv_open(const mk_kv_config* cfg, mk_kv** out) {
  if (!cfg || !out) return fail(MK_ERR_ARG, "null argument");
  *out = nullptr;
  const mk_kv_config& c = *cfg;
  if (c.n_layers < 1 || c.n_kv < 1 || c.num_pages < 1) return fail(MK_ERR_ARG, "empty pools");
  if (c.head_dim != 64 && c.head_dim != 128) return fail(MK_ERR_UNSUPPORTED, "head_dim is 64 or 128");
  if (c.page_size < 16 || c.page_size > 256 || (c.page_size & (c.page_size - 1)))
    return fail(MK_ERR_UNSUPPORTED, "page_size is a power of two from 16 to 256");
  if (c.num_pages >= (int64_t)1 << 31 || c.num_pages * c.n_kv >= (int64_t)1 << 31 ||
      c.num_pages * c.n_kv * c.page_size >= (int64_t)1 << 31)
    return fail(MK_ERR_ARG, "2^31 rows or more in a layer of the pools");
  if (endless(c.n_layers, c.num_pages * c.n_kv * c.page_size * c.head_dim, 2))
    return fail(MK_ERR_ARG, "pools of more than 2^48 bytes");
  if (!c.k_pool || !c.v_pool || misaligned(c.k_pool) || misaligned(c.v_pool))
    return fail(MK_ERR_ARG, "null or misaligned pool");
  if (!(c.rope_base > 1.0) || !std::isfinite(c.rope_base)) return fail(MK_ERR_ARG, "rope_base must be above 1");
  mk_kv* kv = new (std::nothrow) mk_kv;
  if (!kv) return fail(MK_ERR_ARG, "out of host memory");
  kv->cfg = c;
  while ((1 << kv->page_shift) < c.page_size) ++kv->page_shift;
  // base^(-2i/d) / (2 pi) of a turn: below 0.16, so 64 bits hold it without a
  // whole turn; the double's rounding is 2^-53 of it
  for (int i = 0; i < c.head_dim / 2; ++i)
    kv->freq[i] = (uint64_t)std::ldexp(std::pow(c.rope_base, -2.0 * i / c.head_dim) / 6.283185307179586476925, 64);
  *out = kv;
  return MK_OK;
}

void mk_kv_free(mk_kv* kv) { delete kv; }

int mk_kv_append(const mk_kv* kv, int32_t layer, const mk_tokens* tok, const mk_append_io* io, uint32_t* status,
                 void* stream) {
  const int rc = check_tokens(kv, layer, tok);
  if (rc != MK_OK) return rc;
  if (!io) return fail(MK_ERR_ARG, "null argument");
  if (tok->batch == 0 || tok->n_tokens == 0) return MK_OK;
  if (!io->k || !io->v) return fail(MK_ERR_ARG, "null K or V");
  if (misplaced(status)) return fail(MK_ERR_ARG, "misaligned status");
  if (io->dtype != MK_BF16 && io->dtype != MK_F32) return fail(MK_ERR_ARG, "dtype is MK_BF16 or MK_F32");
  const mk_kv_config& c = kv->cfg;
  const size_t elem = io->dtype == MK_F32 ? 4 : 2;
  const int32_t n_q = io->q ? io->n_q : 0;
  if (io->q && (!io->q_out || n_q < 1)) return fail(MK_ERR_ARG, "q without q_out or heads");
  if (io->n_q < 0 || n_q > (1 << 16)) return fail(MK_ERR_ARG, "bad number of query heads");
  const int64_t kv_row = (int64_t)c.n_kv * c.head_dim, q_row = (int64_t)n_q * c.head_dim;
  auto bad = [&](const void* p, int64_t stride, int64_t row, size_t e) {
    return misaligned(p) || stride < row || (stride * e) % 16 != 0 || endless(tok->n_tokens, stride, e);
  };
  if (bad(io->k, io->k_stride, kv_row, elem) || bad(io->v, io->v_stride, kv_row, elem) ||
      (n_q && (bad(io->q, io->q_stride, q_row, elem) || bad(io->q_out, io->q_out_stride, q_row, 2))))
    return fail(MK_ERR_ARG, "misaligned token array, or a stride that is too small, too large or no multiple of 16 bytes");
  const int64_t T = tok->n_tokens;
  if (n_q) {
    // q_out is q itself (k and v may be other columns of the same rows), or
    // apart from every input
    const bool itself = io->q_out == io->q && io->dtype == MK_BF16 && io->q_out_stride == io->q_stride;
    const size_t out = span(T, io->q_out_stride, q_row, 2);
    auto collides = [&](const void* p, int64_t stride) {
      if (!overlap(io->q_out, out, p, span(T, stride, kv_row, elem))) return false;
      if (!itself || stride != io->q_stride) return true;
      const int64_t apart = (static_cast<const uint16_t*>(p) - static_cast<const uint16_t*>(io->q_out)) % stride;
      const int64_t col = apart < 0 ? apart + stride : apart;
      return col < q_row || col + kv_row > stride;
    };
    if ((!itself && overlap(io->q_out, out, io->q, span(T, io->q_stride, q_row, elem))) ||
        collides(io->k, io->k_stride) || collides(io->v, io->v_stride) || over_batch(tok, io->q_out, out) ||
        over_pools(kv, status, io->q_out, out))
      return fail(MK_ERR_ARG, "q_out overlaps another argument or the pools");
  }
  AppendArgs a;
  a.pools = pools_of(kv, layer);
  a.b = batch_of(tok);
  a.q = io->q, a.k = io->k, a.v = io->v, a.q_out = static_cast<uint16_t*>(io->q_out);
  a.q_stride = io->q_stride, a.k_stride = io->k_stride, a.v_stride = io->v_stride, a.q_out_stride = io->q_out_stride;
  a.n_q = n_q;
  a.status = status;
  for (int i = 0; i < 64; ++i) a.freq[i] = kv->freq[i];
  auto kernel = c.head_dim == 128 ? (io->dtype == MK_F32 ? append_kernel<128, true> : append_kernel<128, false>)
                                  : (io->dtype == MK_F32 ? append_kernel<64, true> : append_kernel<64, false>);
  return launch("append", kernel, dim3((unsigned)T + 1), kAppend, 0, static_cast<cudaStream_t>(stream), a);
}

int mk_kv_commit(const mk_kv* kv, int32_t batch, const int32_t* cache_lens, const int32_t* path,
                 const int32_t* path_lens, int32_t max_path, const int32_t* block_tables, int32_t max_pages,
                 int32_t* new_lens, uint32_t* status, void* stream) {
  if (!kv) return fail(MK_ERR_ARG, "null argument");
  if (batch < 0 || max_path < 0 || max_pages < 1) return fail(MK_ERR_ARG, "negative batch or path width, or no page columns");
  if (!table_fits(kv, max_pages)) return fail(MK_ERR_ARG, "block tables of more than 2^30 slots");
  if (batch == 0) return MK_OK;
  if (!cache_lens || !path_lens || !block_tables || (max_path > 0 && !path)) return fail(MK_ERR_ARG, "null argument");
  if (batch > 65535) return fail(MK_ERR_ARG, "batch above 65535");
  if (misplaced(cache_lens, path, path_lens, block_tables, new_lens, status)) return fail(MK_ERR_ARG, "misaligned argument");
  if (overlap(new_lens, 4 * (size_t)batch, cache_lens, 4 * (size_t)batch) ||
      overlap(new_lens, 4 * (size_t)batch, path_lens, 4 * (size_t)batch) ||
      overlap(new_lens, 4 * (size_t)batch, path, 4 * (size_t)batch * max_path) ||
      overlap(new_lens, 4 * (size_t)batch, block_tables, 4 * (size_t)batch * max_pages) ||
      over_pools(kv, status, new_lens, 4 * (size_t)batch))
    return fail(MK_ERR_ARG, "new_lens overlaps another argument or the pools");
  CommitArgs a;
  a.pools = pools_of(kv, 0);
  a.ctx = cache_lens, a.path = path, a.path_lens = path_lens, a.tables = block_tables, a.new_lens = new_lens;
  a.max_path = max_path, a.max_pages = max_pages, a.row_chunks = kv->cfg.head_dim / 8;
  a.status = status;
  const int64_t chunks = (int64_t)2 * kv->cfg.n_kv * a.row_chunks * kv->cfg.n_layers;
  if (chunks > INT32_MAX) return fail(MK_ERR_ARG, "more than 2^31 chunks in a token's rows");
  const dim3 grid((unsigned)((chunks + kThreads - 1) / kThreads), (unsigned)batch);
  return launch("commit", commit_kernel, grid, kThreads, 0, static_cast<cudaStream_t>(stream), a);
}

int mk_beam_reorder(const mk_kv* kv, int32_t requests, int32_t beams, const int32_t* lens, const int32_t* parents,
                    const int32_t* tables_in, int32_t* tables_out, int32_t max_pages, uint32_t* status, void* stream) {
  if (!kv) return fail(MK_ERR_ARG, "null argument");
  if (requests < 0 || beams < 1 || beams > kMaxBeams || max_pages < 1)
    return fail(MK_ERR_ARG, "bad number of requests, beams (1 to 64) or page columns");
  if (!table_fits(kv, max_pages)) return fail(MK_ERR_ARG, "block tables of more than 2^30 slots");
  if (requests == 0) return MK_OK;
  if (!lens || !parents || !tables_in || !tables_out) return fail(MK_ERR_ARG, "null argument");
  if (misplaced(lens, parents, tables_in, tables_out, status)) return fail(MK_ERR_ARG, "misaligned argument");
  const size_t bytes = 4 * (size_t)requests * beams * max_pages;
  if (overlap(tables_out, bytes, tables_in, bytes) || overlap(tables_out, bytes, parents, 4 * (size_t)requests * beams) ||
      overlap(tables_out, bytes, lens, 4 * (size_t)requests) || over_pools(kv, status, tables_out, bytes))
    return fail(MK_ERR_ARG, "tables_out overlaps another argument or the pools");
  ReorderArgs a;
  a.pools = pools_of(kv, 0);
  a.lens = lens, a.parents = parents, a.tables_in = tables_in, a.tables_out = tables_out;
  a.beams = beams, a.max_pages = max_pages, a.row_chunks = kv->cfg.head_dim / 8;
  a.status = status;
  const int64_t units = (int64_t)2 * kv->cfg.n_kv * kv->cfg.n_layers * beams;
  if (units > 1 << 30) return fail(MK_ERR_ARG, "more than 2^30 runs to copy");
  const dim3 grid((unsigned)requests, reorder_blocks(requests, units / beams));
  return launch("reorder", reorder_kernel, grid, kThreads, 0, static_cast<cudaStream_t>(stream), a);
}

int mk_check_status(const uint32_t* status, void* stream) {
  if (!status || misplaced(status)) return fail(MK_ERR_ARG, "null or misaligned status");
  uint32_t r[8] = {};
  cudaStream_t st = static_cast<cudaStream_t>(stream);
  cudaError_t e = cudaMemcpyAsync(r, status, sizeof r, cudaMemcpyDeviceToHost, st);
  if (e == cudaSuccess) e = cudaStreamSynchronize(st);
  if (e != cudaSuccess) return fail(MK_ERR_CUDA, std::string("status: ") + cudaGetErrorString(e));
  if (r[0] == 0) return MK_OK;
  static const char* const names[] = {"?", "kv_append", "tree_attn", "kv_commit", "beam_reorder"};
  const std::string at = std::string(names[r[1] < 5 ? r[1] : 0]) + ", row " + std::to_string(r[2]);
  if (r[0] == mk::dev::ERR_TIMEOUT) return fail(MK_ERR_TIMEOUT, at + ": a wait on the device gave up");
  const char* what = r[0] == mk::dev::ERR_PAGE ? "page id" : r[0] == mk::dev::ERR_INDEX ? "index" : "length or position";
  return fail(MK_ERR_DEVICE, at + ", index " + std::to_string(r[3]) + ": " + what + " " +
                                 std::to_string((int32_t)r[4]) + " out of range (limit " + std::to_string(r[5]) + ")");
}

}  // extern "C"
