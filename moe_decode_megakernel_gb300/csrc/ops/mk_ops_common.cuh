// mk_ops_common.cuh -- what the operators of include/mk_ops.h share: the
// handle on the pools, the status record, host checks, the ragged batch.
#pragma once

#include <cuda_runtime.h>
#include <stdint.h>

#include <atomic>
#include <mutex>
#include <string>

#include "../../../include/mk_ops.h"
#include "../mk_host.h"
#include "../mk_kernel.cuh"

struct mk_kv {
  mk_kv_config cfg;
  int page_shift = 0;
  // turns per position of each rotated pair, as a fraction of 2^64
  uint64_t freq[64] = {};
  // tensor maps of the pools, made by the first call that reads through them
  std::mutex tm_lock;
  std::atomic<bool> tm_ready{false};
  CUtensorMap tm_k, tm_v;
};

namespace mk {
namespace ops {

enum OpId : uint32_t { OP_APPEND = 1, OP_ATTN = 2, OP_COMMIT = 3, OP_REORDER = 4 };

// The pools as the kernels see them.
struct Pools {
  uint16_t* k;  // of the call's first layer
  uint16_t* v;
  int64_t num_pages;
  int64_t layer_elems;  // elements of one layer
  int32_t n_kv, page_shift, n_layers;
};

struct Batch {
  const int32_t* cu;
  const int32_t* ctx;
  const int32_t* tables;
  const int32_t* positions;
  int32_t batch, n_tokens, max_pages;
};

// All earlier work of the stream is done and visible behind this.
__device__ __forceinline__ void wait_before() { asm volatile("griddepcontrol.wait;" ::: "memory"); }
// The next kernel may become resident once every block has passed this.
__device__ __forceinline__ void let_next_in() { asm volatile("griddepcontrol.launch_dependents;" ::: "memory"); }

// The first record stays: {code, operator, row, index, value, limit}.
__device__ inline void record(uint32_t* status, uint32_t code, uint32_t op, uint32_t row, uint32_t index, uint32_t value,
                              uint32_t limit) {
  if (!status || atomicCAS(status, 0u, code) != 0u) return;
  status[1] = op;
  status[2] = row;
  status[3] = index;
  status[4] = value;
  status[5] = limit;
}

// Sequence b of a ragged batch: its rows [t0, t0 + n) and its cache length;
// n = 0 (and the fault recorded) where the batch's numbers cannot be.
struct Seq {
  int t0, n, ctx;
};
__device__ inline Seq seq_of(const Batch& a, int b, int page_shift, uint32_t* status, uint32_t op) {
  Seq s;
  s.t0 = a.cu[b];
  const int t1 = a.cu[b + 1];
  s.ctx = a.ctx[b];
  s.n = t1 - s.t0;
  if (s.t0 < 0 || s.n < 0 || t1 > a.n_tokens) {
    record(status, dev::ERR_INDEX, op, b, 0, t1, a.n_tokens);
    s.n = 0;
  } else if (s.n > 0 && (s.ctx < 0 || (int64_t)s.ctx + s.n > ((int64_t)a.max_pages << page_shift))) {
    record(status, dev::ERR_RANGE, op, b, 1, s.ctx, a.max_pages << page_shift);
    s.n = 0;
  }
  return s;
}

// ---------------------------------------------------------------- arithmetic
__device__ __forceinline__ float ex2(float x) {
  float r;
  asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(r) : "f"(x));
  return r;
}
// Two fp32 at a time (each half rounded as the scalar operation).
__device__ __forceinline__ uint64_t pair(uint32_t lo, uint32_t hi) {
  uint64_t r;
  asm("mov.b64 %0, {%1, %2};" : "=l"(r) : "r"(lo), "r"(hi));
  return r;
}
__device__ __forceinline__ float2 halves(uint64_t v) {
  float a, b;
  asm("mov.b64 {%0, %1}, %2;" : "=f"(a), "=f"(b) : "l"(v));
  return make_float2(a, b);
}
__device__ __forceinline__ uint64_t fma2(uint64_t a, uint64_t b, uint64_t c) {
  uint64_t r;
  asm("fma.rn.f32x2 %0, %1, %2, %3;" : "=l"(r) : "l"(a), "l"(b), "l"(c));
  return r;
}
__device__ __forceinline__ uint64_t mul2(uint64_t a, uint64_t b) {
  uint64_t r;
  asm("mul.rn.f32x2 %0, %1, %2;" : "=l"(r) : "l"(a), "l"(b));
  return r;
}
__device__ __forceinline__ uint64_t add2(uint64_t a, uint64_t b) {
  uint64_t r;
  asm("add.rn.f32x2 %0, %1, %2;" : "=l"(r) : "l"(a), "l"(b));
  return r;
}
// Two bf16 in a word, each rounded to nearest even.
__device__ __forceinline__ uint32_t pack_bf16(float lo, float hi) {
  uint32_t r;
  asm("cvt.rn.bf16x2.f32 %0, %1, %2;" : "=r"(r) : "f"(hi), "f"(lo));
  return r;
}

// ---------------------------------------------------------------- host side
inline bool misaligned(const void* p, uintptr_t a = 16) { return (reinterpret_cast<uintptr_t>(p) & (a - 1)) != 0; }

// Whether an address (NULL aside) does not fit its elements.
template <typename... T>
inline bool misplaced(const T*... p) {
  return (misaligned(p, sizeof(T)) || ...);
}

inline bool overlap(const void* a, size_t an, const void* b, size_t bn) {
  const uintptr_t x = reinterpret_cast<uintptr_t>(a), y = reinterpret_cast<uintptr_t>(b);
  return a && b && an && bn && x < y + bn && y < x + an;
}

// Whether an array of so many strided rows is longer than addresses reach (2^48
// bytes), where its offsets would pass 64 bits.
inline bool endless(int64_t rows, int64_t stride, size_t elem) {
  return rows > 1 && stride > (int64_t)(((uint64_t)1 << 48) / ((uint64_t)rows * elem));
}

// Bytes of a strided token array: the last row counts its own elements only.
inline size_t span(int64_t rows, int64_t stride, int64_t row_elems, size_t elem) {
  return rows > 0 ? (size_t)((rows - 1) * stride + row_elems) * elem : 0;
}

// Launches a kernel that may become resident while the one before it in the
// stream ends; every such kernel waits (wait_before) before it touches memory.
template <typename... P, typename... A>
inline int launch(const char* what, void (*kernel)(P...), dim3 grid, int threads, size_t smem, cudaStream_t st, const A&... args) {
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = grid;
  cfg.blockDim = dim3((unsigned)threads);
  cfg.dynamicSmemBytes = smem;
  cfg.stream = st;
  cudaLaunchAttribute early;
  early.id = cudaLaunchAttributeProgrammaticStreamSerialization;
  early.val.programmaticStreamSerializationAllowed = 1;
  cfg.attrs = &early;
  cfg.numAttrs = 1;
  const cudaError_t e = cudaLaunchKernelEx(&cfg, kernel, args...);
  if (e != cudaSuccess) {
    cudaGetLastError();
    return fail(MK_ERR_CUDA, std::string(what) + " launch: " + cudaGetErrorString(e));
  }
  return MK_OK;
}

// A kernel's shared memory limit, raised once per device (the call costs about
// as much as a launch).  done: a bit per device of one kernel.
inline int allow_smem(std::atomic<uint64_t>& done, const void* kernel, int bytes, const char* what) {
  int dev = 0;
  cudaError_t e = cudaGetDevice(&dev);
  if (e == cudaSuccess && dev < 64 && (done.load(std::memory_order_relaxed) >> dev & 1)) return MK_OK;
  if (e == cudaSuccess) e = cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, bytes);
  if (e != cudaSuccess) {
    cudaGetLastError();
    return fail(MK_ERR_CUDA, std::string(what) + ": " + cudaGetErrorString(e));
  }
  if (dev < 64) done.fetch_or((uint64_t)1 << dev, std::memory_order_relaxed);
  return MK_OK;
}

inline Pools pools_of(const mk_kv* kv, int32_t layer) {
  const mk_kv_config& c = kv->cfg;
  Pools p;
  p.layer_elems = c.num_pages * c.n_kv * c.page_size * c.head_dim;
  p.k = static_cast<uint16_t*>(c.k_pool) + layer * p.layer_elems;
  p.v = static_cast<uint16_t*>(c.v_pool) + layer * p.layer_elems;
  p.num_pages = c.num_pages;
  p.n_kv = c.n_kv;
  p.page_shift = kv->page_shift;
  p.n_layers = c.n_layers;
  return p;
}

// A sequence's slots (and a tile behind them) are counted in 32 bits.
constexpr int32_t kMaxSlots = 1 << 30;
inline bool table_fits(const mk_kv* kv, int32_t max_pages) { return ((int64_t)max_pages << kv->page_shift) <= kMaxSlots; }

// The checks that append and attention share.
inline int check_tokens(const mk_kv* kv, int32_t layer, const mk_tokens* t) {
  if (!kv || !t) return fail(MK_ERR_ARG, "null argument");
  if (layer < 0 || layer >= kv->cfg.n_layers) return fail(MK_ERR_ARG, "layer outside the pools");
  if (t->batch < 0 || t->n_tokens < 0 || t->max_pages < 1) return fail(MK_ERR_ARG, "negative batch or token count, or no page columns");
  if (!table_fits(kv, t->max_pages)) return fail(MK_ERR_ARG, "block tables of more than 2^30 slots");
  if (t->batch > 0 && (!t->cu_seqlens || !t->cache_lens || !t->block_tables)) return fail(MK_ERR_ARG, "null batch array");
  if (misplaced(t->cu_seqlens, t->cache_lens, t->block_tables, t->positions)) return fail(MK_ERR_ARG, "misaligned batch array");
  return MK_OK;
}

// Whether an array that a call writes lies over the pools, the status record or
// the arrays of the batch.
inline bool over_pools(const mk_kv* kv, const uint32_t* status, const void* p, size_t bytes) {
  const mk_kv_config& c = kv->cfg;
  const size_t pool = (size_t)c.n_layers * c.num_pages * c.n_kv * c.page_size * c.head_dim * 2;
  return overlap(p, bytes, c.k_pool, pool) || overlap(p, bytes, c.v_pool, pool) || overlap(p, bytes, status, 32);
}
inline bool over_batch(const mk_tokens* t, const void* p, size_t bytes) {
  const size_t b = (size_t)t->batch * 4;
  return overlap(p, bytes, t->cu_seqlens, b + 4) || overlap(p, bytes, t->cache_lens, b) ||
         overlap(p, bytes, t->block_tables, b * t->max_pages) || overlap(p, bytes, t->positions, (size_t)t->n_tokens * 4);
}

inline Batch batch_of(const mk_tokens* t) {
  return {t->cu_seqlens, t->cache_lens, t->block_tables, t->positions, t->batch, t->n_tokens, t->max_pages};
}

int encode_pools(mk_kv* kv);  // the handle's tensor maps, once

}  // namespace ops
}  // namespace mk
