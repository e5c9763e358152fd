// mk_tree_attn.cu -- attention of new tokens (a drafted tree, or a run) over
// the paged pools.
#include <cmath>

#include "mk_ops_common.cuh"

namespace mk {
namespace ops {
namespace {

struct AttnArgs {
  Pools pools;
  Batch b;
  const uint16_t* q;
  uint16_t* out;
  float* lse;
  const uint64_t* mask;
  int64_t q_stride, out_stride;
  int32_t n_q, group, mask_words, window;
  float scale;
  uint32_t* status;
};

constexpr int kThreads = 128;

// One block per (token, query head): each warp takes every fourth slot, a lane
// D / 32 elements of the head.
template <int D>
__global__ void __launch_bounds__(kThreads) attn_simple(const __grid_constant__ AttnArgs a) {
  constexpr int E = D / 32;
  __shared__ int found;
  __shared__ float sm[4], sl[4], so[4][D];
  const int t = blockIdx.x, h = blockIdx.y, tid = threadIdx.x, lane = tid % 32, warp = tid / 32;
  if (tid == 0) found = -1;
  __syncthreads();
  for (int b = tid; b < a.b.batch; b += kThreads)
    if (a.b.cu[b] <= t && t < a.b.cu[b + 1]) found = b;
  __syncthreads();
  const int b = found;
  if (b < 0) return;
  Seq s = seq_of(a.b, b, a.pools.page_shift, a.status, OP_ATTN);
  if (a.mask && s.n > 64 * a.mask_words) {
    record(a.status, dev::ERR_RANGE, OP_ATTN, b, 2, s.n, 64 * a.mask_words);
    s.n = 0;
  }
  if (s.n == 0) return;
  const int i = t - s.t0, g = h / a.group, P = 1 << a.pools.page_shift;
  auto position = [&](int j) {
    const int slot = s.ctx + j;
    if (!a.b.positions) return slot;
    const int p = a.b.positions[s.t0 + j];
    if (p < s.ctx || p >= s.ctx + s.n) {
      if (a.window) record(a.status, dev::ERR_RANGE, OP_ATTN, b, 3, p, s.ctx + s.n);
      return p < s.ctx ? s.ctx : s.ctx + s.n - 1;
    }
    return p;
  };
  const int pos = a.window ? position(i) : 0;
  float q[E], o[E] = {}, m = -INFINITY, l = 0;
  for (int e = 0; e < E; ++e)
    q[e] = a.scale * __uint_as_float((uint32_t)a.q[t * a.q_stride + h * D + lane * E + e] << 16);
  const int end = s.ctx + s.n;
  for (int slot = warp; slot < end; slot += 4) {
    const int j = slot - s.ctx;
    bool see = true;
    if (j >= 0) see = a.mask ? (a.mask[(int64_t)t * a.mask_words + j / 64] >> (j % 64)) & 1 : j <= i;
    if (a.window) see = see && pos - (j >= 0 ? position(j) : slot) < a.window;
    if (!see) continue;
    int64_t page = a.b.tables[(int64_t)b * a.b.max_pages + (slot >> a.pools.page_shift)];
    if (page < 0 || page >= a.pools.num_pages) {
      record(a.status, dev::ERR_PAGE, OP_ATTN, b, slot, (uint32_t)page, (uint32_t)a.pools.num_pages);
      page = 0;
    }
    const int64_t row = ((page * a.pools.n_kv + g) << a.pools.page_shift) + (slot & (P - 1));
    float d = 0;
    for (int e = 0; e < E; ++e) d += q[e] * __uint_as_float((uint32_t)a.pools.k[row * D + lane * E + e] << 16);
    for (int x = 16; x > 0; x >>= 1) d += __shfl_xor_sync(0xffffffffu, d, x);
    const float mn = fmaxf(m, d), z = mn == -INFINITY ? 0.0f : mn;
    const float c = expf(m - z), p = expf(d - z);
    l = l * c + p;
    for (int e = 0; e < E; ++e)
      o[e] = o[e] * c + p * __uint_as_float((uint32_t)a.pools.v[row * D + lane * E + e] << 16);
    m = mn;
  }
  if (lane == 0) sm[warp] = m, sl[warp] = l;
  for (int e = 0; e < E; ++e) so[warp][lane * E + e] = o[e];
  __syncthreads();
  float M = fmaxf(fmaxf(sm[0], sm[1]), fmaxf(sm[2], sm[3])), L = 0;
  const float z = M == -INFINITY ? 0.0f : M;
  for (int w = 0; w < 4; ++w) L += sl[w] * expf(sm[w] - z);
  for (int e = tid; e < D; e += kThreads) {
    float x = 0;
    for (int w = 0; w < 4; ++w) x += so[w][e] * expf(sm[w] - z);
    uint32_t r;
    asm("cvt.rn.bf16x2.f32 %0, %1, %2;" : "=r"(r) : "f"(0.0f), "f"(L == 0 ? 0.0f : x / L));
    a.out[t * a.out_stride + h * D + e] = (uint16_t)r;
  }
  if (a.lse && tid == 0) a.lse[(int64_t)t * a.n_q + h] = M + logf(L);
}

}  // namespace
}  // namespace ops
}  // namespace mk

using mk::fail;
using namespace mk::ops;

extern "C" {

size_t mk_tree_attn_workspace_bytes(const mk_kv* kv) {
  if (!kv || mk::query_num_sms() < 1) return 0;
  return 16;
}

int mk_tree_attn(mk_kv* kv, int32_t layer, const mk_tokens* tok, const mk_attn_io* io, void* workspace,
                 size_t workspace_bytes, uint32_t* status, void* stream) {
  int rc = check_tokens(kv, layer, tok);
  if (rc != MK_OK) return rc;
  const mk_kv_config& c = kv->cfg;
  if (!io || !io->q || !io->out) return fail(MK_ERR_ARG, "null q or out");
  if (io->n_q < c.n_kv || io->n_q % c.n_kv != 0 || io->n_q > (1 << 16)) return fail(MK_ERR_ARG, "n_q must be a multiple of n_kv");
  const int64_t row = (int64_t)io->n_q * c.head_dim;
  if (misaligned(io->q) || misaligned(io->out) || io->q_stride < row || io->out_stride < row || io->q_stride % 8 ||
      io->out_stride % 8)
    return fail(MK_ERR_ARG, "misaligned q or out, or a stride that is too small or no multiple of 16 bytes");
  if (overlap(io->out, span(tok->n_tokens, io->out_stride, row, 2), io->q, span(tok->n_tokens, io->q_stride, row, 2)))
    return fail(MK_ERR_ARG, "out overlaps q");
  if (io->tree_mask ? io->mask_words < 1 : io->mask_words != 0)
    return fail(MK_ERR_ARG, "mask_words must be positive with a tree_mask and 0 without");
  if (io->window < 0) return fail(MK_ERR_ARG, "negative window");
  if (!(io->scale >= 0) || !std::isfinite(io->scale)) return fail(MK_ERR_ARG, "scale must be positive (0: 1 / sqrt(head_dim))");
  if (!workspace || misaligned(workspace)) return fail(MK_ERR_ARG, "workspace null or misaligned");
  if (tok->batch == 0 || tok->n_tokens == 0) return MK_OK;
  const size_t need = mk_tree_attn_workspace_bytes(kv);
  if (need == 0) return fail(MK_ERR_CUDA, "no device");
  if (workspace_bytes < need) return fail(MK_ERR_ARG, "workspace smaller than mk_tree_attn_workspace_bytes");
  AttnArgs a;
  a.pools = pools_of(kv, layer);
  a.b = batch_of(tok);
  a.q = static_cast<const uint16_t*>(io->q), a.out = static_cast<uint16_t*>(io->out), a.lse = io->lse;
  a.mask = io->tree_mask;
  a.q_stride = io->q_stride, a.out_stride = io->out_stride;
  a.n_q = io->n_q, a.group = io->n_q / c.n_kv, a.mask_words = io->mask_words, a.window = io->window;
  a.scale = io->scale > 0 ? io->scale : 1.0f / std::sqrt((float)c.head_dim);
  a.status = status;
  const dim3 grid((unsigned)tok->n_tokens, (unsigned)io->n_q);
  if (c.head_dim == 128)
    attn_simple<128><<<grid, kThreads, 0, static_cast<cudaStream_t>(stream)>>>(a);
  else
    attn_simple<64><<<grid, kThreads, 0, static_cast<cudaStream_t>(stream)>>>(a);
  return launched("tree_attn");
}

}  // extern "C"
