// aq_attention.cu -- aq_tree_attention: attention of each sequence's newest (drafted) tokens over its
// paged cache.
//   o_i = sum_j p_ij v_j,  p_i = softmax over the visible j of scale * (q_i . k_j)
// One pass over the keys with the running maximum m and sum l of the softmax: on a larger maximum the
// sums so far are scaled by exp(m_old - m_new).
#include <math.h>

#include <algorithm>

#include "aq_serve.h"

namespace aq {
namespace {

struct AttnParams {
  const uint8_t* kc;
  const uint8_t* vc;
  const float* ks;
  const float* vs;
  int32_t pages, page_shift, hk, group;
  const uint16_t* q;
  int64_t q_tok, q_head;
  uint16_t* o;
  int64_t o_tok, o_head;
  float* lse;
  const int32_t* cu;
  const int32_t* ctx;
  const int32_t* table;
  int64_t ld_table;
  int32_t pages_per_seq;
  const uint64_t* mask;
  int64_t ld_mask;
  const int32_t* depth;
  int32_t batch, max_q, window;
  int64_t total_q;
  float scale;
};

// One block per row and query head; each of four warps takes every fourth key, its lanes the elements.
template <int D, bool E4M3>
__global__ void __launch_bounds__(128) aq_tree_attention_kernel(const __grid_constant__ AttnParams p) {
  constexpr int N = D / 32;
  __shared__ float sm[4], sl[4], so[4][D];
  pdl_wait_prior_grid();
  pdl_launch_dependents();
  const int lane = threadIdx.x & 31, w = threadIdx.x >> 5;
  const int64_t row = blockIdx.x;
  const int h = blockIdx.y, kh = h / p.group;
  int b = 0;
  while (b < p.batch && !(p.cu[b] <= row && row < p.cu[b + 1])) ++b;
  if (b == p.batch) return;
  const int64_t first = p.cu[b];
  const int i = static_cast<int>(row - first);
  if (first < 0 || i >= p.max_q) return;
  const int T = static_cast<int>(min(static_cast<int64_t>(min(p.cu[b + 1], static_cast<int32_t>(p.total_q))) - first, static_cast<int64_t>(p.max_q)));
  const int ctx = max(p.ctx[b], 0);
  const bool dep = p.mask && p.depth;
  const int64_t pos = static_cast<int64_t>(ctx) + (dep ? p.depth[row] : i);
  float q[N], o[N], m = -INFINITY, l = 0.0f;
  for (int e = 0; e < N; ++e) {
    q[e] = bf16_to_f32(p.q[row * p.q_tok + h * p.q_head + lane * N + e]);
    o[e] = 0.0f;
  }
  for (int64_t j = w; j < static_cast<int64_t>(ctx) + T; j += 4) {
    const int t = static_cast<int>(j - ctx);
    bool seen = true;
    if (t >= 0) seen = p.mask ? (p.mask[row * p.ld_mask + t / 64] >> (t & 63)) & 1 : t <= i;
    if (p.window > 0) {
      const int64_t at = t < 0 ? j : static_cast<int64_t>(ctx) + (dep ? p.depth[first + t] : t);
      seen = seen && pos - at < p.window;
    }
    const int64_t pg = j >> p.page_shift;
    if (!seen || pg >= p.pages_per_seq) continue;
    const int page = p.table[b * p.ld_table + pg];
    if (page < 0 || page >= p.pages) continue;
    const int64_t cell = ((static_cast<int64_t>(page) * p.hk + kh) << p.page_shift) + (j & ((1 << p.page_shift) - 1));
    float k[N], v[N], s = 0.0f;
    for (int e = 0; e < N; ++e) {
      const int64_t at = cell * D + lane * N + e;
      if (E4M3) {
        const uint32_t kk = f16x2_from_e4m3x2(p.kc[at]), vv = f16x2_from_e4m3x2(p.vc[at]);
        k[e] = __low2float(*reinterpret_cast<const __half2*>(&kk)) * p.ks[cell];
        v[e] = __low2float(*reinterpret_cast<const __half2*>(&vv)) * p.vs[cell];
      } else {
        k[e] = bf16_to_f32(reinterpret_cast<const uint16_t*>(p.kc)[at]);
        v[e] = bf16_to_f32(reinterpret_cast<const uint16_t*>(p.vc)[at]);
      }
      s = fmaf(q[e], k[e], s);
    }
    for (int off = 16; off; off >>= 1) s += __shfl_xor_sync(0xffffffffu, s, off);
    s *= p.scale;
    if (s == -INFINITY) continue;
    const float mn = fmaxf(m, s), f = m == -INFINITY ? 0.0f : expf(m - mn), x = expf(s - mn);
    for (int e = 0; e < N; ++e) o[e] = o[e] * f + x * v[e];
    l = l * f + x;
    m = mn;
    if (isnan(s)) l = s;
  }
  for (int e = 0; e < N; ++e) so[w][lane * N + e] = o[e];
  if (lane == 0) {
    sm[w] = m;
    sl[w] = l;
  }
  __syncthreads();
  float mt = -INFINITY, lt = 0.0f;
  for (int k = 0; k < 4; ++k) mt = fmaxf(mt, sm[k]);
  for (int k = 0; k < 4; ++k) lt += sm[k] == -INFINITY ? 0.0f : sl[k] * expf(sm[k] - mt);
  for (int d = threadIdx.x; d < D; d += 128) {
    float x = 0.0f;
    for (int k = 0; k < 4; ++k) x += sm[k] == -INFINITY ? 0.0f : so[k][d] * expf(sm[k] - mt);
    p.o[row * p.o_tok + h * p.o_head + d] = f32_to_bf16_rn(mt == -INFINITY ? 0.0f : x / lt);
  }
  if (p.lse && threadIdx.x == 0) p.lse[row * (p.hk * p.group) + h] = mt == -INFINITY ? -INFINITY : mt + logf(lt);
}

template <int D>
cudaError_t launch_attention(const AttnParams& p, bool e4m3, dim3 grid, cudaStream_t st) {
  return e4m3 ? launch_serve(aq_tree_attention_kernel<D, true>, p, grid, 128, 0, st)
              : launch_serve(aq_tree_attention_kernel<D, false>, p, grid, 128, 0, st);
}

aq_status check_batch(const aq_kv_cache* c, const aq_draft_batch* d, int32_t q_heads, const char* who) {
  aq_status st = check_kv_cache(c, who);
  if (st != AQ_OK) return st;
  if (!d) return serve_fail(AQ_ERR_INVALID_ARG, "%s: batch is NULL", who);
  if (c->head_dim != 64 && c->head_dim != 128 && c->head_dim != 256)
    return serve_fail(AQ_ERR_UNSUPPORTED, "%s: head_dim=%d is not 64, 128 or 256", who, c->head_dim);
  if (q_heads < 1 || q_heads % c->kv_heads)
    return serve_fail(AQ_ERR_SHAPE, "%s: q_heads=%d must be a multiple of kv_heads=%d", who, q_heads, c->kv_heads);
  if (d->batch < 0 || d->max_q < 0 || d->total_q < 0 || d->total_q > 0x7fffffffLL || d->pages_per_seq < 0)
    return serve_fail(AQ_ERR_SHAPE, "%s: batch=%d max_q=%d total_q=%lld pages_per_seq=%d out of range", who, d->batch,
                      d->max_q, (long long)d->total_q, d->pages_per_seq);
  if (d->window < 0) return serve_fail(AQ_ERR_INVALID_ARG, "%s: window=%d is negative", who, d->window);
  return AQ_OK;
}

}  // namespace
}  // namespace aq

using namespace aq;

extern "C" size_t aq_tree_attention_workspace_bytes(const aq_kv_cache* cache, const aq_draft_batch* batch, int32_t q_heads) {
  if (check_batch(cache, batch, q_heads, "aq_tree_attention_workspace_bytes") != AQ_OK) return static_cast<size_t>(-1);
  return 0;
}

extern "C" aq_status aq_tree_attention(const aq_kv_cache* cache, const aq_draft_batch* batch, const void* q,
                                       int32_t q_heads, int64_t q_tok, int64_t q_head, float scale, void* o, int64_t o_tok,
                                       int64_t o_head, float* lse, void* workspace, size_t workspace_bytes, void* stream) {
  const char* who = "aq_tree_attention";
  aq_status st = check_batch(cache, batch, q_heads, who);
  if (st != AQ_OK) return st;
  const int D = cache->head_dim;
  const aq_draft_batch& d = *batch;
  if (d.batch == 0 || d.total_q == 0 || d.max_q == 0) return AQ_OK;
  if (!d.cu_q || !d.ctx || !q || !o || (d.pages_per_seq > 0 && !d.page_table))
    return serve_fail(AQ_ERR_INVALID_ARG, "%s: NULL argument", who);
  if (d.pages_per_seq > 0 && d.ld_table < d.pages_per_seq)
    return serve_fail(AQ_ERR_SHAPE, "%s: ld_table=%lld < pages_per_seq=%d", who, (long long)d.ld_table, d.pages_per_seq);
  if (d.mask && d.ld_mask < (static_cast<int64_t>(d.max_q) + 63) / 64)
    return serve_fail(AQ_ERR_SHAPE, "%s: ld_mask=%lld holds no %d bits", who, (long long)d.ld_mask, d.max_q);
  if (!serve_aligned(d.cu_q, 4) || !serve_aligned(d.ctx, 4) || !serve_aligned(d.page_table, 4) || !serve_aligned(d.depth, 4) ||
      !serve_aligned(d.mask, 8) || !serve_aligned(lse, 4))
    return serve_fail(AQ_ERR_ALIGNMENT, "%s: index arrays, mask and lse must be aligned to their elements", who);
  const int64_t nq = d.total_q;
  auto heads = [&](const void* x, int64_t tok, int64_t head, const char* name) {
    if (!serve_aligned(x, 16) || tok % 8 || head % 8)
      return serve_fail(AQ_ERR_ALIGNMENT, "%s: %s must be 16-byte aligned with strides that are multiples of 8", who, name);
    const bool tok_outer = nq <= 1 || tok >= (q_heads - 1) * head + D;
    const bool head_outer = q_heads <= 1 || head >= (nq - 1) * tok + D;
    if ((q_heads > 1 && head < D) || (nq > 1 && tok < D) || (!tok_outer && !head_outer))
      return serve_fail(AQ_ERR_SHAPE, "%s: %s strides (token %lld, head %lld) do not hold heads of %d", who, name,
                        (long long)tok, (long long)head, D);
    return AQ_OK;
  };
  if ((st = heads(q, q_tok, q_head, "q")) != AQ_OK || (st = heads(o, o_tok, o_head, "o")) != AQ_OK) return st;
  const ByteSpan outs[] = {byte_span(o, 1, 0, (nq - 1) * o_tok + (q_heads - 1) * o_head + D, 2),
                           byte_span(lse, 1, 0, nq * q_heads, 4)};
  const ByteSpan ins[] = {byte_span(q, 1, 0, (nq - 1) * q_tok + (q_heads - 1) * q_head + D, 2),
                          byte_span(cache->k, 1, 0, kv_cells(cache) * D, kv_elem_bytes(cache)),
                          byte_span(cache->v, 1, 0, kv_cells(cache) * D, kv_elem_bytes(cache)),
                          byte_span(cache->k_scale, 1, 0, kv_cells(cache), 4),
                          byte_span(cache->v_scale, 1, 0, kv_cells(cache), 4),
                          byte_span(d.cu_q, 1, 0, d.batch + 1, 4),
                          byte_span(d.ctx, 1, 0, d.batch, 4),
                          byte_span(d.page_table, d.batch, d.ld_table, d.pages_per_seq, 4),
                          byte_span(d.mask, nq, d.ld_mask, (d.max_q + 63) / 64, 8),
                          byte_span(d.depth, 1, 0, nq, 4)};
  for (int i = 0; i < 2; ++i)
    for (const ByteSpan& in : ins)
      if (byte_overlap(outs[i], in)) return serve_fail(AQ_ERR_OVERLAP, "%s: an output overlaps an input", who);
  if (byte_overlap(outs[0], outs[1])) return serve_fail(AQ_ERR_OVERLAP, "%s: o and lse overlap", who);
  (void)workspace;
  (void)workspace_bytes;
  ServeDev dev;
  if ((st = serve_device(&dev)) != AQ_OK) return st;
  AttnParams p = {};
  p.kc = static_cast<const uint8_t*>(cache->k);
  p.vc = static_cast<const uint8_t*>(cache->v);
  p.ks = cache->k_scale;
  p.vs = cache->v_scale;
  p.pages = cache->pages;
  while ((1 << p.page_shift) < cache->page_size) ++p.page_shift;
  p.hk = cache->kv_heads;
  p.group = q_heads / cache->kv_heads;
  p.q = static_cast<const uint16_t*>(q);
  p.q_tok = q_tok;
  p.q_head = q_head;
  p.o = static_cast<uint16_t*>(o);
  p.o_tok = o_tok;
  p.o_head = o_head;
  p.lse = lse;
  p.cu = d.cu_q;
  p.ctx = d.ctx;
  p.table = d.page_table;
  p.ld_table = d.ld_table;
  p.pages_per_seq = d.pages_per_seq;
  p.mask = d.mask;
  p.ld_mask = d.ld_mask;
  p.depth = d.depth;
  p.batch = d.batch;
  p.max_q = d.max_q;
  p.window = d.window;
  p.total_q = nq;
  p.scale = scale;
  const dim3 grid(static_cast<unsigned>(nq), q_heads);
  const bool e4m3 = cache->type == AQ_KV_E4M3;
  const cudaStream_t cs = static_cast<cudaStream_t>(stream);
  const cudaError_t e = D == 64    ? launch_attention<64>(p, e4m3, grid, cs)
                        : D == 128 ? launch_attention<128>(p, e4m3, grid, cs)
                                   : launch_attention<256>(p, e4m3, grid, cs);
  return serve_launched(e, who);
}
