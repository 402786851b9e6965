// aq_norm.cu -- aq_qk_norm_rope_backward: the gradient of the head norms with the rotation behind them (their forward is in
// aq_positions.cu, beside the rotation and the cache's write).
//
// With r = 1 / sqrt(mean(x^2) + eps), n = x r, f = offset + w and y = R (n f):
//   g = R^T dy,  dx = r (g f - n mean(g f n)),  dw_i = sum over tokens and heads of g_i n_i.
// Bound by memory: x and dy are read once, dx is written once, and a head needs two sums over its elements. A group of lanes
// holds a head as in the forward, 16 elements a lane. The weight's gradient stays in 16 registers a lane over all
// the heads that the lane sees, so a block is given heads of q alone or of k alone; the groups' sums meet in shared memory, the
// blocks' in the workspace, and a second launch adds those up, all in an order fixed by the sizes.
#include <algorithm>

#include "aq_positions.cuh"

namespace aq {
namespace {

constexpr int kNormThreads = 256, kNormPerSm = 2;

struct NormSet {
  const uint16_t* dy;
  const uint16_t* x;
  uint16_t* dx;
  const uint16_t* w;
  float* part;         // [blocks][D], or NULL
  int64_t dy_tok, dy_head, x_tok, x_head, dx_tok, dx_head;
  int32_t heads, hl_shift;   // log2 of the groups that share a token
  int32_t blocks;
  float eps, offset;
};
struct NormGradParams {
  NormSet set[2];
  const int32_t* pos;
  const uint64_t* freq;   // NULL: no rotation
  int64_t T;
  int32_t D, rot16;
  float magnitude;
};

template <bool HALF, int GW>
__global__ void __launch_bounds__(kNormThreads, kNormPerSm) aq_norm_grad_kernel(const __grid_constant__ NormGradParams p) {
  pdl_wait_prior_grid();
  pdl_launch_dependents();
  constexpr int kGroups = kNormThreads / GW;
  __shared__ float sums[kGroups][GW * 16 + 1];
  const int which = static_cast<int>(blockIdx.x) >= p.set[0].blocks;
  const NormSet& s = p.set[which];
  const int block = static_cast<int>(blockIdx.x) - (which ? p.set[0].blocks : 0);
  const int lane = threadIdx.x & 31, u = threadIdx.x % GW;
  const Chunks<HALF> ch(u, p.rot16, p.D / 16);
  const uint32_t group = (GW == 32 ? 0xffffffffu : (1u << GW) - 1) << (lane & ~(GW - 1));
  const bool mine = u * 16 < p.D;
  const int k0 = mine ? ch.c0 * 8 : 0, k1 = mine ? ch.c1 * 8 : 0;
  const int hl = 1 << s.hl_shift;
  const float inv_dim = 1.0f / p.D;
  float f0[8], f1[8], w0[8], w1[8];
  norm_factor(s.w, k0 / 8, s.offset, f0);
  norm_factor(s.w, k1 / 8, s.offset, f1);
#pragma unroll
  for (int i = 0; i < 8; ++i) w0[i] = w1[i] = 0.0f;

  const int64_t items = p.T << s.hl_shift, step = static_cast<int64_t>(s.blocks) * kGroups;
  // a warp's groups walk together: every lane is there when angles are passed round
  for (int64_t first = static_cast<int64_t>(block) * kGroups + (threadIdx.x / 32) * (32 / GW); first < items; first += step) {
    const int64_t item = first + lane / GW;
    const bool live = item < items && mine;
    const int64_t t = live ? item >> s.hl_shift : 0;
    float c[8], sn[8];
    angles<HALF, GW, false>(ch, u, p.freq, p.freq && live ? p.pos[t] : 0, p.magnitude, -p.magnitude, c, sn);
    const bool turns = p.freq && live && (ch.turns0 || ch.turns1);
    for (int h = static_cast<int>(item & (hl - 1)); h < s.heads; h += hl) {
      const uint16_t* xs = s.x + t * s.x_tok + h * s.x_head;
      const uint16_t* ys = s.dy + t * s.dy_tok + h * s.dy_head;
      const uint4 r0 = ld_stream(xs + k0), r1 = ld_stream(xs + k1), r2 = ld_stream(ys + k0), r3 = ld_stream(ys + k1);
      float a[8], b[8], ga[8], gb[8];
      const uint4 none = make_uint4(0, 0, 0, 0);
      unpack8(live ? r0 : none, a);
      unpack8(live ? r1 : none, b);
      unpack8(live ? r2 : none, ga);
      unpack8(live ? r3 : none, gb);
      if (turns) rotate16<HALF>(ga, gb, c, sn, ch.turns1);
      const float r = head_rstd<GW>(a, b, group, inv_dim, s.eps);
      float dot = 0.0f;
#pragma unroll
      for (int i = 0; i < 8; ++i) {
        a[i] *= r;
        b[i] *= r;
        w0[i] = fmaf(ga[i], a[i], w0[i]);
        w1[i] = fmaf(gb[i], b[i], w1[i]);
        ga[i] *= f0[i];
        gb[i] *= f1[i];
        dot = fmaf(ga[i], a[i], dot);
        dot = fmaf(gb[i], b[i], dot);
      }
#pragma unroll
      for (int o = GW / 2; o > 0; o >>= 1) dot += __shfl_xor_sync(group, dot, o);
      dot *= inv_dim;
#pragma unroll
      for (int i = 0; i < 8; ++i) {
        a[i] = r * fmaf(-a[i], dot, ga[i]);
        b[i] = r * fmaf(-b[i], dot, gb[i]);
      }
      if (live) {
        uint16_t* d = s.dx + t * s.dx_tok + h * s.dx_head;
        *reinterpret_cast<uint4*>(d + k0) = pack8(a);
        *reinterpret_cast<uint4*>(d + k1) = pack8(b);
      }
    }
  }
  if (!s.part) return;
  float* row = sums[threadIdx.x / GW];
  if (mine) {
#pragma unroll
    for (int i = 0; i < 8; ++i) {
      row[k0 + i] = w0[i];
      row[k1 + i] = w1[i];
    }
  }
  __syncthreads();
  for (int d = threadIdx.x; d < p.D; d += kNormThreads) {
    float v = 0.0f;
    for (int i = 0; i < kGroups; ++i) v += sums[i][d];
    s.part[static_cast<int64_t>(block) * p.D + d] = v;
  }
}

// dw = the blocks' sums, 32 elements of one set a block: eight threads an element, each every eighth block.
struct NormJoinParams {
  const float* part[2];
  float* dw[2];
  int32_t blocks[2];
  int32_t D, tiles;    // tiles of 32 elements of a set
};
__global__ void __launch_bounds__(256) aq_norm_join_kernel(const __grid_constant__ NormJoinParams p) {
  pdl_wait_prior_grid();
  pdl_launch_dependents();
  __shared__ float sums[8][33];
  const int which = static_cast<int>(blockIdx.x) / p.tiles, d = (static_cast<int>(blockIdx.x) % p.tiles) * 32 + (threadIdx.x & 31);
  const int part = threadIdx.x / 32;
  if (!p.dw[which]) return;
  float v = 0.0f;
  if (d < p.D) {
#pragma unroll 8
    for (int i = part; i < p.blocks[which]; i += 8) v += p.part[which][static_cast<int64_t>(i) * p.D + d];
  }
  sums[part][threadIdx.x & 31] = v;
  __syncthreads();
  if (part == 0 && d < p.D) {
    for (int i = 1; i < 8; ++i) v += sums[i][threadIdx.x];
    p.dw[which][d] = v;
  }
}

// Blocks of the two sets: what fills the GPU, shared out by their heads; no more than their groups of work.
void norm_blocks(int64_t T, int32_t D, int32_t hq, int32_t hk, int sms, int32_t* hl_shift, int32_t* blocks) {
  const int gw = group_width(D), groups = kNormThreads / gw, heads[2] = {hq, hk};
  const int fill = sms * kNormPerSm;
  for (int i = 0; i < 2; ++i) {
    hl_shift[i] = 0;
    blocks[i] = 0;
    if (!heads[i]) continue;
    // groups that share a token: a warp's, more while the call does not fill the GPU, and never more than heads
    int most = 0;
    while ((2 << most) <= heads[i] && (2 << most) <= groups) ++most;
    hl_shift[i] = std::min(log2_of(32 / gw), most);
    while (hl_shift[i] < most && (T << hl_shift[i]) < static_cast<int64_t>(fill) * groups / 2) ++hl_shift[i];
    const int64_t need = ((T << hl_shift[i]) + groups - 1) / groups;
    const int64_t share = std::max<int64_t>(1, static_cast<int64_t>(fill) * heads[i] / (hq + hk));
    blocks[i] = static_cast<int32_t>(std::min(need, share));
  }
}
constexpr int kNormSmsBound = 256;   // SMs that the workspace's size allows for

template <bool HALF>
cudaError_t launch_norm_grad(const NormGradParams& p, int gw, cudaStream_t st) {
  const unsigned grid = static_cast<unsigned>(p.set[0].blocks + p.set[1].blocks);
  switch (gw) {
    case 1: return launch_serve(aq_norm_grad_kernel<HALF, 1>, p, grid, kNormThreads, 0, st);
    case 2: return launch_serve(aq_norm_grad_kernel<HALF, 2>, p, grid, kNormThreads, 0, st);
    case 4: return launch_serve(aq_norm_grad_kernel<HALF, 4>, p, grid, kNormThreads, 0, st);
    case 8: return launch_serve(aq_norm_grad_kernel<HALF, 8>, p, grid, kNormThreads, 0, st);
    default: return launch_serve(aq_norm_grad_kernel<HALF, 16>, p, grid, kNormThreads, 0, st);
  }
}

}  // namespace
}  // namespace aq

using namespace aq;

extern "C" size_t aq_qk_norm_rope_backward_workspace_bytes(int64_t T, int32_t head_dim, int32_t q_heads, int32_t k_heads) {
  if (T < 0 || head_dim < 16 || head_dim % 16 || head_dim > kServeMaxHeadDim || q_heads < 1 || k_heads < 0) {
    serve_fail(AQ_ERR_INVALID_ARG, "aq_qk_norm_rope_backward_workspace_bytes: invalid arguments");
    return static_cast<size_t>(-1);
  }
  // at most kNormPerSm blocks an SM, one more where both sets are there
  return (static_cast<size_t>(kNormSmsBound) * kNormPerSm + 1) * head_dim * sizeof(float);
}

extern "C" aq_status aq_qk_norm_rope_backward(const aq_head_norm* q_norm, const aq_head_norm* k_norm, const aq_rope_spec* rope,
                                              const int32_t* pos, int64_t T, int32_t head_dim, const aq_heads* dq_out, const aq_heads* q,
                                              const aq_heads* dq, float* dq_weight, const aq_heads* dk_out, const aq_heads* k,
                                              const aq_heads* dk, float* dk_weight, void* workspace, size_t workspace_bytes, void* stream) {
  const char* who = "aq_qk_norm_rope_backward";
  const int D = head_dim;
  if (T < 0) return serve_fail(AQ_ERR_SHAPE, "%s: T=%lld is negative", who, (long long)T);
  if (D < 16 || D % 16 || D > kServeMaxHeadDim)
    return serve_fail(AQ_ERR_SHAPE, "%s: head_dim=%d must be a multiple of 16 up to %d", who, D, kServeMaxHeadDim);
  if (!q_norm || !dq_out || !q || !dq) return serve_fail(AQ_ERR_INVALID_ARG, "%s: q_norm, dq_out, q and dq must be non-NULL", who);
  if (!k != !dk_out || !k != !dk || !k != !k_norm || (!k && dk_weight))
    return serve_fail(AQ_ERR_INVALID_ARG, "%s: k_norm, dk_out, k and dk go together", who);
  aq_status st;
  if (rope && (st = check_rope_spec(rope, D, who)) != AQ_OK) return st;
  if ((st = check_head_norm(q_norm, "q_norm", who)) != AQ_OK || (st = check_head_norm(k_norm, "k_norm", who)) != AQ_OK) return st;
  const aq_head_norm* const norm[2] = {q_norm, k_norm};
  const aq_heads* const set[2][3] = {{dq_out, q, dq}, {dk_out, k, dk}};
  const char* const names[2][3] = {{"dq_out", "q", "dq"}, {"dk_out", "k", "dk"}};
  float* const dw[2] = {dq_weight, dk_weight};
  const int sets = k ? 2 : 1;
  for (int i = 0; i < sets; ++i) {
    if (dw[i] && !norm[i]->weight) return serve_fail(AQ_ERR_INVALID_ARG, "%s: a gradient of a weight that is not there", who);
    if (!serve_aligned(dw[i], 4)) return serve_fail(AQ_ERR_ALIGNMENT, "%s: the weights' gradients must be 4-byte aligned", who);
    for (int j = 0; j < 3; ++j)
      if (set[i][j]->heads < 1 || set[i][j]->heads != set[i][0]->heads)
        return serve_fail(AQ_ERR_SHAPE, "%s: heads of %s, %s and %s must be >= 1 and equal", who, names[i][0], names[i][1], names[i][2]);
  }
  const cudaStream_t cs = static_cast<cudaStream_t>(stream);
  if (T == 0) {
    for (int i = 0; i < sets; ++i)
      if (dw[i]) {
        const cudaError_t e = cudaMemsetAsync(dw[i], 0, D * sizeof(float), cs);
        if (e != cudaSuccess) return serve_launched(e, who);
      }
    return AQ_OK;
  }
  if (rope && !pos) return serve_fail(AQ_ERR_INVALID_ARG, "%s: rope needs pos", who);
  for (int i = 0; i < sets; ++i) {
    for (int j = 0; j < 3; ++j)
      if ((st = check_heads(set[i][j]->data, set[i][j]->tok, set[i][j]->head, set[i][j]->heads, D, names[i][j], who)) != AQ_OK) return st;
    if ((st = check_out_heads(dq->tok, dq->head, T, dq->heads, D, "dq", who)) != AQ_OK) return st;
    if (k && (st = check_out_heads(dk->tok, dk->head, T, dk->heads, D, "dk", who)) != AQ_OK) return st;
  }
  const bool sums = dw[0] || dw[1];
  const size_t need = aq_qk_norm_rope_backward_workspace_bytes(T, D, q->heads, k ? k->heads : 0);
  if (sums) {
    if (!workspace) return serve_fail(AQ_ERR_INVALID_ARG, "%s: workspace is NULL", who);
    if (workspace_bytes < need) return serve_fail(AQ_ERR_WORKSPACE, "%s: workspace of %zu bytes < %zu", who, workspace_bytes, need);
    if (!serve_aligned(workspace, 16)) return serve_fail(AQ_ERR_ALIGNMENT, "%s: workspace must be 16-byte aligned", who);
  }
  const int64_t wbytes = D * 2, gbytes = D * 4;
  const ByteRows outs[] = {heads_rows(dq, T, D), heads_rows(dk, T, D), ByteRows(dw[0], 1, gbytes, gbytes), ByteRows(dw[1], 1, gbytes, gbytes),
                           ByteRows(sums ? workspace : nullptr, 1, static_cast<int64_t>(need), static_cast<int64_t>(need))};
  const ByteRows ins[] = {heads_rows(dq_out, T, D), heads_rows(dk_out, T, D), heads_rows(q, T, D), heads_rows(k, T, D),
                          ByteRows(q_norm->weight, 1, wbytes, wbytes), ByteRows(k ? k_norm->weight : nullptr, 1, wbytes, wbytes),
                          ByteRows(rope ? pos : nullptr, 1, T * 4, T * 4), ByteRows(rope ? rope->freq : nullptr, 1, D * 4, rope ? rope->rotary_dim * 4 : 0)};
  for (int i = 0; i < 5; ++i) {
    for (int j = 0; j < 8; ++j) {
      const bool same = i < 2 && i == j && i < sets && set[i][0]->data == set[i][2]->data && (T == 1 || set[i][0]->tok == set[i][2]->tok) &&
                        (set[i][0]->heads == 1 || set[i][0]->head == set[i][2]->head);
      if (!same && outs[i].meets(ins[j])) return serve_fail(AQ_ERR_OVERLAP, "%s: an output overlaps an input", who);
    }
    for (int j = 0; j < i; ++j)
      if (outs[i].meets(outs[j])) return serve_fail(AQ_ERR_OVERLAP, "%s: two outputs overlap", who);
  }
  ServeDev dev;
  if ((st = serve_device(&dev)) != AQ_OK) return st;
  NormGradParams p = {};
  int32_t hl[2], blocks[2];
  norm_blocks(T, D, q->heads, k ? k->heads : 0, std::min(dev.sms, kNormSmsBound), hl, blocks);
  float* part = static_cast<float*>(workspace);
  for (int i = 0; i < sets; ++i) {
    NormSet& s = p.set[i];
    s.dy = static_cast<const uint16_t*>(set[i][0]->data);
    s.dy_tok = set[i][0]->tok;
    s.dy_head = set[i][0]->head;
    s.x = static_cast<const uint16_t*>(set[i][1]->data);
    s.x_tok = set[i][1]->tok;
    s.x_head = set[i][1]->head;
    s.dx = static_cast<uint16_t*>(set[i][2]->data);
    s.dx_tok = set[i][2]->tok;
    s.dx_head = set[i][2]->head;
    s.w = static_cast<const uint16_t*>(norm[i]->weight);
    s.heads = set[i][0]->heads;
    s.hl_shift = hl[i];
    s.blocks = blocks[i];
    s.eps = norm[i]->eps;
    s.offset = norm[i]->offset;
    if (dw[i]) s.part = part + (i ? static_cast<int64_t>(blocks[0]) * D : 0);
  }
  p.T = T;
  p.D = D;
  if (rope) {
    p.pos = pos;
    p.freq = rope->freq;
    p.rot16 = rope->rotary_dim / 16;
    p.magnitude = rope->magnitude;
  }
  const cudaError_t e = rope && rope->layout == AQ_ROPE_HALF ? launch_norm_grad<true>(p, group_width(D), cs) : launch_norm_grad<false>(p, group_width(D), cs);
  if (e != cudaSuccess || !sums) return serve_launched(e, who);
  NormJoinParams j = {};
  for (int i = 0; i < sets; ++i) {
    j.part[i] = p.set[i].part;
    j.dw[i] = dw[i];
    j.blocks[i] = blocks[i];
  }
  j.D = D;
  j.tiles = (D + 31) / 32;
  return serve_launched(launch_serve(aq_norm_join_kernel, j, dim3(static_cast<unsigned>(sets * j.tiles)), 256, 0, cs), who);
}
