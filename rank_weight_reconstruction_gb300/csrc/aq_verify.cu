// aq_verify.cu -- aq_verify_drafts: speculative sampling's accept / reject walk over a chain or a tree
// of drafted tokens, and the draw of the token after it.
//
// Walk: at a node with target probabilities r = p[row], its children are tried in index order; child c
// with token x is accepted when u_c q(x) < r(x), else r <- max(r - q, 0) / sum(max(r - q, 0)) (q a point
// mass where the drafts were taken for certain: r(x) <- 0, and with the removed mass s the test reads
// u (1 - s) < p(x), so nothing is summed). The draw is an exponential race: argmax r(v) / E(v) with E ~
// Exp(1) given has P(v) = r(v) / sum r whatever r's scale, so the last residual needs no normaliser, the
// result does not hang on an order of summation, and one pass over the vocabulary is enough.
//
// Bound by memory: one row of p (and of q after a refusal) and of the noise per sequence, 12 bytes a word
// of the vocabulary in fp32. A thread-block cluster takes one sequence: every CTA makes the (short) walk by
// itself from the same few gathered values, passes over its slices of the vocabulary, and the CTAs exchange
// their maxima (packed value and index, so the order does not matter and the lowest index wins) through
// distributed shared memory: one launch, no workspace. Measured on 262144 words: one sequence of 5 in fp32 7.6 us, 48
// with sampled drafts 25.3 us (5970 GB/s); 48 trees of 12 in bf16 20.7 us (3650 GB/s: there the walk and the exchange, about
// 8 us, weigh as much as the 75 MB). Only a refused child that has siblings left, with
// q given, needs a normaliser in between: one more pass, its partial sums added in rank order by every CTA.
#include <atomic>
#include <type_traits>

#include "aq_serve.h"

namespace aq {
namespace {

// Three CTAs of 256 threads an SM (80 registers: with four, the rows of q spill: 61 us for 48 sequences against 41 at the
// time). CTAs of 1024 threads take one to four sequences no faster (7.6 and 8.1 us against 7.6 and 8.0 on 262144 words of
// fp32 p) and eight slower (15.1 against 8.7): as few such clusters fit at once.
constexpr int kVerThreads = 256, kVerPerSm = 3;
constexpr int kVerMaxCluster = 16;

struct VerifyParams {
  const int32_t* cu;
  const int32_t* tokens;
  const int32_t* parent;
  const void* p;
  const void* q;
  const float* u;
  const float* noise;
  int64_t ld_p, ld_q, ld_noise, ld_path;
  int64_t nodes, rows;
  int32_t* n_accepted;
  int32_t* path;
  int32_t* token;
  int32_t vocab, max_nodes, path_cap, cluster, device;
};

__device__ __forceinline__ float prob(const float* p, int64_t i) { return p[i]; }
__device__ __forceinline__ float prob(const uint16_t* p, int64_t i) { return bf16_to_f32(p[i]); }

// r(v) after `k` refusals with the row q: the normalisers zinv[0 .. norm) applied.
__device__ __forceinline__ float residual(float w, float q, int k, int norm, const float* zinv) {
  for (int j = 0; j < k; ++j) {
    w = fmaxf(w - q, 0.0f);
    if (j < norm) w *= zinv[j];
  }
  return w;
}

template <typename T, int N>
struct Vec;
template <>
struct Vec<float, 4> {
  float x[4];
  __device__ __forceinline__ void load(const float* p) {
    const float4 r = __ldg(reinterpret_cast<const float4*>(p));
    x[0] = r.x; x[1] = r.y; x[2] = r.z; x[3] = r.w;
  }
};
template <>
struct Vec<uint16_t, 8> {
  float x[8];
  __device__ __forceinline__ void load(const uint16_t* p) {
    const uint4 r = __ldg(reinterpret_cast<const uint4*>(p));
    const uint32_t w[4] = {r.x, r.y, r.z, r.w};
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      x[2 * i] = __uint_as_float(w[i] << 16);
      x[2 * i + 1] = __uint_as_float(w[i] & 0xffff0000u);
    }
  }
};
template <>
struct Vec<float, 8> {
  float x[8];
  __device__ __forceinline__ void load(const float* p) {
    const float4 r = __ldg(reinterpret_cast<const float4*>(p)), s = __ldg(reinterpret_cast<const float4*>(p) + 1);
    x[0] = r.x; x[1] = r.y; x[2] = r.z; x[3] = r.w;
    x[4] = s.x; x[5] = s.y; x[6] = s.z; x[7] = s.w;
  }
};
template <>
struct Vec<float, 1> {
  float x[1];
  __device__ __forceinline__ void load(const float* p) { x[0] = __ldg(p); }
};
template <>
struct Vec<uint16_t, 1> {
  float x[1];
  __device__ __forceinline__ void load(const uint16_t* p) { x[0] = bf16_to_f32(__ldg(p)); }
};

struct VerShared {
  float px[AQ_MAX_DRAFT_NODES], qx[AQ_MAX_DRAFT_NODES], u[AQ_MAX_DRAFT_NODES], zinv[AQ_MAX_DRAFT_NODES];
  int32_t parent[AQ_MAX_DRAFT_NODES], tok[AQ_MAX_DRAFT_NODES], gone[AQ_MAX_DRAFT_NODES];
  unsigned long long best[2][kVerMaxCluster];
  float sum[2][kVerMaxCluster];
  unsigned long long wbest[kVerThreads / 32];
  float wsum[kVerThreads / 32];
  int32_t cur, refused, next, count, done;
};

// What the draw's weights are made of: p with `k` refused tokens left out, max(p - q, 0) after one refusal, or the
// residual after several.
enum Draw { kPlain, kOnce, kSeveral };

// Largest r(v) / E(v) of this CTA's share of the vocabulary, N words at a time.
template <typename T, Draw MODE, int N>
__device__ __forceinline__ void race(const T* pr, const T* qr, const float* er, int vocab, int k, const VerShared& sh,
                                     int rank, int cluster, float& best, int& at) {
  // A quotient can pass the warp's best so far only if w > best e (1 - 2^-21), rounding included: one fused product and
  // one comparison a word, and the divisions only where some word of a thread's batch gets that far. Words equal to
  // the best pass too, and the lowest index is sorted out when the threads' bests meet. Where the product is below the
  // normal numbers its rounding has no such bound: 2^-126 less covers that, and changes no product above 2^-102.
  float bar = 0.0f, slack = 0.0f;
  auto weigh = [&](float w, float q) { return MODE == kPlain ? w : MODE == kOnce ? fmaxf(w - q, 0.0f) : residual(w, q, k, k - 1, sh.zinv); };
  auto offer = [&](float w, float e, int v) {
    const float s = __fdiv_rn(w, e);
    if (s > best) {
      if (MODE == kPlain)
        for (int j = 0; j < k; ++j)
          if (sh.gone[j] == v) return;   // a refused token has no mass; looked up only for a new best
      best = s;
      at = v;
    }
  };
  const int step = cluster * kVerThreads * N;
  int v = (rank * kVerThreads + threadIdx.x) * N;
  constexpr int U = N == 1 ? 8 : N == 4 ? 4 : 2;   // loads in flight: 32 to 64 bytes a thread of each operand
  // warps leave this loop together: a warp's words of a round are neighbours
  for (; (v - (static_cast<int>(threadIdx.x) & 31) * N) + (U - 1) * step + 32 * N <= vocab; v += U * step) {
    Vec<T, N> w[U], q[U];
    Vec<float, N> e[U];
#pragma unroll
    for (int j = 0; j < U; ++j) {
      w[j].load(pr + v + j * step);
      if (MODE != kPlain) q[j].load(qr + v + j * step);
      e[j].load(er + v + j * step);
    }
    bool hit = false;
#pragma unroll
    for (int j = 0; j < U; ++j)
#pragma unroll
      for (int i = 0; i < N; ++i) {
        if (MODE != kPlain) w[j].x[i] = weigh(w[j].x[i], q[j].x[i]);
        hit = hit || w[j].x[i] > fmaf(bar, e[j].x[i], slack);
      }
    if (__any_sync(0xffffffffu, hit)) {
      if (hit) {
#pragma unroll
        for (int j = 0; j < U; ++j)
#pragma unroll
          for (int i = 0; i < N; ++i)
            if (w[j].x[i] > fmaf(bar, e[j].x[i], slack)) offer(w[j].x[i], e[j].x[i], v + j * step + i);
      }
      bar = __uint_as_float(__reduce_max_sync(0xffffffffu, __float_as_uint(best))) * (1.0f - 0x1p-21f);
      slack = bar > 0.0f ? -0x1p-126f : 0.0f;
    }
  }
  for (; v < vocab; v += step)
    for (int i = 0; i < N && v + i < vocab; ++i) {
      const float w = weigh(prob(pr, v + i), MODE != kPlain ? prob(qr, v + i) : 0.0f), e = er[v + i];
      if (w > fmaf(bar, e, slack)) offer(w, e, v + i);
    }
}

template <typename T, bool HASQ>
__global__ void __launch_bounds__(kVerThreads, kVerPerSm) aq_verify_kernel(const __grid_constant__ VerifyParams p) {
  __shared__ VerShared sh;
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
  const int C = p.cluster;
  const int rank = C > 1 ? static_cast<int>(cluster_ctarank()) : 0;
  const int b = blockIdx.x / C;
  const T* P = static_cast<const T*>(p.p);
  const T* Q = static_cast<const T*>(p.q);
  // a CTA may write into a peer's shared memory only once that peer runs: waited for before the walk
  asm volatile("barrier.cluster.arrive.relaxed.aligned;" ::: "memory");
  pdl_wait_prior_grid();
  pdl_launch_dependents();

  const int64_t first = p.cu[b];
  int64_t last = p.cu[b + 1];
  const bool ok = first >= 0 && last >= first && last <= p.nodes && first + b < p.rows;
  int n = ok ? static_cast<int>(min(last - first, static_cast<int64_t>(p.max_nodes))) : 0;
  const int64_t row0 = first + b;   // row of p after the context; node i: row0 + 1 + i
  if (ok) n = static_cast<int>(min(static_cast<int64_t>(n), p.rows - row0 - 1));
  for (int i = tid; i < n; i += kVerThreads) {
    const int par = p.parent ? p.parent[first + i] : i - 1;
    const int tok = p.tokens[first + i];
    const bool good = par >= -1 && par < i && tok >= 0 && tok < p.vocab;
    const int64_t row = row0 + 1 + par;
    sh.parent[i] = good ? par : -2;   // no one's child: what was never drafted from q is not refused, either
    sh.tok[i] = tok;
    sh.px[i] = good ? prob(P, row * p.ld_p + tok) : 0.0f;
    sh.qx[i] = HASQ ? (good ? prob(Q, row * p.ld_q + tok) : 0.0f) : 1.0f;
    sh.u[i] = p.u[first + i];
  }
  if (tid == 0) {
    sh.cur = -1;
    sh.refused = 0;
    sh.next = 0;
    sh.count = 0;
    sh.done = 0;
  }
  asm volatile("barrier.cluster.wait.acquire.aligned;" ::: "memory");
  __syncthreads();

  int phase = 0;
  float mass_gone = 0.0f;   // thread 0's, point-mass drafts
  for (;;) {
    if (warp == 0) {
      int cur = sh.cur, refused = sh.refused, count = sh.count, from = sh.next;
      bool stop = count >= p.path_cap, sum = false;
      while (!stop && !sum) {
        // next child of cur at or after `from`
        int c = -1;
        for (int i0 = from; i0 < n && c < 0; i0 += 32) {
          const unsigned m = __ballot_sync(0xffffffffu, i0 + lane < n && sh.parent[min(i0 + lane, n - 1)] == cur);
          if (m) c = i0 + __ffs(m) - 1;
        }
        if (c < 0) {
          stop = true;
          break;
        }
        if (HASQ && refused > 0 && refused > sh.done) {   // the residual this child is tested on is not normalised yet
          from = c;
          sum = true;
          break;
        }
        bool take;
        if (HASQ) {
          const float r = residual(sh.px[c], sh.qx[c], refused, refused, sh.zinv);
          take = __fmul_rn(sh.u[c], sh.qx[c]) < r;
        } else {
          float px = sh.px[c];
          for (int j = 0; j < refused; ++j)
            if (sh.gone[j] == sh.tok[c]) px = 0.0f;
          take = __fmul_rn(sh.u[c], 1.0f - mass_gone) < px;
          if (!take) mass_gone += px;
        }
        if (take) {
          if (rank == 0 && lane == 0) p.path[b * p.ld_path + count] = c;
          ++count;
          cur = c;
          refused = 0;
          mass_gone = 0.0f;
          __syncwarp();
          if (lane == 0) sh.done = 0;
          __syncwarp();
          stop = count >= p.path_cap;
        } else {
          if (!HASQ && lane == 0) sh.gone[refused] = sh.tok[c];
          ++refused;
          __syncwarp();
        }
        from = c + 1;
      }
      __syncwarp();
      if (lane == 0) {
        sh.cur = cur;
        sh.refused = refused;
        sh.count = count;
        sh.next = sum ? from : -1;
      }
    }
    __syncthreads();
    if (!HASQ || sh.next < 0) break;
    // normaliser of the residual after refusal number `done`: this CTA's share, then all in rank order
    const int k = sh.done + 1;
    const T* pr = P + (row0 + 1 + sh.cur) * p.ld_p;
    const T* qr = Q + (row0 + 1 + sh.cur) * p.ld_q;
    float part = 0.0f;
#pragma unroll 8
    for (int v = rank * kVerThreads + tid; v < p.vocab; v += C * kVerThreads)
      part += residual(prob(pr, v), prob(qr, v), k, k - 1, sh.zinv);
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) part += __shfl_xor_sync(0xffffffffu, part, o);
    if (lane == 0) sh.wsum[warp] = part;
    __syncthreads();
    if (tid < C) {
      float s = 0.0f;
      for (int w = 0; w < kVerThreads / 32; ++w) s += sh.wsum[w];
      asm volatile("st.shared::cluster.f32 [%0], %1;" ::"r"(cluster_map(&sh.sum[phase][rank], tid)), "f"(s) : "memory");
    }
    cluster_sync_all();
    if (tid == 0) {
      float s = 0.0f;
      for (int c = 0; c < C; ++c) s += sh.sum[phase][c];
      sh.zinv[k - 1] = s > 0.0f ? __frcp_rn(s) : 0.0f;
      sh.done = k;
    }
    phase ^= 1;
    __syncthreads();
  }

  // the draw
  const int64_t row = row0 + 1 + sh.cur;
  int k = sh.refused;
  float best = 0.0f;
  int at = 0;
  for (int pass = 0; ok && pass < 2; ++pass) {
    const T* pr = P + row * p.ld_p;
    const T* qr = HASQ ? Q + row * p.ld_q : pr;
    const float* er = p.noise + b * p.ld_noise;
    const uintptr_t low = reinterpret_cast<uintptr_t>(pr) | reinterpret_cast<uintptr_t>(qr);
    constexpr int kVec = 16 / sizeof(T);
    const bool whole = ((low | reinterpret_cast<uintptr_t>(er)) & 15) == 0;
    // with q, k counts refusals of the residual; without, tokens that are left out
    auto pass_over = [&](auto mode) {
      constexpr Draw kMode = decltype(mode)::value;
      if (whole) race<T, kMode, kVec>(pr, qr, er, p.vocab, k, sh, rank, C, best, at);
      else race<T, kMode, 1>(pr, qr, er, p.vocab, k, sh, rank, C, best, at);
    };
    if (!HASQ || k == 0) pass_over(std::integral_constant<Draw, kPlain>());
    else if (k == 1) pass_over(std::integral_constant<Draw, kOnce>());
    else pass_over(std::integral_constant<Draw, kSeveral>());
    unsigned long long key = (static_cast<unsigned long long>(__float_as_uint(best)) << 32) | (0xffffffffu - static_cast<uint32_t>(at));
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) {
      const unsigned long long other = __shfl_xor_sync(0xffffffffu, key, o);
      key = other > key ? other : key;
    }
    if (lane == 0) sh.wbest[warp] = key;
    __syncthreads();
    if (tid < C) {
      for (int w = 0; w < kVerThreads / 32; ++w) key = w == 0 || sh.wbest[w] > key ? sh.wbest[w] : key;
      asm volatile("st.shared::cluster.b64 [%0], %1;" ::"r"(cluster_map(&sh.best[phase][rank], tid)), "l"(key) : "memory");
    }
    cluster_sync_all();
    key = 0;
    for (int c = 0; c < C; ++c) key = sh.best[phase][c] > key ? sh.best[phase][c] : key;
    phase ^= 1;
    at = static_cast<int>(0xffffffffu - static_cast<uint32_t>(key));
    if ((key >> 32) != 0 || k == 0) break;   // nothing has mass after the refusals: draw from p itself
    k = 0;
    best = 0.0f;
    at = 0;
  }
  if (rank == 0) {
    for (int i = sh.count + tid; i < p.path_cap; i += kVerThreads) p.path[b * p.ld_path + i] = -1;
    if (tid == 0) {
      p.n_accepted[b] = sh.count;
      p.token[b] = ok ? at : -1;
    }
  }
}

template <typename T, bool HASQ>
cudaError_t launch_verify(const VerifyParams& p, unsigned grid, cudaStream_t st) {
  static std::atomic<uint64_t> ready{0};   // devices on which the kernel may use clusters of 16
  if (p.cluster > 8 && !(ready.load() >> p.device & 1)) {
    const cudaError_t e = cudaFuncSetAttribute(aq_verify_kernel<T, HASQ>, cudaFuncAttributeNonPortableClusterSizeAllowed, 1);
    if (e != cudaSuccess) return e;
    ready.fetch_or(1ull << p.device);
  }
  return launch_serve(aq_verify_kernel<T, HASQ>, p, grid, kVerThreads, 0, st, p.cluster);
}

}  // namespace
}  // namespace aq

using namespace aq;

extern "C" aq_status aq_verify_drafts(int32_t batch, int32_t vocab, const int32_t* cu, const int32_t* tokens,
                                      const int32_t* parent, int64_t nodes, int32_t max_nodes, const void* p,
                                      int64_t ld_p, const void* q, int64_t ld_q, int64_t rows, int32_t p_type,
                                      const float* u, const float* noise, int64_t ld_noise, int32_t* n_accepted,
                                      int32_t* path, int64_t ld_path, int32_t path_cap, int32_t* token, void* stream) {
  const char* who = "aq_verify_drafts";
  if (batch < 0 || nodes < 0 || rows < 0 || path_cap < 0)
    return serve_fail(AQ_ERR_SHAPE, "%s: batch=%d nodes=%lld rows=%lld path_cap=%d must not be negative", who, batch,
                      (long long)nodes, (long long)rows, path_cap);
  if (vocab < 1 || vocab > (1 << 30)) return serve_fail(AQ_ERR_SHAPE, "%s: vocab=%d outside [1, 2^30]", who, vocab);
  if (max_nodes < 0 || max_nodes > AQ_MAX_DRAFT_NODES)
    return serve_fail(AQ_ERR_UNSUPPORTED, "%s: max_nodes=%d outside [0, %d]", who, max_nodes, AQ_MAX_DRAFT_NODES);
  if (p_type != AQ_PROB_F32 && p_type != AQ_PROB_BF16)
    return serve_fail(AQ_ERR_INVALID_ARG, "%s: unknown probability type %d", who, p_type);
  if (batch == 0) return AQ_OK;
  if (!cu || !p || !noise || !n_accepted || !token || (path_cap > 0 && !path) || (nodes > 0 && (!tokens || !u)))
    return serve_fail(AQ_ERR_INVALID_ARG, "%s: NULL argument", who);
  if (rows < nodes + batch)
    return serve_fail(AQ_ERR_SHAPE, "%s: rows=%lld: p needs one row for each node and sequence (%lld)", who,
                      (long long)rows, (long long)(nodes + batch));
  if (ld_p < vocab || (q && ld_q < vocab) || ld_noise < vocab || (path_cap > 0 && ld_path < path_cap))
    return serve_fail(AQ_ERR_SHAPE, "%s: a row stride is smaller than its row", who);
  const uintptr_t size = p_type == AQ_PROB_F32 ? 4 : 2;
  if (!serve_aligned(p, size) || (q && !serve_aligned(q, size)) || !serve_aligned(u, 4) || !serve_aligned(noise, 4) ||
      !serve_aligned(cu, 4) || !serve_aligned(tokens, 4) || !serve_aligned(parent, 4) || !serve_aligned(n_accepted, 4) ||
      !serve_aligned(path, 4) || !serve_aligned(token, 4))
    return serve_fail(AQ_ERR_ALIGNMENT, "%s: pointers must be aligned to their elements", who);
  const ByteSpan outs[] = {byte_span(n_accepted, 1, 0, batch, 4), byte_span(path, batch, ld_path, path_cap, 4),
                           byte_span(token, 1, 0, batch, 4)};
  const ByteSpan ins[] = {byte_span(p, rows, ld_p, vocab, size), byte_span(q, rows, ld_q, vocab, size),
                          byte_span(noise, batch, ld_noise, vocab, 4), byte_span(cu, 1, 0, batch + 1, 4),
                          byte_span(tokens, 1, 0, nodes, 4), byte_span(parent, 1, 0, nodes, 4), byte_span(u, 1, 0, nodes, 4)};
  for (int i = 0; i < 3; ++i) {
    for (const ByteSpan& in : ins)
      if (byte_overlap(outs[i], in)) return serve_fail(AQ_ERR_OVERLAP, "%s: an output overlaps an input", who);
    for (int j = 0; j < i; ++j)
      if (byte_overlap(outs[i], outs[j])) return serve_fail(AQ_ERR_OVERLAP, "%s: two outputs overlap", who);
  }
  ServeDev dev;
  aq_status st = serve_device(&dev);
  if (st != AQ_OK) return st;
  VerifyParams v = {};
  v.cu = cu;
  v.tokens = tokens;
  v.parent = parent;
  v.p = p;
  v.q = q;
  v.u = u;
  v.noise = noise;
  v.ld_p = ld_p;
  v.ld_q = ld_q;
  v.ld_noise = ld_noise;
  v.ld_path = ld_path;
  v.nodes = nodes;
  v.rows = rows;
  v.n_accepted = n_accepted;
  v.path = path;
  v.token = token;
  v.vocab = vocab;
  v.max_nodes = max_nodes;
  v.path_cap = path_cap;
  // the largest cluster that keeps the launch within the CTAs that are resident at once and gives every CTA at
  // least one round of its threads
  int c = kVerMaxCluster;
  while (c > 1 && (static_cast<int64_t>(batch) * c > kVerPerSm * dev.sms || vocab < c * kVerThreads)) c /= 2;
  v.cluster = c;
  v.device = dev.index;
  if (static_cast<int64_t>(batch) * c > 0x7fffffffLL) return serve_fail(AQ_ERR_SHAPE, "%s: batch=%d is too large", who, batch);
  const unsigned grid = static_cast<unsigned>(batch) * c;
  const cudaStream_t cs = static_cast<cudaStream_t>(stream);
  cudaError_t e;
  if (p_type == AQ_PROB_F32)
    e = q ? launch_verify<float, true>(v, grid, cs) : launch_verify<float, false>(v, grid, cs);
  else
    e = q ? launch_verify<uint16_t, true>(v, grid, cs) : launch_verify<uint16_t, false>(v, grid, cs);
  return serve_launched(e, who);
}
