// aq_scores.cu -- aq_token_logprobs and its gradient: from rows of logits the log probability of a given word, the entropy,
// the log of the normaliser and the most likely words.
//
// With z = scale x over a row: lse = log sum e^z, log p(v) = z_v - lse, H = lse - sum p z. One pass holds, for each thread, the
// largest x so far, m, and s = sum 2^d, a = sum 2^d d with d = (x - m) scale log2(e): lse = m scale + ln s, H = ln s - ln2 a / s.
// Threads, warps and the CTAs of a cluster are joined by the same rule in a fixed order.
//
// The most likely words: a warp keeps the best 32 of its words sorted, one a lane, as 64-bit keys (the value's order, then the
// lower index), so equal values need no rule of their own and no order of arrival shows. A batch of words is looked at only where
// a lane's largest beats the k-th of the list; where many do (the first batch, a rising row), the lanes' largest are sorted and
// merged first, which raises the bar for the rest.
//
// Bound by memory: the logits are read once (the gradient: read once, written once).
#include <algorithm>
#include <atomic>
#include <type_traits>

#include "aq_serve.h"

namespace aq {
namespace {

constexpr int kScoreThreads = 256, kScoreWarps = kScoreThreads / 32, kScorePerSm = 3;
constexpr int kScoreMaxCluster = 16;
constexpr float kLog2e = 1.4426950408889634f, kLn2 = 0.6931471805599453f;

struct ScoreParams {
  const void* logits;
  int64_t ld, rows;
  const int32_t* tokens;
  float* logprob;
  float* lse;
  float* entropy;
  float* top_logprob;
  int32_t* top_token;
  float scale;
  int32_t vocab, top, cluster, device;
};

__device__ __forceinline__ float ex2(float x) {
  float r;
  asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(r) : "f"(x));
  return r;
}
// The larger, NaN if either is: keeps a NaN that fmaxf would drop.
__device__ __forceinline__ float max_nan(float a, float b) {
  float r;
  asm("max.NaN.f32 %0, %1, %2;" : "=f"(r) : "f"(a), "f"(b));
  return r;
}

template <typename T>
struct Words;   // 16 bytes of logits
template <>
struct Words<float> {
  static constexpr int N = 4;
  static constexpr uint32_t kNone = 0xff800000u;   // -inf
  static __device__ __forceinline__ void unpack(const uint4& r, float (&x)[4]) {
    x[0] = __uint_as_float(r.x);
    x[1] = __uint_as_float(r.y);
    x[2] = __uint_as_float(r.z);
    x[3] = __uint_as_float(r.w);
  }
  static __device__ __forceinline__ uint4 pack(const float (&x)[4]) {
    return make_uint4(__float_as_uint(x[0]), __float_as_uint(x[1]), __float_as_uint(x[2]), __float_as_uint(x[3]));
  }
  static __device__ __forceinline__ float largest(const uint4& r) {
    return fmaxf(fmaxf(__uint_as_float(r.x), __uint_as_float(r.y)), fmaxf(__uint_as_float(r.z), __uint_as_float(r.w)));
  }
  static __device__ __forceinline__ float one(const float* p) { return *p; }
  static __device__ __forceinline__ void put(float* p, float v) { *p = v; }
};
template <>
struct Words<uint16_t> {
  static constexpr int N = 8;
  static constexpr uint32_t kNone = 0xff80ff80u;
  static __device__ __forceinline__ void unpack(const uint4& r, float (&x)[8]) {
    const uint32_t w[4] = {r.x, r.y, r.z, r.w};
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      x[2 * i] = __uint_as_float(w[i] << 16);
      x[2 * i + 1] = __uint_as_float(w[i] & 0xffff0000u);
    }
  }
  static __device__ __forceinline__ uint4 pack(const float (&x)[8]) {
    return make_uint4(pack_bf16x2_cvt(x[0], x[1]), pack_bf16x2_cvt(x[2], x[3]), pack_bf16x2_cvt(x[4], x[5]), pack_bf16x2_cvt(x[6], x[7]));
  }
  static __device__ __forceinline__ uint32_t max2(uint32_t a, uint32_t b) {
    uint32_t r;
    asm("max.bf16x2 %0, %1, %2;" : "=r"(r) : "r"(a), "r"(b));
    return r;
  }
  static __device__ __forceinline__ float largest(const uint4& r) {
    const uint32_t m = max2(max2(r.x, r.y), max2(r.z, r.w));
    return fmaxf(__uint_as_float(m << 16), __uint_as_float(m & 0xffff0000u));
  }
  static __device__ __forceinline__ float one(const uint16_t* p) { return bf16_to_f32(*p); }
  static __device__ __forceinline__ void put(uint16_t* p, float v) { *p = f32_to_bf16_rn(v); }
};

// Loads of logits: read once, not kept in L1.
__device__ __forceinline__ uint4 ld_words(const void* p) {
  uint4 r;
  asm volatile("ld.global.L1::no_allocate.v4.u32 {%0, %1, %2, %3}, [%4];" : "=r"(r.x), "=r"(r.y), "=r"(r.z), "=r"(r.w) : "l"(p) : "memory");
  return r;
}

// A row's body in whole 16-byte pieces, and the words before and after it.
template <typename T>
struct Row {
  const T* p;
  int head, vecs, tail;
  __device__ __forceinline__ Row(const T* row, int vocab) : p(row) {
    constexpr int N = Words<T>::N;
    const int off = static_cast<int>(reinterpret_cast<uintptr_t>(row) & 15) / sizeof(T);
    head = min(vocab, off ? N - off : 0);
    vecs = (vocab - head) / N;
    tail = vocab - head - vecs * N;
  }
};

// ---- sums ----
struct Sums {
  float m = -INFINITY, at = 0.0f, s = 0.0f, a = 0.0f;   // at: m, or 0 while m is -inf
  // To a new largest value. Differences below -1000 are as good as -inf, whose product with 0 would be NaN; they are taken before
  // the scale, which could carry a mask of the type's lowest value past the range.
  __device__ __forceinline__ void rise(float to, float c) {
    at = to == -INFINITY ? 0.0f : to;
    const float d = fmaxf((m - at) * c, -1000.0f), f = ex2(d);
    a = f * fmaf(s, d, a);
    s *= f;
    m = to;
  }
  __device__ __forceinline__ void add(float x, float c) {
    const float d = max_nan((x - at) * c, -1000.0f), e = ex2(d);
    s += e;
    a = fmaf(e, d, a);
  }
};

// ---- the most likely words ----
typedef unsigned long long Key;
// Order of a value, NaN below all numbers; 0 stands for no word at all.
__device__ __forceinline__ uint32_t order_of(float x) {
  const uint32_t b = __float_as_uint(x + 0.0f);   // -0 is 0
  return x != x ? 1u : (b & 0x80000000u) ? ~b : b | 0x80000000u;
}
__device__ __forceinline__ float value_of(uint32_t order) {
  return order <= 1u ? __uint_as_float(0x7fc00000u) : __uint_as_float((order & 0x80000000u) ? order & 0x7fffffffu : ~order);
}
__device__ __forceinline__ Key key_of(float x, int at) { return (static_cast<Key>(order_of(x)) << 32) | (0xffffffffu - static_cast<uint32_t>(at)); }

struct Best {
  Key key = 0;      // this lane's place in the warp's list, lane 0 the best
  Key kth = 0;
  float bar = 0.0f;
  bool open = true;   // the list's first k places are not all held by numbers: every word may enter
  __device__ __forceinline__ void mark(int k) {
    kth = __shfl_sync(0xffffffffu, key, k - 1);
    open = (kth >> 32) <= 1u;
    bar = value_of(static_cast<uint32_t>(kth >> 32));
  }
  __device__ __forceinline__ void insert(Key x) {
    const Key up = __shfl_up_sync(0xffffffffu, key, 1);
    if (x > key) key = (threadIdx.x & 31) > 0 && x > up ? up : x;
  }
  // The best 32 of the list and one key of every lane.
  __device__ __forceinline__ void merge(Key x) {
    const int lane = threadIdx.x & 31;
    auto exchange = [&](Key v, int o, bool larger) {
      const Key w = __shfl_xor_sync(0xffffffffu, v, o);
      return (v > w) == larger ? v : w;
    };
#pragma unroll
    for (int n = 2; n <= 32; n *= 2)
#pragma unroll
      for (int o = n / 2; o > 0; o /= 2) x = exchange(x, o, ((lane & o) == 0) != ((lane & n) != 0 && n < 32));
    // x descends as the list does: against its reverse, the larger of each pair are the best 32, and rise once
    const Key back = __shfl_xor_sync(0xffffffffu, x, 31);
    key = key > back ? key : back;
#pragma unroll
    for (int o = 16; o > 0; o /= 2) key = exchange(key, o, (lane & o) == 0);
  }
};

// N words a lane, U times: x(u, i) at index at(u, i); `held(u)` whether the lane's words of that piece exist.
template <int U, int N, typename X, typename At, typename Held>
__device__ __forceinline__ void consider(Best& b, int k, float largest, X x, At at, Held held) {
  const unsigned who = __ballot_sync(0xffffffffu, b.open || largest > b.bar);
  if (!who) return;
  Key used = 0;
  if (__popc(who) >= 8) {
#pragma unroll
    for (int u = 0; u < U; ++u)
      if (held(u))
#pragma unroll
        for (int i = 0; i < N; ++i) {
          const Key y = key_of(x(u, i), at(u, i));
          used = y > used ? y : used;
        }
    b.merge(used);
    b.mark(k);
  }
#pragma unroll
  for (int u = 0; u < U; ++u) {
    bool any = false;
#pragma unroll
    for (int i = 0; i < N; ++i) any = any || x(u, i) >= b.bar;
    if (!__any_sync(0xffffffffu, held(u) && (b.open || any))) continue;
#pragma unroll 1
    for (int i = 0; i < N; ++i) {
      const Key y = key_of(x(u, i), at(u, i));
      unsigned in = __ballot_sync(0xffffffffu, held(u) && y > b.kth && y != used);
      while (in) {
        const Key z = __shfl_sync(0xffffffffu, y, __ffs(in) - 1);
        in &= in - 1;
        if (z > b.kth) {
          b.insert(z);
          b.mark(k);
        }
      }
    }
  }
}

struct ScoreShared {
  float m[kScoreMaxCluster * kScoreWarps], s[kScoreMaxCluster * kScoreWarps], a[kScoreMaxCluster * kScoreWarps];   // rank 0's
  Key list[kScoreWarps][32];
  Key lists[kScoreMaxCluster][32];   // rank 0's
  float ln_s, m_all;
};

// How many keys of a descending list of 32 are above x.
__device__ __forceinline__ int above(const Key* list, Key x) {
  int n = 0;
#pragma unroll
  for (int s = 16; s > 0; s /= 2)
    if (list[n + s - 1] > x) n += s;
  return n + (list[n] > x);
}

template <typename T, bool TOP>
__global__ void __launch_bounds__(kScoreThreads, kScorePerSm) aq_scores_kernel(const __grid_constant__ ScoreParams p) {
  using W = Words<T>;
  constexpr int N = W::N, U = 4;
  __shared__ ScoreShared sh;
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
  const int C = p.cluster, rank = C > 1 ? static_cast<int>(cluster_ctarank()) : 0;
  const int64_t r = blockIdx.x / C;
  if (C > 1) asm volatile("barrier.cluster.arrive.relaxed.aligned;" ::: "memory");
  pdl_wait_prior_grid();
  pdl_launch_dependents();
  const T* row = static_cast<const T*>(p.logits) + r * p.ld;
  const Row<T> w(row, p.vocab);
  const float c = p.scale * kLog2e;
  float given = 0.0f;   // the given word's logit, on its way meanwhile
  int token = -1;
  if (rank == 0 && tid == 0 && p.logprob) {
    token = p.tokens[r];
    if (token >= 0 && token < p.vocab) given = W::one(row + token);
  }

  Sums q;
  Best best;
  // the words before the body, one a lane
  if (rank == 0 && warp == 0 && w.head > 0) {
    const bool in = lane < w.head;
    const float x = in ? W::one(row + lane) : -INFINITY;
    q.rise(fmaxf(x, -INFINITY), c);
    if (in) q.add(x, c);
    if (TOP) consider<1, 1>(best, p.top, x, [&](int, int) { return x; }, [&](int, int) { return lane; }, [&](int) { return in; });
  }
  const T* body = row + w.head;
  const int v0 = static_cast<int>(static_cast<int64_t>(w.vecs) * rank / C), v1 = static_cast<int>(static_cast<int64_t>(w.vecs) * (rank + 1) / C);
  for (int vw = v0 + warp * 32; vw < v1; vw += U * kScoreThreads) {   // a warp's words of a round are neighbours
    uint4 raw[U];
#pragma unroll
    for (int u = 0; u < U; ++u) {
      const int v = vw + lane + u * kScoreThreads;
      raw[u] = v < v1 ? ld_words(body + static_cast<int64_t>(v) * N) : make_uint4(W::kNone, W::kNone, W::kNone, W::kNone);
    }
    float top = W::largest(raw[0]);
#pragma unroll
    for (int u = 1; u < U; ++u) top = fmaxf(top, W::largest(raw[u]));
    q.rise(fmaxf(q.m, top), c);
#pragma unroll
    for (int u = 0; u < U; ++u) {
      float x[N];
      W::unpack(raw[u], x);
#pragma unroll
      for (int i = 0; i < N; ++i) q.add(x[i], c);
    }
    if (TOP)
      consider<U, N>(
          best, p.top, top,
          [&](int u, int i) {
            float x[N];
            W::unpack(raw[u], x);
            return x[i];
          },
          [&](int u, int i) { return w.head + (vw + lane + u * kScoreThreads) * N + i; }, [&](int u) { return vw + lane + u * kScoreThreads < v1; });
  }
  if (rank == C - 1 && warp == 0 && w.tail > 0) {
    const bool in = lane < w.tail;
    const int at = w.head + w.vecs * N + lane;
    const float x = in ? W::one(row + at) : -INFINITY;
    q.rise(fmaxf(q.m, x), c);
    if (in) q.add(x, c);
    if (TOP) consider<1, 1>(best, p.top, x, [&](int, int) { return x; }, [&](int, int) { return at; }, [&](int) { return in; });
  }

  // the warp's sums
  float m = q.m;
#pragma unroll
  for (int o = 16; o > 0; o >>= 1) m = fmaxf(m, __shfl_xor_sync(0xffffffffu, m, o));
  q.rise(m, c);
#pragma unroll
  for (int o = 16; o > 0; o >>= 1) {
    q.s += __shfl_xor_sync(0xffffffffu, q.s, o);
    q.a += __shfl_xor_sync(0xffffffffu, q.a, o);
  }
  if (C > 1) asm volatile("barrier.cluster.wait.acquire.aligned;" ::: "memory");   // rank 0 runs
  if (lane == 0) {
    const int i = rank * kScoreWarps + warp;
    if (C > 1) {
      asm volatile("st.shared::cluster.f32 [%0], %1;" ::"r"(cluster_map(&sh.m[i], 0)), "f"(q.m) : "memory");
      asm volatile("st.shared::cluster.f32 [%0], %1;" ::"r"(cluster_map(&sh.s[i], 0)), "f"(q.s) : "memory");
      asm volatile("st.shared::cluster.f32 [%0], %1;" ::"r"(cluster_map(&sh.a[i], 0)), "f"(q.a) : "memory");
    } else {
      sh.m[i] = q.m;
      sh.s[i] = q.s;
      sh.a[i] = q.a;
    }
  }
  if (TOP) {
    sh.list[warp][lane] = best.key;
    if (C == 1 && tid < 32) sh.lists[0][tid] = 0;
  }
  __syncthreads();
  if (TOP) {
    // the CTA's list: a key's place is its own in its warp's list and the number of keys above it in the others
    int place = lane;
#pragma unroll
    for (int i = 0; i < kScoreWarps; ++i)
      if (i != warp) place += above(sh.list[i], best.key);
    if (C > 1) {
      // its 32 places, empty ones (fewer words than places) as no word: those above the number of keys held
      int held = 0;
#pragma unroll
      for (int i = 0; i < kScoreWarps; ++i) held += above(sh.list[i], 0);
      if (best.key && place < 32) asm volatile("st.shared::cluster.u64 [%0], %1;" ::"r"(cluster_map(&sh.lists[rank][place], 0)), "l"(best.key) : "memory");
      if (tid < 32 && tid >= held) asm volatile("st.shared::cluster.u64 [%0], %1;" ::"r"(cluster_map(&sh.lists[rank][tid], 0)), "l"(Key(0)) : "memory");
    } else if (best.key && place < 32) {
      sh.lists[0][place] = best.key;
    }
  }
  if (C > 1) cluster_sync_all();
  else if (TOP) __syncthreads();
  if (rank != 0) return;
  if (warp == 0) {
    // sums over the cluster, C * kScoreWarps of them
    float top = -INFINITY;
    for (int i = lane; i < C * kScoreWarps; i += 32) top = fmaxf(top, sh.m[i]);
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) top = fmaxf(top, __shfl_xor_sync(0xffffffffu, top, o));
    float s = 0.0f, a = 0.0f;
    for (int i = lane; i < C * kScoreWarps; i += 32) {
      Sums one;
      one.m = sh.m[i];
      one.s = sh.s[i];
      one.a = sh.a[i];
      one.rise(top, c);
      s += one.s;
      a += one.a;
    }
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) {
      s += __shfl_xor_sync(0xffffffffu, s, o);
      a += __shfl_xor_sync(0xffffffffu, a, o);
    }
    if (lane == 0) {
      const bool none = top == -INFINITY && s == 0.0f;   // no word has any mass
      const float ln_s = logf(s);
      sh.ln_s = ln_s;
      sh.m_all = top;
      if (p.lse) p.lse[r] = none ? -INFINITY : (top == -INFINITY ? s : fmaf(top, p.scale, ln_s));
      if (p.entropy) p.entropy[r] = none ? 0.0f : ln_s - kLn2 * (a / s);
      if (p.logprob) p.logprob[r] = token < 0 || token >= p.vocab ? 0.0f : none ? -INFINITY : fmaf(given - top, p.scale, -ln_s);
    }
  }
  if (TOP) {
    __syncthreads();
    const float ln_s = sh.ln_s, m_all = sh.m_all;
    const bool none = m_all == -INFINITY && ln_s == -INFINITY;
    for (int i = tid; i < C * 32; i += kScoreThreads) {
      const Key x = sh.lists[i / 32][i % 32];
      if (!x) continue;
      int place = i % 32;
      for (int l = 0; l < C && place < p.top; ++l)
        if (l != i / 32) place += above(sh.lists[l], x);
      if (place >= p.top) continue;
      const float v = value_of(static_cast<uint32_t>(x >> 32));
      p.top_token[r * p.top + place] = static_cast<int32_t>(0xffffffffu - static_cast<uint32_t>(x));
      p.top_logprob[r * p.top + place] = none ? -INFINITY : fmaf(v - m_all, p.scale, -ln_s);
    }
  }
}

// ---------------------------------------------------------------------------------
// gradient
// ---------------------------------------------------------------------------------
struct ScoreGradParams {
  const void* logits;
  void* out;
  int64_t ld, ld_out, rows;
  const int32_t* tokens;
  const float* lse;
  const float* entropy;
  const float* dlogprob;
  const float* dentropy;   // or NULL
  const float* dlse;       // or NULL
  float scale;
  int32_t vocab, parts;
};

template <typename T>
__global__ void __launch_bounds__(kScoreThreads, 4) aq_scores_grad_kernel(const __grid_constant__ ScoreGradParams p) {
  using W = Words<T>;
  constexpr int N = W::N, U = 4;
  pdl_wait_prior_grid();
  pdl_launch_dependents();
  const int64_t r = blockIdx.x / p.parts;
  const int part = static_cast<int>(blockIdx.x - r * p.parts);
  const T* row = static_cast<const T*>(p.logits) + r * p.ld;
  T* out = static_cast<T*>(p.out) + r * p.ld_out;
  const int token = p.tokens ? p.tokens[r] : -1;
  const bool has = token >= 0 && token < p.vocab;
  const float lse = p.lse[r], g = has ? p.dlogprob[r] : 0.0f, gh = p.dentropy ? p.dentropy[r] : 0.0f, gl = p.dlse ? p.dlse[r] : 0.0f;
  const bool none = lse == -INFINITY;   // a row without any mass has no gradient
  // dx = p (A + B d) + [v = token] g scale, with d = log2 p
  const float A = p.scale * (gl - g - (p.dentropy ? gh * p.entropy[r] : 0.0f)), B = -p.scale * gh * kLn2, hit = g * p.scale;
  auto grad = [&](float x) {
    const float d = max_nan(fmaf(x, p.scale, -lse) * kLog2e, -1000.0f);
    return none ? 0.0f : ex2(d) * fmaf(B, d, A);
  };
  const bool whole = ((reinterpret_cast<uintptr_t>(row) ^ reinterpret_cast<uintptr_t>(out)) & 15) == 0;
  if (!whole) {   // rows that start at different places of a 16-byte piece: word by word
    const int c0 = static_cast<int>(static_cast<int64_t>(p.vocab) * part / p.parts), c1 = static_cast<int>(static_cast<int64_t>(p.vocab) * (part + 1) / p.parts);
#pragma unroll 4
    for (int v = c0 + static_cast<int>(threadIdx.x); v < c1; v += kScoreThreads) {
      const float x = grad(W::one(row + v));
      W::put(out + v, v == token && !none ? x + hit : x);
    }
    return;
  }
  const Row<T> w(row, p.vocab);
  const int edge = static_cast<int>(threadIdx.x);
  if ((part == 0 && edge < w.head) || (part == p.parts - 1 && edge >= 32 && edge < 32 + w.tail)) {
    const int v = edge < 32 ? edge : w.head + w.vecs * N + edge - 32;
    const float x = grad(W::one(row + v));
    W::put(out + v, v == token && !none ? x + hit : x);
  }
  const int v0 = static_cast<int>(static_cast<int64_t>(w.vecs) * part / p.parts), v1 = static_cast<int>(static_cast<int64_t>(w.vecs) * (part + 1) / p.parts);
  for (int v = v0 + static_cast<int>(threadIdx.x); v < v1; v += U * kScoreThreads) {
    uint4 raw[U];
#pragma unroll
    for (int u = 0; u < U; ++u) raw[u] = ld_words(row + w.head + static_cast<int64_t>(min(v + u * kScoreThreads, v1 - 1)) * N);
#pragma unroll
    for (int u = 0; u < U; ++u) {
      const int at = v + u * kScoreThreads;
      float x[N];
      W::unpack(raw[u], x);
#pragma unroll
      for (int i = 0; i < N; ++i) x[i] = grad(x[i]);
      const int i0 = token - (w.head + at * N);
      if (i0 >= 0 && i0 < N && !none) {
#pragma unroll
        for (int i = 0; i < N; ++i)
          if (i == i0) x[i] += hit;
      }
      if (at < v1) *reinterpret_cast<uint4*>(out + w.head + static_cast<int64_t>(at) * N) = W::pack(x);
    }
  }
}

template <typename T, bool TOP>
cudaError_t launch_scores(const ScoreParams& p, unsigned grid, cudaStream_t st) {
  static std::atomic<uint64_t> ready{0};   // devices on which the kernel may use clusters of 16
  if (p.cluster > 8 && !(ready.load() >> p.device & 1)) {
    const cudaError_t e = cudaFuncSetAttribute(aq_scores_kernel<T, TOP>, cudaFuncAttributeNonPortableClusterSizeAllowed, 1);
    if (e != cudaSuccess) return e;
    ready.fetch_or(1ull << p.device);
  }
  return launch_serve(aq_scores_kernel<T, TOP>, p, grid, kScoreThreads, 0, st, p.cluster);
}

aq_status check_logits(const void* logits, int64_t ld, int64_t rows, int32_t vocab, int32_t type, float scale, const char* who) {
  if (rows < 0) return serve_fail(AQ_ERR_SHAPE, "%s: rows=%lld is negative", who, (long long)rows);
  if (vocab < 1 || vocab > (1 << 30)) return serve_fail(AQ_ERR_SHAPE, "%s: vocab=%d outside [1, 2^30]", who, vocab);
  if (type != AQ_PROB_F32 && type != AQ_PROB_BF16) return serve_fail(AQ_ERR_INVALID_ARG, "%s: unknown element type %d", who, type);
  if (!(scale > 0.0f) || !(scale < 1e30f)) return serve_fail(AQ_ERR_INVALID_ARG, "%s: scale must be positive and finite", who);
  if (rows > 0 && !logits) return serve_fail(AQ_ERR_INVALID_ARG, "%s: logits must be non-NULL", who);
  if (ld < vocab && rows > 1) return serve_fail(AQ_ERR_SHAPE, "%s: ld=%lld < vocab=%d", who, (long long)ld, vocab);
  if (!serve_aligned(logits, type == AQ_PROB_F32 ? 4 : 2)) return serve_fail(AQ_ERR_ALIGNMENT, "%s: logits must be aligned to their elements", who);
  return AQ_OK;
}

// CTAs that share a row: enough of them to fill the GPU several times over (so that the last wave weighs little), with at least
// one round of loads a thread and more.
int score_parts(int64_t rows, int32_t vocab, int sms, int most) {
  int c = 1;
  while (c < most && rows * c < 6ll * sms && vocab / (2 * c) >= 8192) c *= 2;
  return c;
}

}  // namespace
}  // namespace aq

using namespace aq;

extern "C" aq_status aq_token_logprobs(const void* logits, int64_t ld, int64_t rows, int32_t vocab, int32_t type, const int32_t* tokens,
                                       float scale, float* logprob, float* lse, float* entropy, int32_t top, float* top_logprob,
                                       int32_t* top_token, void* stream) {
  const char* who = "aq_token_logprobs";
  aq_status st = check_logits(logits, ld, rows, vocab, type, scale, who);
  if (st != AQ_OK) return st;
  if (top < 0 || top > AQ_MAX_TOP || top > vocab)
    return serve_fail(AQ_ERR_UNSUPPORTED, "%s: top=%d outside [0, %d], or past vocab=%d", who, top, AQ_MAX_TOP, vocab);
  if (rows == 0) return AQ_OK;
  if (logprob && !tokens) return serve_fail(AQ_ERR_INVALID_ARG, "%s: logprob needs tokens", who);
  if (top > 0 && (!top_logprob || !top_token)) return serve_fail(AQ_ERR_INVALID_ARG, "%s: top=%d needs top_logprob and top_token", who, top);
  if (!logprob && !lse && !entropy && top == 0) return serve_fail(AQ_ERR_INVALID_ARG, "%s: no output is asked for", who);
  if (!serve_aligned(tokens, 4) || !serve_aligned(logprob, 4) || !serve_aligned(lse, 4) || !serve_aligned(entropy, 4) || !serve_aligned(top_logprob, 4) ||
      !serve_aligned(top_token, 4))
    return serve_fail(AQ_ERR_ALIGNMENT, "%s: pointers must be aligned to their elements", who);
  const int64_t size = type == AQ_PROB_F32 ? 4 : 2;
  const ByteSpan ins[] = {byte_span(logits, rows, ld, vocab, size), byte_span(tokens, 1, 0, rows, 4)};
  const ByteSpan outs[] = {byte_span(logprob, 1, 0, rows, 4), byte_span(lse, 1, 0, rows, 4), byte_span(entropy, 1, 0, rows, 4),
                           byte_span(top ? top_logprob : nullptr, 1, 0, rows * top, 4), byte_span(top ? top_token : nullptr, 1, 0, rows * top, 4)};
  for (int i = 0; i < 5; ++i) {
    for (const ByteSpan& in : ins)
      if (byte_overlap(outs[i], in)) return serve_fail(AQ_ERR_OVERLAP, "%s: an output overlaps an input", who);
    for (int j = 0; j < i; ++j)
      if (byte_overlap(outs[i], outs[j])) return serve_fail(AQ_ERR_OVERLAP, "%s: two outputs overlap", who);
  }
  ServeDev dev;
  if ((st = serve_device(&dev)) != AQ_OK) return st;
  ScoreParams p = {};
  p.logits = logits;
  p.ld = ld;
  p.rows = rows;
  p.tokens = tokens;
  p.logprob = logprob;
  p.lse = lse;
  p.entropy = entropy;
  p.top_logprob = top_logprob;
  p.top_token = top_token;
  p.scale = scale;
  p.vocab = vocab;
  p.top = top;
  p.device = dev.index;
  p.cluster = score_parts(rows, vocab, dev.sms, kScoreMaxCluster);
  if (rows * p.cluster > 0x7fffffffLL) return serve_fail(AQ_ERR_SHAPE, "%s: rows=%lld is too large", who, (long long)rows);
  const unsigned grid = static_cast<unsigned>(rows * p.cluster);
  const cudaStream_t cs = static_cast<cudaStream_t>(stream);
  cudaError_t e;
  if (type == AQ_PROB_F32) e = top ? launch_scores<float, true>(p, grid, cs) : launch_scores<float, false>(p, grid, cs);
  else e = top ? launch_scores<uint16_t, true>(p, grid, cs) : launch_scores<uint16_t, false>(p, grid, cs);
  return serve_launched(e, who);
}

extern "C" aq_status aq_token_logprobs_backward(const void* logits, int64_t ld, int64_t rows, int32_t vocab, int32_t type,
                                                const int32_t* tokens, float scale, const float* lse, const float* entropy,
                                                const float* dlogprob, const float* dentropy, const float* dlse, void* dlogits,
                                                int64_t ld_out, void* stream) {
  const char* who = "aq_token_logprobs_backward";
  aq_status st = check_logits(logits, ld, rows, vocab, type, scale, who);
  if (st != AQ_OK) return st;
  if (rows == 0) return AQ_OK;
  if (!lse || !dlogits) return serve_fail(AQ_ERR_INVALID_ARG, "%s: lse and dlogits must be non-NULL", who);
  if (!tokens != !dlogprob) return serve_fail(AQ_ERR_INVALID_ARG, "%s: tokens and dlogprob go together", who);
  if (!dlogprob && !dentropy && !dlse) return serve_fail(AQ_ERR_INVALID_ARG, "%s: no gradient is given", who);
  if (dentropy && !entropy) return serve_fail(AQ_ERR_INVALID_ARG, "%s: dentropy needs entropy", who);
  if (ld_out < vocab && rows > 1) return serve_fail(AQ_ERR_SHAPE, "%s: ld_out=%lld < vocab=%d", who, (long long)ld_out, vocab);
  const int64_t size = type == AQ_PROB_F32 ? 4 : 2;
  if (!serve_aligned(dlogits, size) || !serve_aligned(tokens, 4) || !serve_aligned(lse, 4) || !serve_aligned(entropy, 4) || !serve_aligned(dlogprob, 4) ||
      !serve_aligned(dentropy, 4) || !serve_aligned(dlse, 4))
    return serve_fail(AQ_ERR_ALIGNMENT, "%s: pointers must be aligned to their elements", who);
  const ByteSpan out = byte_span(dlogits, rows, ld_out, vocab, size);
  const bool same = dlogits == logits && (rows == 1 || ld == ld_out);
  if (!same && byte_overlap(out, byte_span(logits, rows, ld, vocab, size)))
    return serve_fail(AQ_ERR_OVERLAP, "%s: dlogits overlaps logits (in place needs the same pointer and stride)", who);
  const void* const side[] = {tokens, lse, entropy, dlogprob, dentropy, dlse};
  for (const void* s : side)
    if (byte_overlap(out, byte_span(s, 1, 0, rows, 4))) return serve_fail(AQ_ERR_OVERLAP, "%s: dlogits overlaps an input", who);
  ServeDev dev;
  if ((st = serve_device(&dev)) != AQ_OK) return st;
  ScoreGradParams p = {};
  p.logits = logits;
  p.out = dlogits;
  p.ld = ld;
  p.ld_out = ld_out;
  p.rows = rows;
  p.tokens = tokens;
  p.lse = lse;
  p.entropy = entropy;
  p.dlogprob = dlogprob;
  p.dentropy = dentropy;
  p.dlse = dlse;
  p.scale = scale;
  p.vocab = vocab;
  p.parts = score_parts(rows, vocab, dev.sms, 64);
  if (rows * p.parts > 0x7fffffffLL) return serve_fail(AQ_ERR_SHAPE, "%s: rows=%lld is too large", who, (long long)rows);
  const unsigned grid = static_cast<unsigned>(rows * p.parts);
  const cudaStream_t cs = static_cast<cudaStream_t>(stream);
  return serve_launched(type == AQ_PROB_F32 ? launch_serve(aq_scores_grad_kernel<float>, p, grid, kScoreThreads, 0, cs)
                                            : launch_serve(aq_scores_grad_kernel<uint16_t>, p, grid, kScoreThreads, 0, cs),
                        who);
}
