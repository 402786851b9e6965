// aq_scores.cu -- aq_token_logprobs and its gradient: from rows of logits the log probability of a given word, the entropy,
// the log of the normaliser and the most likely words.
//
// With z = scale x over a row: lse = log sum e^z, log p(v) = z_v - lse, H = lse - sum p z. One pass holds, for each thread, the
// largest x so far, m, and s = sum 2^d, a = sum 2^d d with d = (x - m) scale log2(e): log p(v) = ln2 d_v - ln s, H = ln s - ln2 a / s.
// Threads, warps and the CTAs of a cluster are joined by the same rule in a fixed order.
//
// The most likely words cost the pass next to nothing: it leaves every thread's largest value, the batch of its words where that first
// stood, and the largest of its other batches. Of each warp's 32 the j-th largest, and of the warps' the smallest, is a bar that
// at least `top` words reach; those that do lie in the few threads whose largest does, in that batch alone unless another batch's
// largest reaches the bar too. These words are read once more (from L2) and those that reach the bar collected as 64-bit
// keys (the value's order, then the lower index), whose places are counted: equal values need no rule of their own, and no
// order of arrival shows. Rows with more such words than places to collect them (one value everywhere, hardly a number above
// -inf) go through the row again, each warp keeping the best 32 of its words sorted, one a lane.
//
// Bound by memory: the logits are read once (the gradient: read once, written once). 1024 rows of 262144 words in bf16: 86 us (6250
// GB/s), their gradient 159 us (6750 GB/s). Five such rows with five alternatives, a cluster of 16 CTAs each: 6.9 us, latency. 333 rows of
// 50257 in fp32 with 20 alternatives: 19 us (3520 GB/s): two or three CTAs an SM, whose first loads and last choices stand alone.
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
__device__ __forceinline__ float min_nan(float a, float b) {
  float r;
  asm("min.NaN.f32 %0, %1, %2;" : "=f"(r) : "f"(a), "f"(b));
  return r;
}

__device__ __forceinline__ void fadd2_rn(float& d0, float& d1, float a0, float a1, float b0, float b1) {
  asm("{\n\t.reg .b64 ra, rb, rd;\n\tmov.b64 ra, {%2, %3};\n\tmov.b64 rb, {%4, %5};\n\tadd.rn.f32x2 rd, ra, rb;\n\tmov.b64 {%0, %1}, rd;\n\t}"
      : "=f"(d0), "=f"(d1)
      : "f"(a0), "f"(a1), "f"(b0), "f"(b1));
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
  template <int U>
  static __device__ __forceinline__ float largest(const uint4 (&r)[U]) {
    float m = -INFINITY;
#pragma unroll
    for (int u = 0; u < U; ++u)
      m = fmaxf(m, fmaxf(fmaxf(__uint_as_float(r[u].x), __uint_as_float(r[u].y)), fmaxf(__uint_as_float(r[u].z), __uint_as_float(r[u].w))));
    return m;
  }
  static __device__ __forceinline__ float word(const uint4& r, int i) {
    return __uint_as_float(i < 2 ? (i ? r.y : r.x) : (i == 2 ? r.z : r.w));
  }
  // Nothing below `to` (a NaN stays one).
  static __device__ __forceinline__ uint4 raise(const uint4& r, float to) {
    return make_uint4(__float_as_uint(max_nan(__uint_as_float(r.x), to)), __float_as_uint(max_nan(__uint_as_float(r.y), to)),
                      __float_as_uint(max_nan(__uint_as_float(r.z), to)), __float_as_uint(max_nan(__uint_as_float(r.w), to)));
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
  template <int U>
  static __device__ __forceinline__ float largest(const uint4 (&r)[U]) {
    uint32_t m = max2(max2(r[0].x, r[0].y), max2(r[0].z, r[0].w));
#pragma unroll
    for (int u = 1; u < U; ++u) m = max2(m, max2(max2(r[u].x, r[u].y), max2(r[u].z, r[u].w)));
    return fmaxf(fmaxf(__uint_as_float(m << 16), __uint_as_float(m & 0xffff0000u)), -INFINITY);   // NaN only where nothing else is
  }
  static __device__ __forceinline__ float word(const uint4& r, int i) {
    const uint32_t w = i < 4 ? (i < 2 ? r.x : r.y) : (i < 6 ? r.z : r.w);
    return __uint_as_float(i & 1 ? w & 0xffff0000u : w << 16);
  }
  static __device__ __forceinline__ uint4 raise(const uint4& r, float to) {
    const uint32_t b = pack_bf16x2_cvt(to, to);
    auto up = [&](uint32_t w) {
      uint32_t o;
      asm("max.NaN.bf16x2 %0, %1, %2;" : "=r"(o) : "r"(w), "r"(b));
      return o;
    };
    return make_uint4(up(r.x), up(r.y), up(r.z), up(r.w));
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
// Weights are 2^(x c - ref), c = scale log2(e), with ref the rounded m c, so that a word costs one fused product and ref's rounding
// cancels where log probabilities are taken. Beyond 2^26 that rounding passes 2, and soon 2^128 of a weight: there (a row of nothing but
// a type's lowest value, scales far from one) they are 2^((x - m) c).
struct Sums {
  float m = -INFINITY, ref = 0.0f;   // ref: 0 while m is -inf
  float s0 = 0.0f, s1 = 0.0f, a0 = 0.0f, a1 = 0.0f;
  static __device__ __forceinline__ bool beyond(float r) { return !(fabsf(r) < 0x1p26f); }
  // Not one product with the differences below: to the same largest value they are 0.
  static __device__ __forceinline__ float ref_of(float m, float c) { return m == -INFINITY ? 0.0f : __fmul_rn(m, c); }
  __device__ __forceinline__ bool wild() const { return beyond(ref); }
  // To a new largest value. Differences below -1000 are as good as -inf, whose product with 0 would be NaN.
  __device__ __forceinline__ void rise(float to, float c) {
    const float was = m, from = ref;
    m = to;
    ref = ref_of(to, c);
    float d = from - ref;
    if (beyond(from) || wild()) d = !wild() ? fmaf(was, c, -ref) : beyond(from) ? (was - to) * c : fmaf(-to, c, from);
    d = was == -INFINITY ? -1000.0f : fmaxf(d, -1000.0f);
    const float f = ex2(d);
    a0 = f * fmaf(s0, d, a0);
    a1 = f * fmaf(s1, d, a1);
    s0 *= f;
    s1 *= f;
  }
  // Where words weigh nothing, and may be taken for larger ones that weigh nothing either: an infinite difference would make NaN of
  // its weight of 0. 2^-7 of m is the least that a bf16 below m tells from it.
  __device__ __forceinline__ float least(float c) const {
    const float at = m == -INFINITY ? 0.0f : m;
    return fmaxf(at - fmaxf(__fdividef(1000.0f, c), fabsf(at) * 0x1p-6f), -3.4028235e38f);
  }
  // Two words, none below least(), of a row that is not wild.
  __device__ __forceinline__ void add2(float x0, float x1, float c) {
    float d0, d1;
    ffma2_rn(d0, d1, x0, x1, c, c, -ref, -ref);
    const float e0 = ex2(d0), e1 = ex2(d1);
    fadd2_rn(s0, s1, s0, s1, e0, e1);
    ffma2_rn(a0, a1, e0, e1, d0, d1, a0, a1);
  }
  __device__ __forceinline__ void add(float x, float c) {
    const float d = max_nan(distance(x, c), -1000.0f), e = ex2(d);
    s0 += e;
    a0 = fmaf(e, d, a0);
  }
  // log2 of a word's weight.
  __device__ __forceinline__ float distance(float x, float c) const { return wild() ? (x - m) * c : fmaf(x, c, -ref); }
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

// U pieces of N words a lane, those of piece u at index at[u] and on (-1: none), `largest` of all: what reaches the bar `tau` (an order)
// goes into the list. Later calls bring later words, so a word equal to the k-th of the list when the call begins is out.
template <typename W, int U>
__device__ __forceinline__ void consider(Best& b, int k, uint32_t tau, const uint4 (&raw)[U], const int (&at)[U], int words, float largest) {
  constexpr int N = W::N;
  const unsigned who = __ballot_sync(0xffffffffu, (b.open || largest > b.bar) && order_of(largest) >= tau);
  if (!who) return;
  Key used = 0;
  if (__popc(who) >= 8) {   // the lanes' best first: they raise the bar for the rest
#pragma unroll
    for (int u = 0; u < U; ++u)
      for (int i = 0; i < words; ++i) {
        const Key y = at[u] < 0 ? 0 : key_of(W::word(raw[u], i), at[u] + i);
        used = y > used ? y : used;
      }
    b.merge(used);
    b.mark(k);
  }
#pragma unroll
  for (int u = 0; u < U; ++u) {
    const float bar = b.bar;
    const bool open = b.open;
    uint32_t hits = 0;
#pragma unroll
    for (int i = 0; i < N; ++i) {
      const float x = W::word(raw[u], i);
      hits |= (i < words && (open || x >= bar) && order_of(x) >= tau ? 1u : 0u) << i;
    }
    if (at[u] < 0) hits = 0;
    for (uint32_t any = __reduce_or_sync(0xffffffffu, hits); any; any &= any - 1) {
      const int i = __ffs(any) - 1;
      const Key y = key_of(W::word(raw[u], i), at[u] + i);
      unsigned in = __ballot_sync(0xffffffffu, (hits >> i & 1) && y > b.kth && y != used);
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

constexpr int kScoreKeys = 512;   // keys of one CTA, or of the cluster's lists, that are ranked against each other
static_assert(kScoreKeys >= kScoreMaxCluster * AQ_MAX_TOP, "the cluster's lists fit");

template <int WARPS>
struct ScoreShared {
  Key keys[kScoreKeys];
  Key lists[WARPS < kScoreWarps ? 1 : kScoreMaxCluster][32];   // rank 0's
  float cta_m[kScoreMaxCluster], cta_s[kScoreMaxCluster], cta_a[kScoreMaxCluster];   // rank 0's
  float m[WARPS], s[WARPS], a[WARPS];
  uint32_t bar[WARPS];
  int32_t n_keys;
};

// The sums of n parts (n <= N, a power of two up to 32), every lane of a warp the same, in a fixed order: s0 and a0 of the result hold them.
template <int N>
__device__ __forceinline__ Sums join(const float* m, const float* s, const float* a, int n, float c) {
  const int i = threadIdx.x & (N - 1);
  Sums one;
  if (i < n) {
    one.m = m[i];
    one.ref = Sums::ref_of(one.m, c);
    one.s0 = s[i];
    one.a0 = a[i];
  }
  float top = one.m;
#pragma unroll
  for (int o = N / 2; o > 0; o >>= 1) top = fmaxf(top, __shfl_xor_sync(0xffffffffu, top, o));
  one.rise(top, c);
#pragma unroll
  for (int o = N / 2; o > 0; o >>= 1) {
    one.s0 += __shfl_xor_sync(0xffffffffu, one.s0, o);
    one.a0 += __shfl_xor_sync(0xffffffffu, one.a0, o);
  }
  return one;
}

// WARPS: eight, or two or four for many rows of few words (a cluster of one).
template <typename T, bool TOP, int WARPS>
__global__ void __launch_bounds__(32 * WARPS, (TOP ? kScorePerSm : kScorePerSm + 1) * kScoreWarps / WARPS) aq_scores_kernel(const __grid_constant__ ScoreParams p) {
  using W = Words<T>;
  constexpr int N = W::N, U = 4, kThreads = 32 * WARPS;
  __shared__ ScoreShared<WARPS> sh;
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
  // the words before and after the body, one a lane
  const bool before = rank == 0 && warp == 0 && lane < w.head, after = rank == C - 1 && warp == 0 && lane < w.tail;
  const int after_at = w.head + w.vecs * N + lane;
  const float x_before = before ? W::one(row + lane) : -INFINITY, x_after = after ? W::one(row + after_at) : -INFINITY;
  if (warp == 0) {
    q.rise(fmaxf(x_before, fmaxf(x_after, -INFINITY)), c);
    if (before) q.add(x_before, c);
    if (after) q.add(x_after, c);
  }
  const T* body = row + w.head;
  const int v0 = static_cast<int>(static_cast<int64_t>(w.vecs) * rank / C), v1 = static_cast<int>(static_cast<int64_t>(w.vecs) * (rank + 1) / C);
  const int vw = v0 + warp * 32;   // a warp's words of a round are neighbours
  // A batch of the warp's words: U pieces of 16 bytes a lane, b batches from its first.
  constexpr int kStep = U * kThreads;
  const int batches = v1 > vw ? (v1 - vw + kStep - 1) / kStep : 0;
  auto fetch = [&](uint4 (&raw)[U], int b) {
    const int v = vw + lane + b * kStep;
    if (v - lane + 32 + (U - 1) * kThreads <= v1) {
#pragma unroll
      for (int u = 0; u < U; ++u) raw[u] = ld_words(body + static_cast<int64_t>(v + u * kThreads) * N);
    } else {
#pragma unroll
      for (int u = 0; u < U; ++u)
        raw[u] = v + u * kThreads < v1 ? ld_words(body + static_cast<int64_t>(v + u * kThreads) * N) : make_uint4(W::kNone, W::kNone, W::kNone, W::kNone);
    }
  };
  float second = -INFINITY;   // the largest of all batches but the one that holds the thread's largest
  int best_v = -1;            // that batch's first piece
  auto take = [&](const uint4 (&raw)[U], int v) {
    const float top = W::largest(raw);
    if (TOP) {
      second = fmaxf(second, fminf(q.m, top));
      best_v = top > q.m ? v : best_v;
    }
    q.rise(fmaxf(q.m, top), c);
    if (!q.wild()) {
      const float least = q.least(c);
#pragma unroll
      for (int u = 0; u < U; ++u) {
        float x[N];
        W::unpack(W::raise(raw[u], least), x);
#pragma unroll
        for (int i = 0; i < N; i += 2) q.add2(x[i], x[i + 1], c);
      }
    } else {   // a largest word of plus infinity, or at the very ends of the range
#pragma unroll
      for (int u = 0; u < U; ++u)
#pragma unroll 1
        for (int i = 0; i < N; ++i) q.add(W::word(raw[u], i), c);
    }
  };
  {
    uint4 even[U], odd[U];   // the next batch is on its way under each
    if (batches > 0) fetch(even, 0);
#pragma unroll 1
    for (int b = 0; b < batches; b += 2) {
      if (b + 1 < batches) fetch(odd, b + 1);
      take(even, vw + lane + b * kStep);
      if (b + 1 >= batches) break;
      if (b + 2 < batches) fetch(even, b + 2);
      take(odd, vw + lane + (b + 1) * kStep);
    }
  }

  // the warp's sums, and its bar: of the warps whose lanes all have words, each has at least ceil(top / warps) threads with a word that
  // reaches it
  uint32_t left = order_of(q.m);   // of this thread's largest, before it becomes the warp's
  const bool mine = best_v >= 0;
  const int full = min(WARPS, (v1 - v0) / 32), share = full ? (p.top + full - 1) / full : 33;
  const uint32_t largest = left;
  float m = q.m;
#pragma unroll
  for (int o = 16; o > 0; o >>= 1) m = fmaxf(m, __shfl_xor_sync(0xffffffffu, m, o));
  q.rise(m, c);
  float qs = q.s0 + q.s1, qa = q.a0 + q.a1;
#pragma unroll
  for (int o = 16; o > 0; o >>= 1) {
    qs += __shfl_xor_sync(0xffffffffu, qs, o);
    qa += __shfl_xor_sync(0xffffffffu, qa, o);
  }
  if (TOP) {
    uint32_t bar = 0;
    for (int i = 0; i < share && share <= 32; ++i) {
      bar = __reduce_max_sync(0xffffffffu, left);
      if (lane == __ffs(__ballot_sync(0xffffffffu, left == bar)) - 1) left = 0;
    }
    if (lane == 0) sh.bar[warp] = warp < full ? bar : 0xffffffffu;
    if (tid == 0) sh.n_keys = 0;
  }
  if (lane == 0) {
    sh.m[warp] = q.m;
    sh.s[warp] = qs;
    sh.a[warp] = qa;
  }
  __syncthreads();

  // What reaches the bar, on its way; every warp adds up the CTA's sums meanwhile.
  uint32_t tau = 0;
  float bar = 0.0f;
  bool all = false;
  uint4 raw[U];
  int at[U];
  if (TOP) {
    tau = sh.bar[0];
#pragma unroll
    for (int i = 1; i < WARPS; ++i) tau = min(tau, sh.bar[i]);
    if (full == 0 || share > 32 || tau <= order_of(-INFINITY)) tau = 0;   // too few threads with a number above -inf
    bar = value_of(tau);
    all = tau && order_of(second) >= tau;
    const bool one = tau && !all && mine && largest >= tau;   // in one batch alone
#pragma unroll
    for (int u = 0; u < U; ++u) {
      const int v = best_v + u * kThreads;
      at[u] = w.head + v * N;
      raw[u] = one && v < v1 ? *reinterpret_cast<const uint4*>(body + static_cast<int64_t>(v) * N) : make_uint4(W::kNone, W::kNone, W::kNone, W::kNone);
    }
  }
  Sums sum = join<WARPS>(sh.m, sh.s, sh.a, WARPS, c);

  int n = 0;
  if (TOP) {
    auto note_pieces = [&] {
#pragma unroll
      for (int u = 0; u < U; ++u) {
        uint32_t hits = 0;
#pragma unroll
        for (int i = 0; i < N; ++i) hits |= (W::word(raw[u], i) >= bar ? 1u : 0u) << i;
        if (!hits) continue;
        for (int k = atomicAdd(&sh.n_keys, __popc(hits)); hits; hits &= hits - 1, ++k) {
          const int i = __ffs(hits) - 1;
          if (k < kScoreKeys) sh.keys[k] = key_of(W::word(raw[u], i), at[u] + i);
        }
      }
    };
    if (tau) {
      note_pieces();
      auto note = [&](float x, int where) {
        if (!(x >= bar)) return;
        const int k = atomicAdd(&sh.n_keys, 1);
        if (k < kScoreKeys) sh.keys[k] = key_of(x, where);
      };
      if (before) note(x_before, lane);
      if (after) note(x_after, after_at);
      // threads with several such batches: all of their words, by the warp
      const int rounds = v1 > vw ? (v1 - vw + kThreads - 1) / kThreads : 0;   // pieces of a thread, at most
      for (unsigned whole = __ballot_sync(0xffffffffu, all); whole; whole &= whole - 1) {
        const int first = vw + __ffs(whole) - 1;
        for (int i0 = lane; i0 - lane < rounds; i0 += U * 32) {
#pragma unroll
          for (int u = 0; u < U; ++u) {
            const int v = first + (i0 + u * 32) * kThreads;
            at[u] = w.head + v * N;
            raw[u] = i0 + u * 32 < rounds && v < v1 ? *reinterpret_cast<const uint4*>(body + static_cast<int64_t>(v) * N) : make_uint4(W::kNone, W::kNone, W::kNone, W::kNone);
          }
          note_pieces();
        }
      }
    }
    __syncthreads();
    n = sh.n_keys;
    if (!tau || n > kScoreKeys) {   // through the words again, in their order
      Best best;
      if (rank == 0 && warp == 0 && w.head > 0) {
        const uint4 one[1] = {make_uint4(sizeof(T) == 4 ? __float_as_uint(x_before) : __float_as_uint(x_before) >> 16, 0, 0, 0)};
        const int where[1] = {before ? lane : -1};
        consider<W, 1>(best, p.top, tau, one, where, 1, x_before);
      }
#pragma unroll 1
      for (int b = 0; b < batches; ++b) {
        const int v = vw + lane + b * kStep;
        fetch(raw, b);
#pragma unroll
        for (int u = 0; u < U; ++u) at[u] = v + u * kThreads < v1 ? w.head + (v + u * kThreads) * N : -1;
        consider<W, U>(best, p.top, tau, raw, at, N, W::largest(raw));
      }
      if (rank == C - 1 && warp == 0 && w.tail > 0) {
        const uint4 one[1] = {make_uint4(sizeof(T) == 4 ? __float_as_uint(x_after) : __float_as_uint(x_after) >> 16, 0, 0, 0)};
        const int where[1] = {after ? after_at : -1};
        consider<W, 1>(best, p.top, tau, one, where, 1, x_after);
      }
      __syncthreads();
      sh.keys[tid] = best.key;   // none where a warp has fewer words
      n = kThreads;
      __syncthreads();
    }
  }
  // The number of keys above one is its place.
  auto place_of = [&](Key x) {
    int place = 0;
#pragma unroll 8
    for (int i = 0; i < n; ++i) place += sh.keys[i] > x;
    return place;
  };

  if (C > 1) {
    asm volatile("barrier.cluster.wait.acquire.aligned;" ::: "memory");   // rank 0 runs
    if (tid == 0) {
      asm volatile("st.shared::cluster.f32 [%0], %1;" ::"r"(cluster_map(&sh.cta_m[rank], 0)), "f"(sum.m) : "memory");
      asm volatile("st.shared::cluster.f32 [%0], %1;" ::"r"(cluster_map(&sh.cta_s[rank], 0)), "f"(sum.s0) : "memory");
      asm volatile("st.shared::cluster.f32 [%0], %1;" ::"r"(cluster_map(&sh.cta_a[rank], 0)), "f"(sum.a0) : "memory");
    }
    if (TOP) {   // this CTA's list; its end is filled up with none where it has fewer words than places
      auto put = [&](int place, Key x) { asm volatile("st.shared::cluster.u64 [%0], %1;" ::"r"(cluster_map(&sh.lists[rank][place], 0)), "l"(x) : "memory"); };
      for (int k = tid; k < n; k += kThreads) {
        const Key x = sh.keys[k];
        if (!x) continue;
        const int place = place_of(x);
        if (place < p.top) put(place, x);
      }
      if (n < p.top || n == kThreads) {
        const int held = place_of(0);
        if (tid >= held && tid < p.top) put(tid, 0);
      }
    }
    cluster_sync_all();
    if (rank != 0) return;
    sum = join<kScoreMaxCluster>(sh.cta_m, sh.cta_s, sh.cta_a, C, c);
    if (TOP) {
      // Of the CTAs' lists what reaches the larger of two bars, each of which `top` words do: the largest of their last places, and the
      // smallest of the places that make up `top` together (16 lists of 32: hundreds of words reach the first, some 70 the second).
      const uint32_t last = lane < C ? static_cast<uint32_t>(sh.lists[lane][p.top - 1] >> 32) : 0u;
      const uint32_t shared = lane < C ? static_cast<uint32_t>(sh.lists[lane][(p.top + C - 1) / C - 1] >> 32) : 0xffffffffu;
      const uint32_t floor = max(__reduce_max_sync(0xffffffffu, last), __reduce_min_sync(0xffffffffu, shared));
      if (tid == 0) sh.n_keys = 0;
      __syncthreads();
      for (int i = tid; i < C * 32; i += kThreads) {
        const Key x = i % 32 < p.top ? sh.lists[i / 32][i % 32] : 0;
        if (x && static_cast<uint32_t>(x >> 32) >= floor) sh.keys[atomicAdd(&sh.n_keys, 1)] = x;
      }
      __syncthreads();
      n = sh.n_keys;
    }
  }
  const bool none = sum.m == -INFINITY && sum.s0 == 0.0f;   // no word has any mass
  const float ln_s = logf(sum.s0);
  auto logp = [&](float x) {
    const float d = sum.distance(x, c) * kLn2;   // past the range, where log2(e) takes it, the difference itself
    return none ? -INFINITY : (fabsf(d) < 1e37f ? d : (x - sum.m) * p.scale) - ln_s;
  };
  if (tid == 0) {
    if (p.lse) p.lse[r] = none ? -INFINITY : sum.m == -INFINITY ? sum.s0 : sum.wild() ? fmaf(sum.m, p.scale, ln_s) : fmaf(sum.ref, kLn2, ln_s);
    if (p.entropy) p.entropy[r] = none ? 0.0f : ln_s - kLn2 * (sum.a0 / sum.s0);
    if (p.logprob) p.logprob[r] = token < 0 || token >= p.vocab ? 0.0f : logp(given);
  }
  if (TOP) {
    for (int k = tid; k < n; k += kThreads) {
      const Key x = sh.keys[k];
      if (!x) continue;
      const int place = place_of(x);
      if (place >= p.top) continue;
      const float v = value_of(static_cast<uint32_t>(x >> 32));
      p.top_token[r * p.top + place] = static_cast<int32_t>(0xffffffffu - static_cast<uint32_t>(x));
      p.top_logprob[r * p.top + place] = logp(v);
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
    const float d = min_nan(max_nan(fmaf(x, p.scale, -lse) * kLog2e, -1000.0f), 0.0f);   // lse is rounded: no p above one
    return none ? 0.0f : ex2(d) * fmaf(B, d, A);
  };
  const bool whole = ((reinterpret_cast<uintptr_t>(row) ^ reinterpret_cast<uintptr_t>(out)) & 15) == 0;
  // Rows that start at different places of a 16-byte piece go word by word: 1024 rows of 50257 out of rows of 50304, us, gradient apart
  // and alike: bf16 159 and 38.5, fp32 142 and 65.5.
  if (!whole) {
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
cudaError_t launch_scores(const ScoreParams& p, unsigned grid, int warps, cudaStream_t st) {
  if (warps == 2) return launch_serve(aq_scores_kernel<T, TOP, 2>, p, grid, 64, 0, st);
  if (warps == 4) return launch_serve(aq_scores_kernel<T, TOP, 4>, p, grid, 128, 0, st);
  static std::atomic<uint64_t> ready{0};   // devices on which the kernel may use clusters of 16
  if (p.cluster > 8 && !(ready.load() >> p.device & 1)) {
    const cudaError_t e = cudaFuncSetAttribute(aq_scores_kernel<T, TOP, kScoreWarps>, cudaFuncAttributeNonPortableClusterSizeAllowed, 1);
    if (e != cudaSuccess) return e;
    ready.fetch_or(1ull << p.device);
  }
  return launch_serve(aq_scores_kernel<T, TOP, kScoreWarps>, p, grid, kScoreThreads, 0, st, p.cluster);
}

aq_status check_logits(const void* logits, int64_t ld, int64_t rows, int32_t vocab, int32_t type, float scale, const char* who) {
  if (rows < 0) return serve_fail(AQ_ERR_SHAPE, "%s: rows=%lld is negative", who, (long long)rows);
  if (vocab < 1 || vocab > (1 << 30)) return serve_fail(AQ_ERR_SHAPE, "%s: vocab=%d outside [1, 2^30]", who, vocab);
  if (type != AQ_PROB_F32 && type != AQ_PROB_BF16) return serve_fail(AQ_ERR_INVALID_ARG, "%s: unknown element type %d", who, type);
  if (!(scale >= 1e-30f) || !(scale <= 1e30f)) return serve_fail(AQ_ERR_INVALID_ARG, "%s: scale must lie between 1e-30 and 1e30", who);
  if (rows > 0 && !logits) return serve_fail(AQ_ERR_INVALID_ARG, "%s: logits must be non-NULL", who);
  if (ld < vocab && rows > 1) return serve_fail(AQ_ERR_SHAPE, "%s: ld=%lld < vocab=%d", who, (long long)ld, vocab);
  if (!serve_aligned(logits, type == AQ_PROB_F32 ? 4 : 2)) return serve_fail(AQ_ERR_ALIGNMENT, "%s: logits must be aligned to their elements", who);
  return AQ_OK;
}

// CTAs that share a row. Three CTAs an SM are what fills the GPU once (four without alternatives); a row's part is no smaller than 8192
// words, as what comes after its words weighs as much as 4000 of them. One CTA a row, two and four, us: fp32, 300 rows of 151936 words 32.0,
// 29.8, 36.9, with 20 alternatives 40.8, 47.0, 50.6; 120 rows 23.8, 17.3, 15.4, with 20 31.4, 23.4, 27.2; 246 rows of 50257 12.7, 12.0,
// 14.4, with 20 17.8, 22.1, 26.1.
int score_cluster(int64_t rows, int32_t vocab, int32_t top, int sms) {
  int c = 1;
  while (c < kScoreMaxCluster && 2 * rows * c <= (top ? 3ll : 4ll) * sms && vocab / (2 * c) >= 8192) c *= 2;
  return c;
}
// Warps of a CTA: two or four where there are rows enough and a row's bytes are few, so that what comes before and after the words (the
// row's sums joined, its best words placed) goes on in four or two times as many rows at once; alternatives make more of that, but of
// the warps' work too. Eight, four and two warps, us: 4096 rows of 1000 words, fp32, 18.7, -, 6.9; 1000 of 8000 10.4, 7.9, 8.5, with 5
// alternatives 16.3, 13.7, 11.9, with 20 18.0, 15.0, 15.8; bf16, 500 of 16000 5.7, 5.7, 7.4, with 5 10.9, 9.8, 9.6; 1750 of 32000
// with 5 35, 27.9, 25.1, with 20 42, 33, 34; 1000 of 50257 23.2, 21.2, 23.3, with 20 35.6, 33.4, 38, with 32 38.6, 40, 47; fp32, 500 of
// 50257 19.4, 21.1, 30, with 5 28.2, 25.2, 34; 2500 with 20 108, 102, 129; bf16, 1000 of 151936 with 5 64, 71, 81.
// Two without alternatives is for the shortest rows; 1000 of 8000 in fp32 would be 7 % faster with four. Between 20 and 32 alternatives, and between
// 201 and 304 KB a row, nothing was measured: the bounds stand next to the lower of each.
int score_warps(int64_t rows, int64_t bytes, int32_t top, int cluster, int sms) {
  const int64_t fills = rows / sms;   // rows an SM
  if (cluster > 1 || fills < 3 || bytes > 208 * 1024 || (top == 0 && fills < 6 && bytes > 32 * 1024)) return kScoreWarps;
  if (bytes <= 32 * 1024 && (top ? top <= 8 || fills >= 16 : fills >= 6)) return 2;
  if (bytes <= 64 * 1024 && fills >= 8 && top >= 1 && top <= 8) return 2;
  return bytes > 64 * 1024 && top > 20 && fills < 8 ? kScoreWarps : 4;
}
// Blocks that share a row of the gradient: pieces of 48 KB and more, smaller ones while they would not fill the GPU (1024 rows of
// 262144 words in bf16, us: 166 in one piece, 159 in eight; one row 21 and 2.3 in 64).
int score_parts(int64_t rows, int32_t vocab, int size, int sms) {
  int c = 1;
  while (c < 64 && (static_cast<int64_t>(vocab) * size / (2 * c) >= 48 * 1024 || (2 * rows * c <= 2ll * sms && vocab / (2 * c) >= 4096))) c *= 2;
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
  p.cluster = score_cluster(rows, vocab, top, dev.sms);
  if (rows * p.cluster > 0x7fffffffLL) return serve_fail(AQ_ERR_SHAPE, "%s: rows=%lld is too large", who, (long long)rows);
  const unsigned grid = static_cast<unsigned>(rows * p.cluster);
  const cudaStream_t cs = static_cast<cudaStream_t>(stream);
  cudaError_t e;
  const int warps = score_warps(rows, static_cast<int64_t>(vocab) * (type == AQ_PROB_F32 ? 4 : 2), top, p.cluster, dev.sms);
  if (type == AQ_PROB_F32) e = top ? launch_scores<float, true>(p, grid, warps, cs) : launch_scores<float, false>(p, grid, warps, cs);
  else e = top ? launch_scores<uint16_t, true>(p, grid, warps, cs) : launch_scores<uint16_t, false>(p, grid, warps, cs);
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
  p.parts = score_parts(rows, vocab, static_cast<int>(size), dev.sms);
  if (rows * p.parts > 0x7fffffffLL) return serve_fail(AQ_ERR_SHAPE, "%s: rows=%lld is too large", who, (long long)rows);
  const unsigned grid = static_cast<unsigned>(rows * p.parts);
  const cudaStream_t cs = static_cast<cudaStream_t>(stream);
  return serve_launched(type == AQ_PROB_F32 ? launch_serve(aq_scores_grad_kernel<float>, p, grid, kScoreThreads, 0, cs)
                                            : launch_serve(aq_scores_grad_kernel<uint16_t>, p, grid, kScoreThreads, 0, cs),
                        who);
}
