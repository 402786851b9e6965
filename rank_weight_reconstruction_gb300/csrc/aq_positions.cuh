// aq_positions.cuh -- what the kernels that turn heads share (positions, the cache's write, the head norms and their gradient):
// how a group of lanes holds a head, the sines and cosines of a token, and the checks of [T, heads, head_dim] tensors. Not
// part of the public ABI.
#pragma once

#include "aq_serve.h"

namespace aq {

// Not through the read-only path: in place, the same lane writes the chunk back.
__device__ __forceinline__ uint4 ld_stream(const void* p) {
  uint4 r;
  asm volatile("ld.global.L1::no_allocate.v4.u32 {%0, %1, %2, %3}, [%4];"
               : "=r"(r.x), "=r"(r.y), "=r"(r.z), "=r"(r.w)
               : "l"(p)
               : "memory");
  return r;
}
__device__ __forceinline__ void unpack8(const uint4& r, float (&x)[8]) {
  const uint32_t w[4] = {r.x, r.y, r.z, r.w};
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    x[2 * i] = __uint_as_float(w[i] << 16);
    x[2 * i + 1] = __uint_as_float(w[i] & 0xffff0000u);
  }
}
__device__ __forceinline__ uint4 pack8(const float (&x)[8]) {
  return make_uint4(pack_bf16x2_cvt(x[0], x[1]), pack_bf16x2_cvt(x[2], x[3]), pack_bf16x2_cvt(x[4], x[5]),
                    pack_bf16x2_cvt(x[6], x[7]));
}

// The two chunks of eight elements that lane u of a vector holds: load 0 of the lanes covers one stretch of
// memory, load 1 another. In the half layout a rotating lane's chunks rotate against each other.
template <bool HALF>
struct Chunks {
  int c0, c1;        // chunk indices (element / 8)
  bool turns0, turns1;
  __device__ __forceinline__ Chunks(int u, int rot16, int d16) {
    if (HALF) {
      c0 = u < rot16 ? u : u + rot16;
      c1 = u < rot16 ? u + rot16 : u + d16;
      turns0 = turns1 = u < rot16;
    } else {
      c0 = u;
      c1 = u + d16;
      turns0 = c0 < 2 * rot16;
      turns1 = c1 < 2 * rot16;
    }
  }
  // index of pair i (of eight) among the frequencies
  __device__ __forceinline__ int pair(int u, int i) const { return HALF ? u * 8 + i : (i < 4 ? c0 * 4 + i : c1 * 4 + i - 4); }
};

// second: whether b turns (interleaved, part of a head: a lane's second chunk may lie past rotary_dim, where a sine of 0 would
// still make NaN of an infinity's neighbour).
template <bool HALF>
__device__ __forceinline__ void rotate16(float (&a)[8], float (&b)[8], const float (&c)[8], const float (&s)[8], bool second) {
  if (HALF) {
#pragma unroll
    for (int i = 0; i < 8; ++i) {
      const float x = a[i], y = b[i];
      a[i] = fmaf(x, c[i], -(y * s[i]));
      b[i] = fmaf(y, c[i], x * s[i]);
    }
  } else {
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      const float x = a[2 * i], y = a[2 * i + 1];
      a[2 * i] = fmaf(x, c[i], -(y * s[i]));
      a[2 * i + 1] = fmaf(y, c[i], x * s[i]);
      const float z = b[2 * i], w = b[2 * i + 1];
      const float z1 = fmaf(z, c[4 + i], -(w * s[4 + i])), w1 = fmaf(w, c[4 + i], z * s[4 + i]);
      b[2 * i] = second ? z1 : z;
      b[2 * i + 1] = second ? w1 : w;
    }
  }
}

// The sines and cosines of a token at pos, times the magnitude, for the eight pairs the lane rotates. SPLIT: the groups of a
// warp are at one token, and each works out its part of the eight and passes it round (every lane of the warp comes here).
template <bool HALF, int GW, bool SPLIT>
__device__ __forceinline__ void angles(const Chunks<HALF>& ch, int u, const uint64_t* freq, int64_t pos, float magnitude, float sin_sign,
                                       float (&c)[8], float (&s)[8]) {
  constexpr int kShare = SPLIT ? (32 / GW < 8 ? 32 / GW : 8) : 1;
  const int lane = threadIdx.x & 31, part = SPLIT ? (lane / GW) % kShare : 0;
  float cm[8 / kShare], sm[8 / kShare];
#pragma unroll
  for (int k = 0; k < 8 / kShare; ++k) {
    const int i = k * kShare + part;
    cm[k] = 1.0f;
    sm[k] = 0.0f;
    if (freq && (i < 4 ? ch.turns0 : ch.turns1)) {   // half layout: both or neither
      const uint64_t phase = static_cast<uint64_t>(pos) * freq[ch.pair(u, i)];
      float sn, cs;
      sincospif(static_cast<float>(static_cast<int32_t>(phase >> 32)) * 0x1p-31f, &sn, &cs);
      cm[k] = cs * magnitude;
      sm[k] = sn * sin_sign;
    }
  }
#pragma unroll
  for (int i = 0; i < 8; ++i) {
    const int from = (lane & ~(GW * kShare - 1)) + (i % kShare) * GW + u;
    c[i] = SPLIT ? __shfl_sync(0xffffffffu, cm[i / kShare], from) : cm[i / kShare];
    s[i] = SPLIT ? __shfl_sync(0xffffffffu, sm[i / kShare], from) : sm[i / kShare];
  }
}

inline int group_width(int D) {
  int gw = 1;
  while (gw * 16 < D) gw *= 2;
  return gw;
}
inline int log2_of(int v) {
  int s = 0;
  while ((1 << s) < v) ++s;
  return s;
}

// log2 of the groups that share a token, taking neighbouring heads, each walking the rest of them with its angles: as many as a warp
// holds, so that the angles are worked out once a warp (and 512 bytes to 2 KB read in one stretch where heads are the inner
// dimension), more while the call has fewer than `fill` groups, and never more than heads or a block of 256 threads.
inline int share_token(int64_t T, int heads, int gw, int64_t fill) {
  int most = 0;
  while ((2 << most) <= heads && (2 << most) <= 256 / gw) ++most;
  int s = log2_of(32 / gw) < most ? log2_of(32 / gw) : most;
  while (s < most && (T << s) < fill) ++s;
  return s;
}

// Heads of all of a call's tensors together: the kernels walk them as one list, a block's groups at a time.
inline aq_status check_head_count(int64_t heads, const char* who) {
  if (heads > (1 << 30)) return serve_fail(AQ_ERR_SHAPE, "%s: %lld heads of a token are more than 2^30", who, (long long)heads);
  return AQ_OK;
}
// x [T, heads, D] with the given strides: shape, alignment.
inline aq_status check_heads(const void* x, int64_t tok, int64_t head, int32_t heads, int32_t D, const char* name,
                      const char* who) {
  if (!x) return serve_fail(AQ_ERR_INVALID_ARG, "%s: %s must be non-NULL", who, name);
  if (!serve_aligned(x, 16) || tok % 8 || head % 8)
    return serve_fail(AQ_ERR_ALIGNMENT, "%s: %s must be 16-byte aligned with strides that are multiples of 8", who, name);
  if (tok < 0 || head < 0 || (heads > 1 && head < D))
    return serve_fail(AQ_ERR_SHAPE, "%s: %s strides (token %lld, head %lld) do not hold heads of %d", who, name,
                      (long long)tok, (long long)head, D);
  return AQ_OK;
}
// An output's rows may not fall on each other.
inline aq_status check_out_heads(int64_t tok, int64_t head, int64_t T, int32_t heads, int32_t D, const char* name,
                          const char* who) {
  const bool tok_outer = T <= 1 || tok >= (heads - 1) * head + D;
  const bool head_outer = heads <= 1 ? (T <= 1 || tok >= D) : (head >= (T - 1) * tok + D && (T <= 1 || tok >= D));
  if (!tok_outer && !head_outer)
    return serve_fail(AQ_ERR_SHAPE, "%s: rows of %s overlap (token stride %lld, head stride %lld)", who, name,
                      (long long)tok, (long long)head);
  return AQ_OK;
}
inline ByteSpan heads_span(const void* x, int64_t tok, int64_t head, int64_t T, int32_t heads, int32_t D) {
  if (!x || T < 1 || heads < 1) return ByteSpan();
  return byte_span(x, 1, 0, (T - 1) * tok + (heads - 1) * head + D, 2);
}

// The same with its rows told apart, where its heads lie within a token's row.
inline ByteRows heads_rows(const aq_heads* x, int64_t T, int32_t D) {
  if (!x || T < 1) return ByteRows();
  const int64_t row = (x->heads - 1) * x->head + D;
  if (row <= x->tok) return ByteRows(x->data, T, x->tok * 2, row * 2);
  const int64_t all = ((T - 1) * x->tok + row) * 2;
  return ByteRows(x->data, 1, all, all);
}
// Checks of an aq_head_norm (NULL: no norm).
inline aq_status check_head_norm(const aq_head_norm* n, const char* name, const char* who) {
  if (!n) return AQ_OK;
  if (!(n->eps > 0.0f) || !(n->eps < 1e30f)) return serve_fail(AQ_ERR_INVALID_ARG, "%s: %s.eps must be positive and finite", who, name);
  if (!(n->offset - n->offset == 0.0f)) return serve_fail(AQ_ERR_INVALID_ARG, "%s: %s.offset must be finite", who, name);
  if (!serve_aligned(n->weight, 16)) return serve_fail(AQ_ERR_ALIGNMENT, "%s: %s.weight must be 16-byte aligned", who, name);
  return AQ_OK;
}

// The head norms' launch (checked arguments): q into q_out, and k into k_out or, with the values, into the cache.
aq_status run_head_norm(const aq_head_norm* q_norm, const aq_head_norm* k_norm, const aq_rope_spec* rope, const int32_t* pos, int64_t T,
                        int32_t D, const aq_heads* q, const aq_heads* q_out, const aq_heads* k, const aq_heads* k_out, const aq_heads* v,
                        const aq_kv_cache* cache, const int64_t* slots, cudaStream_t st, const char* who);

}  // namespace aq
