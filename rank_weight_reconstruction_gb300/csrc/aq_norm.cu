// aq_norm.cu -- head norms with the rotation behind them: aq_qk_norm_rope, the cache's write with norms, and the gradient
// aq_qk_norm_rope_backward.
//
// With r = 1 / sqrt(mean(x^2) + eps), n = x r, f = offset + w:  y = R (n f), and from dy
//   g = R^T dy,  dx = r (g f - n mean(g f n)),  dw_i = sum over tokens and heads of g_i n_i.
// Bound by memory: every element is read once (the gradient: x and dy) and written once. 16385 tokens of 16 + 4 heads of 128 take
// 29.6 us (5670 GB/s), the gradient of 8195 tokens of 32 + 8 heads 45 us (5600 GB/s); issue slots are 60 % used. A group of lanes holds a head as in the
// rotation, 16 elements a lane, kept as the eight pairs that turn against each other in either order, so that squares, scales and
// turns are packed products of two; a head's sums are a few shuffles. The factors f stay in registers while a group walks the heads
// of q, then those of k. In the gradient the weight's sums stay in 16 registers a lane over all the heads that the lane sees,
// so a block is given heads of q alone or of k alone; the groups' sums meet in shared memory, the blocks' in their cluster's where
// they are few, otherwise in the workspace, where a second launch adds them up, all in an order fixed by the sizes and the device's SM count.
#include <algorithm>

#include "aq_positions.cuh"

namespace aq {
namespace {

// Loads go through shared memory, each lane's own 16 bytes: they hold no registers, so many are in flight, over the ends of tokens too.
__device__ __forceinline__ void cp_async_own(uint32_t dst, const void* src) {
  asm volatile("cp.async.cg.shared.global [%0], [%1], 16;" ::"r"(dst), "l"(src) : "memory");
}
template <int N>
__device__ __forceinline__ void cp_async_wait() {
  asm volatile("cp.async.wait_group %0;" ::"n"(N) : "memory");
}
__device__ __forceinline__ uint4 lds_own(uint32_t a) {
  uint4 r;
  asm volatile("ld.shared.v4.u32 {%0, %1, %2, %3}, [%4];" : "=r"(r.x), "=r"(r.y), "=r"(r.z), "=r"(r.w) : "r"(a) : "memory");
  return r;
}

// Two chunks of a lane as pairs that turn against each other: (a[i], b[i]).
template <bool HALF>
__device__ __forceinline__ void unpack_pairs(const uint4& r0, const uint4& r1, float (&a)[8], float (&b)[8]) {
  if (HALF) {
    unpack8(r0, a);
    unpack8(r1, b);
  } else {
    const uint32_t w[8] = {r0.x, r0.y, r0.z, r0.w, r1.x, r1.y, r1.z, r1.w};
#pragma unroll
    for (int i = 0; i < 8; ++i) {
      a[i] = __uint_as_float(w[i] << 16);
      b[i] = __uint_as_float(w[i] & 0xffff0000u);
    }
  }
}
template <bool HALF>
__device__ __forceinline__ void pack_pairs(const float (&a)[8], const float (&b)[8], uint4& r0, uint4& r1) {
  if (HALF) {
    r0 = pack8(a);
    r1 = pack8(b);
  } else {
    r0 = make_uint4(pack_bf16x2_cvt(a[0], b[0]), pack_bf16x2_cvt(a[1], b[1]), pack_bf16x2_cvt(a[2], b[2]), pack_bf16x2_cvt(a[3], b[3]));
    r1 = make_uint4(pack_bf16x2_cvt(a[4], b[4]), pack_bf16x2_cvt(a[5], b[5]), pack_bf16x2_cvt(a[6], b[6]), pack_bf16x2_cvt(a[7], b[7]));
  }
}
// The rotation, pairs FROM .. FROM + 3, each product rounded as in aq_rope.
template <int FROM>
__device__ __forceinline__ void turn4(float (&a)[8], float (&b)[8], const float (&c)[8], const float (&s)[8]) {
#pragma unroll
  for (int i = FROM; i < FROM + 4; i += 2) {
    float t0, t1, u0, u1;
    fmul2_rn(t0, t1, b[i], b[i + 1], s[i], s[i + 1]);
    fmul2_rn(u0, u1, a[i], a[i + 1], s[i], s[i + 1]);
    a[i] = fmaf(a[i], c[i], -t0);
    a[i + 1] = fmaf(a[i + 1], c[i + 1], -t1);
    ffma2_rn(b[i], b[i + 1], b[i], b[i + 1], c[i], c[i + 1], u0, u1);
  }
}
__device__ __forceinline__ void scale8(float (&x)[8], const float (&y)[8]) {
#pragma unroll
  for (int i = 0; i < 8; i += 2) fmul2_rn(x[i], x[i + 1], x[i], x[i + 1], y[i], y[i + 1]);
}
__device__ __forceinline__ void scale8(float (&x)[8], float y) {
#pragma unroll
  for (int i = 0; i < 8; i += 2) fmul2_rn(x[i], x[i + 1], x[i], x[i + 1], y, y);
}
__device__ __forceinline__ void dot8(float& s0, float& s1, const float (&x)[8], const float (&y)[8]) {
#pragma unroll
  for (int i = 0; i < 8; i += 2) ffma2_rn(s0, s1, x[i], x[i + 1], y[i], y[i + 1], s0, s1);
}
template <int GW>
__device__ __forceinline__ float group_sum(float s, uint32_t group) {
#pragma unroll
  for (int o = GW / 2; o > 0; o >>= 1) s += __shfl_xor_sync(group, s, o);
  return s;
}

// 1 / sqrt(mean(x^2) + eps) of a head held by a group of GW lanes, 16 elements a lane (zeros past the head). Squares of numbers
// past 2^60 could leave fp32: such a head is measured at 2^-70 of its size, and eps with it.
template <int GW>
__device__ __forceinline__ float head_rstd(const float (&a)[8], const float (&b)[8], uint32_t group, float inv_dim, float eps) {
  float s0 = 0.0f, s1 = 0.0f;
  dot8(s0, s1, a, a);
  dot8(s0, s1, b, b);
  float s = group_sum<GW>(s0 + s1, group);
  if (s < 0x1p120f) return rsqrtf(fmaf(s, inv_dim, eps));
  s0 = 0.0f;
#pragma unroll
  for (int i = 0; i < 8; ++i) {
    const float x = a[i] * 0x1p-70f, y = b[i] * 0x1p-70f;
    s0 = fmaf(x, x, s0);
    s0 = fmaf(y, y, s0);
  }
  return rsqrtf(fmaf(group_sum<GW>(s0, group), inv_dim, eps * 0x1p-140f)) * 0x1p-70f;
}

// As share_token, but at least a warp's groups, heads or not: those without one work out their part of the angles too.
int warp_token(int64_t T, int heads, int gw, int64_t fill) { return std::max(share_token(T, heads, gw, fill), log2_of(32 / gw)); }

// offset + weight for a lane's pairs; ones without a weight.
template <bool HALF>
__device__ __forceinline__ void norm_factors(const uint16_t* w, int k0, int k1, float offset, float (&f)[8], float (&h)[8]) {
  if (w) {
    unpack_pairs<HALF>(__ldg(reinterpret_cast<const uint4*>(w + k0)), __ldg(reinterpret_cast<const uint4*>(w + k1)), f, h);
#pragma unroll
    for (int i = 0; i < 8; ++i) {
      f[i] += offset;
      h[i] += offset;
    }
  } else {
#pragma unroll
    for (int i = 0; i < 8; ++i) f[i] = h[i] = 1.0f;
  }
}

// ---------------------------------------------------------------------------------
// forward
// ---------------------------------------------------------------------------------
struct HeadSet {
  const uint16_t* x;
  uint16_t* y;            // NULL: to the cache
  const uint16_t* w;
  int64_t x_tok, x_head, y_tok, y_head;
  float eps, offset;
  int32_t heads, normed;
};
struct HeadNormParams {
  HeadSet set[3];         // q, k, v (v: no norm, not turned)
  const int32_t* pos;
  const uint64_t* freq;   // NULL: nothing is turned
  const int64_t* slots;
  uint8_t* c[2];          // the cache's keys and values
  float* sc[2];
  int64_t T, n_slots;
  int32_t D, rot16, page_shift, hl_shift;
  float magnitude;
};

enum To { kTensor, kCacheBf16, kCacheE4m3 };

// Blocks an SM and heads in flight of a group, us for these 16385 tokens, and for 8192 of 32 + 8 heads into an E4M3 cache and back: 1 and 3 41, 78; 2 and 2 30.2,
// 48.9; 2 and 3 29.6, 47.5; 2 and 4 30.5, 47.6; 3 and 3 30.8, 53; 4 and 4 39.7, 64 (more blocks get in each other's way in DRAM).
constexpr int kHeadThreads = 256, kHeadPerSm = 2, kHeadDepth = 3;

template <bool HALF, int GW, To TO>
__global__ void __launch_bounds__(kHeadThreads, kHeadPerSm) aq_head_norm_kernel(const __grid_constant__ HeadNormParams p) {
  __shared__ __align__(16) uint4 ring[kHeadDepth][2][kHeadThreads];
  pdl_wait_prior_grid();
  pdl_launch_dependents();
  constexpr int kGroups = kHeadThreads / GW;
  const int u = threadIdx.x % GW, lane = threadIdx.x & 31;
  const Chunks<HALF> ch(u, p.rot16, p.D / 16);
  const bool mine = u * 16 < p.D;
  // groups of one warp may be at different heads, so each shuffles by itself
  const uint32_t group = (GW == 32 ? 0xffffffffu : (1u << GW) - 1) << (lane & ~(GW - 1));
  const int k0 = mine ? ch.c0 * 8 : 0, k1 = mine ? ch.c1 * 8 : 0;   // lanes without work load lane 0's chunks
  const float inv_dim = 1.0f / p.D;
  const int hl = 1 << p.hl_shift;
  // The groups of a token take its heads in turn, the sets' as one list; a warp's groups walk tokens together, so that angles can be
  // passed round.
  const int64_t items = p.T << p.hl_shift, step = static_cast<int64_t>(gridDim.x) * kGroups;
  const int64_t start = static_cast<int64_t>(blockIdx.x) * kGroups + (threadIdx.x / 32) * (32 / GW);
  const int h0 = static_cast<int>((start + lane / GW) & (hl - 1));   // step is a multiple of hl
  const int n0 = p.set[0].heads, n1 = n0 + p.set[1].heads, n = n1 + (TO == kTensor ? 0 : p.set[2].heads);

  int64_t f_item = h0 < n ? start + lane / GW : items;   // a group may have no head at all
  int f_h = h0, f_slot = 0;
  const uint32_t mine_at = smem_u32(&ring[0][0][threadIdx.x]);
  constexpr uint32_t kSlot = 2 * kHeadThreads * 16;
  auto fetch = [&] {
    if (f_item < items) {
      const int which = f_h < n0 ? 0 : TO == kTensor || f_h < n1 ? 1 : 2;
      const HeadSet& q = p.set[which];
      const uint16_t* x = q.x + (f_item >> p.hl_shift) * q.x_tok + (f_h - (which == 0 ? 0 : which == 1 ? n0 : n1)) * q.x_head;
      const uint32_t to = mine_at + f_slot * kSlot;
      cp_async_own(to, x + k0);
      cp_async_own(to + kHeadThreads * 16, x + k1);
      f_h += hl;
      if (f_h >= n) {
        f_h = h0;
        f_item += step;
      }
    }
    f_slot = f_slot == kHeadDepth - 1 ? 0 : f_slot + 1;
    cp_async_commit();
  };
#pragma unroll
  for (int i = 0; i < kHeadDepth; ++i) fetch();

  float f0[8], f1[8];   // the factors of one set
  int held = -1;        // which
  uint32_t at_slot = mine_at;
  const uint32_t last_slot = mine_at + (kHeadDepth - 1) * kSlot;
  int32_t next_pos = p.freq && start + lane / GW < items ? p.pos[(start + lane / GW) >> p.hl_shift] : 0;
  int64_t next_slot = TO != kTensor && start + lane / GW < items ? p.slots[(start + lane / GW) >> p.hl_shift] : -1;
  for (int64_t first = start; first < items; first += step) {
    const int64_t item = first + lane / GW;
    const bool there = item < items, live = there && mine;
    const int64_t t = there ? item >> p.hl_shift : 0;
    const int32_t pos = next_pos;
    if (p.freq && item + step < items) next_pos = p.pos[(item + step) >> p.hl_shift];
    float c[8], s[8];
    angles<HALF, GW, true>(ch, u, p.freq, pos, p.magnitude, p.magnitude, c, s);
    const bool turn0 = p.freq && live && ch.turns0, turn1 = p.freq && live && ch.turns1;
    int64_t cell0 = -1;
    if (TO != kTensor) {
      const int64_t slot = next_slot;
      if (item + step < items) next_slot = p.slots[(item + step) >> p.hl_shift];
      if (live && slot >= 0 && slot < p.n_slots)
        cell0 = (((slot >> p.page_shift) * p.set[1].heads) << p.page_shift) + (slot & ((1 << p.page_shift) - 1));
    }
    if (there) {
#pragma unroll 1
      for (int h = h0; h < n; h += hl) {
        const int which = h < n0 ? 0 : TO == kTensor || h < n1 ? 1 : 2;
        const HeadSet& q = p.set[which];
        const int at = h - (which == 0 ? 0 : which == 1 ? n0 : n1);
        const bool normed = which < 2 && q.normed;
        if (normed && held != which) {
          norm_factors<HALF>(q.w, k0, k1, q.offset, f0, f1);
          held = which;
        }
        cp_async_wait<kHeadDepth - 1>();
        float a[8], b[8];
        {
          const uint4 none = make_uint4(0, 0, 0, 0), r0 = lds_own(at_slot), r1 = lds_own(at_slot + kHeadThreads * 16);
          unpack_pairs<HALF>(mine ? r0 : none, mine ? r1 : none, a, b);
        }
        at_slot = at_slot == last_slot ? mine_at : at_slot + kSlot;
        fetch();   // over what has just been read
        if (normed) {
          const float r = head_rstd<GW>(a, b, group, inv_dim, q.eps);
          scale8(a, r);
          scale8(b, r);
          scale8(a, f0);
          scale8(b, f1);
        }
        if (which < 2) {
          if (turn0) turn4<0>(a, b, c, s);
          if (turn1) turn4<4>(a, b, c, s);
        }
        if (which == 0 || TO != kCacheE4m3) {
          uint4 y0, y1;
          pack_pairs<HALF>(a, b, y0, y1);
          uint16_t* dst;
          if (which == 0 || TO == kTensor) {
            dst = q.y + t * q.y_tok + at * q.y_head;
          } else {
            if (cell0 < 0) continue;
            dst = reinterpret_cast<uint16_t*>(p.c[which - 1]) + (cell0 + (static_cast<int64_t>(at) << p.page_shift)) * p.D;
          }
          if (live) *reinterpret_cast<uint4*>(dst + k0) = y0;
          if (live) *reinterpret_cast<uint4*>(dst + k1) = y1;
          continue;
        }
        // as the cache's write without norms: max|x| on the bit patterns, a NaN or infinity stays the largest
        uint32_t top = 0;
#pragma unroll
        for (int i = 0; i < 8; ++i) top = max(top, max(__float_as_uint(a[i]) & 0x7fffffffu, __float_as_uint(b[i]) & 0x7fffffffu));
#pragma unroll
        for (int o = GW / 2; o > 0; o >>= 1) top = max(top, __shfl_xor_sync(group, top, o));
        if (cell0 < 0) continue;
        const int64_t cell = cell0 + (static_cast<int64_t>(at) << p.page_shift);
        const bool finite = top < 0x7f800000u;
        const float scale = finite ? fmaxf(__uint_as_float(top) * (1.0f / kE4m3Max), kKvScaleFloor) : __uint_as_float(0x7fc00000u);
        const float inv = finite ? __frcp_rn(scale) : 0.0f;
        uint8_t* dst = p.c[which - 1] + cell * p.D;
        scale8(a, inv);
        scale8(b, inv);
        auto two = [&](float lo, float hi) { return static_cast<uint32_t>(e4m3x2_from_f32(lo, hi)); };
        uint2 d0, d1;
        if (HALF) {
          d0 = make_uint2(two(a[0], a[1]) | (two(a[2], a[3]) << 16), two(a[4], a[5]) | (two(a[6], a[7]) << 16));
          d1 = make_uint2(two(b[0], b[1]) | (two(b[2], b[3]) << 16), two(b[4], b[5]) | (two(b[6], b[7]) << 16));
        } else {
          d0 = make_uint2(two(a[0], b[0]) | (two(a[1], b[1]) << 16), two(a[2], b[2]) | (two(a[3], b[3]) << 16));
          d1 = make_uint2(two(a[4], b[4]) | (two(a[5], b[5]) << 16), two(a[6], b[6]) | (two(a[7], b[7]) << 16));
        }
        if (!finite) d0 = d1 = make_uint2(0, 0);
        if (live) *reinterpret_cast<uint2*>(dst + k0) = d0;
        if (live) *reinterpret_cast<uint2*>(dst + k1) = d1;
        if (u == 0) p.sc[which - 1][cell] = scale;
      }
    }
    __syncwarp();
  }
}

template <bool HALF, To TO>
cudaError_t launch_head_norm(const HeadNormParams& p, unsigned blocks, int gw, cudaStream_t st) {
  switch (gw) {
    case 1: return launch_serve(aq_head_norm_kernel<HALF, 1, TO>, p, blocks, kHeadThreads, 0, st);
    case 2: return launch_serve(aq_head_norm_kernel<HALF, 2, TO>, p, blocks, kHeadThreads, 0, st);
    case 4: return launch_serve(aq_head_norm_kernel<HALF, 4, TO>, p, blocks, kHeadThreads, 0, st);
    case 8: return launch_serve(aq_head_norm_kernel<HALF, 8, TO>, p, blocks, kHeadThreads, 0, st);
    default: return launch_serve(aq_head_norm_kernel<HALF, 16, TO>, p, blocks, kHeadThreads, 0, st);
  }
}
template <bool HALF>
cudaError_t launch_head_norm(const HeadNormParams& p, unsigned blocks, int gw, To to, cudaStream_t st) {
  switch (to) {
    case kTensor: return launch_head_norm<HALF, kTensor>(p, blocks, gw, st);
    case kCacheBf16: return launch_head_norm<HALF, kCacheBf16>(p, blocks, gw, st);
    default: return launch_head_norm<HALF, kCacheE4m3>(p, blocks, gw, st);
  }
}

// ---------------------------------------------------------------------------------
// gradient
// ---------------------------------------------------------------------------------
// As above, us for the gradient at the top: 1 and 2 53.2, 2 and 2 44.7, 2 and 3 46.2, 3 and 2 63.6, 4 and 2 86.5.
constexpr int kNormThreads = 256, kNormPerSm = 2, kNormDepth = 2;

struct NormSet {
  const uint16_t* dy;
  const uint16_t* x;
  uint16_t* dx;
  const uint16_t* w;
  float* part;         // [blocks][D], or NULL
  float* dw;           // with a cluster: where the sums go, or NULL
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
  int32_t cluster;        // blocks of a set, which are a cluster and join their sums themselves; 0: a second launch does
  float magnitude;
};
constexpr int kNormCluster = 8;

template <bool HALF, int GW>
__global__ void __launch_bounds__(kNormThreads, kNormPerSm) aq_norm_grad_kernel(const __grid_constant__ NormGradParams p) {
  pdl_wait_prior_grid();
  pdl_launch_dependents();
  constexpr int kGroups = kNormThreads / GW, kRow = GW * 16 + 1;
  __shared__ __align__(16) uint4 ring[kNormDepth][4][kNormThreads];   // and the groups' sums in the end
  static_assert(sizeof(ring) >= sizeof(float) * kGroups * kRow, "the sums fit");
  const int which = static_cast<int>(blockIdx.x) >= p.set[0].blocks;
  const NormSet& s = p.set[which];
  if (p.cluster > 1 && s.dw) asm volatile("barrier.cluster.arrive.relaxed.aligned;" ::: "memory");
  const int block = static_cast<int>(blockIdx.x) - (which ? p.set[0].blocks : 0);
  const int lane = threadIdx.x & 31, u = threadIdx.x % GW;
  const Chunks<HALF> ch(u, p.rot16, p.D / 16);
  const uint32_t group = (GW == 32 ? 0xffffffffu : (1u << GW) - 1) << (lane & ~(GW - 1));
  const bool mine = u * 16 < p.D;
  const int k0 = mine ? ch.c0 * 8 : 0, k1 = mine ? ch.c1 * 8 : 0;
  const int hl = 1 << s.hl_shift;
  const float inv_dim = 1.0f / p.D;
  float f0[8], f1[8], w0[8], w1[8];
  norm_factors<HALF>(s.w, k0, k1, s.offset, f0, f1);
#pragma unroll
  for (int i = 0; i < 8; ++i) w0[i] = w1[i] = 0.0f;

  // A warp's groups walk tokens together, so that angles can be passed round.
  const int64_t items = p.T << s.hl_shift, step = static_cast<int64_t>(s.blocks) * kGroups;
  const int64_t start = static_cast<int64_t>(block) * kGroups + (threadIdx.x / 32) * (32 / GW);
  const int h0 = static_cast<int>((start + lane / GW) & (hl - 1));   // step is a multiple of hl
  int64_t f_item = h0 < s.heads ? start + lane / GW : items;   // a group may have no head at all
  int f_h = h0, f_slot = 0;
  const uint32_t mine_at = smem_u32(&ring[0][0][threadIdx.x]);
  constexpr uint32_t kPiece = kNormThreads * 16, kSlot = 4 * kPiece;
  auto fetch = [&] {
    if (f_item < items) {
      const int64_t t = f_item >> s.hl_shift;
      const uint16_t* xh = s.x + t * s.x_tok + f_h * s.x_head;
      const uint16_t* yh = s.dy + t * s.dy_tok + f_h * s.dy_head;
      const uint32_t to = mine_at + f_slot * kSlot;
      cp_async_own(to, xh + k0);
      cp_async_own(to + kPiece, xh + k1);
      cp_async_own(to + 2 * kPiece, yh + k0);
      cp_async_own(to + 3 * kPiece, yh + k1);
      f_h += hl;
      if (f_h >= s.heads) {
        f_h = h0;
        f_item += step;
      }
    }
    f_slot = f_slot == kNormDepth - 1 ? 0 : f_slot + 1;
    cp_async_commit();
  };
#pragma unroll
  for (int i = 0; i < kNormDepth; ++i) fetch();
  uint32_t at_slot = mine_at;
  const uint32_t last_slot = mine_at + (kNormDepth - 1) * kSlot;
  int32_t next_pos = p.freq && start + lane / GW < items ? p.pos[(start + lane / GW) >> s.hl_shift] : 0;
  for (int64_t first = start; first < items; first += step) {
    const int64_t item = first + lane / GW;
    const bool there = item < items, live = there && mine;
    const int64_t t = there ? item >> s.hl_shift : 0;
    const int32_t pos = next_pos;
    if (p.freq && item + step < items) next_pos = p.pos[(item + step) >> s.hl_shift];
    float c[8], sn[8];
    if (hl < 32 / GW) angles<HALF, GW, false>(ch, u, p.freq, pos, p.magnitude, -p.magnitude, c, sn);   // its groups have a token each
    else angles<HALF, GW, true>(ch, u, p.freq, pos, p.magnitude, -p.magnitude, c, sn);
    const bool turn0 = p.freq && live && ch.turns0, turn1 = p.freq && live && ch.turns1;
    uint16_t* ds = s.dx + t * s.dx_tok;
    if (there) {
#pragma unroll 1
      for (int h = h0; h < s.heads; h += hl) {
        float a[8], b[8], ga[8], gb[8];
        cp_async_wait<kNormDepth - 1>();
        {
          const uint4 none = make_uint4(0, 0, 0, 0);
          const uint4 r0 = lds_own(at_slot), r1 = lds_own(at_slot + kPiece), r2 = lds_own(at_slot + 2 * kPiece), r3 = lds_own(at_slot + 3 * kPiece);
          unpack_pairs<HALF>(mine ? r0 : none, mine ? r1 : none, a, b);
          unpack_pairs<HALF>(mine ? r2 : none, mine ? r3 : none, ga, gb);
        }
        at_slot = at_slot == last_slot ? mine_at : at_slot + kSlot;
        fetch();   // over what has just been read
        if (turn0) turn4<0>(ga, gb, c, sn);
        if (turn1) turn4<4>(ga, gb, c, sn);
        const float r = head_rstd<GW>(a, b, group, inv_dim, s.eps);
        scale8(a, r);
        scale8(b, r);
#pragma unroll
        for (int i = 0; i < 8; i += 2) {
          ffma2_rn(w0[i], w0[i + 1], ga[i], ga[i + 1], a[i], a[i + 1], w0[i], w0[i + 1]);
          ffma2_rn(w1[i], w1[i + 1], gb[i], gb[i + 1], b[i], b[i + 1], w1[i], w1[i + 1]);
        }
        scale8(ga, f0);
        scale8(gb, f1);
        float d0 = 0.0f, d1 = 0.0f;
        dot8(d0, d1, ga, a);
        dot8(d0, d1, gb, b);
        const float dot = -group_sum<GW>(d0 + d1, group) * inv_dim;
#pragma unroll
        for (int i = 0; i < 8; i += 2) {
          ffma2_rn(a[i], a[i + 1], a[i], a[i + 1], dot, dot, ga[i], ga[i + 1]);
          ffma2_rn(b[i], b[i + 1], b[i], b[i + 1], dot, dot, gb[i], gb[i + 1]);
        }
        scale8(a, r);
        scale8(b, r);
        if (mine) {
          uint16_t* d = ds + h * s.dx_head;
          uint4 o0, o1;
          pack_pairs<HALF>(a, b, o0, o1);
          *reinterpret_cast<uint4*>(d + k0) = o0;
          *reinterpret_cast<uint4*>(d + k1) = o1;
        }
      }
    }
    __syncwarp();
  }
  if (!s.part && !s.dw) return;
  cp_async_wait<0>();
  __syncthreads();
  float* sums = reinterpret_cast<float*>(ring);
  float* row = sums + threadIdx.x / GW * kRow;
  if (mine) {
#pragma unroll
    for (int i = 0; i < 8; ++i) {   // pair i: elements i of either chunk, or 2 i and 2 i + 1
      row[HALF ? k0 + i : (i < 4 ? k0 : k1) + 2 * (i & 3)] = w0[i];
      row[HALF ? k1 + i : (i < 4 ? k0 : k1) + 2 * (i & 3) + 1] = w1[i];
    }
  }
  __shared__ float met[kNormCluster][kServeMaxHeadDim];   // the first block's: every block's sums
  if (p.cluster > 1) asm volatile("barrier.cluster.wait.acquire.aligned;" ::: "memory");   // it runs
  __syncthreads();
  for (int d = threadIdx.x; d < p.D; d += kNormThreads) {
    float v = 0.0f;
    for (int i = 0; i < kGroups; ++i) v += sums[i * kRow + d];
    if (p.cluster == 0) s.part[static_cast<int64_t>(block) * p.D + d] = v;
    else if (p.cluster == 1) s.dw[d] = v;
    else asm volatile("st.shared::cluster.f32 [%0], %1;" ::"r"(cluster_map(&met[block][d], 0)), "f"(v) : "memory");
  }
  if (p.cluster <= 1) return;
  cluster_sync_all();
  if (block != 0) return;
  for (int d = threadIdx.x; d < p.D; d += kNormThreads) {
    float v = 0.0f;
    for (int i = 0; i < p.cluster; ++i) v += met[i][d];
    s.dw[d] = v;
  }
}

// dw = the blocks' sums, 32 elements of one set a block: 32 threads an element, each every 32nd block.
struct NormJoinParams {
  const float* part[2];
  float* dw[2];
  int32_t blocks[2];
  int32_t D, tiles;    // tiles of 32 elements of a set
};
__global__ void __launch_bounds__(1024) aq_norm_join_kernel(const __grid_constant__ NormJoinParams p) {
  pdl_wait_prior_grid();
  pdl_launch_dependents();
  __shared__ float sums[32][33];
  const int which = static_cast<int>(blockIdx.x) / p.tiles, d = (static_cast<int>(blockIdx.x) % p.tiles) * 32 + (threadIdx.x & 31);
  const int part = threadIdx.x / 32;
  if (!p.dw[which]) return;
  float v = 0.0f;
  if (d < p.D) {
#pragma unroll 4
    for (int i = part; i < p.blocks[which]; i += 32) v += p.part[which][static_cast<int64_t>(i) * p.D + d];
  }
  sums[threadIdx.x & 31][part] = v;
  __syncthreads();
  v = sums[part][threadIdx.x & 31];   // a warp an element
#pragma unroll
  for (int o = 16; o > 0; o >>= 1) v += __shfl_xor_sync(0xffffffffu, v, o);
  const int at = (static_cast<int>(blockIdx.x) % p.tiles) * 32 + part;
  if ((threadIdx.x & 31) == 0 && at < p.D) p.dw[which][at] = v;
}

// Blocks of the two sets: what fills the GPU, shared out by their work (a token's angles weigh as much as a head, and every
// group works them out; to itself, twice as much); no more than their groups of work.
void norm_blocks(int64_t T, int32_t D, int32_t hq, int32_t hk, int sms, int32_t* hl_shift, int32_t* blocks) {
  const int gw = group_width(D), groups = kNormThreads / gw, heads[2] = {hq, hk};
  const int fill = sms * kNormPerSm;
  int64_t work[2] = {0, 0};
  for (int i = 0; i < 2; ++i) {
    hl_shift[i] = blocks[i] = 0;
    if (!heads[i]) continue;
    // A block has one set's heads, often one: where half of a warp's groups or more would have none, and the tokens are enough without, each
    // group has a token and its angles to itself. Shared and apart, us: 16000 tokens of 1 + 1 heads of 64 22.4 and 8.5, 4000 9.3 and 5.6;
    // 2000 of 2 + 2 6.7 and 5.4; 16000 of 4 + 1 of 128 25.7 and 21.1. (Without the gradient q, k and v make one list, and it costs more
    // than it gives: 16385 tokens of 16 + 4 heads 29.6 and 30.0 for having both.)
    const int64_t fit = static_cast<int64_t>(fill) * groups;
    const int own = share_token(T, heads[i], gw, fit / 2);
    hl_shift[i] = 2 * heads[i] <= 32 / gw && (T << own) >= fit / 8 ? own : warp_token(T, heads[i], gw, fit / 2);
    const int hl = 1 << hl_shift[i];
    work[i] = static_cast<int64_t>(hl) * ((hl < 32 / gw ? 2 : 1) + (heads[i] + hl - 1) / hl);
  }
  for (int i = 0; i < 2; ++i) {
    if (!heads[i]) continue;
    const int64_t need = ((T << hl_shift[i]) + groups - 1) / groups;
    blocks[i] = static_cast<int32_t>(std::min(need, std::max<int64_t>(1, fill * work[i] / (work[0] + work[1]))));
  }
}
// Blocks of a set where each group has one token and they are few enough to be a cluster, which joins their sums itself, or 0. One launch
// against two, us: one token of 32 + 8 heads of 128 3.2 and 4.4, eight 3.8 and 4.6, 60 of 4 + 1 3.8 and 4.6; with two tokens a group no less.
int norm_cluster(int64_t T, int32_t D, int32_t hq, int32_t hk, int32_t* hl_shift, int32_t* blocks) {
  const int gw = group_width(D), groups = kNormThreads / gw, heads[2] = {hq, hk};
  int cluster = 1;
  for (int i = 0; i < 2; ++i) {
    hl_shift[i] = heads[i] ? warp_token(T, heads[i], gw, INT64_MAX) : 0;
    if (T > static_cast<int64_t>(kNormCluster) * groups >> hl_shift[i]) return 0;
    while (heads[i] && static_cast<int64_t>(cluster) * groups < T << hl_shift[i]) cluster *= 2;
  }
  for (int i = 0; i < 2; ++i) blocks[i] = heads[i] ? cluster : 0;
  return cluster;
}
constexpr int kNormSmsBound = 256;   // SMs that the workspace's size allows for

template <bool HALF>
cudaError_t launch_norm_grad(const NormGradParams& p, int gw, cudaStream_t st) {
  const unsigned grid = static_cast<unsigned>(p.set[0].blocks + p.set[1].blocks);
  switch (gw) {
    case 1: return launch_serve(aq_norm_grad_kernel<HALF, 1>, p, grid, kNormThreads, 0, st, p.cluster);
    case 2: return launch_serve(aq_norm_grad_kernel<HALF, 2>, p, grid, kNormThreads, 0, st, p.cluster);
    case 4: return launch_serve(aq_norm_grad_kernel<HALF, 4>, p, grid, kNormThreads, 0, st, p.cluster);
    case 8: return launch_serve(aq_norm_grad_kernel<HALF, 8>, p, grid, kNormThreads, 0, st, p.cluster);
    default: return launch_serve(aq_norm_grad_kernel<HALF, 16>, p, grid, kNormThreads, 0, st, p.cluster);
  }
}

}  // namespace

aq_status run_head_norm(const aq_head_norm* q_norm, const aq_head_norm* k_norm, const aq_rope_spec* rope, const int32_t* pos, int64_t T,
                        int32_t D, const aq_heads* q, const aq_heads* q_out, const aq_heads* k, const aq_heads* k_out, const aq_heads* v,
                        const aq_kv_cache* cache, const int64_t* slots, cudaStream_t st, const char* who) {
  ServeDev dev;
  const aq_status s = serve_device(&dev);
  if (s != AQ_OK) return s;
  HeadNormParams p = {};
  const aq_heads* const in[3] = {q, k, v};
  const aq_heads* const out[3] = {q_out, k_out, nullptr};
  const aq_head_norm* const norm[3] = {q_norm, k_norm, nullptr};
  int heads = 0;
  for (int i = 0; i < 3; ++i) {
    if (!in[i]) continue;
    HeadSet& h = p.set[i];
    h.x = static_cast<const uint16_t*>(in[i]->data);
    h.x_tok = in[i]->tok;
    h.x_head = in[i]->head;
    h.heads = in[i]->heads;
    heads += h.heads;
    if (out[i]) {
      h.y = static_cast<uint16_t*>(out[i]->data);
      h.y_tok = out[i]->tok;
      h.y_head = out[i]->head;
    }
    if (norm[i]) {
      h.normed = 1;
      h.w = static_cast<const uint16_t*>(norm[i]->weight);
      h.eps = norm[i]->eps;
      h.offset = norm[i]->offset;
    }
  }
  if (rope) {
    p.pos = pos;
    p.freq = rope->freq;
    p.rot16 = rope->rotary_dim / 16;
    p.magnitude = rope->magnitude;
  }
  if (cache) {
    p.slots = slots;
    p.c[0] = static_cast<uint8_t*>(cache->k);
    p.c[1] = static_cast<uint8_t*>(cache->v);
    p.sc[0] = cache->k_scale;
    p.sc[1] = cache->v_scale;
    p.n_slots = static_cast<int64_t>(cache->pages) * cache->page_size;
    p.page_shift = log2_of(cache->page_size);
  }
  p.T = T;
  p.D = D;
  const int gw = group_width(D);
  p.hl_shift = warp_token(T, heads, gw, static_cast<int64_t>(dev.sms) * (kHeadPerSm * kHeadThreads) / gw);
  // blocks that are resident at once, each walking over tokens
  const int64_t blocks = std::min<int64_t>(((T << p.hl_shift) + kHeadThreads / gw - 1) / (kHeadThreads / gw), static_cast<int64_t>(dev.sms) * kHeadPerSm);
  const To to = !cache ? kTensor : cache->type == AQ_KV_BF16 ? kCacheBf16 : kCacheE4m3;
  const unsigned g = static_cast<unsigned>(blocks);
  return serve_launched(rope && rope->layout == AQ_ROPE_HALF ? launch_head_norm<true>(p, g, gw, to, st) : launch_head_norm<false>(p, g, gw, to, st), who);
}

}  // namespace aq

using namespace aq;

extern "C" aq_status aq_qk_norm_rope(const aq_head_norm* q_norm, const aq_head_norm* k_norm, const aq_rope_spec* rope, const int32_t* pos,
                                     int64_t T, int32_t head_dim, const aq_heads* q, const aq_heads* q_out, const aq_heads* k,
                                     const aq_heads* k_out, void* stream) {
  const char* who = "aq_qk_norm_rope";
  if (T < 0) return serve_fail(AQ_ERR_SHAPE, "%s: T=%lld is negative", who, (long long)T);
  if (head_dim < 16 || head_dim % 16 || head_dim > kServeMaxHeadDim)
    return serve_fail(AQ_ERR_SHAPE, "%s: head_dim=%d must be a multiple of 16 up to %d", who, head_dim, kServeMaxHeadDim);
  if (!q || !q_out) return serve_fail(AQ_ERR_INVALID_ARG, "%s: q and q_out must be non-NULL", who);
  if (!k != !k_out) return serve_fail(AQ_ERR_INVALID_ARG, "%s: k and k_out go together", who);
  if (k_norm && !k) return serve_fail(AQ_ERR_INVALID_ARG, "%s: k_norm needs k", who);
  aq_status st;
  if (rope && (st = check_rope_spec(rope, head_dim, who)) != AQ_OK) return st;
  if ((st = check_head_norm(q_norm, "q_norm", who)) != AQ_OK || (st = check_head_norm(k_norm, "k_norm", who)) != AQ_OK) return st;
  const aq_heads* const in[2] = {q, k};
  const aq_heads* const out[2] = {q_out, k_out};
  const int sets = k ? 2 : 1;
  for (int i = 0; i < sets; ++i)
    if (in[i]->heads < 1 || in[i]->heads != out[i]->heads)
      return serve_fail(AQ_ERR_SHAPE, "%s: heads=%d and %d must be >= 1 and equal", who, in[i]->heads, out[i]->heads);
  if ((st = check_head_count(static_cast<int64_t>(q->heads) + (k ? k->heads : 0), who)) != AQ_OK) return st;
  if (T == 0) return AQ_OK;
  if (rope && !pos) return serve_fail(AQ_ERR_INVALID_ARG, "%s: rope needs pos", who);
  const char* const names[2][2] = {{"q", "q_out"}, {"k", "k_out"}};
  for (int i = 0; i < sets; ++i) {
    if ((st = check_heads(in[i]->data, in[i]->tok, in[i]->head, in[i]->heads, head_dim, names[i][0], who)) != AQ_OK) return st;
    if ((st = check_heads(out[i]->data, out[i]->tok, out[i]->head, out[i]->heads, head_dim, names[i][1], who)) != AQ_OK) return st;
    if ((st = check_out_heads(out[i]->tok, out[i]->head, T, out[i]->heads, head_dim, names[i][1], who)) != AQ_OK) return st;
  }
  const ByteRows side[] = {ByteRows(rope ? pos : nullptr, 1, T * 4, T * 4), ByteRows(rope ? rope->freq : nullptr, 1, head_dim * 4, rope ? rope->rotary_dim * 4 : 0),
                           ByteRows(q_norm ? q_norm->weight : nullptr, 1, head_dim * 2, head_dim * 2), ByteRows(k_norm ? k_norm->weight : nullptr, 1, head_dim * 2, head_dim * 2)};
  for (int i = 0; i < sets; ++i) {
    const ByteRows o = heads_rows(out[i], T, head_dim);
    for (const ByteRows& s : side)
      if (o.meets(s)) return serve_fail(AQ_ERR_OVERLAP, "%s: %s overlaps an input", who, names[i][1]);
    for (int j = 0; j < sets; ++j) {
      const bool same = i == j && in[i]->data == out[i]->data && (T == 1 || in[i]->tok == out[i]->tok) && (in[i]->heads == 1 || in[i]->head == out[i]->head);
      if (!same && o.meets(heads_rows(in[j], T, head_dim)))
        return serve_fail(AQ_ERR_OVERLAP, "%s: %s overlaps %s (in place needs the same pointer and strides)", who, names[i][1], names[j][0]);
    }
  }
  if (sets == 2 && heads_rows(q_out, T, head_dim).meets(heads_rows(k_out, T, head_dim)))
    return serve_fail(AQ_ERR_OVERLAP, "%s: q_out and k_out overlap", who);
  return run_head_norm(q_norm, k_norm, rope, pos, T, head_dim, q, q_out, k, k_out, nullptr, nullptr, nullptr, static_cast<cudaStream_t>(stream), who);
}


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
  if ((st = check_head_count(static_cast<int64_t>(q->heads) + (k ? k->heads : 0), who)) != AQ_OK) return st;
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
  p.cluster = sums ? norm_cluster(T, D, q->heads, k ? k->heads : 0, hl, blocks) : 0;
  if (!p.cluster) norm_blocks(T, D, q->heads, k ? k->heads : 0, std::min(dev.sms, kNormSmsBound), hl, blocks);
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
    if (p.cluster) s.dw = dw[i];
    else if (dw[i]) s.part = part + (i ? static_cast<int64_t>(blocks[0]) * D : 0);
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
  if (e != cudaSuccess || !sums || p.cluster) return serve_launched(e, who);
  NormJoinParams j = {};
  for (int i = 0; i < sets; ++i) {
    j.part[i] = p.set[i].part;
    j.dw[i] = dw[i];
    j.blocks[i] = blocks[i];
  }
  j.D = D;
  j.tiles = (D + 31) / 32;
  return serve_launched(launch_serve(aq_norm_join_kernel, j, dim3(static_cast<unsigned>(sets * j.tiles)), 1024, 0, cs), who);
}
