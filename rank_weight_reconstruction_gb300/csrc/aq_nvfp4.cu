// aq_nvfp4.cu -- aq_nvfp4_linear, aq_nvfp4_linear_multi: products of a few tokens with the 4-bit weights that
// aq_precompute_nvfp4 makes.
//
//   y[m, o] = RN_bf16( g * sum_k E2M1(q[o, k]) * E4M3(sf[o, k / 16]) * x[m, k] )
//
// A code times its block scale has six significant bits between 2^-10 and 2688: exact in f16, so the weights are widened
// to f16 in registers (one conversion for two codes, one packed product with the scale) and go to mma.sync as its 16-row
// operand, the tokens as its 8 columns. x enters as f16 too, each token of a CTA's K slice scaled by the power of two that
// brings its largest element to at least 2^15: an element down to 2^-32 of the largest keeps all its bits. Sums are fp32.
//
// Bound by memory: 0.5625 bytes a weight are read once. A cluster of S CTAs takes groups of R row tiles of 16, each CTA a
// K slice whose x it keeps in shared memory; its eight warps share out the group's tiles and the slice's chunks of 128, each
// streaming its chunks through a ring of its own (cp.async: every lane copies what it will itself multiply, the scales
// apart), so no barrier stands in the stream. Sums meet in shared memory once a group, in a fixed order, then over the
// cluster, whose exchange of one group runs under the stream of the next.
#include <algorithm>
#include <atomic>

#include "aq_serve.h"

namespace aq {
namespace {

constexpr int kQWarps = 8, kQThreads = 32 * kQWarps;
constexpr int kQDepth = 6;                      // ring stages of a warp, one chunk each
constexpr int kQChunk = 128;                    // K of a chunk: 64 bytes of codes a row
constexpr int kQCodes = 1024;                   // bytes of a chunk's codes: 16 rows
constexpr int kQStage = kQCodes + 16 * 12;      // and 12 bytes of scales a row: eight, and room for any alignment
constexpr int kQPart = 20;                      // floats a token of a warp's partial sums: 16 rows, spread over the banks
constexpr int kQMaxS = 8;
constexpr int kQHead = 256;                     // bytes: per token the largest element, then the factor back

struct Nvfp4Seg {
  const uint8_t* q;
  const uint8_t* sf;
  const float* g;
  uint16_t* y;
  int64_t ldq, ldy;
  int32_t out;
  int32_t begin;       // first group
};
struct Nvfp4Params {
  Nvfp4Seg seg[AQ_MAX_FAMILIES];
  const uint16_t* x;
  int64_t M, ldx;
  int32_t nseg, in;
  int32_t cols;        // in / 16
  int32_t mode;        // scales: 0 linear, rows on 4 bytes; 1 linear; 2 128x4
  int32_t wide;        // codes move in 16-byte pieces (8 otherwise)
  int32_t groups, clusters, S, R_shift;
  int32_t slice;       // chunks of a CTA's K slice
  int32_t share;       // outputs of a group that one CTA of the cluster finishes
};

__device__ __forceinline__ void mma_f16(float (&d)[4], const uint32_t (&a)[4], uint32_t b0, uint32_t b1) {
  asm volatile("mma.sync.aligned.m16n8k16.row.col.f32.f16.f16.f32 {%0, %1, %2, %3}, {%4, %5, %6, %7}, {%8, %9}, "
               "{%0, %1, %2, %3};"
               : "+f"(d[0]), "+f"(d[1]), "+f"(d[2]), "+f"(d[3])
               : "r"(a[0]), "r"(a[1]), "r"(a[2]), "r"(a[3]), "r"(b0), "r"(b1));
}
// Two E2M1 codes (byte i of w, the low nibble first) as halves.
template <int I>
__device__ __forceinline__ uint32_t f16x2_from_e2m1x2(uint32_t w) {
  uint32_t r;
  asm("{\n\t.reg .b8 b0, b1, b2, b3;\n\tmov.b32 {b0, b1, b2, b3}, %1;\n\tcvt.rn.f16x2.e2m1x2 %0, b0;\n\t}"
      : "=r"(r)
      : "r"(w >> (8 * I)));
  return r;
}
__device__ __forceinline__ uint32_t hmul2(uint32_t a, uint32_t b) {
  uint32_t r;
  asm("mul.rn.f16x2 %0, %1, %2;" : "=r"(r) : "r"(a), "r"(b));
  return r;
}
template <int BYTES>
__device__ __forceinline__ void cp_async_small(uint32_t dst, const void* src, int bytes) {
  asm volatile("cp.async.ca.shared.global [%0], [%1], %2, %3;" ::"r"(dst), "l"(src), "n"(BYTES), "r"(bytes) : "memory");
}
__device__ __forceinline__ uint4 lds128(uint32_t a) {
  uint4 r;
  asm volatile("ld.shared.v4.u32 {%0, %1, %2, %3}, [%4];" : "=r"(r.x), "=r"(r.y), "=r"(r.z), "=r"(r.w) : "r"(a));
  return r;
}
__device__ __forceinline__ uint32_t lds_u8(uint32_t a) {
  uint32_t r;
  asm volatile("ld.shared.u8 %0, [%1];" : "=r"(r) : "r"(a));
  return r;
}
template <int N>
__device__ __forceinline__ void cp_async_wait() {
  asm volatile("cp.async.wait_group %0;" ::"n"(N) : "memory");
}

// The segment and first row of a group of R row tiles.
__device__ __forceinline__ int group_seg(const Nvfp4Params& p, int group) {
  int s = 0;
  if (p.nseg > 1 && group >= p.seg[1].begin) s = 1;
  if (p.nseg > 2 && group >= p.seg[2].begin) s = 2;
  return s;
}

// Where a warp's next chunk comes from.
struct Feed {
  const uint8_t *qa, *qb;   // this lane's 16 bytes of rows g and g + 8, chunk 0
  const uint8_t* q0;        // any readable byte of the codes
  const uint8_t *s0, *s1;   // its word (or two) of the scales, chunk 0
  const uint8_t* sb;        // any readable byte of the scales
  int na, nb;               // code bytes of the rows from this lane's on (0: no such row)
  int64_t left0, left1;     // bytes of scales from s0, s1 on that may be read
};

template <int NT>
__global__ void __launch_bounds__(kQThreads, NT <= 2 ? 2 : 1) aq_nvfp4_kernel(const __grid_constant__ Nvfp4Params p) {
  extern __shared__ __align__(1024) uint8_t smem[];
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5, g = lane >> 2, t = lane & 3;
  const int S = p.S;
  const int rank = S > 1 ? static_cast<int>(cluster_ctarank()) : 0;
  const int cluster = static_cast<int>(blockIdx.x) / S;
  if (S > 1) asm volatile("barrier.cluster.arrive.relaxed.aligned;" ::: "memory");
  const int R = 1 << p.R_shift, ksplit = kQWarps >> p.R_shift;
  const int tile = warp & (R - 1), kpart = warp >> p.R_shift;
  const int rounds = (p.groups - cluster + p.clusters - 1) / p.clusters;
  const int c_first = rank * p.slice;
  const int chunks = (p.in + kQChunk - 1) / kQChunk;
  const int nc = max(0, min(p.slice, chunks - c_first));
  const int64_t m0 = static_cast<int64_t>(blockIdx.y) * (8 * NT);
  const int M = static_cast<int>(min(p.M - m0, static_cast<int64_t>(8 * NT)));

  uint32_t* top = reinterpret_cast<uint32_t*>(smem);
  float* back = reinterpret_cast<float*>(smem + kQHead / 2);
  float* part = reinterpret_cast<float*>(smem + kQHead);
  constexpr int kPartWarp = 8 * NT * kQPart, kPartBuf = kQWarps * kPartWarp;
  float* recv = part + 2 * kPartBuf;
  const int recv_buf = S > 1 ? S * p.share : 0;
  const uint32_t ring = smem_u32(recv + 2 * recv_buf) + warp * (kQDepth * kQStage);
  const uint32_t xs = smem_u32(recv + 2 * recv_buf) + kQWarps * kQDepth * kQStage;

  // ---- the weights' stream ----
  Feed f;
  int f_round = 0, f_c = 0;
  auto enter = [&](int round) {   // the first chunk of a round
    f_round = round;
    f_c = ksplit > 1 ? (kpart + round) & (ksplit - 1) : 0;   // so that no part keeps the longer share
    if (round >= rounds) return;
    const int group = cluster + round * p.clusters;
    const Nvfp4Seg& sg = p.seg[group_seg(p, group)];
    const int row0 = ((group - sg.begin) * R + tile) * 16;
    const int ra = row0 + g, rb = ra + 8;
    f.q0 = sg.q;
    f.na = ra < sg.out ? p.in / 2 - 16 * t : 0;
    f.nb = rb < sg.out ? p.in / 2 - 16 * t : 0;
    f.qa = sg.q + static_cast<int64_t>(min(ra, sg.out - 1)) * sg.ldq + 16 * t;
    f.qb = sg.q + static_cast<int64_t>(min(rb, sg.out - 1)) * sg.ldq + 16 * t;
    f.sb = sg.sf;
    if (p.mode == 1) {
      // three aligned words a row hold its eight scales: 48 words, the second of a lane for the first sixteen
      const int64_t total = static_cast<int64_t>(sg.out) * p.cols;
      auto word = [&](int i, const uint8_t*& s, int64_t& left) {
        const int row = row0 + i / 3;
        const int64_t at = ((static_cast<int64_t>(row) * p.cols) & ~3ll) + 4 * (i % 3);
        s = sg.sf + at;
        left = row < sg.out ? total - at : 0;
      };
      word(lane, f.s0, f.left0);
      if (lane < 16) word(32 + lane, f.s1, f.left1);
      else f.left1 = 0;
    } else {
      const int row = row0 + lane / 2, half = lane & 1;
      const int r = min(row, sg.out - 1);
      if (p.mode == 0) {
        f.s0 = sg.sf + static_cast<int64_t>(r) * p.cols + 4 * half;
        f.left0 = row < sg.out ? p.cols - 4 * half : 0;
      } else {
        const int ktiles = (p.cols + 3) / 4;
        f.s0 = sg.sf + (static_cast<int64_t>(r / 128) * ktiles + half) * 512 + 16 * (r % 32) + 4 * (r % 128 / 32);
        f.left0 = row < sg.out ? 4 * (ktiles - half) : 0;   // in scales of this row: a tile of four 512 bytes on
      }
    }
  };
  // One chunk into stage `slot`, or an empty group where the stream is through.
  auto feed = [&](int slot) {
    while (f_round < rounds && f_c >= nc) enter(f_round + 1);
    if (f_round < rounds) {
      const int c = c_first + f_c;
      const uint32_t dst = ring + slot * kQStage;
      const int off = c * 64;
      const int za = max(0, min(16, f.na - off)), zb = max(0, min(16, f.nb - off));
      const uint8_t* sa = za ? f.qa + off : f.q0;
      const uint8_t* sb = zb ? f.qb + off : f.q0;
      if (p.wide) {
        cp_async_16_zfill(dst + lane * 16, sa, za);
        cp_async_16_zfill(dst + 512 + lane * 16, sb, zb);
      } else {
        cp_async_small<8>(dst + lane * 16, sa, min(za, 8));
        cp_async_small<8>(dst + lane * 16 + 8, za > 8 ? sa + 8 : f.q0, max(za - 8, 0));
        cp_async_small<8>(dst + 512 + lane * 16, sb, min(zb, 8));
        cp_async_small<8>(dst + 512 + lane * 16 + 8, zb > 8 ? sb + 8 : f.q0, max(zb - 8, 0));
      }
      if (p.mode == 1) {
        const int z0 = static_cast<int>(max(0ll, min(4ll, f.left0 - 8ll * c)));
        cp_async_small<4>(dst + kQCodes + lane * 4, z0 ? f.s0 + 8 * static_cast<int64_t>(c) : f.sb, z0);
        if (lane < 16) {
          const int z1 = static_cast<int>(max(0ll, min(4ll, f.left1 - 8ll * c)));
          cp_async_small<4>(dst + kQCodes + (32 + lane) * 4, z1 ? f.s1 + 8 * static_cast<int64_t>(c) : f.sb, z1);
        }
      } else {
        const bool in = f.left0 > 8 * c;
        const int64_t at = p.mode == 0 ? 8 * static_cast<int64_t>(c) : 1024 * static_cast<int64_t>(c);
        cp_async_small<4>(dst + kQCodes + (lane / 2) * 12 + (lane & 1) * 4, in ? f.s0 + at : f.sb, in ? 4 : 0);
      }
      f_c += ksplit;
    }
    cp_async_commit();
  };
  // Weights are not written by a kernel that is still running, so the stream starts before the previous kernel ends.
  enter(0);
  for (int i = 0; i < kQDepth - 1; ++i) feed(i);
  pdl_wait_prior_grid();
  pdl_launch_dependents();

  // ---- x of this slice: f16, in the order in which the lanes read it: [chunk][step pair][token][t][8] ----
  if (tid < 8 * NT) top[tid] = 0;
  __syncthreads();
  {
    const int vecs = nc * 16, k_first = c_first * kQChunk;   // vectors of eight elements a token
    const int spans = (vecs + 31) / 32, items = spans * M;   // a warp takes 32 vectors of one token at a time
    auto dst = [&](int v, int m) {   // chunk v / 16; in it t = v % 16 / 4, step pair v % 4
      return xs + ((((v >> 4) * 4 + (v & 3)) * M + m) * 4 + ((v >> 2) & 3)) * 16;
    };
#pragma unroll 4
    for (int it = warp; it < items; it += kQWarps) {
      const int m = it / spans, v = (it - m * spans) * 32 + lane;
      const int k = k_first + v * 8;
      uint4 r = make_uint4(0, 0, 0, 0);
      if (v < vecs && k < p.in) r = *reinterpret_cast<const uint4*>(p.x + (m0 + m) * p.ldx + k);
      uint32_t most = 0;
      const uint32_t w[4] = {r.x, r.y, r.z, r.w};
#pragma unroll
      for (int i = 0; i < 4; ++i) {   // the largest finite magnitude
        const uint32_t lo = w[i] & 0x7fffu, hi = (w[i] >> 16) & 0x7fffu;
        most = max(most, max(lo < 0x7f80u ? lo : 0u, hi < 0x7f80u ? hi : 0u));
      }
      most = __reduce_max_sync(0xffffffffu, most);
      if (lane == 0) atomicMax(&top[m], most);
      if (v < vecs) asm volatile("st.shared.v4.u32 [%0], {%1, %2, %3, %4};" ::"r"(dst(v, m)), "r"(r.x), "r"(r.y), "r"(r.z), "r"(r.w) : "memory");
    }
    __syncthreads();
#pragma unroll 2
    for (int it = warp; it < items; it += kQWarps) {
      const int m = it / spans, v = (it - m * spans) * 32 + lane;
      if (v >= vecs) continue;
      const int e = static_cast<int>(top[m] >> 7) - 127;   // -127: zeros and numbers below the normal ones
      const float up = __uint_as_float(static_cast<uint32_t>(min(15 - e, 120) + 127) << 23);
      const uint4 r = lds128(dst(v, m));
      const uint32_t w[4] = {r.x, r.y, r.z, r.w};
      uint32_t h[4];
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        const float lo = __uint_as_float(w[i] << 16) * up, hi = __uint_as_float(w[i] & 0xffff0000u) * up;
        asm("cvt.rn.f16x2.f32 %0, %1, %2;" : "=r"(h[i]) : "f"(hi), "f"(lo));
      }
      asm volatile("st.shared.v4.u32 [%0], {%1, %2, %3, %4};" ::"r"(dst(v, m)), "r"(h[0]), "r"(h[1]), "r"(h[2]), "r"(h[3]) : "memory");
    }
    if (tid < M) {
      const int e = static_cast<int>(top[tid] >> 7) - 127;
      back[tid] = __uint_as_float(static_cast<uint32_t>(127 - min(15 - e, 120)) << 23);
    }
    __syncthreads();
  }

  // ---- rounds ----
  const int E = (16 << p.R_shift) * M;   // outputs of a group: token-major, its rows innermost
  auto store = [&](int round, int e, float v) {
    const int group = cluster + round * p.clusters;
    const Nvfp4Seg& sg = p.seg[group_seg(p, group)];
    const int m = e >> (4 + p.R_shift), row = (group - sg.begin) * (16 << p.R_shift) + (e & ((16 << p.R_shift) - 1));
    if (row < sg.out) sg.y[(m0 + m) * sg.ldy + row] = f32_to_bf16_rn(v);
  };
  auto finish = [&](int round) {   // the cluster's sums of a group: this CTA's share
    const float* from = recv + (round & 1) * recv_buf;
    for (int i = tid; i < p.share; i += kQThreads) {
      const int e = rank * p.share + i;
      if (e >= E) break;
      float v = 0.0f;
      for (int s = 0; s < S; ++s) v += from[s * p.share + i];
      store(round, e, v);
    }
  };
  int slot = 0;
  uint32_t b_at[NT];
#pragma unroll
  for (int n = 0; n < NT; ++n) b_at[n] = xs + (min(n * 8 + g, M - 1) * 4 + t) * 16;   // columns past M repeat the last: unread
  for (int round = 0; round < rounds; ++round) {
    const int group = cluster + round * p.clusters;
    const Nvfp4Seg& sg = p.seg[group_seg(p, group)];
    uint32_t sh_a = 12 * g + 2 * t, sh_b = sh_a + 96;   // this lane's two scales in a stage
    if (p.mode == 1) {
      const int64_t ra = static_cast<int64_t>((group - sg.begin) * R + tile) * 16 + g;
      sh_a += static_cast<uint32_t>(ra * p.cols) & 3u;
      sh_b += static_cast<uint32_t>((ra + 8) * p.cols) & 3u;
    }
    float acc[NT][4];
#pragma unroll
    for (int n = 0; n < NT; ++n) acc[n][0] = acc[n][1] = acc[n][2] = acc[n][3] = 0.0f;
    for (int c = ksplit > 1 ? (kpart + round) & (ksplit - 1) : 0; c < nc; c += ksplit) {
      cp_async_wait<kQDepth - 2>();
      __syncwarp();
      feed(slot == 0 ? kQDepth - 1 : slot - 1);
      const uint32_t st = ring + slot * kQStage;
      slot = slot == kQDepth - 1 ? 0 : slot + 1;
      const uint4 wa = lds128(st + lane * 16), wb = lds128(st + 512 + lane * 16);
      uint32_t ca = lds_u8(st + kQCodes + sh_a) | (lds_u8(st + kQCodes + sh_a + 1) << 8);
      uint32_t cb = lds_u8(st + kQCodes + sh_b) | (lds_u8(st + kQCodes + sh_b + 1) << 8);
      const int col = (c_first + c) * 8 + 2 * t;
      if (col + 1 >= p.cols) {   // past the row's end stand the next row's scales
        const uint32_t keep = col >= p.cols ? 0u : 0xffu;
        ca &= keep;
        cb &= keep;
      }
      const uint32_t fa = f16x2_from_e4m3x2(static_cast<uint16_t>(ca)), fb = f16x2_from_e4m3x2(static_cast<uint16_t>(cb));
      const uint32_t pa[4] = {wa.x, wa.y, wa.z, wa.w}, pb[4] = {wb.x, wb.y, wb.z, wb.w};
      const uint32_t xc = static_cast<uint32_t>(c * 4 * M) * 64;
#pragma unroll
      for (int j = 0; j < 4; ++j) {
        const uint32_t s_a = __byte_perm(fa, fa, j < 2 ? 0x1010 : 0x3232), s_b = __byte_perm(fb, fb, j < 2 ? 0x1010 : 0x3232);
        uint4 b[NT];
#pragma unroll
        for (int n = 0; n < NT; ++n) b[n] = lds128(b_at[n] + xc + j * M * 64);
        const uint32_t a0[4] = {hmul2(f16x2_from_e2m1x2<0>(pa[j]), s_a), hmul2(f16x2_from_e2m1x2<0>(pb[j]), s_b),
                                hmul2(f16x2_from_e2m1x2<1>(pa[j]), s_a), hmul2(f16x2_from_e2m1x2<1>(pb[j]), s_b)};
        const uint32_t a1[4] = {hmul2(f16x2_from_e2m1x2<2>(pa[j]), s_a), hmul2(f16x2_from_e2m1x2<2>(pb[j]), s_b),
                                hmul2(f16x2_from_e2m1x2<3>(pa[j]), s_a), hmul2(f16x2_from_e2m1x2<3>(pb[j]), s_b)};
#pragma unroll
        for (int n = 0; n < NT; ++n) {
          mma_f16(acc[n], a0, b[n].x, b[n].y);
          mma_f16(acc[n], a1, b[n].z, b[n].w);
        }
      }
    }
    float* mine = part + (round & 1) * kPartBuf + warp * kPartWarp;
#pragma unroll
    for (int n = 0; n < NT; ++n)
#pragma unroll
      for (int i = 0; i < 4; ++i) mine[(n * 8 + 2 * t + (i & 1)) * kQPart + g + (i >> 1) * 8] = acc[n][i];
    __syncthreads();
    if (S > 1) {
      asm volatile("barrier.cluster.wait.acquire.aligned;" ::: "memory");   // every CTA runs, or the exchange of the round before is in
      if (round > 0) finish(round - 1);
    }
    const float scale = *sg.g;
    const float* from = part + (round & 1) * kPartBuf;
    for (int e = tid; e < E; e += kQThreads) {
      const int m = e >> (4 + p.R_shift), rr = e & ((16 << p.R_shift) - 1);
      const float* at = from + (rr >> 4) * kPartWarp + m * kQPart + (rr & 15);
      float v = 0.0f;
      for (int k = 0; k < ksplit; ++k) v += at[(k << p.R_shift) * kPartWarp];
      v = (v * scale) * back[m];
      if (S > 1) {
        const int owner = e / p.share;
        asm volatile("st.shared::cluster.f32 [%0], %1;" ::"r"(cluster_map(recv + (round & 1) * recv_buf + rank * p.share + (e - owner * p.share), owner)), "f"(v) : "memory");
      } else {
        store(round, e, v);
      }
    }
    if (S > 1) asm volatile("barrier.cluster.arrive.release.aligned;" ::: "memory");
  }
  if (S > 1) {
    asm volatile("barrier.cluster.wait.acquire.aligned;" ::: "memory");
    finish(rounds - 1);
  }
}

// ---------------------------------------------------------------------------------
// host
// ---------------------------------------------------------------------------------
struct Nvfp4Plan {
  int S = 0, R_shift = 0, groups = 0, clusters = 0, slice = 0, share = 0;
  size_t smem = 0;
};

// The largest bytes of shared memory of a launch with NT token tiles, S CTAs a cluster and R row tiles a group.
size_t nvfp4_smem(int NT, int M, int S, int R_shift, int slice, int* share) {
  *share = ((16 << R_shift) * M + S - 1) / S;
  const size_t part = 2ull * kQWarps * 8 * NT * kQPart * 4;
  const size_t recv = S > 1 ? (2ull * S * *share * 4 + 15) / 16 * 16 : 0;
  return kQHead + part + recv + static_cast<size_t>(kQWarps) * kQDepth * kQStage + static_cast<size_t>(slice) * kQChunk * 2 * M;
}

// Cluster size and row tiles a group, by an estimate of the call's time in ns: the weights' stream, x into every CTA's shared
// memory, and what each round and an exchange cost.
bool plan_nvfp4(const int32_t* outs, int n, int in, int M, int NT, const ServeDev& dev, Nvfp4Plan* best) {
  const int chunks = (in + kQChunk - 1) / kQChunk;
  double least = 0;
  bool found = false;
  for (int S = 1; S <= kQMaxS && S <= chunks; S *= 2) {
    const int slice = (chunks + S - 1) / S;
    for (int r = 0; r <= 3; ++r) {
      Nvfp4Plan c;
      c.S = S;
      c.R_shift = r;
      c.slice = slice;
      c.smem = nvfp4_smem(NT, M, S, r, slice, &c.share);
      if (c.smem > dev.smem_optin) continue;
      for (int i = 0; i < n; ++i) c.groups += (outs[i] + (16 << r) - 1) / (16 << r);
      const int fit = NT <= 2 ? static_cast<int>(std::min<size_t>(2, (dev.smem_optin + 1024) / (c.smem + 1024))) : 1;
      c.clusters = std::max(1, std::min(c.groups, dev.sms * fit / S));
      const int rounds = (c.groups + c.clusters - 1) / c.clusters, ksplit = kQWarps >> r;
      const int ctas = c.clusters * S, per_sm = (ctas + dev.sms - 1) / dev.sms, busy = std::min(ctas, dev.sms);
      const double bytes = static_cast<double>(per_sm) * rounds * ((slice + ksplit - 1) / ksplit) * kQWarps * kQStage;
      const double rate = std::min(90.0, 6600.0 / busy);   // bytes a ns of one SM
      const double t = bytes / rate + per_sm * static_cast<double>(slice) * kQChunk * 2 * M / 40.0 + rounds * (S > 1 ? 250.0 : 120.0) + (S > 1 ? 700.0 : 0.0);
      if (!found || t < least) {
        least = t;
        *best = c;
        found = true;
      }
    }
  }
  return found;
}

template <int NT>
cudaError_t launch_nvfp4(const Nvfp4Params& p, dim3 grid, size_t smem, const ServeDev& dev, cudaStream_t st) {
  static std::atomic<uint64_t> ready{0};   // devices on which the kernel may use all of an SM's shared memory
  const uint64_t bit = 1ull << dev.index;
  if (!(ready.load() & bit)) {
    const cudaError_t e = cudaFuncSetAttribute(aq_nvfp4_kernel<NT>, cudaFuncAttributeMaxDynamicSharedMemorySize, static_cast<int>(dev.smem_optin));
    if (e != cudaSuccess) return e;
    ready.fetch_or(bit);
  }
  return launch_serve(aq_nvfp4_kernel<NT>, p, grid, kQThreads, smem, st, p.S);
}

}  // namespace
}  // namespace aq

using namespace aq;

extern "C" aq_status aq_nvfp4_linear_multi(const aq_nvfp4_weight* w, int32_t n, const void* x, int64_t M, int64_t ldx,
                                           void* const* y, const int64_t* ldy, void* stream) {
  const char* who = "aq_nvfp4_linear";
  if (!w || !y || !ldy) return serve_fail(AQ_ERR_INVALID_ARG, "%s: NULL argument", who);
  if (n < 1 || n > AQ_MAX_FAMILIES) return serve_fail(AQ_ERR_INVALID_ARG, "%s: n=%d outside [1, %d]", who, n, AQ_MAX_FAMILIES);
  if (M < 0) return serve_fail(AQ_ERR_SHAPE, "%s: M=%lld is negative", who, (long long)M);
  const int32_t in = w[0].in;
  if (in < 16 || in % 16 || in > AQ_NVFP4_MAX_IN)
    return serve_fail(in > AQ_NVFP4_MAX_IN ? AQ_ERR_UNSUPPORTED : AQ_ERR_SHAPE, "%s: in=%d must be a multiple of 16 up to %d", who, in, AQ_NVFP4_MAX_IN);
  bool wide = true;
  ByteRows outs[AQ_MAX_FAMILIES], ins[1 + 3 * AQ_MAX_FAMILIES];
  for (int i = 0; i < n; ++i) {
    const aq_nvfp4_weight& a = w[i];
    if (!a.q || !a.sf || !a.global_scale) return serve_fail(AQ_ERR_INVALID_ARG, "%s: q, sf and global_scale must be non-NULL", who);
    if (a.in != in) return serve_fail(AQ_ERR_SHAPE, "%s: the weights' in differ (%d and %d)", who, in, a.in);
    if (a.sf_layout != w[0].sf_layout || (a.sf_layout != AQ_SF_LINEAR && a.sf_layout != AQ_SF_128X4))
      return serve_fail(AQ_ERR_INVALID_ARG, "%s: sf_layout must be AQ_SF_LINEAR or AQ_SF_128X4, one for all", who);
    if (a.out < 1) return serve_fail(AQ_ERR_SHAPE, "%s: out=%d must be >= 1", who, a.out);
    if (a.ldq < in / 2) return serve_fail(AQ_ERR_SHAPE, "%s: ldq=%lld < in/2=%d", who, (long long)a.ldq, in / 2);
    if (a.ldq % 8 || !serve_aligned(a.q, 8) || !serve_aligned(a.sf, 16) || !serve_aligned(a.global_scale, 4))
      return serve_fail(AQ_ERR_ALIGNMENT, "%s: q and ldq must be 8-byte aligned, sf 16-byte, global_scale 4-byte", who);
    wide = wide && a.ldq % 16 == 0 && serve_aligned(a.q, 16);
  }
  if (M == 0) return AQ_OK;
  if (!x) return serve_fail(AQ_ERR_INVALID_ARG, "%s: x must be non-NULL", who);
  if (!serve_aligned(x, 16) || (M > 1 && ldx % 8)) return serve_fail(AQ_ERR_ALIGNMENT, "%s: x must be 16-byte aligned and ldx a multiple of 8", who);
  if (ldx < in && M > 1) return serve_fail(AQ_ERR_SHAPE, "%s: ldx=%lld < in=%d", who, (long long)ldx, in);
  const int64_t cols = in / 16;
  int k = 0;
  ins[k++] = ByteRows(x, M, ldx * 2, in * 2);
  for (int i = 0; i < n; ++i) {
    if (!y[i]) return serve_fail(AQ_ERR_INVALID_ARG, "%s: y must be non-NULL", who);
    if (!serve_aligned(y[i], 2)) return serve_fail(AQ_ERR_ALIGNMENT, "%s: y must be aligned to its elements", who);
    if (ldy[i] < w[i].out && M > 1) return serve_fail(AQ_ERR_SHAPE, "%s: ldy=%lld < out=%d", who, (long long)ldy[i], w[i].out);
    outs[i] = ByteRows(y[i], M, ldy[i] * 2, static_cast<int64_t>(w[i].out) * 2);
    ins[k++] = ByteRows(w[i].q, w[i].out, w[i].ldq, in / 2);
    const int64_t sf = w[i].sf_layout == AQ_SF_LINEAR ? w[i].out * cols : (w[i].out + 127ll) / 128 * 128 * ((cols + 3) / 4 * 4);
    ins[k++] = ByteRows(w[i].sf, 1, sf, sf);
    ins[k++] = ByteRows(w[i].global_scale, 1, 4, 4);
  }
  for (int i = 0; i < n; ++i) {
    for (int j = 0; j < k; ++j)
      if (outs[i].meets(ins[j])) return serve_fail(AQ_ERR_OVERLAP, "%s: an output overlaps an input", who);
    for (int j = 0; j < i; ++j)
      if (outs[i].meets(outs[j])) return serve_fail(AQ_ERR_OVERLAP, "%s: two outputs overlap", who);
  }
  ServeDev dev;
  aq_status st = serve_device(&dev);
  if (st != AQ_OK) return st;
  // Token tiles of 8, 16 or 32: the largest that the tokens fill and whose x a cluster's shared memory holds.
  int32_t rows[AQ_MAX_FAMILIES];
  for (int i = 0; i < n; ++i) rows[i] = w[i].out;
  Nvfp4Plan plan;
  int NT = M <= 8 ? 1 : M <= 16 ? 2 : 4;
  for (; NT >= 1; NT /= 2)
    if (plan_nvfp4(rows, n, in, static_cast<int>(std::min<int64_t>(M, 8 * NT)), NT, dev, &plan)) break;
  if (NT < 1) return serve_fail(AQ_ERR_UNSUPPORTED, "%s: in=%d does not fit this device's shared memory", who, in);
  const int64_t tiles = (M + 8 * NT - 1) / (8 * NT);
  if (tiles > 65535) return serve_fail(AQ_ERR_SHAPE, "%s: M=%lld is too large", who, (long long)M);
  Nvfp4Params p = {};
  for (int i = 0, at = 0; i < n; ++i) {
    p.seg[i] = {static_cast<const uint8_t*>(w[i].q), static_cast<const uint8_t*>(w[i].sf), w[i].global_scale, static_cast<uint16_t*>(y[i]),
                w[i].ldq, ldy[i], w[i].out, at};
    at += (w[i].out + (16 << plan.R_shift) - 1) / (16 << plan.R_shift);
  }
  p.x = static_cast<const uint16_t*>(x);
  p.M = M;
  p.ldx = ldx;
  p.nseg = n;
  p.in = in;
  p.cols = static_cast<int32_t>(cols);
  p.mode = w[0].sf_layout == AQ_SF_128X4 ? 2 : cols % 4 ? 1 : 0;
  p.wide = wide;
  p.groups = plan.groups;
  p.clusters = plan.clusters;
  p.S = plan.S;
  p.R_shift = plan.R_shift;
  p.slice = plan.slice;
  p.share = plan.share;
  const dim3 grid(static_cast<unsigned>(plan.clusters) * plan.S, static_cast<unsigned>(tiles));
  const cudaStream_t cs = static_cast<cudaStream_t>(stream);
  const cudaError_t e = NT == 1 ? launch_nvfp4<1>(p, grid, plan.smem, dev, cs) : NT == 2 ? launch_nvfp4<2>(p, grid, plan.smem, dev, cs)
                                                                               : launch_nvfp4<4>(p, grid, plan.smem, dev, cs);
  return serve_launched(e, who);
}

extern "C" aq_status aq_nvfp4_linear(const aq_nvfp4_weight* w, const void* x, int64_t M, int64_t ldx, void* y, int64_t ldy, void* stream) {
  return aq_nvfp4_linear_multi(w, 1, x, M, ldx, &y, &ldy, stream);
}
