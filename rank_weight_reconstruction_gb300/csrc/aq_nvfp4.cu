// aq_nvfp4.cu -- aq_nvfp4_linear, aq_nvfp4_linear_multi: products of a few tokens with the 4-bit weights that
// aq_precompute_nvfp4 makes.
//
//   y[m, o] = RN_bf16( g * sum_k E2M1(q[o, k]) * E4M3(sf[o, k / 16]) * x[m, k] )
//
// A code times its block scale has six significant bits between 2^-10 and 2688: exact in f16, so the weights are widened
// to f16 in registers (one conversion for two codes, one packed product with the scale) and go to mma.sync as its 16-row
// operand, the tokens as its 8 columns. x enters as f16 too, each token's chunk of 256 K scaled by the power of two that
// brings its largest element to at least 2^15: an element down to 2^-32 of the largest keeps all its bits. Sums are fp32.
//
// Bound by memory (0.5625 bytes a weight are read once) and, near it, by instructions: a chunk of 16 rows and 256 K is 2304 bytes, about
// 300 instructions of a warp, of which 64 conversions (half an ALU clock of the SM each), 64 products by the scale and 16 mma.sync (2.5
// clocks each): the SM's share of the copy rate allows 100 clocks a chunk, and 110 to 125 are taken. Scales behind the product instead
// of before it would need each instruction's 16 K within one block, and so codes in pieces of two bytes; the matrix instructions
// that take both operands' block scales want x in 4 bits as well. 262144 rows of 1152, five tokens: 34.2 us (4970 GB/s); 21504 rows of
// 5376, one token 14.2 us (4580 GB/s), eight 16.2, 16 22.9, 32 44.
//
// A cluster of S CTAs, one an SM, takes a stretch of row tiles of 16, each CTA a K slice whose x it keeps in shared memory. Its sixteen
// warps share out the tiles' chunks, and each streams its own through a ring of its own (cp.async), so no barrier stands in the stream.
// Either a warp takes whole tiles, or the chunks laid end to end are cut into equal runs. A tile's sums leave from the registers of the
// warp whose run begins it, which adds those of the runs that go on with it, in their order. The cluster's CTAs are added in their
// order, through distributed shared memory.
#include <algorithm>
#include <atomic>
#include <type_traits>

#include "aq_serve.h"

namespace aq {
namespace {

constexpr int kQChunk = 256;                    // K of a chunk: 128 bytes of codes a row, 16 scales
constexpr int kQCodes = 16 * 128;               // bytes of a chunk's codes
constexpr int kQStage = kQCodes + 16 * 32;      // and up to 32 bytes of scales a row (two pieces of 16 hold 16 bytes at any alignment)
constexpr int kQRow = 4 * 144;                  // bytes of a chunk of a token of x

struct Nvfp4Seg {
  const uint8_t* q;
  const uint8_t* sf;
  const float* g;
  uint16_t* y;
  int64_t ldq, ldy;
  int32_t out;
  int32_t begin;       // first tile
};
struct Nvfp4Params {
  Nvfp4Seg seg[AQ_MAX_FAMILIES];
  const uint16_t* x;
  int64_t M, ldx;
  int32_t nseg, in;
  int32_t cols;        // in / 16
  int32_t wide;        // codes move in 16-byte pieces (8 otherwise)
  int32_t tiles, clusters, S;
  int32_t round;       // tiles of a round: the cluster's sums of a round meet together
  int32_t whole;       // a warp takes whole tiles
  int32_t tokens;      // of a launch row: up to 8 NT
  int32_t slice;       // chunks of a CTA's K slice
};

__device__ __forceinline__ void mma_f16(float (&d)[4], const uint32_t (&a)[4], uint32_t b0, uint32_t b1) {
  asm volatile("mma.sync.aligned.m16n8k16.row.col.f32.f16.f16.f32 {%0, %1, %2, %3}, {%4, %5, %6, %7}, {%8, %9}, "
               "{%0, %1, %2, %3};"
               : "+f"(d[0]), "+f"(d[1]), "+f"(d[2]), "+f"(d[3])
               : "r"(a[0]), "r"(a[1]), "r"(a[2]), "r"(a[3]), "r"(b0), "r"(b1));
}
// The same onto nothing.
__device__ __forceinline__ void mma_f16_first(float (&d)[4], const uint32_t (&a)[4], uint32_t b0, uint32_t b1) {
  asm volatile("mma.sync.aligned.m16n8k16.row.col.f32.f16.f16.f32 {%0, %1, %2, %3}, {%4, %5, %6, %7}, {%8, %9}, {%10, %10, %10, %10};"
               : "=f"(d[0]), "=f"(d[1]), "=f"(d[2]), "=f"(d[3])
               : "r"(a[0]), "r"(a[1]), "r"(a[2]), "r"(a[3]), "r"(b0), "r"(b1), "f"(0.0f));
}
// Eight E2M1 codes, the low nibbles first, as four pairs of halves. All four bytes in one statement: each conversion then picks its
// byte itself (3.2 clocks a warp and SM; with a shift for each 4.5, by masks and shifts 5.5).
__device__ __forceinline__ void f16_from_e2m1x8(uint32_t w, uint32_t (&h)[4]) {
  asm("{\n\t.reg .b8 b0, b1, b2, b3;\n\tmov.b32 {b0, b1, b2, b3}, %4;\n\tcvt.rn.f16x2.e2m1x2 %0, b0;\n\tcvt.rn.f16x2.e2m1x2 %1, b1;\n\t"
      "cvt.rn.f16x2.e2m1x2 %2, b2;\n\tcvt.rn.f16x2.e2m1x2 %3, b3;\n\t}"
      : "=r"(h[0]), "=r"(h[1]), "=r"(h[2]), "=r"(h[3])
      : "r"(w));
}
__device__ __forceinline__ uint32_t max_u16x2(uint32_t a, uint32_t b) {
  uint32_t r;
  asm("max.u16x2 %0, %1, %2;" : "=r"(r) : "r"(a), "r"(b));
  return r;
}
__device__ __forceinline__ uint32_t hmul2(uint32_t a, uint32_t b) {
  uint32_t r;
  asm("mul.rn.f16x2 %0, %1, %2;" : "=r"(r) : "r"(a), "r"(b));
  return r;
}
__device__ __forceinline__ void cp_async_16(uint32_t dst, const void* src) {
  asm volatile("cp.async.cg.shared.global [%0], [%1], 16;" ::"r"(dst), "l"(src) : "memory");
}
template <int BYTES>
__device__ __forceinline__ void cp_async_small(uint32_t dst, const void* src) {
  asm volatile("cp.async.ca.shared.global [%0], [%1], %2;" ::"r"(dst), "l"(src), "n"(BYTES) : "memory");
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
__device__ __forceinline__ uint32_t lds32(uint32_t a) {
  uint32_t r;
  asm volatile("ld.shared.u32 %0, [%1];" : "=r"(r) : "r"(a));
  return r;
}
__device__ __forceinline__ uint16_t lds16(uint32_t a) {
  uint16_t r;
  asm volatile("ld.shared.u16 %0, [%1];" : "=h"(r) : "r"(a));
  return r;
}
__device__ __forceinline__ float2 lds64f(uint32_t a) {
  float2 r;
  asm volatile("ld.shared.v2.f32 {%0, %1}, [%2];" : "=f"(r.x), "=f"(r.y) : "r"(a));
  return r;
}
template <int N>
__device__ __forceinline__ void cp_async_wait() {
  asm volatile("cp.async.wait_group %0;" ::"n"(N) : "memory");
}

__device__ __forceinline__ const Nvfp4Seg& tile_seg(const Nvfp4Params& p, int tile) {
  int s = 0;
  if (p.nseg > 1 && tile >= p.seg[1].begin) s = 1;
  if (p.nseg > 2 && tile >= p.seg[2].begin) s = 2;
  return p.seg[s];
}

// NW warps a CTA; DEPTH: ring stages of a warp, one chunk each; MODE of the scales: 0 linear, rows on 8 bytes; 1 linear, anywhere;
// 2 128x4. (Four tiles of tokens, two stages and mode 1 together pass 128 registers by four: 16 bytes a thread are spilled.)
template <int NT, int DEPTH, int NW, int MODE>
__global__ void __launch_bounds__(32 * NW, 16 / NW) aq_nvfp4_kernel(const __grid_constant__ Nvfp4Params p) {
  extern __shared__ __align__(1024) uint8_t smem[];
  const int tid = threadIdx.x, lane = tid & 31, warp = __shfl_sync(0xffffffffu, tid >> 5, 0), g = lane >> 2, t = lane & 3;
  const int S = p.S;
  const int rank = S > 1 ? static_cast<int>(cluster_ctarank()) : 0;
  const int cluster = static_cast<int>(blockIdx.x) / S;
  if (S > 1) asm volatile("barrier.cluster.arrive.relaxed.aligned;" ::: "memory");
  const int t_first = static_cast<int>(static_cast<int64_t>(p.tiles) * cluster / p.clusters);
  const int t_last = static_cast<int>(static_cast<int64_t>(p.tiles) * (cluster + 1) / p.clusters);
  const int rounds = (t_last - t_first + p.round - 1) / p.round;
  // Of a chunk of a row lane t of four takes two pieces of 16 bytes: side by side, or, where its scales' bytes can be read in twos, one of
  // either half, so that a last chunk of half a row's chunk is half the work.
  constexpr bool kHalves = MODE != 1;
  const int c_first = rank * p.slice, c_whole = p.in / kQChunk;   // chunks before c_whole lie within K
  const int nc = max(0, min(p.slice, (p.in + kQChunk - 1) / kQChunk - c_first));
  const int64_t m0 = static_cast<int64_t>(blockIdx.y) * p.tokens;
  const int M = static_cast<int>(min(p.M - m0, static_cast<int64_t>(p.tokens)));

  const uint32_t part = smem_u32(smem) + (tid & 31) * 16;                  // [NW][NT][lane] four sums, unless whole
  const int recv_tiles = (p.round + S - 1) / S;                           // tiles that one CTA of the cluster finishes
  const int recv_src = recv_tiles * 16 * p.tokens, recv_buf = S > 1 ? S * recv_src : 0;
  float* recv = reinterpret_cast<float*>(smem) + (p.whole ? 0 : NW * NT * 128);   // [2 or 1][S][recv_tiles][tokens][16]
  float* back = recv + (p.clusters * p.round >= p.tiles ? 1 : 2) * recv_buf;   // [slice][8 NT]
  const uint32_t ring = smem_u32(back + p.slice * 8 * NT) + warp * (DEPTH * kQStage);
  const uint32_t xs = smem_u32(back + p.slice * 8 * NT) + NW * DEPTH * kQStage;

  // A warp's run in a round, in chunks of the round's tiles laid end to end.
  auto run = [&](int round, int& first, int& count) {
    const int n = min(p.round, t_last - t_first - round * p.round);
    const int lo = p.whole ? ((n * warp) / NW) * nc : (n * nc * warp) / NW;
    first = lo;
    count = (p.whole ? ((n * (warp + 1)) / NW) * nc : (n * nc * (warp + 1)) / NW) - lo;
  };

  // ---- the weights' stream ----
  int f_round = -1, f_left = 0, f_tile = 0, f_c = 0;
  const uint8_t* f_q = nullptr;   // this lane's 16 bytes of row lane / 8 of the tile, chunk f_c; the others 4, 8 and 12 rows on
  const uint8_t* f_s = nullptr;   // its scales there
  int64_t f_row4 = 0;
  int f_safe = 0;                 // tiles of this segment before f_safe have all 16 rows, and room behind their scales
  int64_t f_skip = 0;             // from a tile's chunk behind the slice to the next tile's first
  const int s_step = MODE == 2 ? 2048 : 16;
  auto aim = [&] {
    const Nvfp4Seg& sg = tile_seg(p, f_tile);
    const int row0 = (f_tile - sg.begin) * 16, rows = min(16, sg.out - row0);
    f_safe = sg.begin + (sg.out - (MODE == 1 ? (31 + p.cols) / p.cols : 0)) / 16;
    f_skip = 16 * sg.ldq - nc * 128;
    f_row4 = 4 * sg.ldq;
    f_q = sg.q + static_cast<int64_t>(row0 + min(lane / 8, rows - 1)) * sg.ldq + (lane & 7) * 16 + static_cast<int64_t>(f_c) * 128;
    if (MODE <= 1) {   // row lane / 2: half of its 16 scales, or one of the two aligned pieces that hold them
      const int64_t at = static_cast<int64_t>(row0 + min(lane / 2, rows - 1)) * p.cols;
      f_s = sg.sf + f_c * 16 + (MODE == 0 ? at + (lane & 1) * 8 : (at & ~15ll) + (lane & 1) * 16);
    } else {             // 128x4: word lane & 3 (four scales: a tile of 512 bytes each) of rows lane / 4 and 8 more
      const int r = row0 + min(lane / 4, rows - 1);
      f_s = sg.sf + (static_cast<int64_t>(r / 128) * ((p.cols + 3) / 4) + (lane & 3)) * 512 + 16 * (r % 32) + 4 * (r % 128 / 32) + static_cast<int64_t>(f_c) * 2048;
    }
  };
  auto next_run = [&] {
    while (f_left == 0 && f_round + 1 < rounds) {
      int first;
      run(++f_round, first, f_left);
      if (f_left == 0) continue;
      f_tile = t_first + f_round * p.round + first / nc;
      f_c = c_first + first % nc;
      aim();
    }
  };
  auto next_tile = [&] {   // the slice's first chunk, a tile on
    f_c = c_first;
    if (++f_tile >= f_safe) return aim();
    f_q += f_skip;
    if (MODE <= 1) {
      f_s += 16 * (p.cols - nc);
    } else {
      const int i = f_tile - tile_seg(p, f_tile).begin;   // rows 16 apart stand 256 bytes apart, or 4 on in the 16 bytes of the row 32 before
      f_s += (i & 1 ? 256 : i & 7 ? -252 : (p.cols + 3) / 4 * 512 - 268) - nc * 2048ll;
    }
  };
  // Rows or bytes that are not there: zeros.
  auto copy_some = [&](uint32_t st, uint32_t dq) {
    const Nvfp4Seg& sg = tile_seg(p, f_tile);
    const int rows = min(16, sg.out - (f_tile - sg.begin) * 16);
    const int held = max(0, min(16, p.in / 2 - f_c * 128 - (lane & 7) * 16));   // bytes of the rows in this piece
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      const int z = lane / 8 + 4 * i < rows ? held : 0;
      const uint8_t* from = z ? f_q + i * f_row4 : sg.q;
      if (p.wide) {
        cp_async_16_zfill(dq + i * 512, from, z);
      } else {
        cp_async_small<8>(dq + i * 512, from, min(z, 8));
        cp_async_small<8>(dq + i * 512 + 8, z > 8 ? from + 8 : sg.q, max(z - 8, 0));
      }
    }
    const uint32_t ds = st + kQCodes;
    const int col = f_c * 16;
    if (MODE == 0) {
      const int z = lane / 2 < rows && col + (lane & 1) * 8 < p.cols ? 8 : 0;
      cp_async_small<8>(ds + lane * 8, z ? f_s : sg.sf, z);
    } else if (MODE == 1) {
      const int64_t left = static_cast<int64_t>(sg.out) * p.cols - (f_s - sg.sf);
      const int z = lane / 2 < rows ? static_cast<int>(max(int64_t(0), min(int64_t(16), left))) : 0;
      cp_async_16_zfill(ds + lane * 16, z ? f_s : sg.sf, z);
    } else {
#pragma unroll
      for (int i = 0; i < 2; ++i) {
        const int z = lane / 4 + 8 * i < rows && col + (lane & 3) * 4 < p.cols ? 4 : 0;
        cp_async_small<4>(ds + lane * 4 + 128 * i, z ? f_s + 128 * i : sg.sf, z);
      }
    }
  };
  const uint32_t to_q = (lane / 8) * 128 + (((lane & 7) ^ (((lane / 8) & 1) * (kHalves ? 4 : 1))) * 16);   // rows 4 apart keep their parity
  auto feed = [&](uint32_t st) {
    if (f_left > 0) {
      const uint32_t dq = st + to_q;
      if (f_tile < f_safe && f_c < c_whole) {
        if (p.wide) {
          cp_async_16(dq, f_q);
          cp_async_16(dq + 512, f_q + f_row4);
          cp_async_16(dq + 1024, f_q + 2 * f_row4);
          cp_async_16(dq + 1536, f_q + 3 * f_row4);
        } else {
#pragma unroll
          for (int i = 0; i < 4; ++i) {
            cp_async_small<8>(dq + i * 512, f_q + i * f_row4);
            cp_async_small<8>(dq + i * 512 + 8, f_q + i * f_row4 + 8);
          }
        }
        if (MODE == 0) {
          cp_async_small<8>(st + kQCodes + lane * 8, f_s);
        } else if (MODE == 1) {
          cp_async_16(st + kQCodes + lane * 16, f_s);
        } else {
          cp_async_small<4>(st + kQCodes + lane * 4, f_s);
          cp_async_small<4>(st + kQCodes + lane * 4 + 128, f_s + 128);
        }
      } else if (f_tile < f_safe && p.wide) {   // a row's last bytes: a piece with none of them reads at the chunk's first
        const int held = max(0, min(16, p.in / 2 - f_c * 128 - (lane & 7) * 16));
        const uint8_t* from = f_q - (held ? 0 : (lane & 7) * 16);
#pragma unroll
        for (int i = 0; i < 4; ++i) cp_async_16_zfill(dq + i * 512, from + i * f_row4, held);
        if (MODE == 0) {
          const bool is = f_c * 16 + (lane & 1) * 8 < p.cols;
          cp_async_small<8>(st + kQCodes + lane * 8, f_s - (is ? 0 : (lane & 1) * 8), is ? 8 : 0);
        } else if (MODE == 1) {
          cp_async_16(st + kQCodes + lane * 16, f_s);
        } else {
          const bool is = f_c * 16 + (lane & 3) * 4 < p.cols;
          const uint8_t* at = f_s - (is ? 0 : (lane & 3) * 512);
          cp_async_small<4>(st + kQCodes + lane * 4, at, is ? 4 : 0);
          cp_async_small<4>(st + kQCodes + lane * 4 + 128, at + 128, is ? 4 : 0);
        }
      } else {
        copy_some(st, dq);
      }
      f_q += 128;
      f_s += s_step;
      ++f_c;
      if (--f_left == 0) {
        next_run();
      } else if (f_c == c_first + nc) {
        next_tile();
      }
    }
    cp_async_commit();
  };
  // Weights are not written by a kernel that is still running, so the stream starts before the previous kernel ends.
  next_run();
  for (int i = 0; i < DEPTH - 1; ++i) feed(ring + i * kQStage);
  // A warp's first piece of x, [token][chunk] from a place of the CTA's own on, and the way from one to its next.
  const int items = nc * M;
  int m = 0, c = 0, by_m = 0, by_c = 0;
  if (items) {
    const int at = static_cast<int>(__umulhi(blockIdx.x * 0x9e3779b9u, static_cast<uint32_t>(items))) + warp;
    m = at / nc;
    c = at - m * nc;
    by_m = NW / nc;
    by_c = NW - by_m * nc;
    while (m >= M) m -= M;
  }
  pdl_wait_prior_grid();
  pdl_launch_dependents();

  // ---- x of this slice: f16, [chunk][token][t][word of codes][8], the lanes' rows of 128 bytes 144 apart, so that what eight lanes read
  // together lies in eight places of the banks. A warp takes a chunk of a token at a time; the CTAs start at different ones, or all would ask the same
  // part of L2 at once ----
  const uint32_t x_chunk = static_cast<uint32_t>(M) * kQRow;
  {
    const uint32_t x_lane = xs + (kHalves ? ((lane >> 2) & 3) * 144 + (lane >> 4) * 64 + (lane & 3) * 16 : (lane >> 3) * 144 + (lane & 7) * 16);
    constexpr int kBatch = 8;   // loads in flight
    for (int i0 = warp; i0 < items; i0 += kBatch * NW) {
      uint4 r[kBatch];
      int mc[kBatch];
#pragma unroll
      for (int j = 0; j < kBatch; ++j) {
        const int k = (c_first + c) * kQChunk + lane * 8;
        const bool there = i0 + j * NW < items;
        mc[j] = there ? (m << 16) | c : -1;
        r[j] = make_uint4(0, 0, 0, 0);
        if (there && k < p.in) r[j] = *reinterpret_cast<const uint4*>(p.x + (m0 + m) * p.ldx + k);
        m += by_m;
        c += by_c;
        if (c >= nc) {
          c -= nc;
          ++m;
        }
        while (m >= M) m -= M;   // by_m may pass M: a slice of few chunks of few tokens
      }
#pragma unroll
      for (int j = 0; j < kBatch; ++j) {
        if (mc[j] < 0) continue;
        const int m = mc[j] >> 16, c = mc[j] & 0xffff;
        const uint32_t w[4] = {r[j].x, r[j].y, r[j].z, r[j].w};
        // The largest magnitude. A token with an infinity or a NaN has no finite output, so what becomes of its numbers is all one.
        uint32_t most = max_u16x2(max_u16x2(w[0] & 0x7fff7fffu, w[1] & 0x7fff7fffu), max_u16x2(w[2] & 0x7fff7fffu, w[3] & 0x7fff7fffu));
        most = max(most & 0xffffu, most >> 16);
        const int e = static_cast<int>(__reduce_max_sync(0xffffffffu, most) >> 7) - 127;   // -127: zeros and numbers below the normal ones
        const int lift = min(15 - e, 120);
        const float up = __uint_as_float(static_cast<uint32_t>(lift + 127) << 23);
        uint32_t h[4];
#pragma unroll
        for (int i = 0; i < 4; ++i) {
          float lo, hi;
          fmul2_rn(lo, hi, __uint_as_float(w[i] << 16), __uint_as_float(w[i] & 0xffff0000u), up, up);
          asm("cvt.rn.f16x2.f32 %0, %1, %2;" : "=r"(h[i]) : "f"(hi), "f"(lo));
        }
        asm volatile("st.shared.v4.u32 [%0], {%1, %2, %3, %4};" ::"r"(x_lane + c * x_chunk + m * kQRow), "r"(h[0]), "r"(h[1]), "r"(h[2]), "r"(h[3]) : "memory");
        if (lane == 0) back[c * 8 * NT + m] = __uint_as_float(static_cast<uint32_t>(127 - lift) << 23);
      }
    }
    __syncthreads();
  }

  // ---- rounds ----
  auto put = [&](int tile, int m, int r, const float4& v) {   // four outputs: rows r.. of a tile
    const Nvfp4Seg& sg = tile_seg(p, tile);
    const int row = (tile - sg.begin) * 16 + r;
    uint16_t* to = sg.y + (m0 + m) * sg.ldy + row;
    const uint16_t h[4] = {f32_to_bf16_rn(v.x), f32_to_bf16_rn(v.y), f32_to_bf16_rn(v.z), f32_to_bf16_rn(v.w)};
    if (row + 4 <= sg.out && (reinterpret_cast<uintptr_t>(to) & 7) == 0) {
      *reinterpret_cast<uint2*>(to) = make_uint2(h[0] | static_cast<uint32_t>(h[1]) << 16, h[2] | static_cast<uint32_t>(h[3]) << 16);
    } else {
#pragma unroll
      for (int i = 0; i < 4; ++i)
        if (row + i < sg.out) to[i] = h[i];
    }
  };
  auto add = [](float4& v, const float* at) {
    const float4 x = *reinterpret_cast<const float4*>(at);
    v.x += x.x, v.y += x.y, v.z += x.z, v.w += x.w;
  };
  const int eights = (M + 7) / 8;   // the sums that warps share go by eight tokens of a tile, four rows a lane
  const int l_m = lane >> 2, l_r = 4 * (lane & 3);
  // Tile i of a round is finished by CTA i % S of the cluster, as its tile i / S: the sums of all CTAs with a part of K in their order.
  const int parts = (p.in + kQChunk * p.slice - 1) / (kQChunk * p.slice);
  auto finish = [&](int round) {
    const float* from = recv + (round & 1) * recv_buf;
    const int n = min(p.round, t_last - t_first - round * p.round), mine = (n - rank + S - 1) / S;
    for (int e = warp; e < mine * eights; e += NW) {
      const int i = e / eights, m = 8 * (e - i * eights) + l_m;
      if (m >= M) continue;
      const float* at = from + i * 16 * p.tokens + m * 16 + l_r;
      float4 v = make_float4(0.0f, 0.0f, 0.0f, 0.0f);
      for (int s = 0; s < parts; ++s) add(v, at + s * recv_src);
      put(t_first + round * p.round + i * S + rank, m, l_r, v);
    }
  };
  uint32_t b_at[NT];
#pragma unroll
  for (int n = 0; n < NT; ++n) b_at[n] = min(n * 8 + g, M - 1) * kQRow + t * 144;   // columns past M repeat the last: unread
  const uint32_t at_a = g * 128 + (kHalves ? (t ^ ((g & 1) * 4)) : ((2 * t) ^ (g & 1))) * 16, at_s = kQCodes + (kHalves ? 16 * g + 2 * t : 32 * g + 4 * t);
  const uint32_t back_at = smem_u32(back) + 8 * t;
  if (S > 1) asm volatile("barrier.cluster.wait.acquire.aligned;" ::: "memory");   // the cluster's other CTAs run
  const int last_left = p.in - c_whole * kQChunk;   // K of a chunk that is not whole
  uint32_t st = ring, st_feed = ring + (DEPTH - 1) * kQStage;
  int seg_end = 0;              // first tile behind the segment of:
  float scale = 0.0f;
  uint16_t* y_lane = nullptr;   // row g of its first tile, token 2 t
  int64_t ldy = 0;
  int seg_begin = 0, seg_out = 0;
  for (int round = 0; round < rounds; ++round) {
    const int tile0 = t_first + round * p.round;
    int first, left;
    run(round, first, left);
    int tile = nc ? first / nc : 0, c = nc ? first - tile * nc : 0;
    if (!p.whole && round > 0) __syncthreads();   // the sums of the round before have been taken
    const int units = min(p.round, t_last - tile0) * nc;
    float tot[NT][4];
    // A tile's sums on their way out of this CTA: over the cluster to the one that adds them up, or rounded.
    auto leave = [&](int tile) {
      const uint32_t to = S > 1 ? cluster_map(recv + (round & 1) * recv_buf + rank * recv_src + (tile / S) * 16 * p.tokens, tile % S) : 0;
      const int row0 = (tile0 + tile - seg_begin) * 16, rows = seg_out - row0 - g;   // from row g on
#pragma unroll
      for (int n = 0; n < NT; ++n)
#pragma unroll
        for (int i = 0; i < 4; ++i) {
          const int m = n * 8 + 2 * t + (i & 1), r = g + (i >> 1) * 8;
          if (m >= M) continue;
          if (S > 1) asm volatile("st.shared::cluster.f32 [%0], %1;" ::"r"(to + (m * 16 + r) * 4), "f"(tot[n][i]) : "memory");
          else if ((i >> 1) * 8 < rows) y_lane[(n * 8 + (i & 1)) * ldy + row0 + (i >> 1) * 8] = f32_to_bf16_rn(tot[n][i]);
        }
    };
    int kept = -1;   // tile that this warp's run begins and does not end, its last
    while (left > 0) {
      const int here = min(left, nc - c);   // chunks of this tile
      if (tile0 + tile >= seg_end) {
        const Nvfp4Seg& sg = tile_seg(p, tile0 + tile);
        scale = *sg.g;
        seg_begin = sg.begin;
        seg_out = sg.out;
        seg_end = sg.begin + (sg.out + 15) / 16;
        ldy = sg.ldy;
        y_lane = sg.y + (m0 + 2 * t) * ldy + g;
      }
      uint32_t sa = 0, sb = 0;   // where the rows' scales stand in their pieces
      if (MODE == 1) {
        const uint32_t r = static_cast<uint32_t>((tile0 + tile - seg_begin) * 16 + g) * static_cast<uint32_t>(p.cols);
        sa = r & 15u;
        sb = (r + 8u * static_cast<uint32_t>(p.cols)) & 15u;
      }
#pragma unroll
      for (int n = 0; n < NT; ++n) tot[n][0] = tot[n][1] = tot[n][2] = tot[n][3] = 0.0f;
      uint32_t xc = xs + c * x_chunk, bk = back_at + c * 32 * NT;
      const int c_end = c_first + c + here;
#pragma unroll 1
      for (int ca = c_first + c; ca < c_end; ++ca) {
        cp_async_wait<DEPTH - 2>();
        __syncwarp();
        feed(st_feed);
        st_feed = st;
        uint32_t sc[2][2];   // [row g, g + 8][half]: two scales
        if (MODE == 1) {
          const uint32_t wa = st + at_s + (sa & ~3u), wb = st + at_s + 256 + (sb & ~3u);
          const uint32_t a = __funnelshift_r(lds32(wa), lds32(wa + 4), (sa & 3u) * 8), b = __funnelshift_r(lds32(wb), lds32(wb + 4), (sb & 3u) * 8);
          sc[0][0] = a, sc[0][1] = a >> 16, sc[1][0] = b, sc[1][1] = b >> 16;
        } else {
#pragma unroll
          for (int i = 0; i < 4; ++i) sc[i >> 1][i & 1] = lds16(st + at_s + (i >> 1) * 128 + (i & 1) * 8);
        }
        if (ca >= c_whole) {   // behind a row's scales stand the next row's, or what the layout is filled up with
#pragma unroll
          for (int h = 0; h < 2; ++h) {
            const int over = ca * 16 + (kHalves ? 8 * h + 2 * t : 4 * t + 2 * h) + 2 - p.cols;
            const uint32_t keep = over <= 0 ? 0xffffu : over == 1 ? 0xffu : 0u;
            sc[0][h] &= keep;
            sc[1][h] &= keep;
          }
        }
        uint32_t xb[NT];
#pragma unroll
        for (int n = 0; n < NT; ++n) xb[n] = xc + b_at[n];
        float acc[NT][4], odd[4];   // one tile of tokens: two chains, so that a product does not wait for the one before
        // Up to two tiles of tokens the products of a word of codes stand behind the next word's widening, and the two run side by side
        // (the loop by itself: 3.9 clocks a word, warp and SM, 4.5 with the products first). With four the products take longest.
        constexpr bool kBehind = NT <= 2;
        uint32_t a0[4], a1[4];
        uint4 b[NT];
        auto products = [&](bool first) {
#pragma unroll
          for (int n = 0; n < NT; ++n) {
            if (first) mma_f16_first(acc[n], a0, b[n].x, b[n].y);
            else mma_f16(acc[n], a0, b[n].x, b[n].y);
          }
          if (NT == 1) {
            if (first) mma_f16_first(odd, a1, b[0].z, b[0].w);
            else mma_f16(odd, a1, b[0].z, b[0].w);
          } else {
#pragma unroll
            for (int n = 0; n < NT; ++n) mma_f16(acc[n], a1, b[n].z, b[n].w);
          }
        };
        auto half = [&](auto which) {   // sixteen bytes of codes a row: two blocks
          constexpr int h = decltype(which)::value;
          const uint4 wa = lds128(st + (at_a ^ (h * (kHalves ? 64 : 16)))), wb = lds128(st + 1024 + (at_a ^ (h * (kHalves ? 64 : 16))));
          const uint32_t pa[4] = {wa.x, wa.y, wa.z, wa.w}, pb[4] = {wb.x, wb.y, wb.z, wb.w};
          const uint32_t fa = f16x2_from_e4m3x2(static_cast<uint16_t>(sc[0][h])), fb = f16x2_from_e4m3x2(static_cast<uint16_t>(sc[1][h]));
#pragma unroll
          for (int j = 0; j < 4; ++j) {
            const uint32_t s_a = __byte_perm(fa, 0, j < 2 ? 0x1010 : 0x3232), s_b = __byte_perm(fb, 0, j < 2 ? 0x1010 : 0x3232);
            uint32_t ha[4], hb[4];
            f16_from_e2m1x8(pa[j], ha);
            f16_from_e2m1x8(pb[j], hb);
            const uint32_t n0[4] = {hmul2(ha[0], s_a), hmul2(hb[0], s_b), hmul2(ha[1], s_a), hmul2(hb[1], s_b)};
            const uint32_t n1[4] = {hmul2(ha[2], s_a), hmul2(hb[2], s_b), hmul2(ha[3], s_a), hmul2(hb[3], s_b)};
            if (kBehind && h + j) products(h == 0 && j == 1);
#pragma unroll
            for (int i = 0; i < 4; ++i) a0[i] = n0[i], a1[i] = n1[i];
#pragma unroll
            for (int n = 0; n < NT; ++n) b[n] = lds128(xb[n] + (h * 4 + j) * 16);
            if (!kBehind) products(h == 0 && j == 0);
          }
        };
        half(std::integral_constant<int, 0>());
        if (!kHalves || ca < c_whole || last_left > kQChunk / 2) half(std::integral_constant<int, 1>());
        if (kBehind) products(false);
#pragma unroll
        for (int n = 0; n < NT; ++n) {
          const float2 f = lds64f(bk + 32 * n);
#pragma unroll
          for (int i = 0; i < 4; ++i) tot[n][i] = fmaf((NT == 1 ? acc[n][i] + odd[i] : acc[n][i]) * scale, i & 1 ? f.y : f.x, tot[n][i]);
        }
        st = st == ring + (DEPTH - 1) * kQStage ? ring : st + kQStage;
        xc += x_chunk;
        bk += 32 * NT;
      }
      if (here == nc) {
        leave(tile);
      } else if (c == 0) {
        kept = tile;
      } else {   // a part of a tile that an earlier warp's run begins: the first of this run
#pragma unroll
        for (int n = 0; n < NT; ++n)
          asm volatile("st.shared.v4.f32 [%0], {%1, %2, %3, %4};" ::"r"(part + (warp * NT + n) * 512), "f"(tot[n][0]), "f"(tot[n][1]), "f"(tot[n][2]), "f"(tot[n][3]) : "memory");
      }
      left -= here;
      c += here;
      if (c == nc) {
        c = 0;
        ++tile;
      }
    }
    if (!p.whole) {
      __syncthreads();
      if (kept >= 0) {   // the runs that begin within the tile, in their order (one may be empty)
        for (int w = warp + 1; w < NW && (units * w) / NW < (kept + 1) * nc; ++w) {
          if ((units * w) / NW == (units * (w + 1)) / NW) continue;
#pragma unroll
          for (int n = 0; n < NT; ++n) {
            const uint4 x = lds128(part + (w * NT + n) * 512);
            tot[n][0] += __uint_as_float(x.x);
            tot[n][1] += __uint_as_float(x.y);
            tot[n][2] += __uint_as_float(x.z);
            tot[n][3] += __uint_as_float(x.w);
          }
        }
        leave(kept);
      }
    }
    if (S > 1) {
      // Sums of a round are read behind its barrier; those of the next go to the other buffer, and the ones after that come behind
      // the next barrier, which every CTA reaches with this reading done.
      cluster_sync_all();
      finish(round);
    }
  }
}

// ---------------------------------------------------------------------------------
// host
// ---------------------------------------------------------------------------------
// What a ring of three chunks leaves of an SM's shared memory: x comes through L1, which has what is left (21504 rows of 5376, us, K in one
// slice: 18.6 with three chunks in 228 KB, 17.4 with two in 187; 16 tokens, four slices 26.1 and 24.3).
constexpr size_t kQFree = 20 * 1024;
struct Nvfp4Plan {
  int S = 0, clusters = 0, slice = 0, round = 0, whole = 0, depth = 0, warps = 0;
  size_t smem = 0;
  double ns = 0;   // estimated
};

// Shared memory of a launch, in the kernel's order.
size_t nvfp4_smem(int NT, int M, int tok, int tiles, const Nvfp4Plan& c) {
  const size_t part = c.whole ? 0 : static_cast<size_t>(c.warps) * NT * 512;
  const size_t recv = c.S > 1 ? static_cast<size_t>(c.S) * ((c.round + c.S - 1) / c.S) * 16 * tok * 4 * (c.clusters * c.round >= tiles ? 1 : 2) : 0;
  return part + recv + static_cast<size_t>(c.slice) * 8 * NT * 4 + static_cast<size_t>(c.warps) * c.depth * kQStage +
         static_cast<size_t>(c.slice) * kQRow * M;
}

// Cluster size, warps a CTA, tiles a round and how the warps share them, by an estimate of the call's time in ns: the chunks that the
// busiest warp takes, x into every CTA's shared memory, what a round and an exchange cost, and the tokens' launch rows after one another
// (of CTAs of eight warps two run beside each other). Its figures are fitted to 39 products timed under every plan (M 1 to 32, K 80 to
// 21504, rows 100 to 262144); what it picks for these is within 1 % of the fastest on average, 14 % at worst (19451 + 181 + 25353 rows of
// 1936, M=15). It ranks plans: its times themselves are up to a third too low. CTAs of eight warps that leave half an SM
// free may begin under the tail of the kernel before. Some of them, us (S, runs or whole tiles, warps): 21504 rows of 5376, M=8: (2,
// runs, 16) 16.4, (1, runs, 16) 17.3, (4, whole, 16) 18.6, (1, whole, 16) 21.9, (1, runs, 8) 25.6; 262144 rows of 1152, M=5: (1, runs,
// 16) 33.7, (1, whole, 16) 34.2, (1, runs, 8) 42.6; 1536 rows of 1152, M=1: (1, runs, 8) 3.6, (1, runs, 16) 4.5, (2, runs, 8) 4.6; 5376
// rows of 21504, M=8: (4, runs, 16) 19.1, (8, whole, 16) 20.3, (1, runs, 16) 76.
bool plan_nvfp4(int tiles, int in, int M, int tok, int64_t rows_of_tokens, const ServeDev& dev, const int (&fit)[4], Nvfp4Plan* best) {
  const int NT = std::max(1, tok / 8), chunks = (in + kQChunk - 1) / kQChunk;
  const size_t half = (dev.smem_optin + 1024) / 2 - 1024;
  bool found = false;
  for (int i = 0, S = 1; i < 4 && S <= chunks; ++i, S *= 2)
    for (int way = 0; way < 4; ++way) {
      Nvfp4Plan c;
      c.S = S;
      c.whole = way & 1;
      c.warps = way & 2 ? 8 : 16;
      const size_t room = c.warps == 8 ? half : dev.smem_optin;
      c.slice = (chunks + S - 1) / S;
      c.clusters = std::max(1, std::min(tiles, fit[i]));
      const int each = (tiles + c.clusters - 1) / c.clusters;   // tiles of a cluster
      int rounds = 1;
      for (bool fits = false; !fits; ++rounds) {   // the fewest rounds and the deepest ring that fit
        c.round = (each + rounds - 1) / rounds;
        if (c.whole && rounds > 1) c.round = (c.round + c.warps - 1) / c.warps * c.warps;
        for (c.depth = NT > 1 && c.warps == 8 ? 2 : 3; c.depth >= (NT > 1 || c.warps == 16 ? 2 : 3) && !fits; --c.depth)
          fits = (c.smem = nvfp4_smem(NT, M, tok, tiles, c)) <= (c.depth == 3 && c.warps == 16 ? room - kQFree : room);
        ++c.depth;
        if (fits || c.round <= (c.whole ? c.warps : 1)) break;
      }
      if (c.smem > room) continue;
      rounds = (each + c.round - 1) / c.round;
      const double mine = c.whole ? (c.round + c.warps - 1) / c.warps * c.slice : (c.round * c.slice + c.warps - 1) / c.warps;   // chunks of a warp and round
      const bool eight = c.warps == 8;
      const double chunk = (NT == 1 ? 49.0 : NT == 2 ? 66.0 : 91.0) * (eight ? 1.56 : c.depth == 2 ? 1.16 : 1.0);
      const int pieces = c.slice * M, turns = (pieces + 8 * c.warps - 1) / (8 * c.warps);   // of x; a warp has eight on their way at once
      c.ns = mine * rounds * c.warps * chunk + (eight ? 1170.0 : 2210.0) + pieces * (eight ? 6.7 : 10.9) + 380.0 * (turns - 1) +
             (S > 1 ? 930.0 * rounds + each * 4.8 * M : 0.0) + (c.whole ? 0.0 : 460.0 * rounds + each * 3.2 * M);
      c.ns *= 1.0 + (rows_of_tokens - 1) * (eight ? 0.44 : 1.0);
      if (!found || c.ns < best->ns) *best = c;
      found = true;
    }
  return found;
}

// Clusters of 1, 2, 4 and 8 CTAs, one an SM, that the device holds at once (groups of SMs that a cluster may span bound them).
cudaError_t clusters_at_once(const ServeDev& dev, int (&fit)[4]) {
  static std::atomic<int> known[64][4];
  fit[0] = dev.sms;
  for (int i = 1; i < 4; ++i) {
    if (!(fit[i] = known[dev.index][i].load())) {
      cudaError_t e = cudaFuncSetAttribute(aq_nvfp4_kernel<1, 3, 16, 0>, cudaFuncAttributeMaxDynamicSharedMemorySize, static_cast<int>(dev.smem_optin));
      if (e != cudaSuccess) return e;
      cudaLaunchConfig_t cfg = {};
      cfg.gridDim = dim3(static_cast<unsigned>(dev.sms) & ~7u);
      cfg.blockDim = dim3(512);
      cfg.dynamicSmemBytes = dev.smem_optin;
      cudaLaunchAttribute at[1] = {};
      at[0].id = cudaLaunchAttributeClusterDimension;
      at[0].val.clusterDim.x = 1u << i;
      at[0].val.clusterDim.y = at[0].val.clusterDim.z = 1;
      cfg.attrs = at;
      cfg.numAttrs = 1;
      int n = 0;
      if ((e = cudaOccupancyMaxActiveClusters(&n, aq_nvfp4_kernel<1, 3, 16, 0>, &cfg)) != cudaSuccess) return e;
      known[dev.index][i].store(fit[i] = std::max(1, n));
    }
  }
  return cudaSuccess;
}

template <int NT, int DEPTH, int NW, int MODE>
cudaError_t launch_nvfp4(const Nvfp4Params& p, dim3 grid, size_t smem, const ServeDev& dev, cudaStream_t st) {
  static std::atomic<uint64_t> ready{0};   // devices on which the kernel may use all of an SM's shared memory
  const uint64_t bit = 1ull << dev.index;
  if (!(ready.load() & bit)) {
    const cudaError_t e = cudaFuncSetAttribute(aq_nvfp4_kernel<NT, DEPTH, NW, MODE>, cudaFuncAttributeMaxDynamicSharedMemorySize, static_cast<int>(dev.smem_optin));
    if (e != cudaSuccess) return e;
    ready.fetch_or(bit);
  }
  return launch_serve(aq_nvfp4_kernel<NT, DEPTH, NW, MODE>, p, grid, 32 * NW, smem, st, p.S);
}
template <int MODE>
cudaError_t launch_nvfp4(const Nvfp4Params& p, dim3 grid, const Nvfp4Plan& c, int tok, const ServeDev& dev, cudaStream_t st) {
  if (tok <= 8) {
    if (c.warps == 8) return launch_nvfp4<1, 3, 8, MODE>(p, grid, c.smem, dev, st);
    return c.depth == 3 ? launch_nvfp4<1, 3, 16, MODE>(p, grid, c.smem, dev, st) : launch_nvfp4<1, 2, 16, MODE>(p, grid, c.smem, dev, st);
  }
  if (tok == 16) {
    if (c.warps == 8) return launch_nvfp4<2, 2, 8, MODE>(p, grid, c.smem, dev, st);
    return c.depth == 3 ? launch_nvfp4<2, 3, 16, MODE>(p, grid, c.smem, dev, st) : launch_nvfp4<2, 2, 16, MODE>(p, grid, c.smem, dev, st);
  }
  if (c.warps == 8) return launch_nvfp4<4, 2, 8, MODE>(p, grid, c.smem, dev, st);
  return c.depth == 3 ? launch_nvfp4<4, 3, 16, MODE>(p, grid, c.smem, dev, st) : launch_nvfp4<4, 2, 16, MODE>(p, grid, c.smem, dev, st);
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
  int64_t row_tiles = 0;
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
    row_tiles += (a.out + 15ll) / 16;
  }
  if (row_tiles > 0x7fffffffLL / 16) return serve_fail(AQ_ERR_SHAPE, "%s: the weights have too many rows for one call", who);   // rows of a tile count in 32 bits
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
  int fit[4];
  cudaError_t e = clusters_at_once(dev, fit);
  if (e != cudaSuccess) return serve_launched(e, who);
  // Tokens of a launch row: 32, 16 or 8 by the estimate (21504 rows of 5376, 32 tokens, us: 49.8 at once, 44.4 in two rows; 1152 of 6912
  // 10.6 and 8.7; 49567 of 5264, 20 tokens: 97 and 134), or fewer where a cluster's shared memory does not hold so many.
  Nvfp4Plan plan;
  int tok = 0;
  for (int t = M <= 8 ? 8 : M <= 16 ? 16 : 32; t >= 1 && (t >= 8 || !tok); t /= 2) {
    Nvfp4Plan c;
    if (!plan_nvfp4(static_cast<int>(row_tiles), in, static_cast<int>(std::min<int64_t>(M, t)), t, (M + t - 1) / t, dev, fit, &c)) continue;
    if (!tok || c.ns < plan.ns) {
      tok = t;
      plan = c;
    }
  }
  const int64_t tiles = (M + tok - 1) / tok;
  if (tiles > 65535) return serve_fail(AQ_ERR_SHAPE, "%s: M=%lld is too large", who, (long long)M);
  Nvfp4Params p = {};
  for (int i = 0, at = 0; i < n; ++i) {
    p.seg[i] = {static_cast<const uint8_t*>(w[i].q), static_cast<const uint8_t*>(w[i].sf), w[i].global_scale, static_cast<uint16_t*>(y[i]),
                w[i].ldq, ldy[i], w[i].out, at};
    at += (w[i].out + 15) / 16;
  }
  p.x = static_cast<const uint16_t*>(x);
  p.M = M;
  p.ldx = ldx;
  p.nseg = n;
  p.in = in;
  p.cols = static_cast<int32_t>(cols);
  p.wide = wide;
  p.tiles = static_cast<int32_t>(row_tiles);
  p.clusters = plan.clusters;
  p.S = plan.S;
  p.round = plan.round;
  p.tokens = tok;
  p.slice = plan.slice;
  p.whole = plan.whole;
  const dim3 grid(static_cast<unsigned>(plan.clusters) * plan.S, static_cast<unsigned>(tiles));
  const cudaStream_t cs = static_cast<cudaStream_t>(stream);
  if (w[0].sf_layout == AQ_SF_128X4) e = launch_nvfp4<2>(p, grid, plan, tok, dev, cs);
  else e = cols % 8 == 0 ? launch_nvfp4<0>(p, grid, plan, tok, dev, cs) : launch_nvfp4<1>(p, grid, plan, tok, dev, cs);
  return serve_launched(e, who);
}

extern "C" aq_status aq_nvfp4_linear(const aq_nvfp4_weight* w, const void* x, int64_t M, int64_t ldx, void* y, int64_t ldy, void* stream) {
  return aq_nvfp4_linear_multi(w, 1, x, M, ldx, &y, &ldy, stream);
}
