// aq_attention.cu -- aq_tree_attention: attention of each sequence's newest (drafted) tokens over its
// paged cache.
//   o_i = sum_j p_ij v_j,  p_i = softmax over the visible j of scale * (q_i . k_j)
//
// Work. The rows of one sequence that read one key/value head (drafted tokens x group of query heads) form
// row tiles; a tile against its visible keys is an item, its keys cut into tiles of KS. The items' key
// tiles, laid end to end, are shared out evenly over a persistent grid, so that every CTA streams the same
// number of keys whatever the sequences' lengths; an item that ends up in several CTAs leaves fp32
// partial sums (at most two a CTA) that a second launch adds in order.
//
// One pass over the keys with the running maximum and sum of the softmax. A producer warp streams K and V
// pages through a ring of shared-memory stages with TMA (128-byte swizzle); consumer warps split a stage by
// keys (KG ways) and the tile by rows (RG ways), 16 rows a warp. With keys split over the warps each cache
// byte is read from shared memory once per 16 rows, no warp waits for another, and their softmax states meet
// once per item. The products are mma.sync: at 1 to 64 rows a byte of cache meets few rows, the kernel is
// bound by HBM, and the rows would fill a small part of a 128-lane tcgen05 accumulator.
//
// E4M3 codes become halves on their way into the registers (exact; mma.sync on E4M3 operands is no
// shortcut: it is carried out as the same conversions and f16 products, repeated for every use of a
// fragment). A query row is scaled by a power of two to [2^14, 2^15), so that its bf16 elements are exact in f16 down to
// 2^-28 of the largest; keys' scales multiply the scores. The weights against the running maximum, times the
// values' scales against the largest of them so far (a power of two), fill the range of f16 from 2^15 down to
// 2^-24: 11 bits each down to 2^-22 of the largest, and nothing below 2^-32 is kept (kTop and kLag). With a
// bf16 cache the weights are rounded to bf16 (2^-9).
//
// Measured, 32 query and 8 key/value heads of 128: 48 sequences of one token over 750 to 6000 E4M3 keys 64 us
// (343 MB: 5390 GB/s), over bf16 keys 106 us (665 MB: 6300 GB/s), 32 trees of 8 over 1024 to 8192 bf16 keys 126 us (609 MB: 4820
// GB/s); eight sequences of one token over 7500 to 60000 E4M3 keys 94 us (6090 GB/s), over 60000 each 158 us (6410). What the short calls pay beside the stream is the start (locating the work and the first loads, about
// 6 us) and the joining launch (about 4).
#include <math.h>

#include <algorithm>
#include <atomic>
#include <type_traits>

#include "aq_attention.cuh"

namespace aq {

aq_status attention_cache_map(CUtensorMap* m, const void* base, const aq_kv_cache* c, int box_cols, int box_rows, const char* who) {
  const bool e4m3 = c->type == AQ_KV_E4M3;
  const cuuint64_t es = e4m3 ? 1 : 2, row = c->head_dim * es;
  const cuuint64_t dims[3] = {static_cast<cuuint64_t>(c->head_dim), static_cast<cuuint64_t>(c->page_size),
                              static_cast<cuuint64_t>(c->pages) * c->kv_heads};
  const cuuint64_t strides[2] = {row, row * c->page_size};
  const cuuint32_t box[3] = {static_cast<cuuint32_t>(box_cols), static_cast<cuuint32_t>(box_rows), 1};
  const cuuint32_t unit[3] = {1, 1, 1};
  const serve_encode_fn fn = serve_encode();
  if (!fn) return serve_fail(AQ_ERR_CUDA, "%s: cuTensorMapEncodeTiled is not available from the driver", who);
  const CUresult r = fn(m, e4m3 ? CU_TENSOR_MAP_DATA_TYPE_UINT8 : CU_TENSOR_MAP_DATA_TYPE_BFLOAT16, 3, const_cast<void*>(base),
                        dims, strides, box, unit, CU_TENSOR_MAP_INTERLEAVE_NONE,
                        box_cols * es == 128 ? CU_TENSOR_MAP_SWIZZLE_128B : CU_TENSOR_MAP_SWIZZLE_64B,
                        CU_TENSOR_MAP_L2_PROMOTION_L2_256B, CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE);
  if (r != CUDA_SUCCESS) return serve_fail(AQ_ERR_CUDA, "%s: cuTensorMapEncodeTiled failed (%d)", who, static_cast<int>(r));
  return AQ_OK;
}

namespace {

// ---------------------------------------------------------------------------------
// instructions
// ---------------------------------------------------------------------------------
__device__ __forceinline__ void ldsm4(uint32_t (&r)[4], uint32_t addr) {
  asm volatile("ldmatrix.sync.aligned.m8n8.x4.shared.b16 {%0, %1, %2, %3}, [%4];"
               : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3])
               : "r"(addr)
               : "memory");
}
__device__ __forceinline__ void ldsm4_t(uint32_t (&r)[4], uint32_t addr) {
  asm volatile("ldmatrix.sync.aligned.m8n8.x4.trans.shared.b16 {%0, %1, %2, %3}, [%4];"
               : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3])
               : "r"(addr)
               : "memory");
}
__device__ __forceinline__ void mma_bf16(float (&d)[4], const uint32_t (&a)[4], uint32_t b0, uint32_t b1) {
  asm volatile("mma.sync.aligned.m16n8k16.row.col.f32.bf16.bf16.f32 {%0, %1, %2, %3}, {%4, %5, %6, %7}, {%8, %9}, "
               "{%0, %1, %2, %3};"
               : "+f"(d[0]), "+f"(d[1]), "+f"(d[2]), "+f"(d[3])
               : "r"(a[0]), "r"(a[1]), "r"(a[2]), "r"(a[3]), "r"(b0), "r"(b1));
}
__device__ __forceinline__ void mma_f16(float (&d)[4], const uint32_t (&a)[4], uint32_t b0, uint32_t b1) {
  asm volatile("mma.sync.aligned.m16n8k16.row.col.f32.f16.f16.f32 {%0, %1, %2, %3}, {%4, %5, %6, %7}, {%8, %9}, "
               "{%0, %1, %2, %3};"
               : "+f"(d[0]), "+f"(d[1]), "+f"(d[2]), "+f"(d[3])
               : "r"(a[0]), "r"(a[1]), "r"(a[2]), "r"(a[3]), "r"(b0), "r"(b1));
}
// Transposes an 8 x 8 matrix of 16-bit elements held one row pair a lane.
__device__ __forceinline__ uint32_t transpose8(uint32_t x) {
  uint32_t r;
  asm volatile("movmatrix.sync.aligned.m8n8.trans.b16 %0, %1;" : "=r"(r) : "r"(x));
  return r;
}
constexpr int kAttnStages = 6;          // most stages of the ring
constexpr int kAttnMaxWarps = 8;        // most consumer warps
constexpr int kAttnMaxRows = 32;        // rows of the largest tile
// ---------------------------------------------------------------------------------
// shapes: D elements a head; a warp takes 8 NR rows against CK keys at a time; NW warps are RG row groups by
// KG key groups. Keys are the matrix instruction's 16 lanes and rows its 8 columns, in both products: S^T = K Q^T
// and O^T = V^T P^T. So 1 to 8 rows (a single token's group of query heads) cost half of what they would as the
// 16 lanes, and a fragment of the cache, converted once, meets all rows of the warp.
// ---------------------------------------------------------------------------------
template <int D_, bool E4M3_, int NR_, int RG_, int NW_, int PER_SM_>
struct Shape {
  static constexpr int D = D_;
  static constexpr bool E4M3 = E4M3_;
  static constexpr int NR = NR_, RG = RG_, NW = NW_, KG = NW_ / RG_;
  static constexpr int kPerSm = PER_SM_;
  // eight consumer warps take the registers of the producer's warpgroup, of which one warp works
  static constexpr bool kSplitRegs = NW == 8;
  static constexpr int kThreads = (NW + (kSplitRegs ? 4 : 1)) * 32;
  static constexpr int M = 8 * NR * RG;                    // rows of a tile
  static constexpr int ES = E4M3 ? 1 : 2;
  // 16 KB to 64 KB a stage, so that three fit a CTA's share of shared memory
  static constexpr int CK = (E4M3 ? D * KG * kPerSm >= 2048 : D * KG >= 512) ? 16 : 32;
  static constexpr int KT = CK / 16;
  static constexpr int NI = CK * KG * D * ES >= 16384 || CK * KG >= 128 ? 1 : 2;
  static constexpr int KS = CK * KG * NI;                  // keys of a stage
  static constexpr int RB = D * ES < 128 ? D * ES : 128;   // bytes of a row of one column block
  static constexpr int kCode = KS * D * ES;                // bytes of K (or V) in a stage
  static constexpr int NC = D * ES / RB;
  static constexpr int kStage = 2 * kCode;
  static constexpr int kScale = E4M3 ? KS * 4 : 0;         // bytes of K's (or V's) scales in a stage
  static constexpr int kQ = M * D * 2;                     // queries, in the order of fragments
  static constexpr bool kQRegs = NR * D <= 256;            // ... and in registers
  static constexpr int kCols = D == 256 && NW == 8 ? 64 : 32;   // columns joined at a time
  static constexpr int kJoinLd = kCols + 4;
  static constexpr int kJoin = NW * 8 * NR * kJoinLd * 4;
  static_assert(M <= kAttnMaxRows && 8 * NR <= 32, "shared arrays");
};

struct AttnShared {
  uint64_t full[kAttnStages], empty[kAttnStages];
  uint32_t valid[kAttnStages];
  int32_t abort;
  AttnWork work;
  float m[kAttnMaxWarps][32], l[kAttnMaxWarps][32];
  float fac[kAttnMaxRows];                       // of a row's raw products, to base-2 logits; not negative
  int64_t pos[kAttnMaxRows];                  // of a row
  int32_t i[kAttnMaxRows];                     // its drafted index
};

template <class S>
__device__ __forceinline__ void produce(const AttnParams& p, AttnShared& sh, uint8_t* stage0, uint8_t* scale0,
                                        const int64_t (&range)[2], int stages, const AbortCtl& ctl) {
  const int lane = threadIdx.x & 31;
  const int page = 1 << p.page_shift;
  const int box = min(page, S::KS), np = S::KS / box;   // rows of a page in a tile; pages a tile touches
  int st = 0, issued = 0;
  uint32_t parity = 1;
  Walk<S::M, S::KS> w(p, sh.work, range);
  bool ok = true;
  while (ok && w.left > 0) {
    const int32_t* table = p.table + w.b * p.ld_table;
    auto page_id = [&](int64_t i) {   // -1: left out
      if (i >= p.pages_per_seq || (i << p.page_shift) >= w.s.hi || ((i + 1) << p.page_shift) <= w.s.lo) return -1;
      const int id = table[i];
      return id >= 0 && id < p.pages ? id : -1;
    };
    // page numbers of this sequence, 32 at a time and 32 ahead
    int64_t base = (static_cast<int64_t>(w.tile0) * S::KS) >> p.page_shift;
    int cur = page_id(base + lane), ahead = page_id(base + 32 + lane);
    for (int i = 0; i < w.n; ++i) {
      const int64_t key = static_cast<int64_t>(w.tile0 + i) * S::KS;
      const int64_t first = key >> p.page_shift;
      if (first >= base + 32) {
        base += 32;
        cur = ahead;
        ahead = page_id(base + 32 + lane);
      }
      const int id = __shfl_sync(0xffffffffu, cur, static_cast<int>(first - base) + (lane < np ? lane : 0));
      const bool valid = lane < np && id >= 0 && key + static_cast<int64_t>(lane) * box < w.s.hi;
      const uint32_t mask = __ballot_sync(0xffffffffu, valid);
      ok = mbar_wait(&sh.empty[st], parity, ctl);
      if (!__all_sync(0xffffffffu, ok)) {
        ok = false;
        break;
      }
      if (lane == 0) {
        sh.valid[st] = mask;
        mbar_arrive_expect_tx(&sh.full[st], __popc(mask) * box * (2 * S::D * S::ES + (S::E4M3 ? 8 : 0)));
      }
      __syncwarp();
      if (valid) {
        uint8_t* kd = stage0 + st * S::kStage + lane * box * S::RB;
        const int off = static_cast<int>(key & (page - 1));
        const int row = id * p.hk + w.head;
#pragma unroll
        for (int c = 0; c < S::NC; ++c) {
          tma_load_3d(kd + c * S::KS * S::RB, &p.tm_k, c * (S::RB / S::ES), off, row, &sh.full[st]);
          tma_load_3d(kd + S::kCode + c * S::KS * S::RB, &p.tm_v, c * (S::RB / S::ES), off, row, &sh.full[st]);
        }
        if (S::E4M3) {
          const int64_t cell = (static_cast<int64_t>(row) << p.page_shift) + off;
          uint8_t* sd = scale0 + st * 2 * S::kScale + lane * box * 4;
          bulk_load(sd, p.ks + cell, box * 4, &sh.full[st]);
          bulk_load(sd + S::kScale, p.vs + cell, box * 4, &sh.full[st]);
        }
      }
      ++issued;
      if (++st == stages) {
        st = 0;
        parity ^= 1;
      }
    }
    if (ok) w.next(p);
  }
  if (!ok) {   // a wait ran out: let the copies already issued land before the CTA may end
    for (int i = 0; i < min(issued, stages); ++i) {
      st = st == 0 ? stages - 1 : st - 1;
      const uint32_t use = (issued - 1 - i) / stages;
      const uint64_t t0 = global_timer_ns();
      while (!mbar_try_wait(&sh.full[st], use & 1))
        if (global_timer_ns() - t0 > ctl.timeout_ns) break;
    }
  }
}

// Shared-memory address of 16 bytes of a key: column block x / (RB / 16), swizzled as TMA writes it.
template <class S>
__device__ __forceinline__ uint32_t cell_addr(uint32_t base, int key, int x) {
  constexpr int XB = S::RB / 16;
  const int c = x / XB, xi = x % XB;
  const int sw = S::RB == 128 ? (key & 7) : ((key >> 1) & 3);
  return base + c * S::KS * S::RB + key * S::RB + ((xi ^ sw) << 4);
}

// Loads the item's queries into shared memory in the order of B fragments, uint2 [D / 16][M][4]: bf16 elements
// 16 k + 2 t + {0, 1} and 8 more; for E4M3 keys f16 elements 16 k + 4 t + {0, 1, 2, 3} (the order in which a key's
// codes are loaded), scaled by the row's power of two. The sign of the logits' scale goes into them.
template <class S>
__device__ __forceinline__ void load_queries(const AttnParams& p, AttnShared& sh, uint2* qs, const KeySpan& s, int head, int rt) {
  const int tid = threadIdx.x, lane = tid & 31;
  const float scale2 = p.scale * 1.4426950408889634f;
  const uint32_t sign = scale2 < 0.0f ? 0x80008000u : 0u;
  constexpr int L = S::D / 8;                  // lanes a row, 16 bytes each: 8, 16 or 32
  constexpr int kStep = S::NW * (32 / L);      // rows the warps take at once
  constexpr int kRounds = (S::M + kStep - 1) / kStep;
  const int c = lane % L;                      // elements 8 c .. 8 c + 7
  const uint32_t rows = static_cast<uint32_t>(s.T) * p.group, group = p.group;
  if (tid < S::M) {
    const uint32_t rr = static_cast<uint32_t>(rt) * S::M + tid;
    const int i = rr < rows ? p.by_group.quot(rr) : 0;
    sh.i[tid] = i;
    sh.pos[tid] = static_cast<int64_t>(s.ctx) + (p.mask && p.depth ? max(p.depth[s.first + i], 0) : i);
  }
  uint4 v[kRounds];                            // every round's load in flight
#pragma unroll
  for (int k = 0; k < kRounds; ++k) {
    const int r = (tid >> 5) * (32 / L) + lane / L + k * kStep;
    // rows past the last load the last and are zeroed on use: a load under a condition would be waited for at once
    const uint32_t rr = min(static_cast<uint32_t>(rt) * S::M + r, rows - 1), i = p.by_group.quot(rr);
    v[k] = *reinterpret_cast<const uint4*>(p.q + (static_cast<int64_t>(s.first) + i) * p.q_tok + (head * group + (rr - i * group)) * p.q_head + c * 8);
  }
#pragma unroll
  for (int k = 0; k < kRounds; ++k) {
    const int r = (tid >> 5) * (32 / L) + lane / L + k * kStep;
    if (r >= S::M) break;                      // whole groups of L lanes
    float fac = fabsf(scale2);
    uint32_t x[4] = {v[k].x ^ sign, v[k].y ^ sign, v[k].z ^ sign, v[k].w ^ sign};
    if (static_cast<uint32_t>(rt) * S::M + r >= rows) x[0] = x[1] = x[2] = x[3] = 0;
    if constexpr (S::E4M3) {
      uint32_t top = 0;
#pragma unroll
      for (int e = 0; e < 4; ++e) top = max(top, max((x[e] << 16) & 0x7fff0000u, x[e] & 0x7fff0000u));
      const uint32_t lanes = (L == 32 ? 0xffffffffu : (1u << L) - 1) << (lane & ~(L - 1));
#pragma unroll
      for (int o = L / 2; o > 0; o >>= 1) top = max(top, __shfl_xor_sync(lanes, top, o));
      const bool finite = top < 0x7f800000u;
      const int e = finite ? top_exponent(__uint_as_float(top)) : 0;
      const float f = pow2(14 - e);
      fac = finite ? pow2(e - 14) * fac : __uint_as_float(0x7fc00000u);   // a row with an infinity or a NaN has no finite score
#pragma unroll
      for (int y = 0; y < 4; ++y)
        x[y] = finite ? pack_f16x2(__uint_as_float(x[y] << 16) * f, __uint_as_float(x[y] & 0xffff0000u) * f) : 0u;
      uint2* dst = qs + ((c >> 1) * S::M + r) * 4 + (c & 1) * 2;
      dst[0] = make_uint2(x[0], x[1]);
      dst[1] = make_uint2(x[2], x[3]);
    } else {
      uint32_t* dst = reinterpret_cast<uint32_t*>(qs + ((c >> 1) * S::M + r) * 4) + (c & 1);
#pragma unroll
      for (int y = 0; y < 4; ++y) dst[2 * y] = x[y];
    }
    if (c == 0) sh.fac[r] = fac;
  }
}

// A warp's sums for its rows 2 t + {0, 1} of each of NR groups of eight.
template <class S>
struct Sums {
  // o[x][n]: O^T fragment, lanes the columns: E4M3 16 x + 2 g + {0: first half, 1: second}, bf16 16 x + g + {0, 8}
  float o[S::D / 16][S::NR][4];
  float m[S::NR][2], l[S::NR][2];   // the reference (base 2), the sum of the weights against it
};

// Adds the infinities and NaN among a step's values to the rows that see them (weights in w [row][key], -1: masked).
template <class S>
__device__ __forceinline__ void reach_rows(Sums<S>& a, const float* w, uint32_t vb, int k0) {
  const int lane = threadIdx.x & 31, g = lane >> 2, t = lane & 3;
#pragma unroll 1
  for (int k = 0; k < S::CK; ++k) {
#pragma unroll
    for (int x = 0; x < S::D / 16; ++x)
#pragma unroll
      for (int h = 0; h < 2; ++h) {
        const int d = S::E4M3 ? 16 * x + 2 * g + h : 16 * x + g + 8 * h;
        const uint32_t addr = cell_addr<S>(vb, k0 + k, d * S::ES / 16) + d * S::ES % 16;
        uint32_t v;
        bool special;
        if (S::E4M3) {
          asm volatile("ld.shared.u8 %0, [%1];" : "=r"(v) : "r"(addr) : "memory");
          special = (v & 0x7f) == 0x7f;
          v = 0x7fc00000u;
        } else {
          asm volatile("ld.shared.u16 %0, [%1];" : "=r"(v) : "r"(addr) : "memory");
          special = (v & 0x7f80) == 0x7f80;
          v <<= 16;
        }
        if (special) {
#pragma unroll
          for (int n = 0; n < S::NR; ++n)
#pragma unroll
            for (int c = 0; c < 2; ++c) {
              const float q = w[(8 * n + 2 * t + c) * S::kJoinLd + k];
              if (q >= 0.0f) a.o[x][n][2 * h + c] += q * __uint_as_float(v);
            }
        }
      }
  }
}

struct StepInfo {          // what a step that not every row sees in full needs besides
  uint32_t pages;
  int box_shift;
  int64_t key0;            // first key of the tile
  int rg;
};

// CK keys, the first being key k0 of the stage, against the warp's rows. WHOLE: every row sees every key.
template <class S, bool WHOLE>
__device__ __forceinline__ void step(const AttnParams& p, const AttnShared& sh, const KeySpan& span, const StepInfo& info, Sums<S>& a,
                                     const uint2* qs, const uint2 (&qr)[S::kQRegs ? S::D / 16 : 1][S::NR], uint32_t kb,
                                     uint32_t vb, const float* ksc, const float* vsc, float* mine, int k0,
                                     const float (&fac)[S::NR][2]) {
  constexpr int D = S::D, NR = S::NR, KT = S::KT;
  const int lane = threadIdx.x & 31, g = lane >> 2, t = lane & 3;
  // scores, in the units of fac: sc[j][n]: keys 16 j + g + {0, 8}, rows 8 n + 2 t + {0, 1}
  float sc[KT][NR][4];
#pragma unroll
  for (int j = 0; j < KT; ++j)
#pragma unroll
    for (int n = 0; n < NR; ++n) sc[j][n][0] = sc[j][n][1] = sc[j][n][2] = sc[j][n][3] = 0.0f;
  auto query = [&](int k, int n) { return S::kQRegs ? qr[S::kQRegs ? k : 0][n] : qs[(k * S::M + 8 * n + g) * 4 + t]; };
  if constexpr (S::E4M3) {
#pragma unroll
    for (int k = 0; k < D / 16; k += 2)
#pragma unroll
      for (int j = 0; j < KT; ++j) {
        uint32_t r[4];   // keys 0-7 and 8-15 of columns k, then of columns k + 1
        ldsm4(r, cell_addr<S>(kb, k0 + 16 * j + (lane & 15), k + (lane >> 4)));
#pragma unroll
        for (int i = 0; i < 2; ++i) {
          uint32_t f[4];
          widen(r[2 * i], f[0], f[2]);
          widen(r[2 * i + 1], f[1], f[3]);
#pragma unroll
          for (int n = 0; n < NR; ++n) {
            const uint2 b = query(k + i, n);
            mma_f16(sc[j][n], f, b.x, b.y);
          }
        }
      }
  } else {
#pragma unroll
    for (int k = 0; k < D / 16; ++k)
#pragma unroll
      for (int j = 0; j < KT; ++j) {
        uint32_t f[4];
        ldsm4(f, cell_addr<S>(kb, k0 + 16 * j + (lane & 15), 2 * k + (lane >> 4)));
#pragma unroll
        for (int n = 0; n < NR; ++n) {
          const uint2 b = query(k, n);
          mma_bf16(sc[j][n], f, b.x, b.y);
        }
      }
  }
  float vs[KT][2], ve[KT][2];   // values' scales; what they add to their keys' logits in the reference
#pragma unroll
  for (int j = 0; j < KT; ++j)
#pragma unroll
    for (int h = 0; h < 2; ++h) {
      vs[j][h] = 1.0f;
      ve[j][h] = 0.0f;
      if constexpr (S::E4M3) {
        const float ks = ksc[k0 + 16 * j + 8 * h + g];
        vs[j][h] = vsc[k0 + 16 * j + 8 * h + g];
        ve[j][h] = scale_log2(vs[j][h]) - kTop;
#pragma unroll
        for (int n = 0; n < NR; ++n) {
          sc[j][n][2 * h] *= ks;
          sc[j][n][2 * h + 1] *= ks;
        }
      }
    }
  // What the reference has to cover: the logits, and with E4M3 the values' scales on them. Looked at by each lane for
  // itself, put together only where one lane's passes the reference.
  float mt[NR][2];
  if constexpr (WHOLE) {
#pragma unroll
    for (int n = 0; n < NR; ++n)
#pragma unroll
      for (int c = 0; c < 2; ++c) {
        if constexpr (S::E4M3) {
          mt[n][c] = -INFINITY;
#pragma unroll
          for (int j = 0; j < KT; ++j)
            mt[n][c] = fmaxf(mt[n][c], fmaxf(fmaf(sc[j][n][c], fac[n][c], ve[j][0]), fmaf(sc[j][n][2 + c], fac[n][c], ve[j][1])));
        } else {
          float x = fmaxf(sc[0][n][c], sc[0][n][2 + c]);
#pragma unroll
          for (int j = 1; j < KT; ++j) x = fmaxf(x, fmaxf(sc[j][n][c], sc[j][n][2 + c]));
          mt[n][c] = x == -INFINITY ? x : x * fac[n][c];
        }
      }
  } else {
    const uint32_t bits = seen_bits(p, span, sh.i[info.rg * 8 * NR + min(lane, 8 * NR - 1)], sh.pos[info.rg * 8 * NR + min(lane, 8 * NR - 1)],
                                    info.key0 + k0, k0, S::CK, info.pages, info.box_shift);
#pragma unroll
    for (int n = 0; n < NR; ++n)
#pragma unroll
      for (int c = 0; c < 2; ++c) {
        const uint32_t mine_bits = __shfl_sync(0xffffffffu, bits, 8 * n + 2 * t + c) >> g;
        mt[n][c] = -INFINITY;
#pragma unroll
        for (int j = 0; j < KT; ++j)
#pragma unroll
          for (int h = 0; h < 2; ++h) {
            float& x = sc[j][n][2 * h + c];
            if (!((mine_bits >> (16 * j + 8 * h)) & 1)) x = -INFINITY;
            if (x != -INFINITY) mt[n][c] = fmaxf(mt[n][c], fmaf(x, fac[n][c], ve[j][h]));
          }
      }
  }
  bool grown = false;
#pragma unroll
  for (int n = 0; n < NR; ++n)
#pragma unroll
    for (int c = 0; c < 2; ++c) grown = grown || mt[n][c] > a.m[n][c] + kLag;
  if (__any_sync(0xffffffffu, grown)) {
#pragma unroll
    for (int n = 0; n < NR; ++n)
#pragma unroll
      for (int c = 0; c < 2; ++c) {
#pragma unroll
        for (int off = 4; off < 32; off *= 2) mt[n][c] = fmaxf(mt[n][c], __shfl_xor_sync(0xffffffffu, mt[n][c], off));
        const float mx = fmaxf(a.m[n][c], mt[n][c]);
        const float keep = ex2(a.m[n][c] - (mx == -INFINITY ? 0.0f : mx));
        a.m[n][c] = mx;
        a.l[n][c] *= keep;
#pragma unroll
        for (int x = 0; x < D / 16; ++x) {
          a.o[x][n][c] *= keep;
          a.o[x][n][2 + c] *= keep;
        }
      }
  }
  float mz[NR][2];   // the reference, 0 while every score was minus infinity
#pragma unroll
  for (int n = 0; n < NR; ++n)
#pragma unroll
    for (int c = 0; c < 2; ++c) mz[n][c] = a.m[n][c] == -INFINITY ? 0.0f : a.m[n][c];
  // weights
  uint32_t pw[KT][NR][2];
#pragma unroll
  for (int j = 0; j < KT; ++j)
#pragma unroll
    for (int n = 0; n < NR; ++n) {
#pragma unroll
      for (int c = 0; c < 4; ++c) {
        const bool off = !WHOLE && sc[j][n][c] == -INFINITY;
        float e = ex2(fmaf(sc[j][n][c], fac[n][c & 1], -mz[n][c & 1]));
        if (off) e = 0.0f;
        a.l[n][c & 1] += e;
        if (S::E4M3) e *= vs[j][c >> 1];
        if (S::E4M3 && off) e = 0.0f;   // whatever scale lies there
        if (!WHOLE) mine[(8 * n + 2 * t + (c & 1)) * S::kJoinLd + 16 * j + 8 * (c >> 1) + g] = off ? -1.0f : e;
        sc[j][n][c] = e;
      }
#pragma unroll
      for (int h = 0; h < 2; ++h)
        pw[j][n][h] = transpose8(S::E4M3 ? pack_f16x2(sc[j][n][2 * h], sc[j][n][2 * h + 1])
                                         : pack_bf16x2_cvt(sc[j][n][2 * h], sc[j][n][2 * h + 1]));
    }
  // values
  uint32_t bad = 0;   // infinities and NaN where not every row sees every key: they take no part in the product
  if constexpr (S::E4M3) {
    // 32 keys by 16 columns, or 16 keys by 32 columns at a time
#pragma unroll
    for (int y = 0; y < D / 16; y += 3 - KT) {
      uint32_t r[4];
      ldsm4_t(r, KT == 2 ? cell_addr<S>(vb, k0 + lane, y) : cell_addr<S>(vb, k0 + (lane & 15), y + (lane >> 4)));
#pragma unroll
      for (int u = 0; u < 2; ++u) {
        const int x = KT == 2 ? y : y + u, j = KT == 2 ? u : 0;
        uint32_t f[4];
#pragma unroll
        for (int i = 0; i < 2; ++i) {
          uint32_t& c = r[2 * u + i];
          if (!WHOLE) {
            const uint32_t nan = ((((c & 0x7f7f7f7fu) + 0x01010101u) & 0x80808080u) >> 7) * 255u;
            bad |= nan;
            c &= ~nan;
          }
          widen(__byte_perm(c, 0, 0x3120), f[2 * i], f[2 * i + 1]);   // keys 2 t, 2 t + 1: column 2 g, then 2 g + 1
        }
#pragma unroll
        for (int n = 0; n < NR; ++n) mma_f16(a.o[x][n], f, pw[j][n][0], pw[j][n][1]);
      }
    }
  } else {
#pragma unroll
    for (int j = 0; j < KT; ++j)
#pragma unroll
      for (int x = 0; x < D / 16; ++x) {
        uint32_t f[4];
        ldsm4_t(f, cell_addr<S>(vb, k0 + 16 * j + (lane & 7) + 8 * (lane >> 4), 2 * x + ((lane >> 3) & 1)));
        if (!WHOLE) {
#pragma unroll
          for (int i = 0; i < 4; ++i) {
            const uint32_t off = __vcmpeq2(f[i] & 0x7f807f80u, 0x7f807f80u);
            bad |= off;
            f[i] &= ~off;
          }
        }
#pragma unroll
        for (int n = 0; n < NR; ++n) mma_bf16(a.o[x][n], f, pw[j][n][0], pw[j][n][1]);
      }
  }
  if (!WHOLE) {
    __syncwarp();
    if (__any_sync(0xffffffffu, bad != 0)) reach_rows<S>(a, mine, vb, k0);
    __syncwarp();
  }
}

template <class S>
__device__ __forceinline__ void consume(const AttnParams& p, AttnShared& sh, const uint8_t* stage0, const uint8_t* scale0,
                                        uint2* qs, float* join, const int64_t (&range)[2], int stages, const AbortCtl& ctl) {
  constexpr int D = S::D, NR = S::NR;
  constexpr int kConsumers = S::NW * 32;
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
  const int g = lane >> 2, t = lane & 3;
  const int rg = warp / S::KG, kg = warp % S::KG;
  StepInfo info;
  info.box_shift = min(p.page_shift, 31 - __clz(S::KS));
  info.rg = rg;
  const uint32_t all_pages = S::KS >> info.box_shift >= 32 ? 0xffffffffu : (1u << (S::KS >> info.box_shift)) - 1;
  int st = 0;
  uint32_t parity = 0;
  Walk<S::M, S::KS> w(p, sh.work, range);
  float* mine = join + warp * 8 * NR * S::kJoinLd;
  bool ok = true;
  while (w.left > 0) {
    const int rt = w.rt;
    load_queries<S>(p, sh, qs, w.s, w.head, rt);
    named_bar_sync(1, kConsumers);
    const uint2* qw = qs + rg * 8 * NR * 4;
    uint2 qr[S::kQRegs ? D / 16 : 1][NR];
    if constexpr (S::kQRegs) {
#pragma unroll
      for (int k = 0; k < D / 16; ++k)
#pragma unroll
        for (int n = 0; n < NR; ++n) qr[k][n] = qw[(k * S::M + 8 * n + g) * 4 + t];
    }
    float fac[NR][2];
    Sums<S> a;
    int64_t top = 0;         // largest position of the warp's rows
#pragma unroll
    for (int n = 0; n < NR; ++n)
#pragma unroll
      for (int c = 0; c < 2; ++c) {
        const int r = rg * 8 * NR + 8 * n + 2 * t + c;
        fac[n][c] = sh.fac[r];
        top = max(top, sh.pos[r]);
        a.m[n][c] = -INFINITY;
        a.l[n][c] = 0.0f;
#pragma unroll
        for (int x = 0; x < D / 16; ++x) a.o[x][n][c] = a.o[x][n][2 + c] = 0.0f;
      }
#pragma unroll
    for (int off = 1; off < 4; off *= 2) top = max(top, __shfl_xor_sync(0xffffffffu, top, off));
    // keys [whole0, whole1) are seen by every row
    const int64_t whole1 = min(static_cast<int64_t>(w.s.ctx), w.s.hi), whole0 = p.window > 0 ? top - p.window + 1 : 0;

    for (int it = 0; it < w.n; ++it) {
      ok = ok && mbar_wait(&sh.full[st], parity, ctl);
      ok = __all_sync(0xffffffffu, ok);
      if (!ok) break;
      info.pages = sh.valid[st];
      const uint32_t kb = smem_u32(stage0 + st * S::kStage), vb = kb + S::kCode;
      const float* ksc = reinterpret_cast<const float*>(scale0 + st * 2 * S::kScale);
      const float* vsc = reinterpret_cast<const float*>(scale0 + st * 2 * S::kScale + S::kScale);
      info.key0 = static_cast<int64_t>(w.tile0 + it) * S::KS;
#pragma unroll 1
      for (int ni = 0; ni < S::NI; ++ni) {
        const int k0 = (kg * S::NI + ni) * S::CK;            // the step's first key within the tile
        const int64_t ka = info.key0 + k0;
        if (ka >= w.s.hi || ka + S::CK <= w.s.lo) continue;
        if (ka >= whole0 && ka + S::CK <= whole1 && info.pages == all_pages)
          step<S, true>(p, sh, w.s, info, a, qw, qr, kb, vb, ksc, vsc, mine, k0, fac);
        else
          step<S, false>(p, sh, w.s, info, a, qw, qr, kb, vb, ksc, vsc, mine, k0, fac);
      }
      __syncwarp();
      if (lane == 0) mbar_arrive(&sh.empty[st]);
      if (++st == stages) {
        st = 0;
        parity ^= 1;
      }
    }
    // the item's rows: the warps of a row group put their sums together
#pragma unroll
    for (int n = 0; n < NR; ++n)
#pragma unroll
      for (int c = 0; c < 2; ++c) {
#pragma unroll
        for (int off = 4; off < 32; off *= 2) a.l[n][c] += __shfl_xor_sync(0xffffffffu, a.l[n][c], off);
        if (g == 0) {
          sh.m[warp][8 * n + 2 * t + c] = a.m[n][c];
          sh.l[warp][8 * n + 2 * t + c] = a.l[n][c];
        }
      }
    named_bar_sync(1, kConsumers);
    const bool complete = w.n == w.len;
    const int slot = w.offset > 0 ? 0 : 1;   // partial sums: an item begun elsewhere, or one that goes on elsewhere
    float fold[NR][2];
#pragma unroll
    for (int n = 0; n < NR; ++n)
#pragma unroll
      for (int c = 0; c < 2; ++c) {
        float mx = -INFINITY;
        for (int k = 0; k < S::KG; ++k) mx = fmaxf(mx, sh.m[rg * S::KG + k][8 * n + 2 * t + c]);
        fold[n][c] = ex2(a.m[n][c] - (mx == -INFINITY ? 0.0f : mx));
      }
    for (int c0 = 0; c0 < D; c0 += S::kCols) {
#pragma unroll
      for (int x = 0; x < D / 16; ++x) {
        if (x * 16 < c0 || x * 16 >= c0 + S::kCols) continue;
#pragma unroll
        for (int n = 0; n < NR; ++n)
#pragma unroll
          for (int c = 0; c < 2; ++c) {
            float* dst = mine + (8 * n + 2 * t + c) * S::kJoinLd + x * 16 - c0;
            const float v0 = a.o[x][n][c] * fold[n][c], v1 = a.o[x][n][2 + c] * fold[n][c];
            if (S::E4M3) {
              *reinterpret_cast<float2*>(dst + 2 * g) = make_float2(v0, v1);
            } else {
              dst[g] = v0;
              dst[g + 8] = v1;
            }
          }
      }
      named_bar_sync(1, kConsumers);
      for (int u = tid; u < S::M * (S::kCols / 4); u += kConsumers) {
        const int r = u / (S::kCols / 4), c = u % (S::kCols / 4) * 4;
        const int g0 = r / (8 * NR) * S::KG, rr = r % (8 * NR);
        const uint32_t row = static_cast<uint32_t>(rt) * S::M + r;
        if (row >= static_cast<uint32_t>(w.s.T) * p.group || !ok) continue;
        float mx = -INFINITY, lt = 0.0f;
        float4 v = make_float4(0.0f, 0.0f, 0.0f, 0.0f);
#pragma unroll
        for (int k = 0; k < S::KG; ++k) mx = fmaxf(mx, sh.m[g0 + k][rr]);
        const float mz = mx == -INFINITY ? 0.0f : mx;
#pragma unroll
        for (int k = 0; k < S::KG; ++k) {
          lt += sh.l[g0 + k][rr] * ex2(sh.m[g0 + k][rr] - mz);
          const float4 y = *reinterpret_cast<const float4*>(join + ((g0 + k) * 8 * NR + rr) * S::kJoinLd + c);
          v.x += y.x;
          v.y += y.y;
          v.z += y.z;
          v.w += y.w;
        }
        if (complete) {
          const int i = sh.i[r];
          const int head = w.head * p.group + static_cast<int>(row - static_cast<uint32_t>(i) * p.group);
          const bool none = mx == -INFINITY && lt == 0.0f;
          const float inv = none ? 0.0f : 1.0f / lt;
          uint16_t* dst = p.o + (static_cast<int64_t>(w.s.first) + i) * p.o_tok + head * p.o_head + c0 + c;
          *reinterpret_cast<uint2*>(dst) = none ? make_uint2(0, 0)
                                                : make_uint2(pack_bf16x2_cvt(v.x * inv, v.y * inv), pack_bf16x2_cvt(v.z * inv, v.w * inv));
          if (p.lse && c0 == 0 && c == 0)
            p.lse[(static_cast<int64_t>(w.s.first) + i) * (p.hk * p.group) + head] = none ? -INFINITY : (mz + log2f(lt)) * 0.6931471805599453f;
        } else {
          const int64_t at = (static_cast<int64_t>(blockIdx.x) * 2 + slot) * S::M + r;
          *reinterpret_cast<float4*>(p.part_o + at * D + c0 + c) = v;
          if (c0 == 0 && c == 0) p.part_ml[at] = make_float2(mx, lt);
        }
      }
      named_bar_sync(1, kConsumers);
    }
    w.next(p);
  }
}

template <class S>
__global__ void __launch_bounds__(S::kThreads, S::kPerSm) aq_tree_attention_kernel(const __grid_constant__ AttnParams p) {
  extern __shared__ uint8_t raw[];
  __shared__ AttnShared sh;
  uint8_t* stage0 = raw + ((1024 - (smem_u32(raw) & 1023)) & 1023);
  uint8_t* scale0 = stage0 + p.stages * S::kStage;
  uint2* qs = reinterpret_cast<uint2*>(scale0 + p.stages * 2 * S::kScale);
  float* join = reinterpret_cast<float*>(qs) + S::kQ / 4;
  if (threadIdx.x == 0) {
    for (int i = 0; i < p.stages; ++i) {
      mbar_init(&sh.full[i], 1);
      mbar_init(&sh.empty[i], S::NW);
    }
    sh.abort = 0;
    fence_barrier_init();
    tma_prefetch_desc(&p.tm_k);
    tma_prefetch_desc(&p.tm_v);
  }
  pdl_wait_prior_grid();
  int64_t range[2];
  locate<S::M, S::KS>(p, sh.work, blockIdx.x == 0, range);
  pdl_launch_dependents();   // the joining blocks find their rows meanwhile; they wait for this grid before its results
  const AbortCtl ctl = {&sh.abort, p.status, p.timeout_ns};
  if (threadIdx.x >= S::NW * 32) {
    // 384 threads at 168 registers: 256 at 232 and 128 at 40
    if (S::kSplitRegs) asm volatile("setmaxnreg.dec.sync.aligned.u32 40;");
    if (threadIdx.x < S::NW * 32 + 32) produce<S>(p, sh, stage0, scale0, range, p.stages, ctl);
  } else {
    if (S::kSplitRegs) asm volatile("setmaxnreg.inc.sync.aligned.u32 232;");
    consume<S>(p, sh, stage0, scale0, qs, join, range, p.stages, ctl);
  }
}

// Adds the partial sums of the items that were shared between CTAs, in the CTAs' order. W warps to a row and query head,
// each taking every W-th part: one where an item has few parts (up to about eight: two rounds of loads), as the rows are then
// many and the blocks' waves are what they cost; four where a few items are cut into many. Measured, calls whole: 16384
// rows and heads of three parts 255 us with four warps and 247 with one, 256 of five parts 19.5 and 18.9, 512 of
// nineteen parts 29.2 and 41.6.
template <int D, int W>
__global__ void __launch_bounds__(128) aq_attention_join_kernel(const __grid_constant__ AttnParams p) {
  constexpr int N = D / 32;
  __shared__ float sm[4], sl[4], so[W == 1 ? 1 : 4][D];
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
  const int heads = p.hk * p.group;
  const uint32_t unit = blockIdx.x * (4u / W) + (W == 1 ? warp : 0), part = W == 1 ? 0 : warp;
  const int row = p.by_heads.quot(unit), head = unit - row * heads, kv_head = p.by_group.quot(head);
  // Before the wait: the batch's layout is an input that was complete when the main grid, whose blocks all got past their
  // own wait before these could start, began to read it.
  int b = -1;
  if (row < p.total_q) {
    for (int k = lane; k < p.batch; k += 32) {
      const int c0 = p.cu[k], c1 = p.cu[k + 1];
      if (c0 >= 0 && c0 <= row && row < c1 && row - c0 < p.max_q) b = k;
    }
  }
  b = __reduce_max_sync(0xffffffffu, b);
  const int in_seq = b < 0 ? 0 : row - p.cu[b];
  pdl_wait_prior_grid();
  pdl_launch_dependents();
  if (b < 0) return;
  const uint32_t r = static_cast<uint32_t>(in_seq) * p.group + (head - kv_head * p.group);
  const int shift = 31 - __clz(p.rows_per_tile);   // a power of two
  const AttnShare own = p.shares[b * p.row_tiles + (r >> shift)];
  const int rr = r & (p.rows_per_tile - 1);
  const int64_t t0 = own.first + static_cast<int64_t>(kv_head) * own.step;
  const int c0 = own.base + static_cast<int>(quot(t0, own.share)), c1 = own.base + static_cast<int>(quot(t0 + own.len - 1, own.share));
  if (c0 == c1) return;   // one CTA had it all
  float m = -INFINITY, l = 0.0f, o[N];
#pragma unroll
  for (int e = 0; e < N; ++e) o[e] = 0.0f;
  constexpr int kParts = 4;   // of each warp in flight at once
  for (int c = c0 + part; c <= c1; c += W * kParts) {
    float2 ml[kParts];
    __align__(8) float v[kParts][N];
#pragma unroll
    for (int k = 0; k < kParts; ++k) {
      const int cc = min(c + W * k, c1);   // past the last: the last again, left out below
      const int64_t at = (static_cast<int64_t>(cc) * 2 + (cc > c0 ? 0 : 1)) * p.rows_per_tile + rr;
      ml[k] = p.part_ml[at];
      const float* src = p.part_o + at * D + lane * N;
#pragma unroll
      for (int e = 0; e < N; e += 2) *reinterpret_cast<float2*>(&v[k][e]) = *reinterpret_cast<const float2*>(src + e);
    }
#pragma unroll
    for (int k = 0; k < kParts; ++k)
      if (c + W * k > c1) {
        ml[k] = make_float2(-INFINITY, 0.0f);
#pragma unroll
        for (int e = 0; e < N; ++e) v[k][e] = 0.0f;
      }
    float mx = m;
#pragma unroll
    for (int k = 0; k < kParts; ++k) mx = fmaxf(mx, ml[k].x);
    const float mz = mx == -INFINITY ? 0.0f : mx, a = ex2(m - mz);
    l *= a;
#pragma unroll
    for (int e = 0; e < N; ++e) o[e] *= a;
#pragma unroll
    for (int k = 0; k < kParts; ++k) {
      const float f = ex2(ml[k].x - mz);
      l += ml[k].y * f;
#pragma unroll
      for (int e = 0; e < N; ++e) o[e] += v[k][e] * f;
    }
    m = mx;
  }
  uint16_t* out = p.o + static_cast<int64_t>(row) * p.o_tok + head * p.o_head;
  auto finish = [&](float mt, float lt) {   // the row's factor; its logarithm's sum by the first lane
    const bool none = mt == -INFINITY && lt == 0.0f;
    if (p.lse && lane == 0 && part == 0)
      p.lse[static_cast<int64_t>(row) * heads + head] = none ? -INFINITY : ((mt == -INFINITY ? 0.0f : mt) + log2f(lt)) * 0.6931471805599453f;
    return none ? 0.0f : 1.0f / lt;
  };
  if constexpr (W == 1) {
    const float inv = finish(m, l);
    const bool none = m == -INFINITY && l == 0.0f;
#pragma unroll
    for (int e = 0; e < N; e += 2)
      *reinterpret_cast<uint32_t*>(out + lane * N + e) = none ? 0u : pack_bf16x2_cvt(o[e] * inv, o[e + 1] * inv);
  } else {
#pragma unroll
    for (int e = 0; e < N; ++e) so[warp][lane * N + e] = o[e];
    if (lane == 0) {
      sm[warp] = m;
      sl[warp] = l;
    }
    __syncthreads();
    float mt = -INFINITY, lt = 0.0f, f[4];
#pragma unroll
    for (int k = 0; k < 4; ++k) mt = fmaxf(mt, sm[k]);
    const float mz = mt == -INFINITY ? 0.0f : mt;
#pragma unroll
    for (int k = 0; k < 4; ++k) {
      f[k] = ex2(sm[k] - mz);
      lt += sl[k] * f[k];
    }
    const float inv = finish(mt, lt);
    const bool none = mt == -INFINITY && lt == 0.0f;
    for (int d = tid; d < D; d += 128) {
      float x = 0.0f;
#pragma unroll
      for (int k = 0; k < 4; ++k) x += so[k][d] * f[k];
      out[d] = f32_to_bf16_rn(none ? 0.0f : x * inv);
    }
  }
}

// ---------------------------------------------------------------------------------
// host
// ---------------------------------------------------------------------------------
// Rows of a tile: the fewest of 8, 16, 32 (mma.sync), 128, 256 (tcgen05; two tiles' sums of D = 256 do not fit tensor
// memory) that hold a sequence's rows of one key/value head. Measured, 32 trees over 8192 keys on 32 query and 8 key/value
// heads of 128, mma.sync against tcgen05: trees of 8 (32 rows) bf16 127 and 127 us, E4M3 120 and 186; trees of 16 (64
// rows: two tiles of 32) bf16 245 and 133, E4M3 216 and 197.
int rows_per_tile(int64_t rows, int D) {
  return rows <= 8 ? 8 : rows <= 16 ? 16 : rows <= 32 ? 32 : rows <= 128 || D == 256 ? 128 : 256;
}

struct AttnLayout {
  int rows = 0, row_tiles = 0;
  size_t part_o = 0, part_ml = 0, total = 0;   // shares at 0
};
// Entries (sequences x row tiles) beyond this are refused: every CTA looks through them.
constexpr int64_t kAttnMaxEntries = 1 << 22;

bool attn_layout(const aq_kv_cache* c, const aq_draft_batch* d, int32_t q_heads, AttnLayout* out) {
  const int64_t rows = static_cast<int64_t>(d->max_q) * (q_heads / c->kv_heads);
  AttnLayout l;
  l.rows = rows_per_tile(rows, c->head_dim);
  const int64_t tiles = std::max<int64_t>((rows + l.rows - 1) / l.rows, 1);
  if (tiles * d->batch > kAttnMaxEntries) return false;
  l.row_tiles = static_cast<int>(tiles);
  const int64_t ctas = kAttnSmsBound * (l.rows >= 128 ? 1 : kAttnMaxPerSm);
  auto up = [](size_t v) { return (v + 255) / 256 * 256; };
  l.part_ml = up(tiles * d->batch * sizeof(AttnShare));
  l.part_o = up(l.part_ml + ctas * 2 * l.rows * 8);
  l.total = up(l.part_o + static_cast<size_t>(ctas) * 2 * l.rows * c->head_dim * 4);
  *out = l;
  return true;
}

template <class S>
aq_status launch_attention(AttnParams& p, const aq_kv_cache* c, const ServeDev& dev, cudaStream_t st, const char* who) {
  aq_status s;
  const int box = std::min(c->page_size, S::KS);
  if ((s = attention_cache_map(&p.tm_k, c->k, c, S::RB / S::ES, box, who)) != AQ_OK) return s;
  if ((s = attention_cache_map(&p.tm_v, c->v, c, S::RB / S::ES, box, who)) != AQ_OK) return s;
  constexpr size_t kStatic = (sizeof(AttnShared) + 127) / 128 * 128;
  constexpr size_t kUnit = S::kStage + 2 * S::kScale, kFixed = 1024 + S::kQ + S::kJoin;
  const size_t room = (dev.smem_optin + 1024) / S::kPerSm - 1024 - kStatic - kFixed;   // 1 KB a CTA is the system's
  p.stages = static_cast<int>(std::min<size_t>(room / kUnit, kAttnStages));
  if (p.stages < 2) return serve_fail(AQ_ERR_UNSUPPORTED, "%s: the device has too little shared memory", who);
  const size_t smem = kFixed + p.stages * kUnit;
  static std::atomic<uint64_t> ready{0};   // devices on which the kernel may use that much
  const uint64_t bit = 1ull << dev.index;
  if (!(ready.load() & bit)) {
    const cudaError_t e = cudaFuncSetAttribute(aq_tree_attention_kernel<S>, cudaFuncAttributeMaxDynamicSharedMemorySize, static_cast<int>(smem));
    if (e != cudaSuccess) return serve_launched(e, who);
    ready.fetch_or(bit);
  }
  p.main_grid = std::min(dev.sms, kAttnSmsBound) * S::kPerSm;
  return serve_launched(launch_serve(aq_tree_attention_kernel<S>, p, dim3(p.main_grid), S::kThreads, smem, st), who);
}

// Registers (O^T takes D NR / 4 a thread) and shared memory decide how many CTAs share an SM.
template <int D, bool E4M3>
aq_status launch_rows(AttnParams& p, const aq_kv_cache* c, const ServeDev& dev, cudaStream_t st, const char* who) {
  constexpr int per1 = D == 256 && !E4M3 ? 1 : 2, per2 = D == 256 ? 1 : 2;
  aq_status s;
  switch (p.rows_per_tile) {
    case 8: s = launch_attention<Shape<D, E4M3, 1, 1, 4, per1>>(p, c, dev, st, who); break;
    case 16: s = launch_attention<Shape<D, E4M3, 2, 1, 4, per2>>(p, c, dev, st, who); break;
    case 32: s = launch_attention<std::conditional_t<D == 256, Shape<D, E4M3, 2, 2, 8, 1>, Shape<D, E4M3, 4, 1, 8, 1>>>(p, c, dev, st, who); break;
    default: s = launch_attention_tc(p, c, dev, st, who);
  }
  if (s != AQ_OK) return s;
  const int64_t units = p.total_q * p.hk * p.group, items = static_cast<int64_t>(p.batch) * p.row_tiles * p.hk;
  if (p.main_grid <= 8 * items) return serve_launched(launch_serve(aq_attention_join_kernel<D, 1>, p, dim3(static_cast<unsigned>((units + 3) / 4)), 128, 0, st), who);
  return serve_launched(launch_serve(aq_attention_join_kernel<D, 4>, p, dim3(static_cast<unsigned>(units)), 128, 0, st), who);
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
  AttnLayout l;
  if (batch->batch == 0 || batch->total_q == 0 || batch->max_q == 0) return 0;
  if (!attn_layout(cache, batch, q_heads, &l)) {
    serve_fail(AQ_ERR_SHAPE, "aq_tree_attention_workspace_bytes: batch * max_q is too large for one call");
    return static_cast<size_t>(-1);
  }
  return l.total;
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
  AttnLayout l;
  if (!attn_layout(cache, batch, q_heads, &l) || nq * q_heads > 0x7fffffffLL)
    return serve_fail(AQ_ERR_SHAPE, "%s: batch * max_q is too large for one call", who);
  if (!workspace || workspace_bytes < l.total || !serve_aligned(workspace, 256))
    return serve_fail(AQ_ERR_WORKSPACE, "%s: workspace of %zu bytes (256-byte aligned) required, got %zu", who, l.total,
                      workspace_bytes);
  const ByteSpan ws = byte_span(workspace, 1, 0, static_cast<int64_t>(l.total), 1);
  for (const ByteSpan& x : ins)
    if (byte_overlap(ws, x)) return serve_fail(AQ_ERR_OVERLAP, "%s: workspace overlaps an input", who);
  if (byte_overlap(ws, outs[0]) || byte_overlap(ws, outs[1]))
    return serve_fail(AQ_ERR_OVERLAP, "%s: workspace overlaps an output", who);
  ServeDev dev;
  if ((st = serve_device(&dev)) != AQ_OK) return st;
  AttnParams p = {};
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
  uint8_t* base = static_cast<uint8_t*>(workspace);
  p.rows_per_tile = l.rows;
  p.by_group = FastDiv(p.group);
  p.by_tiles = FastDiv(l.row_tiles);
  p.by_heads = FastDiv(q_heads);
  p.row_tiles = l.row_tiles;
  p.shares = reinterpret_cast<AttnShare*>(base);
  p.part_ml = reinterpret_cast<float2*>(base + l.part_ml);
  p.part_o = reinterpret_cast<float*>(base + l.part_o);
  p.status = dev.status;
  p.timeout_ns = kServeTimeoutNs;
  const bool e4m3 = cache->type == AQ_KV_E4M3;
  const cudaStream_t cs = static_cast<cudaStream_t>(stream);
  if (D == 64) return e4m3 ? launch_rows<64, true>(p, cache, dev, cs, who) : launch_rows<64, false>(p, cache, dev, cs, who);
  if (D == 128) return e4m3 ? launch_rows<128, true>(p, cache, dev, cs, who) : launch_rows<128, false>(p, cache, dev, cs, who);
  return e4m3 ? launch_rows<256, true>(p, cache, dev, cs, who) : launch_rows<256, false>(p, cache, dev, cs, who);
}
