// aq_attention_tc.cu -- aq_tree_attention for many rows: S = Q K^T and O = P V on tcgen05, accumulators in tensor
// memory.
//
// From about 128 rows a key/value head (64 drafted tokens of a group of four, a chunk of a prefill) a byte of cache
// meets enough rows for the products to weigh as much as the loads, and mma.sync (607 TFLOP/s measured here) falls
// behind HBM. A CTA takes one or two tiles of 128 rows of one item against key tiles of BN: a producer warp streams
// pages with TMA, one warp issues the MMAs, and each row tile has a group of four warps, a thread to a row, that
// turns its scores into weights (no exchange between threads: the row's maximum and sum are the thread's own).
// With two row tiles the groups take turns, so that one's products run under the other's exponentials; with one,
// two score buffers let the next scores form under the weights of this tile. The weights go back to tensor memory
// over the scores they came from and enter P V from there; V is read as stored, [key][column], as the MN-major
// operand. The sums O stay in tensor memory for the item; they are scaled over only when a row's reference is
// passed by 2^kLag.
//
// E4M3 codes are widened to f16 tiles in shared memory by four warps in between (exact), once for all rows; scales
// and f16 scaling as in the mma.sync kernel.
//
// Measured, eight trees of 64 over 32768 keys, 32 query and 8 key/value heads (256 rows an item): D = 128 bf16 220 to 225 us in a
// graph, 240 a call (1150 to 1250 TFLOP/s, 4520 to 4930 GB/s), of which about 190 are the stream at 3330 clocks a pair of 128-key tiles (the products
// alone 2050), the rest starts, ends of items and the joining launch; E4M3 317 us (a scale
// on every score and every weight, beside the widening's instructions), D = 64 173, D = 256 650 (one row tile, and 64-key products that
// re-read Q). Chunks of 512 tokens of four prompts over 4096 keys: bf16 177 us (826 TFLOP/s), E4M3 283; one of 4096 from the start 528
// (260: every key of the chunk is a masked one).
#include <math.h>

#include <algorithm>
#include <atomic>
#include <type_traits>

#include "aq_attention.cuh"

namespace aq {
namespace {

constexpr int kInfo = 8;      // tiles whose scales and page masks are kept
constexpr int kMaxRing = 8;   // most tile buffers
constexpr int kGroup = 128;   // threads (rows) of a row tile

template <int D_, bool E4M3_, int TILES_>
struct TcShape {
  static constexpr int D = D_, TILES = TILES_;
  static constexpr bool E4M3 = E4M3_;
  static constexpr int M = 128 * TILES;
  static constexpr int BN = D == 256 ? 64 : 128;           // keys of a tile
  static constexpr int kTile = BN * D * 2;                 // bytes of a 16-bit K or V tile
  static constexpr int kQ = M * D * 2;
  static constexpr int CB = D < 128 ? D : 128;             // bytes of a row of one column block of codes
  static constexpr int kCode = BN * D;                     // bytes of a tile of codes
  static constexpr int kScale = E4M3 ? kInfo * 2 * BN * 4 : 0;
  static constexpr int kSoftWarps = 4 * TILES;
  static constexpr int kConvWarp = kSoftWarps;             // first of four converting warps (E4M3)
  static constexpr int kTmaWarp = kSoftWarps + (E4M3 ? 4 : 0), kMmaWarp = kTmaWarp + 1;
  // Two row tiles of an E4M3 cache: 16 warps launched with 128 registers a thread, of which the weighing warps take a
  // part from the others (256 x 176 + 128 x 88 + 128 x 72 = 65536 = 512 x 128): 307 to 313 us against 342 without, then.
  static constexpr bool kSplitRegs = E4M3 && TILES == 2;
  static constexpr int kThreads = kSplitRegs ? 512 : (kMmaWarp + 1) * 32;
  // tensor memory: two score buffers, one a row tile or two of one tile (the weights over them), then the sums
  static constexpr int kS(int x) { return x * 128; }
  static constexpr int kO(int t) { return 256 + t * D; }
  static_assert(256 + TILES * D <= 512, "tensor memory");
  // f16 buffers of an E4M3 cache: a fourth lets the next keys be widened under this tile's sums
  static constexpr int NF = !E4M3 ? 0 : kQ + 4 * kTile + 3 * kCode + kScale <= 224 * 1024 ? 4 : 3;
};

struct TcShared {
  uint64_t full[kMaxRing], empty[kMaxRing];     // 16-bit tiles: K of tile n is buffer use 2 n, V use 2 n + 1
  uint64_t cfull[kMaxRing], cempty[kMaxRing];   // codes
  uint64_t info[kInfo];                         // page mask and scales of a tile
  uint64_t q_ready, s_full[2], p_ready[2], o_done[2], item_done, together[2], drain;   // item_done: with one row tile
  uint32_t valid[kInfo];
  int32_t skip[2];                              // the product P V of this score buffer is done by the threads
  int32_t special[2][2];                        // [row tile][tile & 1]
  uint32_t tmem;
  int32_t abort;
  int64_t top[2][4];
  float fac[256];
  AttnWork work;
};

__device__ __forceinline__ void tmem_ld32(uint32_t addr, float (&v)[32]) {
  // one statement: the values exist only past the wait
  asm volatile(
      "tcgen05.ld.sync.aligned.32x32b.x32.b32 "
      "{%0, %1, %2, %3, %4, %5, %6, %7, %8, %9, %10, %11, %12, %13, %14, %15, "
      "%16, %17, %18, %19, %20, %21, %22, %23, %24, %25, %26, %27, %28, %29, %30, %31}, [%32];\n\t"
      "tcgen05.wait::ld.sync.aligned;"
      : "=f"(v[0]), "=f"(v[1]), "=f"(v[2]), "=f"(v[3]), "=f"(v[4]), "=f"(v[5]), "=f"(v[6]), "=f"(v[7]), "=f"(v[8]), "=f"(v[9]),
        "=f"(v[10]), "=f"(v[11]), "=f"(v[12]), "=f"(v[13]), "=f"(v[14]), "=f"(v[15]), "=f"(v[16]), "=f"(v[17]), "=f"(v[18]),
        "=f"(v[19]), "=f"(v[20]), "=f"(v[21]), "=f"(v[22]), "=f"(v[23]), "=f"(v[24]), "=f"(v[25]), "=f"(v[26]), "=f"(v[27]),
        "=f"(v[28]), "=f"(v[29]), "=f"(v[30]), "=f"(v[31])
      : "r"(addr)
      : "memory");
}
// The same in two halves, for loads under other work: the values may be used past tmem_ld32_wait alone.
__device__ __forceinline__ void tmem_ld32_issue(uint32_t addr, float (&v)[32]) {
  asm volatile(
      "tcgen05.ld.sync.aligned.32x32b.x32.b32 "
      "{%0, %1, %2, %3, %4, %5, %6, %7, %8, %9, %10, %11, %12, %13, %14, %15, "
      "%16, %17, %18, %19, %20, %21, %22, %23, %24, %25, %26, %27, %28, %29, %30, %31}, [%32];"
      : "=f"(v[0]), "=f"(v[1]), "=f"(v[2]), "=f"(v[3]), "=f"(v[4]), "=f"(v[5]), "=f"(v[6]), "=f"(v[7]), "=f"(v[8]), "=f"(v[9]),
        "=f"(v[10]), "=f"(v[11]), "=f"(v[12]), "=f"(v[13]), "=f"(v[14]), "=f"(v[15]), "=f"(v[16]), "=f"(v[17]), "=f"(v[18]),
        "=f"(v[19]), "=f"(v[20]), "=f"(v[21]), "=f"(v[22]), "=f"(v[23]), "=f"(v[24]), "=f"(v[25]), "=f"(v[26]), "=f"(v[27]),
        "=f"(v[28]), "=f"(v[29]), "=f"(v[30]), "=f"(v[31])
      : "r"(addr)
      : "memory");
}
__device__ __forceinline__ void tmem_ld32_wait(float (&v)[32]) {
  asm volatile("tcgen05.wait::ld.sync.aligned;" ::: "memory");
#pragma unroll
  for (int i = 0; i < 32; i += 8)   // the values pass through here, so no use of them moves before the wait
    asm volatile("" : "+f"(v[i]), "+f"(v[i + 1]), "+f"(v[i + 2]), "+f"(v[i + 3]), "+f"(v[i + 4]), "+f"(v[i + 5]), "+f"(v[i + 6]), "+f"(v[i + 7])::"memory");
}
__device__ __forceinline__ void tmem_ld16u(uint32_t addr, uint32_t (&v)[16]) {
  asm volatile(
      "tcgen05.ld.sync.aligned.32x32b.x16.b32 "
      "{%0, %1, %2, %3, %4, %5, %6, %7, %8, %9, %10, %11, %12, %13, %14, %15}, [%16];\n\t"
      "tcgen05.wait::ld.sync.aligned;"
      : "=r"(v[0]), "=r"(v[1]), "=r"(v[2]), "=r"(v[3]), "=r"(v[4]), "=r"(v[5]), "=r"(v[6]), "=r"(v[7]), "=r"(v[8]), "=r"(v[9]),
        "=r"(v[10]), "=r"(v[11]), "=r"(v[12]), "=r"(v[13]), "=r"(v[14]), "=r"(v[15])
      : "r"(addr)
      : "memory");
}
__device__ __forceinline__ void tmem_st32(uint32_t addr, const float (&v)[32]) {
  asm volatile(
      "tcgen05.st.sync.aligned.32x32b.x32.b32 [%0], "
      "{%1, %2, %3, %4, %5, %6, %7, %8, %9, %10, %11, %12, %13, %14, %15, %16, "
      "%17, %18, %19, %20, %21, %22, %23, %24, %25, %26, %27, %28, %29, %30, %31, %32};" ::"r"(addr),
      "f"(v[0]), "f"(v[1]), "f"(v[2]), "f"(v[3]), "f"(v[4]), "f"(v[5]), "f"(v[6]), "f"(v[7]), "f"(v[8]), "f"(v[9]), "f"(v[10]),
      "f"(v[11]), "f"(v[12]), "f"(v[13]), "f"(v[14]), "f"(v[15]), "f"(v[16]), "f"(v[17]), "f"(v[18]), "f"(v[19]), "f"(v[20]),
      "f"(v[21]), "f"(v[22]), "f"(v[23]), "f"(v[24]), "f"(v[25]), "f"(v[26]), "f"(v[27]), "f"(v[28]), "f"(v[29]), "f"(v[30]),
      "f"(v[31])
      : "memory");
}
__device__ __forceinline__ void tmem_st16u(uint32_t addr, const uint32_t (&v)[16]) {
  asm volatile(
      "tcgen05.st.sync.aligned.32x32b.x16.b32 [%0], "
      "{%1, %2, %3, %4, %5, %6, %7, %8, %9, %10, %11, %12, %13, %14, %15, %16};" ::"r"(addr),
      "r"(v[0]), "r"(v[1]), "r"(v[2]), "r"(v[3]), "r"(v[4]), "r"(v[5]), "r"(v[6]), "r"(v[7]), "r"(v[8]), "r"(v[9]), "r"(v[10]),
      "r"(v[11]), "r"(v[12]), "r"(v[13]), "r"(v[14]), "r"(v[15])
      : "memory");
}
// (s0, s1) += (a, b), each rounded as a single addition.
__device__ __forceinline__ void fadd2(float& s0, float& s1, float a, float b) {
  asm("{\n .reg .b64 x, y;\n mov.b64 x, {%0, %1};\n mov.b64 y, {%2, %3};\n add.rn.f32x2 x, x, y;\n mov.b64 {%0, %1}, x;\n}"
      : "+f"(s0), "+f"(s1)
      : "f"(a), "f"(b));
}
// One lane of a converged warp. The MMA warp runs its loops and waits as a whole, so that what it computes stays
// uniform, and one lane issues.
__device__ __forceinline__ bool elect_one() {
  uint32_t is;
  asm volatile("{\n\t.reg .pred p;\n\telect.sync _|p, 0xffffffff;\n\tselp.u32 %0, 1, 0, p;\n\t}" : "=r"(is));
  return is != 0;
}
// D (+)= A B^T with A from tensor memory (rows the lanes, two 16-bit elements a column), B from shared memory.
__device__ __forceinline__ void tc_mma_ts(uint32_t d, uint32_t a, uint64_t b_desc, uint32_t idesc, uint32_t accumulate) {
  asm volatile(
      "{\n\t.reg .pred p;\n\t"
      "setp.ne.b32 p, %4, 0;\n\t"
      "tcgen05.mma.cta_group::1.kind::f16 [%0], [%1], %2, %3, p;\n\t}" ::"r"(d),
      "r"(a), "l"(b_desc), "r"(idesc), "r"(accumulate)
      : "memory");
}
// MN-major operand with 128-byte swizzle: 64 elements of the M/N dimension to a 128-byte row, rows along K, eight
// rows (1024 bytes) repeating along K, blocks of 64 elements `block` bytes apart.
__device__ __forceinline__ uint64_t smem_desc_mn128(uint32_t addr, uint32_t block) {
  uint64_t d = 0;
  d |= static_cast<uint64_t>((addr & 0x3FFFFu) >> 4);
  d |= static_cast<uint64_t>(block >> 4) << 16;      // leading byte offset: next block of 64 elements
  d |= static_cast<uint64_t>(1024 >> 4) << 32;       // stride byte offset: next eight rows along K
  d |= static_cast<uint64_t>(1) << 46;
  d |= static_cast<uint64_t>(2) << 61;
  return d;
}
// kind::f16, f16 or bf16 operands, fp32 sums; b_mn: B is MN-major.
constexpr uint32_t tc_idesc(bool f16, bool b_mn, int n) {
  return (1u << 4) | ((f16 ? 0u : 1u) << 7) | ((f16 ? 0u : 1u) << 10) | ((b_mn ? 1u : 0u) << 16) | (static_cast<uint32_t>(n >> 3) << 17) |
         (static_cast<uint32_t>(128 >> 4) << 24);
}

// Byte offset of 16 bytes (eight elements from 8 c on) of a row of a 16-bit tile: column blocks of 64 elements, each
// `rows` rows of 128 swizzled bytes.
__host__ __device__ constexpr uint32_t tile_offset(int rows, int row, int c) {
  return (c >> 3) * rows * 128 + row * 128 + (((c & 7) ^ (row & 7)) << 4);
}
__device__ __forceinline__ uint32_t tile_addr(uint32_t base, int rows, int row, int c) { return base + tile_offset(rows, row, c); }
// Where the epilogue keeps 16 bytes (k of eight) of a row's sums on their way out: in the first column block of that row's
// query, for any D. Nothing stands between one warp's epilogue and another's next queries, so a warp writes to its own rows alone.
__host__ __device__ constexpr uint32_t stage_offset(int row, int k) { return tile_offset(128, row, k); }
constexpr bool stages_in_own_rows() {
  for (int row = 0; row < 128; ++row) {
    for (int c = 0; c < 256 / 8; ++c)
      if (((tile_offset(128, row, c) >> 7) & 127) != static_cast<uint32_t>(row)) return false;   // a query's bytes by their row
    for (int k = 0; k < 8; ++k)
      if (((stage_offset(row, k) >> 7) & 127) != static_cast<uint32_t>(row)) return false;
  }
  return true;
}
static_assert(stages_in_own_rows(), "the epilogue of one warp would meet another warp's queries");

// Whether the phase with the given parity is complete, without waiting.
__device__ __forceinline__ bool mbar_test(uint64_t* bar, uint32_t parity) {
  uint32_t done;
  asm volatile(
      "{\n\t.reg .pred p;\n\t"
      "mbarrier.test_wait.parity.shared::cta.b64 p, [%1], %2;\n\t"
      "selp.u32 %0, 1, 0, p;\n\t}"
      : "=r"(done)
      : "r"(smem_u32(bar)), "r"(parity)
      : "memory");
  return done != 0;
}
// A position in a ring of `n` buffers: index, and the parity of the phase its use completes.
struct Ring {
  int n, i = 0;
  uint32_t phase = 0;
  __device__ __forceinline__ explicit Ring(int size) : n(size) {}
  __device__ __forceinline__ void next() {
    if (++i == n) {
      i = 0;
      phase ^= 1;
    }
  }
};

// ---------------------------------------------------------------------------------
// producer
// ---------------------------------------------------------------------------------
template <class S>
__device__ __forceinline__ void tc_produce(const AttnParams& p, TcShared& sh, uint8_t* ring, uint8_t* scales, int nring,
                                           const int64_t (&range)[2], const AbortCtl& ctl) {
  constexpr int ES = S::E4M3 ? 1 : 2;
  constexpr int kBytes = S::BN * S::D * ES;
  constexpr int RB = S::E4M3 ? S::CB : 128, NC = S::D * ES / RB;
  uint64_t* full = S::E4M3 ? sh.cfull : sh.full;
  uint64_t* empty = S::E4M3 ? sh.cempty : sh.empty;
  const int lane = threadIdx.x & 31;
  const int page = 1 << p.page_shift;
  const int box = min(page, S::BN), np = S::BN / box;
  int uses = 0, tile = 0;
  Ring at(nring);
  Walk<S::M, S::BN> w(p, sh.work, range);
  bool ok = true;
  while (ok && w.left > 0) {
    const int32_t* table = p.table + w.b * p.ld_table;
    auto page_id = [&](int64_t i) {   // -1: left out
      if (i >= p.pages_per_seq || (i << p.page_shift) >= w.s.hi || ((i + 1) << p.page_shift) <= w.s.lo) return -1;
      const int id = table[i];
      return id >= 0 && id < p.pages ? id : -1;
    };
    int64_t base = (static_cast<int64_t>(w.tile0) * S::BN) >> p.page_shift;   // page numbers, 32 at a time and 32 ahead
    int cur = page_id(base + lane), ahead = page_id(base + 32 + lane);
    for (int i = 0; ok && i < w.n; ++i, ++tile) {
      const int64_t key = static_cast<int64_t>(w.tile0 + i) * S::BN;
      const int64_t first = key >> p.page_shift;
      if (first >= base + 32) {
        base += 32;
        cur = ahead;
        ahead = page_id(base + 32 + lane);
      }
      const int id = __shfl_sync(0xffffffffu, cur, static_cast<int>(first - base) + (lane < np ? lane : 0));
      const bool valid = lane < np && id >= 0 && key + static_cast<int64_t>(lane) * box < w.s.hi;
      const uint32_t mask = __ballot_sync(0xffffffffu, valid);
      const int off = static_cast<int>(key & (page - 1));
      const int row = id * p.hk + w.head;
#pragma unroll 1
      for (int kv = 0; kv < 2; ++kv) {
        ok = __all_sync(0xffffffffu, mbar_wait(&empty[at.i], at.phase ^ 1, ctl));
        if (!ok) break;
        const int slot = tile % kInfo;
        if (lane == 0) {
          if (kv == 0) {
            sh.valid[slot] = mask;
            mbar_arrive_expect_tx(&sh.info[slot], S::E4M3 ? __popc(mask) * box * 8 : 0);
          }
          mbar_arrive_expect_tx(&full[at.i], __popc(mask) * box * S::D * ES);
        }
        __syncwarp();
        if (valid) {
          uint8_t* dst = ring + at.i * kBytes + lane * box * RB;
#pragma unroll
          for (int c = 0; c < NC; ++c)
            tma_load_3d(dst + c * S::BN * RB, kv ? &p.tm_v : &p.tm_k, c * (RB / ES), off, row, &full[at.i]);
          if (S::E4M3 && kv == 0) {
            const int64_t cell = (static_cast<int64_t>(row) << p.page_shift) + off;
            uint8_t* sd = scales + slot * 2 * S::BN * 4 + lane * box * 4;
            bulk_load(sd, p.ks + cell, box * 4, &sh.info[slot]);
            bulk_load(sd + S::BN * 4, p.vs + cell, box * 4, &sh.info[slot]);
          }
        }
        ++uses;
        at.next();
      }
    }
    if (ok) w.next(p);
  }
  if (!ok) {   // a wait ran out: let the copies already issued land before the CTA may end
    for (int i = 0; i < min(uses, nring); ++i) {
      const int u = uses - 1 - i;
      const uint64_t t0 = global_timer_ns();
      while (!mbar_try_wait(&full[u % nring], (u / nring) & 1))
        if (global_timer_ns() - t0 > ctl.timeout_ns) break;
    }
    if (S::E4M3)
      for (int i = 0; i < min(tile + 1, kInfo); ++i) {
        const int u = tile - i;
        const uint64_t t0 = global_timer_ns();
        while (u >= 0 && 2 * u < uses && !mbar_try_wait(&sh.info[u % kInfo], (u / kInfo) & 1))
          if (global_timer_ns() - t0 > ctl.timeout_ns) break;
      }
  }
}

// ---------------------------------------------------------------------------------
// converting warps (E4M3): a tile of codes to a tile of halves
// ---------------------------------------------------------------------------------
template <class S>
__device__ __forceinline__ void tc_convert(TcShared& sh, const uint8_t* codes, const uint8_t* tiles, int ncode, int64_t count,
                                           const AbortCtl& ctl) {
  constexpr int XC = S::D / 16;                // 16-byte chunks of a key's codes
  constexpr int NF = S::E4M3 ? S::NF : 1;
  const int tid = threadIdx.x - S::kConvWarp * 32, lane = tid & 31;
  Ring from(ncode), to(NF);
  for (int64_t u = 0; u < 2 * count; ++u, from.next(), to.next()) {
    if (!__all_sync(0xffffffffu, mbar_wait(&sh.cfull[from.i], from.phase, ctl))) return;
    if (!__all_sync(0xffffffffu, mbar_wait(&sh.empty[to.i], to.phase ^ 1, ctl))) return;
    const uint32_t src = smem_u32(codes + from.i * S::kCode), dst = smem_u32(tiles + to.i * S::kTile);
    constexpr int kRounds = S::BN * XC / 128, kBatch = kRounds < 4 ? kRounds : 4, XB = S::CB / 16;
#pragma unroll 1
    for (int k = 0; k < kRounds; k += kBatch) {
      uint32_t q[kBatch][4];
#pragma unroll
      for (int j = 0; j < kBatch; ++j) {
        const int i = (k + j) * 128 + tid, key = i / XC, x = i % XC;
        const uint32_t at = src + (x / XB) * S::BN * S::CB + key * S::CB + (((x % XB) ^ (S::CB == 128 ? key & 7 : (key >> 1) & 3)) << 4);
        asm volatile("ld.shared.v4.u32 {%0, %1, %2, %3}, [%4];" : "=r"(q[j][0]), "=r"(q[j][1]), "=r"(q[j][2]), "=r"(q[j][3]) : "r"(at) : "memory");
      }
#pragma unroll
      for (int j = 0; j < kBatch; ++j) {
        const int i = (k + j) * 128 + tid, key = i / XC, x = i % XC;
        uint32_t h[8];
#pragma unroll
        for (int e = 0; e < 4; ++e) widen(q[j][e], h[2 * e], h[2 * e + 1]);
        // eight neighbouring lanes store to eight different 16-byte columns: every second four begin with the upper half
        const int swap = XC > 4 ? (x >> 2) & 1 : 0;
#pragma unroll
        for (int e = 0; e < 2; ++e) {
          const bool up = (e ^ swap) != 0;
          asm volatile("st.shared.v4.u32 [%0], {%1, %2, %3, %4};" ::"r"(tile_addr(dst, S::BN, key, 2 * x + (up ? 1 : 0))), "r"(up ? h[4] : h[0]),
                       "r"(up ? h[5] : h[1]), "r"(up ? h[6] : h[2]), "r"(up ? h[7] : h[3])
                       : "memory");
        }
      }
    }
    fence_proxy_async_smem();
    __syncwarp();
    if (lane == 0) {
      mbar_arrive(&sh.full[to.i]);
      mbar_arrive(&sh.cempty[from.i]);
    }
  }
}

// ---------------------------------------------------------------------------------
// MMA issue, one warp
// ---------------------------------------------------------------------------------
// The tensor pipe holds about one product more than it runs, and a wait costs this warp some 100 clocks even where its
// phase is long complete (78 on an idle SM): with two row tiles, waits between the bursts of eight products left the pipe
// idle for 1200 of 3830 clocks a pair of tiles (D = 128). So what the next burst waits for is looked at before the
// last products of this one, and waited for only where it was not there yet.
template <class S>
__device__ __forceinline__ bool tc_issue(const AttnParams& p, TcShared& sh, const uint8_t* qbuf, const uint8_t* tiles, int nring,
                                         uint32_t tmem, const int64_t (&range)[2], const AbortCtl& ctl) {
  constexpr uint32_t kIdS = tc_idesc(S::E4M3, false, S::BN), kIdO = tc_idesc(S::E4M3, true, S::D);
  constexpr int kScores = S::D / 16, kSums = S::BN / 16, kLast = kScores > 4 ? 3 : 2;   // products; those behind a look ahead
  Walk<S::M, S::BN> w(p, sh.work, range);
  uint32_t tile = 0, seg = 0;          // so far, of all segments
  // buffers in order of use: K 0, V 0, K 1, V 1, ...; this tile's V, and the K whose scores come next
  Ring k_at(nring), v_at(nring);
  v_at.next();
  bool k_here = false, v_here = false, p_here = false;   // seen: the next scores' K, this tile's V, the next sums' weights
  bool skip = false;                                     // with p_here: those sums are done by the threads
  const uint64_t q0 = smem_desc_k128(smem_u32(qbuf)), k0 = smem_desc_k128(smem_u32(tiles)), v0 = smem_desc_mn128(smem_u32(tiles), S::BN * 128);
  auto wait = [&](uint64_t* bar, uint32_t parity) { return __all_sync(0xffffffffu, mbar_wait(bar, parity, ctl)); };
  auto need = [&](bool& here, uint64_t* bar, uint32_t parity) {
    if (!here) here = wait(bar, parity);
    return here;
  };
  // t: row tile; x: score buffer
  auto scores = [&](auto tc, int x, uint32_t n, bool look) {
    constexpr int t = decltype(tc)::value;
    const uint64_t k = k0 + k_at.i * (S::kTile >> 4);
    const uint32_t d = tmem + S::kS(x);
    auto product = [&](int i) {   // descriptor addresses count 16 bytes
      tc_mma_bf16(d, q0 + ((t * 128 * S::D * 2 + (i >> 2) * 128 * 128 + (i & 3) * 32) >> 4), k + (((i >> 2) * S::BN * 128 + (i & 3) * 32) >> 4), kIdS, i > 0);
    };
    uint64_t* const k_empty = &sh.empty[k_at.i];
    if (t == S::TILES - 1) {
      k_at.next();
      k_at.next();
      k_here = false;
    }
    if (S::TILES == 2) {
      if (elect_one()) {
#pragma unroll
        for (int i = 0; i < kScores - kLast; ++i) product(i);
      }
      __syncwarp();
      if (look) {
        bool vn = true, kn = true;
        const bool pn = mbar_test(&sh.p_ready[1 - t], (t == 0 ? n - 1 : n) & 1);   // the other row tile's weights
        if (t == 1) {
          vn = mbar_test(&sh.full[v_at.i], v_at.phase);
          kn = mbar_test(&sh.full[k_at.i], k_at.phase);
        }
        const bool sn = *reinterpret_cast<volatile int32_t*>(&sh.skip[1 - t]) != 0;
        const uint32_t all = __reduce_and_sync(0xffffffffu, (pn ? 1u : 0u) | (vn ? 2u : 0u) | (kn ? 4u : 0u) | (sn ? 8u : 0u));
        p_here = (all & 1) != 0;
        skip = (all & 8) != 0;
        if (t == 1) {
          v_here = (all & 2) != 0;
          k_here = (all & 4) != 0;
        }
      }
    }
    if (elect_one()) {
#pragma unroll
      for (int i = S::TILES == 2 ? kScores - kLast : 0; i < kScores; ++i) product(i);
      tc_commit(&sh.s_full[x]);
      if (t == S::TILES - 1) tc_commit(k_empty);
    }
    __syncwarp();
  };
  auto sums = [&](auto tc, int x, bool first) {
    constexpr int t = decltype(tc)::value;
    const uint64_t v = v0 + v_at.i * (S::kTile >> 4);
    const uint32_t a = tmem + S::kS(x);
    if (elect_one()) {
      if (!skip) {
#pragma unroll
        for (int i = 0; i < kSums; ++i) tc_mma_ts(tmem + S::kO(t), a + 8 * i, v + ((i * 2048) >> 4), kIdO, !(first && i == 0));
      }
      tc_commit(&sh.o_done[t]);
      if (t == S::TILES - 1) tc_commit(&sh.empty[v_at.i]);
    }
    __syncwarp();
    p_here = false;
    if (t == S::TILES - 1) {
      v_at.next();
      v_at.next();
      v_here = false;
    }
  };
  constexpr std::integral_constant<int, 0> kFirst{};
  constexpr std::integral_constant<int, S::TILES - 1> kSecond{};
  // the weights in score buffer x, their sums, and with `more` the scores of the next tile
  auto turn = [&](auto tc, int x, uint32_t parity, bool first) {
    if (!p_here) {
      if (!need(p_here, &sh.p_ready[x], parity)) return false;
      skip = __any_sync(0xffffffffu, *reinterpret_cast<volatile int32_t*>(&sh.skip[x]) != 0);
    }
    if (!need(v_here, &sh.full[v_at.i], v_at.phase)) return false;
    tc_fence_after();
    sums(tc, x, first);
    return true;
  };
  auto next_keys = [&]() {
    const bool ok = need(k_here, &sh.full[k_at.i], k_at.phase);
    tc_fence_after();
    return ok;
  };
  for (;; w.next(p), ++seg) {
    const int len = __shfl_sync(0xffffffffu, w.left > 0 ? w.n : 0, 0);   // the same in every lane, and known to be
    if (len == 0) return true;
    if (!wait(&sh.q_ready, seg & 1) || !next_keys()) return false;
    scores(kFirst, S::TILES == 2 ? 0 : tile & 1, tile, false);
    if (S::TILES == 2) scores(kSecond, 1, tile, false);
    for (int i = 0; i < len; ++i, ++tile) {
      const bool more = i + 1 < len;
      if (S::TILES == 2) {
        if (!turn(kFirst, 0, tile & 1, i == 0)) return false;
        if (more) {
          if (!next_keys()) return false;
          scores(kFirst, 0, tile + 1, true);
        }
        if (!turn(kSecond, 1, tile & 1, i == 0)) return false;
        if (more) scores(kSecond, 1, tile + 1, i + 2 < len);
      } else {
        if (more) {
          if (!next_keys()) return false;
          scores(kFirst, (tile + 1) & 1, tile + 1, false);
        }
        if (!turn(kFirst, tile & 1, (tile >> 1) & 1, i == 0)) return false;
      }
    }
    if (S::TILES == 1) {
      if (elect_one()) tc_commit(&sh.item_done);
      __syncwarp();
    }
  }
}

// ---------------------------------------------------------------------------------
// weights: a thread to a row
// ---------------------------------------------------------------------------------
// P V of one tile by the threads: taken where V holds infinities or NaN that some row does not see (0 times them would
// reach every row). The weights are read back from tensor memory, masked keys by their bits.
template <class S>
__device__ __noinline__ void sums_by_hand(const AttnParams& p, const KeySpan& s, int i, int64_t pos, int64_t key0, uint32_t pages,
                                          int box_shift, uint32_t p_addr, uint32_t o_addr, uint32_t v, bool first) {
#pragma unroll 1
  for (int d0 = 0; d0 < S::D; d0 += 32) {
    float o[32];
    tmem_ld32(o_addr + d0, o);
    if (first)
      for (int d = 0; d < 32; ++d) o[d] = 0.0f;
#pragma unroll 1
    for (int c = 0; c < S::BN / 32; ++c) {
      const uint32_t bits = seen_bits(p, s, i, pos, key0 + 32 * c, 32 * c, 32, pages, box_shift);
      uint32_t w[16];
      tmem_ld16u(p_addr + 16 * c, w);
#pragma unroll
      for (int k = 0; k < 32; ++k) {
        const uint16_t half = static_cast<uint16_t>(k & 1 ? w[k / 2] >> 16 : w[k / 2]);
        const float wk = S::E4M3 ? __half2float(__ushort_as_half(half)) : bf16_to_f32(half);
        if ((bits >> k) & 1) {
#pragma unroll
          for (int q = 0; q < 4; ++q) {
            uint32_t r[4];
            asm volatile("ld.shared.v4.u32 {%0, %1, %2, %3}, [%4];"
                         : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3])
                         : "r"(tile_addr(v, S::BN, 32 * c + k, d0 / 8 + q))
                         : "memory");
#pragma unroll
            for (int e = 0; e < 4; ++e) {
              float lo, hi;
              if (S::E4M3) {
                const float2 f = __half22float2(*reinterpret_cast<const __half2*>(&r[e]));
                lo = f.x;
                hi = f.y;
              } else {
                lo = __uint_as_float(r[e] << 16);
                hi = __uint_as_float(r[e] & 0xffff0000u);
              }
              o[8 * q + 2 * e] = fmaf(wk, lo, o[8 * q + 2 * e]);
              o[8 * q + 2 * e + 1] = fmaf(wk, hi, o[8 * q + 2 * e + 1]);
            }
          }
        }
      }
    }
    tmem_st32(o_addr + d0, o);
  }
  tmem_st_wait();
}

template <class S>
__device__ __forceinline__ void tc_weigh(const AttnParams& p, TcShared& sh, uint8_t* qbuf, const uint8_t* tiles, const uint8_t* scales,
                                         int nring, uint32_t tmem, const int64_t (&range)[2], const AbortCtl& ctl) {
  constexpr int D = S::D, BN = S::BN;
  const int tid = threadIdx.x, lane = tid & 31, t = tid / kGroup, r = tid % kGroup, wq = r >> 5;
  const uint32_t lanes = static_cast<uint32_t>(wq * 32) << 16;   // this warp's quarter of the tensor memory lanes
  const int box_shift = min(p.page_shift, 31 - __clz(BN));
  const uint32_t all_pages = BN >> box_shift >= 32 ? 0xffffffffu : (1u << (BN >> box_shift)) - 1;
  const float scale2 = p.scale * 1.4426950408889634f;
  const uint32_t sign = scale2 < 0.0f ? 0x80008000u : 0u;
  const uint32_t group = p.group;
  uint32_t tile = 0, item = 0, together = 0;     // tiles and items so far; uses of the group's own barrier
  Ring v_at(nring);                    // this tile's V
  bool ok = true;
  v_at.next();
  auto wait = [&](uint64_t* bar, uint32_t parity) {
    ok = ok && mbar_wait(bar, parity, ctl);
    ok = __all_sync(0xffffffffu, ok);
    return ok;
  };
  auto meet = [&]() {        // the group's 128 threads
    __syncwarp();
    if (lane == 0) mbar_arrive(&sh.together[t]);
    return wait(&sh.together[t], together++ & 1);
  };
  Walk<S::M, BN> w(p, sh.work, range);
  for (; w.left > 0; w.next(p), ++item) {
    const int rt = w.rt;
    // Lane l of warp wq holds row 4 l + wq of the tile: a tile that is not full is spread over all four warps.
    const uint32_t rows = static_cast<uint32_t>(w.s.T) * group, row0 = static_cast<uint32_t>(rt) * S::M + t * 128 + wq;
    const uint32_t row = row0 + 4 * lane;
    const int count = rows > row0 ? min((rows - row0 + 3) / 4, 32u) : 0;   // rows of the warp
    const bool live_warp = count > 0;
    const int i_row = row < rows ? p.by_group.quot(row) : 0;
    const int depth = p.mask && p.depth ? max(p.depth[w.s.first + i_row], 0) : i_row;   // used behind the queries' loads
    // queries of the warp's rows, as the MMA reads them; what lies in lanes without a row reaches no other
    constexpr int L = D / 8, RPW = 32 / L;       // lanes a row, rows at once
    const int c = lane % L;
    auto query = [&](uint32_t rr) {
      const uint32_t i = p.by_group.quot(rr);
      return p.q + (static_cast<int64_t>(w.s.first) + i) * p.q_tok + (w.head * group + (rr - i * group)) * p.q_head + c * 8;
    };
    constexpr int kBatch = 32 / RPW < 16 ? 32 / RPW : 16;   // loads in flight
#pragma unroll 1
    for (int k0 = 0; k0 * RPW < count; k0 += kBatch) {
      uint4 v[kBatch];
#pragma unroll
      for (int k = 0; k < kBatch; ++k)   // rows past the last load the last: a load under a condition would be waited for at once
        v[k] = *reinterpret_cast<const uint4*>(query(min(row0 + 4 * ((k0 + k) * RPW + lane / L), rows - 1)));
      uint32_t top_bits[kBatch];
      if constexpr (S::E4M3) {
#pragma unroll
        for (int k = 0; k < kBatch; ++k) {
          const uint32_t m16 = 0x7fff0000u;
          top_bits[k] = max(max(max((v[k].x << 16) & m16, v[k].x & m16), max((v[k].y << 16) & m16, v[k].y & m16)),
                            max(max((v[k].z << 16) & m16, v[k].z & m16), max((v[k].w << 16) & m16, v[k].w & m16)));
        }
        if constexpr (L == 32) {
#pragma unroll
          for (int k = 0; k < kBatch; ++k) top_bits[k] = __reduce_max_sync(0xffffffffu, top_bits[k]);
        } else {
#pragma unroll
          for (int off = L / 2; off > 0; off >>= 1)
#pragma unroll
            for (int k = 0; k < kBatch; ++k) top_bits[k] = max(top_bits[k], __shfl_xor_sync(0xffffffffu, top_bits[k], off));
        }
      }
#pragma unroll
      for (int k = 0; k < kBatch; ++k) {
        const int lr = wq * 32 + (k0 + k) * RPW + lane / L;   // lane of the tensor memory
        uint32_t x[4] = {v[k].x ^ sign, v[k].y ^ sign, v[k].z ^ sign, v[k].w ^ sign};
        if constexpr (S::E4M3) {
          const bool finite = top_bits[k] < 0x7f800000u;
          const int e = finite ? top_exponent(__uint_as_float(top_bits[k])) : 0;
          const float f = pow2(14 - e);
#pragma unroll
          for (int y = 0; y < 4; ++y) {
            float lo, hi;
            fmul2_rn(lo, hi, __uint_as_float(x[y] << 16), __uint_as_float(x[y] & 0xffff0000u), f, f);
            x[y] = finite ? pack_f16x2(lo, hi) : 0u;
          }
          if (c == 0) sh.fac[t * 128 + lr] = finite ? pow2(e - 14) * fabsf(scale2) : __uint_as_float(0x7fc00000u);   // NaN: no finite score
        }
        asm volatile("st.shared.v4.u32 [%0], {%1, %2, %3, %4};" ::"r"(tile_addr(smem_u32(qbuf) + t * 128 * D * 2, 128, lr, c)), "r"(x[0]),
                     "r"(x[1]), "r"(x[2]), "r"(x[3])
                     : "memory");
      }
    }
    const int64_t pos = static_cast<int64_t>(w.s.ctx) + depth;
    int64_t top = pos;
#pragma unroll
    for (int off = 16; off > 0; off >>= 1) top = max(top, __shfl_xor_sync(0xffffffffu, top, off));
    if (lane == 0) sh.top[t][wq] = top;
    fence_proxy_async_smem();
    tc_fence_before();       // the last item's sums have been read
    __syncwarp();
    if (lane == 0) mbar_arrive(&sh.q_ready);
    if (!meet()) return;
    const float fac = S::E4M3 ? sh.fac[t * 128 + r] : fabsf(scale2);
#pragma unroll
    for (int k = 0; k < 4; ++k) top = max(top, sh.top[t][k]);
    // keys [whole0, whole1) are seen by every row of the tile
    const int64_t whole1 = min(static_cast<int64_t>(w.s.ctx), w.s.hi), whole0 = p.window > 0 ? top - p.window + 1 : 0;

    float m = -INFINITY, l = 0.0f;
    for (int it = 0; it < w.n; ++it, ++tile, v_at.next(), v_at.next()) {
      const int x = S::TILES == 2 ? t : static_cast<int>(tile & 1);
      const uint32_t x_parity = S::TILES == 2 ? tile & 1 : (tile >> 1) & 1;
      const int slot = tile % kInfo;
      const uint32_t s_addr = tmem + lanes + S::kS(x), o_addr = tmem + lanes + S::kO(t);
      if (!wait(&sh.info[slot], (tile / kInfo) & 1)) return;
      const uint32_t pages = *reinterpret_cast<volatile uint32_t*>(&sh.valid[slot]);
      const int64_t ka = static_cast<int64_t>(w.tile0 + it) * BN;
      const bool whole = ka >= whole0 && ka + BN <= whole1 && pages == all_pages;
      const float4* ks = reinterpret_cast<const float4*>(scales + slot * 2 * BN * 4);
      const float4* vs = ks + BN / 4;
      uint32_t seen[BN / 32];   // of a tile that not every row sees in full; looked up while its scores form
      if (live_warp && !whole) {
        // the words of the row's mask that a tile can touch, in one round
        static_assert(BN <= 128, "three words");
        const int last = (w.s.T - 1) >> 6;
        const int first = static_cast<int>(min(max(ka - w.s.ctx, static_cast<int64_t>(0)) >> 6, static_cast<int64_t>(last)));
        uint64_t word[3] = {0, 0, 0};
        if (p.mask && ka + BN > w.s.ctx) {
          const uint64_t* row = mask_row(p, w.s, i_row);
#pragma unroll
          for (int k = 0; k < 3; ++k) word[k] = row[min(first + k, last)];
        }
#pragma unroll 1
        for (int c = 0; c < BN / 32; ++c)
          seen[c] = seen_bits(p, w.s, i_row, pos, ka + 32 * c, 32 * c, 32, pages, box_shift,
                              [&](int k) { return k <= first ? word[0] : k == first + 1 ? word[1] : word[2]; });
      }
      if (!wait(&sh.s_full[x], x_parity)) return;
      tc_fence_after();
      bool done = false;
      if (live_warp && whole && it > 0) {
        // One pass, the weights taken against the reference as it stands; the largest logit (E4M3: with the tile's largest scale
        // of a value, which is no less than any key's own) is looked at afterwards, and where it has passed the reference (rare
        // past an item's first tiles) the tile is done again below. (The largest product of weight and scale itself, as fp32 or
        // in the packed pairs, is known a step later: trees of 64 over 32768 E4M3 keys 323 us against 319.)
        const float mz = m == -INFINITY ? 0.0f : m;
        uint32_t pk[BN / 2];
        float sum[4] = {0.0f, 0.0f, 0.0f, 0.0f}, mx[2] = {-INFINITY, -INFINITY};
        float v[2][32];
        tmem_ld32_issue(s_addr, v[0]);
#pragma unroll
        for (int c = 0; c < BN / 32; ++c) {
          tmem_ld32_wait(v[c & 1]);
          if (c + 1 < BN / 32) tmem_ld32_issue(s_addr + 32 * (c + 1), v[(c + 1) & 1]);
          float(&y)[32] = v[c & 1];
#pragma unroll
          for (int e = 0; e < 32; e += 4) {
            float4 vf = make_float4(1.0f, 1.0f, 1.0f, 1.0f);
            if constexpr (S::E4M3) {
              const float4 kf = ks[8 * c + e / 4];
              vf = vs[8 * c + e / 4];
              fmul2_rn(y[e], y[e + 1], y[e], y[e + 1], kf.x, kf.y);
              fmul2_rn(y[e + 2], y[e + 3], y[e + 2], y[e + 3], kf.z, kf.w);
            }
            mx[0] = fmaxf(mx[0], fmaxf(y[e], y[e + 1]));
            mx[1] = fmaxf(mx[1], fmaxf(y[e + 2], y[e + 3]));
            ffma2_rn(y[e], y[e + 1], y[e], y[e + 1], fac, fac, -mz, -mz);
            ffma2_rn(y[e + 2], y[e + 3], y[e + 2], y[e + 3], fac, fac, -mz, -mz);
#pragma unroll
            for (int k = 0; k < 4; ++k) y[e + k] = ex2(y[e + k]);
            if constexpr (S::E4M3) {   // packed additions cost 5 % here, where registers are short; with bf16 they save 4 to 8 %
#pragma unroll
              for (int k = 0; k < 4; ++k) sum[k] += y[e + k];
              fmul2_rn(y[e], y[e + 1], y[e], y[e + 1], vf.x, vf.y);
              fmul2_rn(y[e + 2], y[e + 3], y[e + 2], y[e + 3], vf.z, vf.w);
            } else {
              fadd2(sum[0], sum[1], y[e], y[e + 1]);
              fadd2(sum[2], sum[3], y[e + 2], y[e + 3]);
            }
            pk[16 * c + e / 2] = S::E4M3 ? pack_f16x2(y[e], y[e + 1]) : pack_bf16x2_cvt(y[e], y[e + 1]);
            pk[16 * c + e / 2 + 1] = S::E4M3 ? pack_f16x2(y[e + 2], y[e + 3]) : pack_bf16x2_cvt(y[e + 2], y[e + 3]);
          }
        }
        const float tile_sum = (sum[0] + sum[1]) + (sum[2] + sum[3]);
        const float big = fmaxf(mx[0], mx[1]);
        float cover = 0.0f;
        if constexpr (S::E4M3) {
          const float* f = reinterpret_cast<const float*>(vs);
          uint32_t most = 0;   // but for NaN
#pragma unroll
          for (int k = 0; k < BN / 32; ++k) {
            const uint32_t bits = __float_as_uint(f[32 * k + lane]);
            most = max(most, bits < 0x7f800000u ? bits : 0u);
          }
          cover = scale_log2(__uint_as_float(__reduce_max_sync(0xffffffffu, most))) - kTop;
        }
        const float want = big == -INFINITY ? big : fmaf(big, fac, cover);
        if (!__any_sync(0xffffffffu, lane < count && want > m + kLag)) {
          l += tile_sum;
#pragma unroll
          for (int c = 0; c < BN / 32; ++c) tmem_st16u(s_addr + 16 * c, reinterpret_cast<const uint32_t(&)[16]>(pk[16 * c]));
          tmem_st_wait();
          done = true;
        }
      }
      if (live_warp && !done) {
        // what the reference has to cover: the row's largest logit, with E4M3 key by key with the values' scales
        float want = -INFINITY;
        if (whole) {
          float mx = -INFINITY;
#pragma unroll 1
          for (int c = 0; c < BN / 32; ++c) {
            float v[32];
            tmem_ld32(s_addr + 32 * c, v);
            if constexpr (S::E4M3) {
#pragma unroll
              for (int e = 0; e < 8; ++e) {
                const float4 kf = ks[8 * c + e], vf = vs[8 * c + e];
                mx = fmaxf(fmaxf(mx, fmaf(v[4 * e] * kf.x, fac, scale_log2(vf.x))), fmaf(v[4 * e + 1] * kf.y, fac, scale_log2(vf.y)));
                mx = fmaxf(fmaxf(mx, fmaf(v[4 * e + 2] * kf.z, fac, scale_log2(vf.z))), fmaf(v[4 * e + 3] * kf.w, fac, scale_log2(vf.w)));
              }
            } else {
#pragma unroll
              for (int e = 0; e < 32; e += 2) mx = fmaxf(mx, fmaxf(v[e], v[e + 1]));
            }
          }
          want = S::E4M3 ? mx - kTop : mx == -INFINITY ? mx : mx * fac;
        } else {
#pragma unroll 1
          for (int c = 0; c < BN / 32; ++c) {
            const uint32_t bits = seen[c];
            float v[32];
            tmem_ld32(s_addr + 32 * c, v);
#pragma unroll
            for (int e = 0; e < 32; e += 4) {   // without branches: what a masked key's scales hold is selected away
              float4 kf = make_float4(1.0f, 1.0f, 1.0f, 1.0f), vf = kf;
              if constexpr (S::E4M3) {
                kf = ks[8 * c + e / 4];
                vf = vs[8 * c + e / 4];
              }
              const float k4[4] = {kf.x, kf.y, kf.z, kf.w}, v4[4] = {vf.x, vf.y, vf.z, vf.w};
#pragma unroll
              for (int k = 0; k < 4; ++k) {
                const float y = S::E4M3 ? v[e + k] * k4[k] : v[e + k];
                const float z = fmaf(y, fac, S::E4M3 ? scale_log2(v4[k]) - kTop : 0.0f);
                const bool in = ((bits >> (e + k)) & 1) != 0 & (y != -INFINITY);
                want = fmaxf(want, in ? z : -INFINITY);
              }
            }
          }
        }
        // a lane without a row has what an earlier item or call left there: it has no say, or bits would hang on that
        const bool grown = lane < count && want > m + kLag;
        if (__any_sync(0xffffffffu, grown)) {
          const float mx = fmaxf(m, want), keep = ex2(m - (mx == -INFINITY ? 0.0f : mx));
          m = mx;
          l *= keep;
          if (it > 0) {   // the sums of the item so far
            if (!wait(&sh.o_done[t], (tile - 1) & 1)) return;
            tc_fence_after();
#pragma unroll 1
            for (int d = 0; d < D; d += 32) {
              float v[32];
              tmem_ld32(o_addr + d, v);
#pragma unroll
              for (int e = 0; e < 32; ++e) v[e] *= keep;
              tmem_st32(o_addr + d, v);
            }
            tmem_st_wait();
          }
        }
        const float mz = m == -INFINITY ? 0.0f : m;
#pragma unroll 1
        for (int c = 0; c < BN / 32; ++c) {
          const uint32_t bits = whole ? 0xffffffffu : seen[c];
          float v[32];
          tmem_ld32(s_addr + 32 * c, v);
          uint32_t pk[16];
          float part = 0.0f;
#pragma unroll
          for (int e = 0; e < 8; ++e) {
            float4 kf = make_float4(1.0f, 1.0f, 1.0f, 1.0f), vf = kf;
            if (S::E4M3) {
              kf = ks[8 * c + e];
              vf = vs[8 * c + e];
            }
            const float k4[4] = {kf.x, kf.y, kf.z, kf.w}, v4[4] = {vf.x, vf.y, vf.z, vf.w};
#pragma unroll
            for (int k = 0; k < 4; ++k) {
              const float y = S::E4M3 ? v[4 * e + k] * k4[k] : v[4 * e + k];
              float u = ex2(fmaf(y, fac, -mz));
              if (!whole && (!((bits >> (4 * e + k)) & 1) || y == -INFINITY)) u = 0.0f;
              part += u;
              if (S::E4M3) {
                u *= v4[k];
                if (!whole && !((bits >> (4 * e + k)) & 1)) u = 0.0f;   // whatever scale lies there
              }
              v[4 * e + k] = u;
            }
            pk[2 * e] = S::E4M3 ? pack_f16x2(v[4 * e], v[4 * e + 1]) : pack_bf16x2_cvt(v[4 * e], v[4 * e + 1]);
            pk[2 * e + 1] = S::E4M3 ? pack_f16x2(v[4 * e + 2], v[4 * e + 3]) : pack_bf16x2_cvt(v[4 * e + 2], v[4 * e + 3]);
          }
          l += part;
          tmem_st16u(s_addr + 16 * c, pk);   // over scores already read
        }
        tmem_st_wait();
      }
      if (!whole) {
        // Values behind the last key and in pages left out may hold anything: zeros in their place. Infinities and NaN in
        // keys that some row sees: the product is done by hand.
        if (!wait(&sh.full[v_at.i], v_at.phase)) return;
        const uint32_t vb = smem_u32(tiles) + v_at.i * S::kTile;
        if (r == 0) sh.special[t][tile & 1] = 0;
        if (!meet()) return;
        bool special = false;
        constexpr int kLook = 8;   // chunks looked at together
#pragma unroll 1
        for (int e0 = r; e0 < BN * D / 8; e0 += kLook * kGroup) {
          uint32_t q[kLook][4];
#pragma unroll
          for (int j = 0; j < kLook; ++j)
            asm volatile("ld.shared.v4.u32 {%0, %1, %2, %3}, [%4];"
                         : "=r"(q[j][0]), "=r"(q[j][1]), "=r"(q[j][2]), "=r"(q[j][3])
                         : "r"(tile_addr(vb, BN, (e0 + j * kGroup) / (D / 8), (e0 + j * kGroup) % (D / 8)))
                         : "memory");
          uint32_t odd[kLook], any = 0;
          const uint32_t exp = S::E4M3 ? 0x7c007c00u : 0x7f807f80u;
#pragma unroll
          for (int j = 0; j < kLook; ++j) {
            odd[j] = 0;
#pragma unroll
            for (int k = 0; k < 4; ++k) odd[j] |= __vcmpeq2(q[j][k] & exp, exp);
            any |= odd[j];
          }
          if (!any) continue;
#pragma unroll
          for (int j = 0; j < kLook; ++j) {
            if (!odd[j]) continue;
            const int key = (e0 + j * kGroup) / (D / 8), c = (e0 + j * kGroup) % (D / 8);
            const int64_t kk = ka + key;
            if (kk < w.s.lo || kk >= w.s.hi || !((pages >> (key >> box_shift)) & 1))
              asm volatile("st.shared.v4.u32 [%0], {%1, %1, %1, %1};" ::"r"(tile_addr(vb, BN, key, c)), "r"(0) : "memory");
            else
              special = true;
          }
        }
        if (special) sh.special[t][tile & 1] = 1;
        fence_proxy_async_smem();
        if (!meet()) return;
        const bool by_hand = *reinterpret_cast<volatile int32_t*>(&sh.special[t][tile & 1]) != 0;
        if (by_hand) {
          if (it > 0 && !wait(&sh.o_done[t], (tile - 1) & 1)) return;
          tc_fence_after();
          if (live_warp) sums_by_hand<S>(p, w.s, i_row, pos, ka, pages, box_shift, s_addr, o_addr, vb, it == 0);
        }
        if (r == 0) sh.skip[x] = by_hand;
      } else if (r == 0) {
        sh.skip[x] = 0;
      }
      tc_fence_before();
      __syncwarp();
      if (lane == 0) mbar_arrive(&sh.p_ready[x]);
    }
    // The item's rows, behind its last sums. A parity tells a phase from the one before alone. With two row tiles a tile's scores
    // are issued behind the sums of the tile before, so those were complete when the scores were. With one they are issued ahead
    // of them: of the last two sums neither may be complete here, or both, and the item has a barrier of its own.
    if (!(S::TILES == 2 ? wait(&sh.o_done[t], (tile - 1) & 1) : wait(&sh.item_done, item & 1))) return;
    tc_fence_after();
    if (live_warp) {
      const bool complete = w.n == w.len;
      const int slot = w.offset > 0 ? 0 : 1;   // partial sums: an item begun elsewhere, or one that goes on elsewhere
      const bool none = m == -INFINITY && l == 0.0f;
      const float inv = complete ? 1.0f / l : 1.0f;
      const int head = w.head * group + static_cast<int>(row - static_cast<uint32_t>(i_row) * group);
      const int64_t out_row = static_cast<int64_t>(w.s.first) + i_row;
      const int64_t at = (static_cast<int64_t>(blockIdx.x) * 2 + slot) * S::M + t * 128 + 4 * lane + wq;
      // 32 columns at a time through the warp's own rows of the query buffer (their last product is done), so that the
      // stores leave in whole lines: row-wise in, swizzled by 16 bytes, four rows of eight chunks out
      const uint32_t stage = smem_u32(qbuf) + t * 128 * D * 2;
      // where this lane's chunk of rows 4 k + lane / 8 goes: the row's own place, known to its lane
      const int64_t place = complete ? out_row * p.o_tok + head * p.o_head : at * D;
      const int q = lane & 7, below = count - (lane >> 3);   // row 4 k + lane / 8 is one of the warp's: 4 k < below
      int64_t to[8];
#pragma unroll
      for (int k = 0; k < 8; ++k) to[k] = __shfl_sync(0xffffffffu, place, 4 * k + (lane >> 3)) + 4 * q;
#pragma unroll 1
      for (int d = 0; d < D; d += 32) {
        float v[32];
        tmem_ld32(tmem + lanes + S::kO(t) + d, v);
#pragma unroll
        for (int k = 0; k < 8; ++k)
          asm volatile("st.shared.v4.f32 [%0], {%1, %2, %3, %4};" ::"r"(stage + stage_offset(r, k)),
                       "f"(none ? 0.0f : v[4 * k] * inv), "f"(none ? 0.0f : v[4 * k + 1] * inv), "f"(none ? 0.0f : v[4 * k + 2] * inv),
                       "f"(none ? 0.0f : v[4 * k + 3] * inv)
                       : "memory");
        __syncwarp();
        float4 f[8];
#pragma unroll
        for (int k = 0; k < 8; ++k) {
          const int lr = wq * 32 + 4 * k + (lane >> 3);
          asm volatile("ld.shared.v4.f32 {%0, %1, %2, %3}, [%4];"
                       : "=f"(f[k].x), "=f"(f[k].y), "=f"(f[k].z), "=f"(f[k].w)
                       : "r"(stage + stage_offset(lr, q))
                       : "memory");
        }
        // one branch for all stores: one at each cost 500 clocks a round
        if (complete) {
#pragma unroll
          for (int k = 0; k < 8; ++k)
            if (4 * k < below) *reinterpret_cast<uint2*>(p.o + to[k] + d) = make_uint2(pack_bf16x2_cvt(f[k].x, f[k].y), pack_bf16x2_cvt(f[k].z, f[k].w));
        } else {
#pragma unroll
          for (int k = 0; k < 8; ++k)
            if (4 * k < below) *reinterpret_cast<float4*>(p.part_o + to[k] + d) = f[k];
        }
        __syncwarp();
      }
      if (lane < count) {
        if (!complete) p.part_ml[at] = make_float2(m, l);
        else if (p.lse) p.lse[out_row * (p.hk * p.group) + head] = none ? -INFINITY : ((m == -INFINITY ? 0.0f : m) + log2f(l)) * 0.6931471805599453f;
      }
    }
  }
}

template <class S>
__global__ void __launch_bounds__(S::kThreads, 1) aq_tree_attention_tc_kernel(const __grid_constant__ AttnParams p) {
  extern __shared__ uint8_t raw[];
  __shared__ TcShared sh;
  uint8_t* qbuf = raw + ((1024 - (smem_u32(raw) & 1023)) & 1023);
  uint8_t* tiles = qbuf + S::kQ;                                     // 16-bit K and V tiles
  const int nring = S::E4M3 ? S::NF : p.stages;
  uint8_t* codes = tiles + nring * S::kTile;                         // E4M3: p.stages tiles of codes
  uint8_t* scales = codes + (S::E4M3 ? p.stages * S::kCode : 0);
  const int warp = threadIdx.x >> 5;
  if (threadIdx.x == 0) {
    for (int i = 0; i < kMaxRing; ++i) {
      mbar_init(&sh.full[i], S::E4M3 ? 4 : 1);
      mbar_init(&sh.empty[i], 1);
      mbar_init(&sh.cfull[i], 1);
      mbar_init(&sh.cempty[i], 4);
    }
    for (int i = 0; i < kInfo; ++i) mbar_init(&sh.info[i], 1);
    mbar_init(&sh.q_ready, S::kSoftWarps);
    for (int i = 0; i < 2; ++i) {
      mbar_init(&sh.s_full[i], 1);
      mbar_init(&sh.p_ready[i], 4);
      mbar_init(&sh.o_done[i], 1);
      mbar_init(&sh.together[i], 4);
      sh.skip[i] = 0;
    }
    mbar_init(&sh.item_done, 1);
    mbar_init(&sh.drain, 1);
    sh.abort = 0;
    fence_barrier_init();
    tma_prefetch_desc(&p.tm_k);
    tma_prefetch_desc(&p.tm_v);
  }
  if (warp == S::kMmaWarp) {
    tmem_alloc(&sh.tmem, 512);
    tmem_relinquish();
  }
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  const uint32_t tmem = sh.tmem;
  pdl_wait_prior_grid();
  int64_t range[2];
  locate<S::M, S::BN>(p, sh.work, blockIdx.x == 0, range);
  pdl_launch_dependents();   // the joining blocks find their rows meanwhile; they wait for this grid before its results
  const AbortCtl ctl = {&sh.abort, p.status, p.timeout_ns};
  if (warp < S::kSoftWarps) {
    if (S::kSplitRegs) asm volatile("setmaxnreg.inc.sync.aligned.u32 176;");
    tc_weigh<S>(p, sh, qbuf, tiles, scales, nring, tmem, range, ctl);
  } else if (S::E4M3 && warp < S::kTmaWarp) {
    if (S::kSplitRegs) asm volatile("setmaxnreg.dec.sync.aligned.u32 88;");
    tc_convert<S>(sh, codes, tiles, p.stages, range[1] - range[0], ctl);
  } else {
    if (S::kSplitRegs) asm volatile("setmaxnreg.dec.sync.aligned.u32 72;");
    if (warp == S::kTmaWarp) {
      tc_produce<S>(p, sh, S::E4M3 ? codes : tiles, scales, p.stages, range, ctl);
    } else if (warp == S::kMmaWarp) {
      if (range[1] > range[0]) {
        tc_issue<S>(p, sh, qbuf, tiles, nring, tmem, range, ctl);
        // nothing is in flight when tensor memory is freed
        __syncwarp();
        if (elect_one()) tc_commit(&sh.drain);
        const uint64_t t0 = global_timer_ns();
        while (!mbar_try_wait(&sh.drain, 0))
          if (global_timer_ns() - t0 > p.timeout_ns) break;
      }
      __syncwarp();
    }
  }
  tc_fence_before();
  __syncthreads();
  if (warp == S::kMmaWarp) {
    tc_fence_after();
    tmem_dealloc(tmem, 512);
  }
}

template <class S>
aq_status launch_tc(AttnParams& p, const aq_kv_cache* c, const ServeDev& dev, cudaStream_t st, const char* who) {
  aq_status s;
  const int box = std::min(c->page_size, S::BN), cols = S::E4M3 ? S::CB : 64;
  if ((s = attention_cache_map(&p.tm_k, c->k, c, cols, box, who)) != AQ_OK) return s;
  if ((s = attention_cache_map(&p.tm_v, c->v, c, cols, box, who)) != AQ_OK) return s;
  constexpr size_t kStatic = (sizeof(TcShared) + 127) / 128 * 128, kFixed = 1024 + S::kQ + S::kScale + S::NF * S::kTile;
  constexpr size_t kUnit = S::E4M3 ? S::kCode : S::kTile;
  if (dev.smem_optin < kStatic + kFixed + 2 * kUnit) return serve_fail(AQ_ERR_UNSUPPORTED, "%s: the device has too little shared memory", who);
  p.stages = static_cast<int>(std::min<size_t>((dev.smem_optin - kStatic - kFixed) / kUnit, S::E4M3 ? 6 : kMaxRing));
  const size_t smem = kFixed + p.stages * kUnit;
  static std::atomic<uint64_t> ready{0};   // devices on which the kernel may use that much
  const uint64_t bit = 1ull << dev.index;
  if (!(ready.load() & bit)) {
    const cudaError_t e = cudaFuncSetAttribute(aq_tree_attention_tc_kernel<S>, cudaFuncAttributeMaxDynamicSharedMemorySize, static_cast<int>(smem));
    if (e != cudaSuccess) return serve_launched(e, who);
    ready.fetch_or(bit);
  }
  p.main_grid = std::min(dev.sms, kAttnSmsBound);
  return serve_launched(launch_serve(aq_tree_attention_tc_kernel<S>, p, dim3(p.main_grid), S::kThreads, smem, st), who);
}

}  // namespace

aq_status launch_attention_tc(AttnParams& p, const aq_kv_cache* c, const ServeDev& dev, cudaStream_t st, const char* who) {
  const bool e4m3 = c->type == AQ_KV_E4M3, two = p.rows_per_tile == 256;
  switch (c->head_dim) {
    case 64:
      if (two) return e4m3 ? launch_tc<TcShape<64, true, 2>>(p, c, dev, st, who) : launch_tc<TcShape<64, false, 2>>(p, c, dev, st, who);
      return e4m3 ? launch_tc<TcShape<64, true, 1>>(p, c, dev, st, who) : launch_tc<TcShape<64, false, 1>>(p, c, dev, st, who);
    case 128:
      if (two) return e4m3 ? launch_tc<TcShape<128, true, 2>>(p, c, dev, st, who) : launch_tc<TcShape<128, false, 2>>(p, c, dev, st, who);
      return e4m3 ? launch_tc<TcShape<128, true, 1>>(p, c, dev, st, who) : launch_tc<TcShape<128, false, 1>>(p, c, dev, st, who);
    default:
      return e4m3 ? launch_tc<TcShape<256, true, 1>>(p, c, dev, st, who) : launch_tc<TcShape<256, false, 1>>(p, c, dev, st, who);
  }
}

}  // namespace aq
