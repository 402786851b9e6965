// aq_attention.cuh -- what the kernels of aq_tree_attention share: their parameters, how the work of a call is
// shared out over the CTAs, which keys a row sees.
#pragma once

#include <cuda_fp16.h>

#include "aq_serve.h"

namespace aq {

// Division of 32-bit numbers by a number known to the host (Granlund and Montgomery, 1994): a product, a subtraction and
// two shifts, where a division by a variable takes some forty dependent instructions.
struct FastDiv {
  uint32_t d = 1, mul = 0;
  int32_t s1 = 0, s2 = 0;
  __host__ __device__ FastDiv() {}
  __host__ explicit FastDiv(uint32_t by) : d(by) {
    int l = 0;
    while (l < 32 && (1ull << l) < by) ++l;
    mul = static_cast<uint32_t>(((1ull << 32) * ((1ull << l) - by)) / by + 1);
    s1 = l < 1 ? l : 1;
    s2 = l > 1 ? l - 1 : 0;
  }
  __device__ __forceinline__ uint32_t quot(uint32_t n) const {
    const uint32_t t = __umulhi(mul, n);
    return (t + ((n - t) >> s1)) >> s2;
  }
};

// How an entry (a sequence's row tile) was shared out, for the joining launch: its item of key/value head h lies in the
// CTAs base + (first + h step + i) / share, i = 0 .. len - 1.
struct AttnShare {
  int64_t first;
  int32_t base, step, len, share;
};

struct AttnParams {
  CUtensorMap tm_k, tm_v;
  const float* ks;
  const float* vs;
  int32_t pages, page_shift, hk, group;
  const uint16_t* q;
  int64_t q_tok, q_head;
  uint16_t* o;
  int64_t o_tok, o_head;
  float* lse;
  const int32_t* cu;
  const int32_t* ctx;
  const int32_t* table;
  int64_t ld_table;
  int32_t pages_per_seq;
  const uint64_t* mask;
  int64_t ld_mask;
  const int32_t* depth;
  int32_t batch, max_q, window;
  int64_t total_q;
  float scale;
  int32_t rows_per_tile, row_tiles;   // rows of a tile, tiles of a sequence
  FastDiv by_group, by_tiles, by_heads;   // query heads a key/value head; row_tiles; query heads
  int32_t main_grid, stages;
  AttnShare* shares;                  // [batch * row_tiles]
  float2* part_ml;                    // [CTA][2][rows of a tile] maximum (base 2) and sum of a partial item
  float* part_o;                      // [CTA][2][rows of a tile][D]
  int32_t* status;
  uint64_t timeout_ns;
};
static_assert(sizeof(AttnParams) <= 4096, "kernel parameters are limited to 4 KB");

// Launches the tcgen05 kernel (rows_per_tile 128 or 256) in place of the mma.sync one; `grid` CTAs.
aq_status launch_attention_tc(AttnParams& p, const aq_kv_cache* c, const ServeDev& dev, cudaStream_t st, const char* who);
// Cache codes as {D, page, pages * heads}: boxes of one column block (128 bytes at most) of up to a tile's rows.
aq_status attention_cache_map(CUtensorMap* m, const void* base, const aq_kv_cache* c, int box_cols, int box_rows, const char* who);

constexpr int kAttnSmsBound = 192;      // SMs (of any sm_103 part) and CTAs an SM, for sizing the
constexpr int kAttnMaxPerSm = 2;        // workspace without a device
// The reference that a row's weights are taken against may lag by this power of two before the sums are scaled over.
constexpr float kLag = 6.0f;
// E4M3: the reference is that of the weights times their values' scales, key by key (the largest logit and the largest scale by
// themselves may be different keys', and their product far above every key's), so that such a product, in f16, stays below
// 2^(kTop + kLag + 1) = 2^15, and the largest is not below 2^kTop. Scales under 2^kLeast count as that: the weights' own sum
// stays finite.
constexpr int kTop = 8;
constexpr int kLeast = -64;


// Four E4M3 codes to two pairs of halves.
__device__ __forceinline__ void widen(uint32_t c, uint32_t& lo, uint32_t& hi) {
  asm("{\n .reg .b16 l, h;\n mov.b32 {l, h}, %2;\n cvt.rn.f16x2.e4m3x2 %0, l;\n cvt.rn.f16x2.e4m3x2 %1, h;\n}"
      : "=r"(lo), "=r"(hi)
      : "r"(c));
}
__device__ __forceinline__ uint32_t pack_f16x2(float lo, float hi) {
  uint32_t r;
  asm("cvt.rn.f16x2.f32 %0, %1, %2;" : "=r"(r) : "f"(hi), "f"(lo));
  return r;
}
__device__ __forceinline__ float ex2(float x) {
  float r;
  asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(r) : "f"(x));
  return r;
}
__device__ __forceinline__ void bulk_load(void* dst, const void* src, uint32_t bytes, uint64_t* bar) {
  asm volatile("cp.async.bulk.shared::cluster.global.mbarrier::complete_tx::bytes [%0], [%1], %2, [%3];" ::"r"(
                   smem_u32(dst)),
               "l"(src), "r"(bytes), "r"(smem_u32(bar))
               : "memory");
}
// Quotient of non-negative numbers, by a 32-bit division where they fit (a 64-bit one costs ten times as much, and
// these stand between a call's dependent loads).
__device__ __forceinline__ int64_t quot(int64_t a, int64_t b) {
  if (((a | b) >> 32) == 0) return static_cast<uint32_t>(a) / static_cast<uint32_t>(b);
  return a / b;
}
// 2^e for e in [-126, 127].
__device__ __forceinline__ float pow2(int e) { return __int_as_float((e + 127) << 23); }
// Exponent of a non-negative value, kept where 2^(14 - e) and 2^(e - 14) are finite; zero counts as 2^-112.
__device__ __forceinline__ int top_exponent(float x) { return min(max(static_cast<int>(__float_as_uint(x) >> 23) - 127, -112), 126); }

// Logarithm (base 2) of a value's scale, for the reference. The scale of a vector that reads as NaN counts as the smallest: its
// key's weight belongs in the row's sum like any other, and against a reference 2^120 above it the sum (and lse) would lose
// the rest.
__device__ __forceinline__ float scale_log2(float x) {
  float r;
  asm("lg2.approx.ftz.f32 %0, %1;" : "=f"(r) : "f"(x));
  return fminf(fmaxf(r, static_cast<float>(kLeast)), 127.0f);
}

// Keys [lo, hi) and tiles [t0, t1) that the rows of entry (sequence b, row tile rt) can see.
struct KeySpan {
  int64_t lo, hi;
  int32_t t0, t1;
  int32_t first, T, ctx;    // first row in q, rows, context
};

// Where a CTA begins: entry, head and tile of the item; what the warps exchange to find it.
struct AttnWork {
  KeySpan span;
  int32_t entry, head, offset, len;
  int64_t left;          // tiles of the CTA
  int64_t part[2][16];
};

template <int M, int KS>
__device__ __forceinline__ KeySpan entry_span(const AttnParams& p, int b, int rt) {
  KeySpan s;
  const int c0 = p.cu[b], c1 = p.cu[b + 1];
  s.first = c0;
  s.ctx = max(p.ctx[b], 0);
  s.T = c0 >= 0 && c1 > c0 && c0 < p.total_q ? static_cast<int>(min(static_cast<int64_t>(min(c1 - c0, p.max_q)), p.total_q - c0)) : 0;
  const uint32_t rows = static_cast<uint32_t>(s.T) * p.group, r0 = static_cast<uint32_t>(rt) * M;   // below 2^31: see the host
  s.t0 = s.t1 = 0;
  s.lo = s.hi = 0;
  if (r0 >= rows) return s;
  const int i0 = p.by_group.quot(r0), i1 = p.by_group.quot(min(r0 + M, rows) - 1);
  s.hi = min(static_cast<int64_t>(s.ctx) + (p.mask ? s.T : i1 + 1), static_cast<int64_t>(p.pages_per_seq) << p.page_shift);
  if (p.window > 0) s.lo = max(static_cast<int64_t>(s.ctx) + (p.mask ? 0 : i0) - p.window + 1, static_cast<int64_t>(0));
  s.lo = min(s.lo, s.hi);
  s.t0 = static_cast<int32_t>(s.lo / KS);
  s.t1 = max(static_cast<int32_t>((s.hi + KS - 1) / KS), s.t0 + 1);   // a row that can see nothing is written too
  return s;
}

// A number's sum over the threads before this one, and over all; `part` is the warps' exchange.
__device__ __forceinline__ void block_scan(int64_t mine, int64_t (&part)[16], int64_t& before, int64_t& total) {
  const int tid = threadIdx.x;
  int64_t upto = mine;
#pragma unroll
  for (int off = 1; off < 32; off *= 2) {
    const int64_t v = __shfl_up_sync(0xffffffffu, upto, off);
    if ((tid & 31) >= off) upto += v;
  }
  if ((tid & 31) == 31) part[tid >> 5] = upto;
  __syncthreads();
  before = upto - mine;
  total = 0;
  for (int i = 0; i < static_cast<int>(blockDim.x) / 32; ++i) {
    if (i < (tid >> 5)) before += part[i];
    total += part[i];
  }
}

// A CTA pays for every item it takes part in with the item's start and its sums' way out, about as long as this many
// tiles: a call of fewer tiles a CTA gives every CTA one item.
constexpr int kItemTiles = 6;

// The CTA's share of the call's tiles, in sh and `range` (tiles range[0] .. range[1]-1 of the CTA's own count); called by
// every thread. CTA 0 also leaves the shares for the joining launch. Either all items' tiles are laid end to end and cut
// into equal pieces, or (short calls) each item has CTAs of its own in proportion to its length.
template <int M, int KS>
__device__ __forceinline__ void locate(const AttnParams& p, AttnWork& sh, bool write, int64_t (&range)[2]) {
  const int n = p.batch * p.row_tiles, tid = threadIdx.x, G = gridDim.x;
  const int threads = blockDim.x;
  const int per = n <= threads ? 1 : (n + threads - 1) / threads;
  const int e0 = min(tid * per, n), e1 = min(e0 + per, n);
  KeySpan s = {};
  auto span_of = [&](int e) {
    const int b = p.by_tiles.quot(e);
    return entry_span<M, KS>(p, b, e - b * p.row_tiles);
  };
  int64_t sum = 0;   // tiles, and above 2^40 items
  for (int e = e0; e < e1; ++e) {
    s = span_of(e);
    const int len = s.t1 - s.t0;
    sum += static_cast<int64_t>(len) * p.hk + (len > 0 ? static_cast<int64_t>(p.hk) << 40 : 0);
  }
  constexpr int64_t kTiles = (1ll << 40) - 1;
  int64_t before, total;
  block_scan(sum, sh.part[0], before, total);
  const int64_t items = total >> 40;
  before &= kTiles;
  total &= kTiles;
  const int64_t share = quot(total + G - 1, G);
  const bool own = items <= G && share <= kItemTiles;   // CTAs of its own for each item
  auto ctas_of = [&](int len) { return 1 + static_cast<int>(quot(len * (G - items), total)); };
  if (own) {
    int64_t mine = 0, all;
    for (int e = e0; e < e1; ++e) {
      if (e1 - e0 > 1) s = span_of(e);
      if (s.t1 > s.t0) mine += p.hk * ctas_of(s.t1 - s.t0);
    }
    block_scan(mine, sh.part[1], before, all);
  }
  range[0] = own ? 0 : min(share * blockIdx.x, total);
  range[1] = own ? 0 : min(range[0] + share, total);
  if (tid == 0) sh.left = 0;
  __syncthreads();
  int64_t at = before;   // of tiles, or of CTAs
  for (int e = e0; e < e1; ++e) {
    if (e1 - e0 > 1) s = span_of(e);     // a thread's one entry is known already
    const int len = s.t1 - s.t0;
    if (len == 0) continue;
    const int ctas = own ? ctas_of(len) : 0, piece = own ? static_cast<int>(quot(len + ctas - 1, ctas)) : 0;
    const int64_t size = static_cast<int64_t>(own ? ctas : len) * p.hk, me = own ? blockIdx.x : range[0];
    if (me >= at && me < at + size) {
      const int64_t in = me - at;
      sh.span = s;
      sh.entry = e;
      sh.len = len;
      sh.head = static_cast<int>(quot(in, own ? ctas : len));
      sh.offset = static_cast<int>(in - static_cast<int64_t>(sh.head) * (own ? ctas : len)) * (own ? piece : 1);
      sh.left = own ? max(min(piece, len - sh.offset), 0) : range[1] - range[0];
    }
    if (write) p.shares[e] = own ? AttnShare{0, static_cast<int32_t>(at), ctas * piece, len, piece} : AttnShare{at, 0, len, len, static_cast<int32_t>(share)};
    at += size;
  }
  __syncthreads();
  if (own) range[1] = sh.left;
}

// Walks the segments of a CTA's range: consecutive tiles of one item.
template <int M, int KS>
struct Walk {
  int64_t left;          // tiles of the CTA's range still to come
  int entry, head;       // entry: sequence b, row tile rt
  int b, rt;
  int tile0, n;          // this segment: first tile (within the sequence) and how many
  int len;               // tiles of the whole item
  int offset;            // of them before this segment
  KeySpan s;
  __device__ __forceinline__ Walk(const AttnParams& p, const AttnWork& sh, const int64_t (&range)[2]) {
    left = range[1] - range[0];
    if (left <= 0) return;
    entry = sh.entry;
    head = sh.head;
    offset = sh.offset;
    len = sh.len;
    s = sh.span;
    place(p);
    cut();
  }
  __device__ __forceinline__ void place(const AttnParams& p) {
    b = p.by_tiles.quot(entry);
    rt = entry - b * p.row_tiles;
  }
  __device__ __forceinline__ void cut() {
    tile0 = s.t0 + offset;
    n = static_cast<int>(min(static_cast<int64_t>(len - offset), left));
  }
  __device__ __forceinline__ void next(const AttnParams& p) {
    left -= n;
    if (left <= 0) return;
    offset = 0;
    if (++head == p.hk) {
      head = 0;
      do {
        ++entry;
        place(p);
        s = entry_span<M, KS>(p, b, rt);
        len = s.t1 - s.t0;
      } while (len == 0);
    }
    cut();
  }
};

// The `count` <= 32 keys from ka on (place k0 of the tile) that a row sees, as bits; i: its drafted index, pos: its
// position; word(w): word w of the row's mask. Called by whole warps, each lane for a row of its own. One round of loads,
// whatever the mask.
template <class Word>
__device__ __forceinline__ uint32_t seen_bits(const AttnParams& p, const KeySpan& s, int i, int64_t pos, int64_t ka, int k0,
                                              int count, uint32_t pages, int box_shift, Word&& word) {
  const int lane = threadIdx.x & 31;
  auto below = [](int64_t n) { return n <= 0 ? 0u : n >= 32 ? 0xffffffffu : (1u << n) - 1; };   // bits [0, n)
  uint32_t bits = below(s.hi - ka) & below(count);
  for (int k = 0; k < count; k += 1 << min(box_shift, 5))
    if (!((pages >> ((k0 + k) >> box_shift)) & 1)) bits &= ~(below(1 << min(box_shift, 5)) << k);
  const int64_t t0 = ka - s.ctx;                  // drafted index of the first key (negative: context)
  const uint32_t drafted = ~below(-t0);           // which keys are drafted ones
  if (drafted) {
    uint32_t see;
    if (p.mask) {
      const int64_t at = max(t0, static_cast<int64_t>(0));
      const int last = (s.T - 1) >> 6, w0 = min(static_cast<int>(min(at >> 6, static_cast<int64_t>(last))), last), w1 = min(w0 + 1, last);
      const uint64_t lo = word(w0), hi = word(w1);
      const int sh0 = static_cast<int>(at & 63);
      const uint64_t v = sh0 ? (lo >> sh0) | (hi << (64 - sh0)) : lo;
      see = t0 < 0 ? static_cast<uint32_t>(v) << static_cast<int>(-t0) : static_cast<uint32_t>(v);
    } else {
      see = below(i - t0 + 1);
    }
    bits &= ~drafted | see;
  }
  if (p.window > 0) {
    // context (and a chain's) keys lie at their index; a tree's drafted ones at their depth
    const bool tree = p.mask && p.depth;
    const uint32_t indexed = tree ? ~drafted : 0xffffffffu;
    bits &= ~indexed | ~below(pos - p.window + 1 - ka);
    if (tree && drafted) {
      const int64_t t = t0 + lane;
      const int d = t >= 0 && t < s.T ? max(p.depth[s.first + t], 0) : 0;
      for (int k = 0; k < count; ++k) {
        const int dk = __shfl_sync(0xffffffffu, d, k);
        if (((drafted >> k) & 1) && pos - (static_cast<int64_t>(s.ctx) + dk) >= p.window) bits &= ~(1u << k);
      }
    }
  }
  return bits;
}

__device__ __forceinline__ const uint64_t* mask_row(const AttnParams& p, const KeySpan& s, int i) {
  return p.mask + (static_cast<int64_t>(s.first) + i) * p.ld_mask;
}
__device__ __forceinline__ uint32_t seen_bits(const AttnParams& p, const KeySpan& s, int i, int64_t pos, int64_t ka, int k0,
                                              int count, uint32_t pages, int box_shift) {
  return seen_bits(p, s, i, pos, ka, k0, count, pages, box_shift, [&](int w) { return mask_row(p, s, i)[w]; });
}

}  // namespace aq
