// aq_positions.cu -- rotary positions and the paged key/value cache: aq_rope, aq_rope_frequencies,
// aq_kv_write, aq_kv_read.
//
// Rotation of the pair (a, b) of a head at position pos by the angle pos * f:
//   (a cos - b sin, b cos + a sin) * magnitude,   inverse: (a cos + b sin, b cos - a sin) * magnitude
// (the inverse is the transpose, so it is the gradient with respect to the input). The angle is kept
// as a fraction of a turn in 64 bits: phase = pos * F mod 2^64 with F = f / (2 pi) * 2^64, one integer
// product that wraps exactly where the angle does. An fp32 product pos * f is off by pos * f * 2^-24
// radians (0.06 at a million positions); the phase is exact, and its top 32 bits give sincospi an
// argument in [-1, 1).
//
// Quantisation of one vector x of D elements (a token's keys or values of one head) to E4M3:
//   scale = max(max|x| * RN(1/448), 2^-100),  code = E4M3(RN(x * RN(1/scale))),  read = RN_bf16(code * scale)
// A vector holding an infinity or a NaN is stored as scale NaN and codes 0: it reads back as NaN, and
// the codes themselves stay finite.
//
// Both are bound by memory: every element is read once and written once. A group of lanes owns one
// token's vector, each lane two 16-byte chunks of it (in the half layout the two that rotate against
// each other), so a vector is loaded in whole 128-byte lines and its maximum is a few shuffles. The
// eight sines and cosines of a lane depend on the token alone, so a group walks several heads of its token
// with them in registers, two heads' loads in flight. Measured: a
// rotation of 8192 tokens x 32 heads of 128 (64 of them turned) 19.3 us in a graph (134 MB, of whose writes most are still in L2 at
// the launch's end; calls one after another 23.3 us: 5770 GB/s), of 4099 x 16, heads outermost, 7.0 us
// (34 MB: 4770 GB/s, start and end included); an E4M3 write of 8192 tokens with 32 query and 8 key/value heads of
// 128 and its read back 44.7 us together (236 MB: 5280 GB/s), of which the write takes about 34; calls of a few tokens 2.2 us.
#include <math.h>

#include <algorithm>
#include <mutex>

#include "aq_positions.cuh"

namespace aq {

aq_status serve_device(ServeDev* out) {
  static std::mutex mu;
  static ServeDev known[64];
  int dev = 0;
  cudaError_t e = cudaGetDevice(&dev);
  if (e != cudaSuccess) return serve_launched(e, "cudaGetDevice");
  if (dev < 0 || dev >= 64) return serve_fail(AQ_ERR_UNSUPPORTED, "device index %d out of range", dev);
  std::lock_guard<std::mutex> lock(mu);
  ServeDev& d = known[dev];
  if (!d.sms) {
    int major = 0, minor = 0, sms = 0, smem = 0;
    if ((e = cudaDeviceGetAttribute(&major, cudaDevAttrComputeCapabilityMajor, dev)) ||
        (e = cudaDeviceGetAttribute(&minor, cudaDevAttrComputeCapabilityMinor, dev)) ||
        (e = cudaDeviceGetAttribute(&sms, cudaDevAttrMultiProcessorCount, dev)) ||
        (e = cudaDeviceGetAttribute(&smem, cudaDevAttrMaxSharedMemoryPerBlockOptin, dev)))
      return serve_launched(e, "cudaDeviceGetAttribute");
    if (major != 10 || minor != 3)
      return serve_fail(AQ_ERR_UNSUPPORTED, "device %d is sm_%d%d; this library is built for sm_103a (GB300)", dev,
                        major, minor);
    int32_t* status = device_status_ptr(dev, &e);
    if (e != cudaSuccess) return serve_launched(e, "cudaGetSymbolAddress(status)");
    d.index = dev;
    d.status = status;
    d.smem_optin = static_cast<size_t>(smem);
    d.sms = sms;
  }
  *out = d;
  return AQ_OK;
}

serve_encode_fn serve_encode() {
  static serve_encode_fn fn = nullptr;
  static std::once_flag once;
  std::call_once(once, [] {
    void* p = nullptr;
    cudaDriverEntryPointQueryResult q;
    if (cudaGetDriverEntryPointByVersion("cuTensorMapEncodeTiled", &p, 12000, cudaEnableDefault, &q) == cudaSuccess &&
        q == cudaDriverEntryPointSuccess)
      fn = reinterpret_cast<serve_encode_fn>(p);
  });
  return fn;
}

aq_status check_kv_cache(const aq_kv_cache* c, const char* who) {
  if (!c) return serve_fail(AQ_ERR_INVALID_ARG, "%s: cache is NULL", who);
  if (c->type != AQ_KV_BF16 && c->type != AQ_KV_E4M3)
    return serve_fail(AQ_ERR_INVALID_ARG, "%s: unknown cache type %d", who, c->type);
  if (!c->k || !c->v) return serve_fail(AQ_ERR_INVALID_ARG, "%s: cache k and v must be non-NULL", who);
  if (c->pages < 1 || c->kv_heads < 1)
    return serve_fail(AQ_ERR_SHAPE, "%s: cache pages=%d kv_heads=%d must be >= 1", who, c->pages, c->kv_heads);
  if (c->page_size < 16 || c->page_size > 256 || (c->page_size & (c->page_size - 1)))
    return serve_fail(AQ_ERR_SHAPE, "%s: page_size=%d must be 16, 32, 64, 128 or 256", who, c->page_size);
  if (c->head_dim < 16 || c->head_dim > kServeMaxHeadDim || c->head_dim % 16)
    return serve_fail(AQ_ERR_SHAPE, "%s: cache head_dim=%d must be a multiple of 16 up to %d", who, c->head_dim,
                      kServeMaxHeadDim);
  if (!serve_aligned(c->k, 16) || !serve_aligned(c->v, 16))
    return serve_fail(AQ_ERR_ALIGNMENT, "%s: cache k and v must be 16-byte aligned", who);
  if (c->type == AQ_KV_E4M3) {
    if (!c->k_scale || !c->v_scale)
      return serve_fail(AQ_ERR_INVALID_ARG, "%s: an E4M3 cache needs k_scale and v_scale", who);
    if (!serve_aligned(c->k_scale, 16) || !serve_aligned(c->v_scale, 16))
      return serve_fail(AQ_ERR_ALIGNMENT, "%s: cache scales must be 16-byte aligned", who);
  } else if (c->k_scale || c->v_scale) {
    return serve_fail(AQ_ERR_INVALID_ARG, "%s: a bf16 cache has no scales", who);
  }
  if (byte_overlap(byte_span(c->k, 1, 0, kv_cells(c) * c->head_dim, kv_elem_bytes(c)),
                   byte_span(c->v, 1, 0, kv_cells(c) * c->head_dim, kv_elem_bytes(c))))
    return serve_fail(AQ_ERR_OVERLAP, "%s: cache k and v overlap", who);
  return AQ_OK;
}

aq_status check_rope_spec(const aq_rope_spec* r, int32_t head_dim, const char* who) {
  if (!r) return serve_fail(AQ_ERR_INVALID_ARG, "%s: rope is NULL", who);
  if (!r->freq) return serve_fail(AQ_ERR_INVALID_ARG, "%s: rope.freq must be non-NULL", who);
  if (!serve_aligned(r->freq, 8)) return serve_fail(AQ_ERR_ALIGNMENT, "%s: rope.freq must be 8-byte aligned", who);
  if (r->layout != AQ_ROPE_HALF && r->layout != AQ_ROPE_INTERLEAVED)
    return serve_fail(AQ_ERR_INVALID_ARG, "%s: unknown rope layout %d", who, r->layout);
  if (r->rotary_dim < 16 || r->rotary_dim % 16 || r->rotary_dim > head_dim)
    return serve_fail(AQ_ERR_SHAPE, "%s: rotary_dim=%d must be a multiple of 16 up to head_dim=%d", who, r->rotary_dim,
                      head_dim);
  return AQ_OK;
}

namespace {

// One call: up to three sets of heads over the same T tokens, walked as one list of heads:
// [0, hq) rotated and written to qo, then hk keys rotated and stored, then hk values stored.
struct PosParams {
  const uint16_t* q;
  int64_t q_tok, q_head;
  uint16_t* qo;
  int64_t qo_tok, qo_head;
  const uint16_t* k;
  int64_t k_tok, k_head;
  const uint16_t* v;
  int64_t v_tok, v_head;
  const int32_t* pos;
  const int64_t* slots;
  const uint64_t* freq;   // NULL: nothing is rotated
  uint8_t* kc;
  uint8_t* vc;
  float* ks;
  float* vs;
  int64_t T;
  int64_t n_slots;
  int32_t hq, hk, D;
  int32_t rot16;          // rotary_dim / 16
  float magnitude, sin_sign;
  int32_t page_shift;
  int32_t hl_shift;       // log2 of the groups that share a token, each taking every hl-th head
};

// GW lanes per vector (a power of two, >= D / 16).
// SPLIT: the groups of a warp are at one token. Four blocks an SM: a rotation of 8192 tokens takes 19.1 us, with three
// blocks 21.7, with five 25.3; the next heads' loads under these heads' work 20.6 (three) and 23.1 (four).
template <bool HALF, int GW, bool E4M3, bool SPLIT>
__global__ void __launch_bounds__(256, 4) aq_positions_kernel(const __grid_constant__ PosParams p) {
  pdl_wait_prior_grid();
  pdl_launch_dependents();
  const int u = threadIdx.x % GW;
  const int64_t item = static_cast<int64_t>(blockIdx.x) * (256 / GW) + threadIdx.x / GW;
  const int64_t t = item >> p.hl_shift;
  const int hl = 1 << p.hl_shift, h0 = static_cast<int>(item & (hl - 1));
  const int heads = p.hq + 2 * p.hk;
  const bool live = t < p.T && u * 16 < p.D;
  const int64_t tt = live ? t : 0;
  const Chunks<HALF> ch(u, p.rot16, p.D / 16);

  float c[8], s[8];
  const bool turn = p.freq != nullptr && (ch.turns0 || ch.turns1) && live && h0 < p.hq + p.hk;
  angles<HALF, GW, SPLIT>(ch, u, p.freq, p.freq && live ? p.pos[tt] : 0, p.magnitude, p.sin_sign, c, s);
  int64_t cell0 = -1;
  if (p.hk > 0 && live) {
    const int64_t slot = p.slots[tt];
    if (slot >= 0 && slot < p.n_slots)
      cell0 = (((slot >> p.page_shift) * p.hk) << p.page_shift) + (slot & ((1 << p.page_shift) - 1));
  }

  // groups of one warp may be at different kinds of heads, so each shuffles by itself
  const uint32_t group = (GW == 32 ? 0xffffffffu : (1u << GW) - 1) << ((threadIdx.x & 31) & ~(GW - 1));
  const int k0 = live ? ch.c0 : 0, k1 = live ? ch.c1 : 0;
  auto source = [&](int h) {
    if (h < p.hq) return p.q + tt * p.q_tok + h * p.q_head;
    if (h < p.hq + p.hk) return p.k + tt * p.k_tok + (h - p.hq) * p.k_head;
    return p.v + tt * p.v_tok + (h - p.hq - p.hk) * p.v_head;
  };
  auto finish = [&](int h, const uint4& r0, const uint4& r1) {
    const bool is_v = h >= p.hq + p.hk;
    const bool turns = turn && !is_v;
    if (h < p.hq && !turns) {   // nothing rotates in this lane's part
      uint16_t* dst = p.qo + tt * p.qo_tok + h * p.qo_head;
      if (live) *reinterpret_cast<uint4*>(dst + ch.c0 * 8) = r0;
      if (live) *reinterpret_cast<uint4*>(dst + ch.c1 * 8) = r1;
      return;
    }
    float a[8], b[8];
    unpack8(live ? r0 : make_uint4(0, 0, 0, 0), a);
    unpack8(live ? r1 : make_uint4(0, 0, 0, 0), b);
    if (turns) rotate16<HALF>(a, b, c, s, ch.turns1);
    if (h < p.hq) {
      uint16_t* dst = p.qo + tt * p.qo_tok + h * p.qo_head;
      if (live) *reinterpret_cast<uint4*>(dst + ch.c0 * 8) = pack8(a);
      if (live) *reinterpret_cast<uint4*>(dst + ch.c1 * 8) = pack8(b);
      return;
    }
    const int hh = h - p.hq - (is_v ? p.hk : 0);
    const int64_t cell = cell0 + (static_cast<int64_t>(hh) << p.page_shift);
    uint8_t* base = is_v ? p.vc : p.kc;
    if (!E4M3) {
      if (cell0 < 0) return;
      uint16_t* dst = reinterpret_cast<uint16_t*>(base) + cell * p.D;
      if (live) *reinterpret_cast<uint4*>(dst + ch.c0 * 8) = pack8(a);
      if (live) *reinterpret_cast<uint4*>(dst + ch.c1 * 8) = pack8(b);
      return;
    }
    // max|x| on the bit patterns: a NaN or infinity stays the largest
    uint32_t top = 0;
#pragma unroll
    for (int i = 0; i < 8; ++i)
      top = max(top, max(__float_as_uint(a[i]) & 0x7fffffffu, __float_as_uint(b[i]) & 0x7fffffffu));
#pragma unroll
    for (int o = GW / 2; o > 0; o >>= 1) top = max(top, __shfl_xor_sync(group, top, o));
    if (cell0 < 0) return;
    const bool finite = top < 0x7f800000u;
    const float scale = finite ? fmaxf(__uint_as_float(top) * (1.0f / kE4m3Max), kKvScaleFloor) : __uint_as_float(0x7fc00000u);
    const float inv = finite ? __frcp_rn(scale) : 0.0f;
    uint8_t* dst = base + cell * p.D;
    auto codes = [&](const float (&x)[8]) {
      if (!finite) return make_uint2(0, 0);
      return make_uint2(e4m3x2_from_f32(x[0] * inv, x[1] * inv) | (static_cast<uint32_t>(e4m3x2_from_f32(x[2] * inv, x[3] * inv)) << 16),
                        e4m3x2_from_f32(x[4] * inv, x[5] * inv) | (static_cast<uint32_t>(e4m3x2_from_f32(x[6] * inv, x[7] * inv)) << 16));
    };
    if (live) *reinterpret_cast<uint2*>(dst + ch.c0 * 8) = codes(a);
    if (live) *reinterpret_cast<uint2*>(dst + ch.c1 * 8) = codes(b);
    if (u == 0) (is_v ? p.vs : p.ks)[cell] = scale;
  };
  // two heads' loads in flight
  for (int h = h0; h < heads; h += 2 * hl) {
    const bool two = h + hl < heads;
    const uint16_t* s0 = source(h);
    const uint16_t* s1 = source(two ? h + hl : h);
    // lanes without work load lane 0's chunks: a load under a condition would be waited for at once
    const uint4 r0 = ld_stream(s0 + k0 * 8), r1 = ld_stream(s0 + k1 * 8), r2 = ld_stream(s1 + k0 * 8), r3 = ld_stream(s1 + k1 * 8);
    finish(h, r0, r1);
    if (two) finish(h + hl, r2, r3);
  }
}

struct ReadParams {
  const uint8_t* c[2];    // key and value codes
  const float* s[2];
  uint16_t* o[2];
  int64_t o_tok[2], o_head[2];
  const int64_t* slots;
  int64_t T, n_slots;
  int32_t hk, D, page_shift;
};

// One group of GW lanes per token and head, two chunks of eight elements of its key and of its value a lane (chunk u
// and chunk D / 16 + u: each load and store of the group covers one stretch), all four loads in flight. A slot outside the cache reads as zeros.
template <int GW, bool E4M3>
__global__ void __launch_bounds__(256) aq_kv_read_kernel(const __grid_constant__ ReadParams p) {
  pdl_wait_prior_grid();
  pdl_launch_dependents();
  const int u = threadIdx.x % GW;
  const int64_t item = static_cast<int64_t>(blockIdx.x) * (256 / GW) + threadIdx.x / GW;
  const int64_t t = item / p.hk;
  if (t >= p.T || u * 16 >= p.D) return;
  const int h = static_cast<int>(item - t * p.hk);
  const int64_t slot = p.slots[t];
  const bool held = slot >= 0 && slot < p.n_slots;
  const int64_t cell = ((((slot >> p.page_shift) * p.hk) + h) << p.page_shift) + (slot & ((1 << p.page_shift) - 1));
  uint4 r[2][2];
  float s[2];
#pragma unroll
  for (int w = 0; w < 2; ++w) {
    r[w][0] = r[w][1] = make_uint4(0, 0, 0, 0);
    s[w] = 0.0f;
    if (!p.o[w] || !held) continue;
    const uint8_t* src = p.c[w] + (cell * p.D + u * 8) * (E4M3 ? 1 : 2);
    if (E4M3) {
      s[w] = p.s[w][cell];
      const uint2 lo = *reinterpret_cast<const uint2*>(src), hi = *reinterpret_cast<const uint2*>(src + p.D / 2);
      r[w][0] = make_uint4(lo.x, lo.y, hi.x, hi.y);
    } else {
      r[w][0] = *reinterpret_cast<const uint4*>(src);
      r[w][1] = *reinterpret_cast<const uint4*>(src + p.D);
    }
  }
#pragma unroll
  for (int w = 0; w < 2; ++w) {
    if (!p.o[w]) continue;
    uint16_t* dst = p.o[w] + t * p.o_tok[w] + h * p.o_head[w] + u * 8;
    if (E4M3) {
      const uint32_t q[4] = {r[w][0].x, r[w][0].y, r[w][0].z, r[w][0].w};
      uint32_t o[8];
#pragma unroll
      for (int i = 0; i < 8; ++i) {
        const uint32_t f = f16x2_from_e4m3x2(static_cast<uint16_t>(q[i / 2] >> (16 * (i & 1))));
        const float2 v = __half22float2(*reinterpret_cast<const __half2*>(&f));
        o[i] = pack_bf16x2_cvt(v.x * s[w], v.y * s[w]);
      }
      r[w][0] = make_uint4(o[0], o[1], o[2], o[3]);
      r[w][1] = make_uint4(o[4], o[5], o[6], o[7]);
    }
    *reinterpret_cast<uint4*>(dst) = r[w][0];
    *reinterpret_cast<uint4*>(dst + p.D / 2) = r[w][1];
  }
}

template <bool HALF, int GW, bool E4M3>
cudaError_t launch_positions(const PosParams& p, unsigned blocks, cudaStream_t st) {
  if (GW < 32 && (GW << p.hl_shift) >= 32)
    return launch_serve(aq_positions_kernel<HALF, GW, E4M3, true>, p, blocks, 256, 0, st);
  return launch_serve(aq_positions_kernel<HALF, GW, E4M3, false>, p, blocks, 256, 0, st);
}
template <bool HALF, bool E4M3>
cudaError_t launch_positions(const PosParams& p, unsigned blocks, int gw, cudaStream_t st) {
  switch (gw) {
    case 1: return launch_positions<HALF, 1, E4M3>(p, blocks, st);
    case 2: return launch_positions<HALF, 2, E4M3>(p, blocks, st);
    case 4: return launch_positions<HALF, 4, E4M3>(p, blocks, st);
    case 8: return launch_positions<HALF, 8, E4M3>(p, blocks, st);
    default: return launch_positions<HALF, 16, E4M3>(p, blocks, st);
  }
}

template <bool E4M3>
cudaError_t launch_read(const ReadParams& p, unsigned grid, int gw, cudaStream_t st) {
  switch (gw) {
    case 1: return launch_serve(aq_kv_read_kernel<1, E4M3>, p, grid, 256, 0, st);
    case 2: return launch_serve(aq_kv_read_kernel<2, E4M3>, p, grid, 256, 0, st);
    case 4: return launch_serve(aq_kv_read_kernel<4, E4M3>, p, grid, 256, 0, st);
    case 8: return launch_serve(aq_kv_read_kernel<8, E4M3>, p, grid, 256, 0, st);
    default: return launch_serve(aq_kv_read_kernel<16, E4M3>, p, grid, 256, 0, st);
  }
}

// Grid of a positions launch.
aq_status run_positions(PosParams& p, bool half, bool e4m3, cudaStream_t st, const char* who) {
  ServeDev dev;
  aq_status s = serve_device(&dev);
  if (s != AQ_OK) return s;
  const int heads = p.hq + 2 * p.hk;
  const int gw = group_width(p.D);
  const int64_t fill = static_cast<int64_t>(dev.sms) * 1024 / gw;
  p.hl_shift = share_token(p.T, heads, gw, fill);
  const int64_t blocks = ((p.T << p.hl_shift) + 256 / gw - 1) / (256 / gw);
  if (blocks > 0x7fffffffLL) return serve_fail(AQ_ERR_SHAPE, "%s: %lld tokens are too many for one call", who, (long long)p.T);
  const unsigned g = static_cast<unsigned>(blocks);
  cudaError_t e = half ? (e4m3 ? launch_positions<true, true>(p, g, gw, st) : launch_positions<true, false>(p, g, gw, st))
                       : (e4m3 ? launch_positions<false, true>(p, g, gw, st) : launch_positions<false, false>(p, g, gw, st));
  return serve_launched(e, who);
}

}  // namespace
}  // namespace aq

using namespace aq;

extern "C" aq_status aq_rope_frequencies(int32_t rotary_dim, double base, int32_t scaling, const aq_rope_scaling* sc,
                                         uint64_t* freq, float* magnitude) {
  const char* who = "aq_rope_frequencies";
  if (!freq || !magnitude) return serve_fail(AQ_ERR_INVALID_ARG, "%s: NULL argument", who);
  if (rotary_dim < 2 || rotary_dim % 2 || rotary_dim > kServeMaxHeadDim)
    return serve_fail(AQ_ERR_SHAPE, "%s: rotary_dim=%d must be even, up to %d", who, rotary_dim, kServeMaxHeadDim);
  if (!(base > 1.0) || !isfinite(base)) return serve_fail(AQ_ERR_INVALID_ARG, "%s: base must be above 1", who);
  if (scaling < AQ_ROPE_SCALE_NONE || scaling > AQ_ROPE_SCALE_WAVELENGTH)
    return serve_fail(AQ_ERR_INVALID_ARG, "%s: unknown scaling %d", who, scaling);
  const double pi = 3.14159265358979323846, two_pi = 2 * pi;
  if (scaling != AQ_ROPE_SCALE_NONE) {
    if (!sc) return serve_fail(AQ_ERR_INVALID_ARG, "%s: scaling %d needs its parameters", who, scaling);
    if (!(sc->factor >= 1.0) || !isfinite(sc->factor))
      return serve_fail(AQ_ERR_INVALID_ARG, "%s: factor must be at least 1", who);
    if (scaling >= AQ_ROPE_SCALE_YARN &&
        (!(sc->original_len > 0) || !isfinite(sc->original_len) || !(sc->fast > sc->slow) || !(sc->slow > 0) || !isfinite(sc->fast)))
      return serve_fail(AQ_ERR_INVALID_ARG, "%s: need original_len > 0 and fast > slow > 0", who);
    if (scaling == AQ_ROPE_SCALE_NTK && rotary_dim <= 2)
      return serve_fail(AQ_ERR_SHAPE, "%s: AQ_ROPE_SCALE_NTK needs rotary_dim > 2", who);
  }
  const int half = rotary_dim / 2;
  double lo = 0, hi = 0;
  if (scaling == AQ_ROPE_SCALE_NTK) base *= pow(sc->factor, rotary_dim / (rotary_dim - 2.0));
  if (scaling == AQ_ROPE_SCALE_YARN) {
    auto dim_of = [&](double turns) { return rotary_dim * log(sc->original_len / (turns * two_pi)) / (2 * log(base)); };
    lo = std::max(floor(dim_of(sc->fast)), 0.0);
    hi = std::min(ceil(dim_of(sc->slow)), rotary_dim - 1.0);
  }
  for (int i = 0; i < half; ++i) {
    double f = pow(base, -2.0 * i / rotary_dim);
    if (scaling == AQ_ROPE_SCALE_LINEAR) f /= sc->factor;
    if (scaling == AQ_ROPE_SCALE_YARN) {
      const double ramp = std::min(std::max((i - lo) / std::max(hi - lo, 1e-3), 0.0), 1.0);
      f = f / sc->factor * ramp + f * (1 - ramp);
    }
    if (scaling == AQ_ROPE_SCALE_WAVELENGTH) {
      const double turns = sc->original_len * f / two_pi;   // over the original context
      const double keep = std::min(std::max((turns - sc->slow) / (sc->fast - sc->slow), 0.0), 1.0);
      f = f * keep + f / sc->factor * (1 - keep);
    }
    freq[i] = static_cast<uint64_t>(llrint(ldexp(f / two_pi, 64)));   // f <= 1: below 2^62
  }
  *magnitude = scaling == AQ_ROPE_SCALE_YARN ? static_cast<float>(0.1 * log(sc->factor) + 1.0) : 1.0f;
  return AQ_OK;
}

extern "C" aq_status aq_rope(const aq_rope_spec* rope, const int32_t* pos, int64_t T, int32_t heads, int32_t head_dim,
                             const void* x, int64_t x_tok, int64_t x_head, void* y, int64_t y_tok, int64_t y_head,
                             int32_t inverse, void* stream) {
  const char* who = "aq_rope";
  if (T < 0) return serve_fail(AQ_ERR_SHAPE, "%s: T=%lld is negative", who, (long long)T);
  if (heads < 1) return serve_fail(AQ_ERR_SHAPE, "%s: heads=%d must be >= 1", who, heads);
  if (head_dim < 16 || head_dim % 16 || head_dim > kServeMaxHeadDim)
    return serve_fail(AQ_ERR_SHAPE, "%s: head_dim=%d must be a multiple of 16 up to %d", who, head_dim, kServeMaxHeadDim);
  aq_status st = check_rope_spec(rope, head_dim, who);
  if (st != AQ_OK || (st = check_head_count(heads, who)) != AQ_OK) return st;
  if (T == 0) return AQ_OK;
  if (!pos) return serve_fail(AQ_ERR_INVALID_ARG, "%s: pos must be non-NULL", who);
  if ((st = check_heads(x, x_tok, x_head, heads, head_dim, "x", who)) != AQ_OK) return st;
  if ((st = check_heads(y, y_tok, y_head, heads, head_dim, "y", who)) != AQ_OK) return st;
  if ((st = check_out_heads(y_tok, y_head, T, heads, head_dim, "y", who)) != AQ_OK) return st;
  const ByteSpan ys = heads_span(y, y_tok, y_head, T, heads, head_dim);
  const bool same = x == y && (T == 1 || x_tok == y_tok) && (heads == 1 || x_head == y_head);
  if (!same && byte_overlap(heads_span(x, x_tok, x_head, T, heads, head_dim), ys))
    return serve_fail(AQ_ERR_OVERLAP, "%s: y overlaps x (in place needs the same pointer and strides)", who);
  if (byte_overlap(byte_span(pos, 1, 0, T, 4), ys) || byte_overlap(byte_span(rope->freq, 1, 0, rope->rotary_dim / 2, 8), ys))
    return serve_fail(AQ_ERR_OVERLAP, "%s: y overlaps pos or rope.freq", who);
  PosParams p = {};
  p.q = static_cast<const uint16_t*>(x);
  p.q_tok = x_tok;
  p.q_head = x_head;
  p.qo = static_cast<uint16_t*>(y);
  p.qo_tok = y_tok;
  p.qo_head = y_head;
  p.pos = pos;
  p.freq = rope->freq;
  p.T = T;
  p.hq = heads;
  p.D = head_dim;
  p.rot16 = rope->rotary_dim / 16;
  p.magnitude = rope->magnitude;
  p.sin_sign = inverse ? -rope->magnitude : rope->magnitude;
  return run_positions(p, rope->layout == AQ_ROPE_HALF, false, static_cast<cudaStream_t>(stream), who);
}

extern "C" aq_status aq_kv_write(const aq_kv_cache* cache, const int64_t* slots, int64_t T, const void* k, int64_t k_tok,
                                 int64_t k_head, const void* v, int64_t v_tok, int64_t v_head, const aq_rope_spec* rope,
                                 const int32_t* pos, const void* q, int32_t q_heads, int64_t q_tok, int64_t q_head,
                                 void* q_out, int64_t qo_tok, int64_t qo_head, void* stream) {
  return aq_kv_write_norm(cache, slots, T, k, k_tok, k_head, v, v_tok, v_head, rope, pos, q, q_heads, q_tok, q_head, q_out, qo_tok,
                          qo_head, nullptr, nullptr, stream);
}

extern "C" aq_status aq_kv_write_norm(const aq_kv_cache* cache, const int64_t* slots, int64_t T, const void* k, int64_t k_tok,
                                      int64_t k_head, const void* v, int64_t v_tok, int64_t v_head, const aq_rope_spec* rope,
                                      const int32_t* pos, const void* q, int32_t q_heads, int64_t q_tok, int64_t q_head,
                                      void* q_out, int64_t qo_tok, int64_t qo_head, const aq_head_norm* q_norm,
                                      const aq_head_norm* k_norm, void* stream) {
  const char* who = "aq_kv_write";
  aq_status st = check_kv_cache(cache, who);
  if (st != AQ_OK) return st;
  const int D = cache->head_dim;
  if (T < 0) return serve_fail(AQ_ERR_SHAPE, "%s: T=%lld is negative", who, (long long)T);
  if (rope && (st = check_rope_spec(rope, D, who)) != AQ_OK) return st;
  if (!q != !q_out) return serve_fail(AQ_ERR_INVALID_ARG, "%s: q and q_out go together", who);
  if (q && !rope && !q_norm) return serve_fail(AQ_ERR_INVALID_ARG, "%s: q is only normed and rotated here: it needs q_norm or rope", who);
  if (q_norm && !q) return serve_fail(AQ_ERR_INVALID_ARG, "%s: q_norm needs q", who);
  if ((st = check_head_norm(q_norm, "q_norm", who)) != AQ_OK || (st = check_head_norm(k_norm, "k_norm", who)) != AQ_OK) return st;
  if (q && q_heads < 1) return serve_fail(AQ_ERR_SHAPE, "%s: q_heads=%d must be >= 1", who, q_heads);
  if ((st = check_head_count(2ll * cache->kv_heads + (q ? q_heads : 0), who)) != AQ_OK) return st;
  if (T == 0) return AQ_OK;
  if (!slots) return serve_fail(AQ_ERR_INVALID_ARG, "%s: slots must be non-NULL", who);
  if (rope && !pos) return serve_fail(AQ_ERR_INVALID_ARG, "%s: rope needs pos", who);
  if ((st = check_heads(k, k_tok, k_head, cache->kv_heads, D, "k", who)) != AQ_OK) return st;
  if ((st = check_heads(v, v_tok, v_head, cache->kv_heads, D, "v", who)) != AQ_OK) return st;
  ByteSpan outs[5];
  int n = 0;
  outs[n++] = byte_span(cache->k, 1, 0, kv_cells(cache) * D, kv_elem_bytes(cache));
  outs[n++] = byte_span(cache->v, 1, 0, kv_cells(cache) * D, kv_elem_bytes(cache));
  outs[n++] = byte_span(cache->k_scale, 1, 0, kv_cells(cache), 4);
  outs[n++] = byte_span(cache->v_scale, 1, 0, kv_cells(cache), 4);
  bool same = false;
  if (q) {
    if ((st = check_heads(q, q_tok, q_head, q_heads, D, "q", who)) != AQ_OK) return st;
    if ((st = check_heads(q_out, qo_tok, qo_head, q_heads, D, "q_out", who)) != AQ_OK) return st;
    if ((st = check_out_heads(qo_tok, qo_head, T, q_heads, D, "q_out", who)) != AQ_OK) return st;
    outs[n++] = heads_span(q_out, qo_tok, qo_head, T, q_heads, D);
    same = q == q_out && (T == 1 || q_tok == qo_tok) && (q_heads == 1 || q_head == qo_head);
  }
  // In place, q_out may sit inside the stacked [q | k | v] rows of one projection output: its rows
  // are q's own, so k and v only have to lie beside them, which equal token strides make checkable.
  auto beside = [&](const void* x, int64_t x_tok, int64_t x_head) {
    if (!same || x_tok != q_tok || q_head * (q_heads - 1) + D > q_tok || x_head * (cache->kv_heads - 1) + D > x_tok) return false;
    const int64_t diff = (reinterpret_cast<intptr_t>(x) - reinterpret_cast<intptr_t>(q)) / 2;
    const int64_t col = ((diff % q_tok) + q_tok) % q_tok;
    return col >= q_head * (q_heads - 1) + D && col + x_head * (cache->kv_heads - 1) + D <= q_tok;
  };
  struct In {
    ByteSpan s;
    bool by_q;
  } ins[] = {{heads_span(k, k_tok, k_head, T, cache->kv_heads, D), beside(k, k_tok, k_head)},
             {heads_span(v, v_tok, v_head, T, cache->kv_heads, D), beside(v, v_tok, v_head)},
             {q ? heads_span(q, q_tok, q_head, T, q_heads, D) : ByteSpan(), same},
             {byte_span(slots, 1, 0, T, 8), false},
             {rope ? byte_span(pos, 1, 0, T, 4) : ByteSpan(), false},
             {rope ? byte_span(rope->freq, 1, 0, rope->rotary_dim / 2, 8) : ByteSpan(), false},
             {q_norm ? byte_span(q_norm->weight, 1, 0, D, 2) : ByteSpan(), false},
             {k_norm ? byte_span(k_norm->weight, 1, 0, D, 2) : ByteSpan(), false}};
  for (int i = 0; i < n; ++i) {
    for (const In& in : ins)
      if (!(i == 4 && in.by_q) && byte_overlap(outs[i], in.s))
        return serve_fail(AQ_ERR_OVERLAP, "%s: an output overlaps an input", who);
    for (int j = 0; j < i; ++j)
      if (byte_overlap(outs[i], outs[j])) return serve_fail(AQ_ERR_OVERLAP, "%s: two outputs overlap", who);
  }
  if (q_norm || k_norm) {
    const aq_heads hq = {const_cast<void*>(q), q_tok, q_head, q ? q_heads : 0}, ho = {q_out, qo_tok, qo_head, q ? q_heads : 0},
                   hk = {const_cast<void*>(k), k_tok, k_head, cache->kv_heads}, hv = {const_cast<void*>(v), v_tok, v_head, cache->kv_heads};
    return run_head_norm(q_norm, k_norm, rope, pos, T, D, q ? &hq : nullptr, &ho, &hk, nullptr, &hv, cache, slots, static_cast<cudaStream_t>(stream), who);
  }
  PosParams p = {};
  p.q = static_cast<const uint16_t*>(q);
  p.q_tok = q_tok;
  p.q_head = q_head;
  p.qo = static_cast<uint16_t*>(q_out);
  p.qo_tok = qo_tok;
  p.qo_head = qo_head;
  p.k = static_cast<const uint16_t*>(k);
  p.k_tok = k_tok;
  p.k_head = k_head;
  p.v = static_cast<const uint16_t*>(v);
  p.v_tok = v_tok;
  p.v_head = v_head;
  p.pos = pos;
  p.slots = slots;
  p.kc = static_cast<uint8_t*>(cache->k);
  p.vc = static_cast<uint8_t*>(cache->v);
  p.ks = cache->k_scale;
  p.vs = cache->v_scale;
  p.T = T;
  p.n_slots = static_cast<int64_t>(cache->pages) * cache->page_size;
  p.hq = q ? q_heads : 0;
  p.hk = cache->kv_heads;
  p.D = D;
  p.page_shift = log2_of(cache->page_size);
  if (rope) {
    p.freq = rope->freq;
    p.rot16 = rope->rotary_dim / 16;
    p.magnitude = rope->magnitude;
    p.sin_sign = rope->magnitude;
  }
  return run_positions(p, rope && rope->layout == AQ_ROPE_HALF, cache->type == AQ_KV_E4M3,
                       static_cast<cudaStream_t>(stream), who);
}

extern "C" aq_status aq_kv_read(const aq_kv_cache* cache, const int64_t* slots, int64_t T, void* k, int64_t k_tok,
                                int64_t k_head, void* v, int64_t v_tok, int64_t v_head, void* stream) {
  const char* who = "aq_kv_read";
  aq_status st = check_kv_cache(cache, who);
  if (st != AQ_OK) return st;
  const int D = cache->head_dim, hk = cache->kv_heads;
  if (T < 0) return serve_fail(AQ_ERR_SHAPE, "%s: T=%lld is negative", who, (long long)T);
  if (!k && !v) return serve_fail(AQ_ERR_INVALID_ARG, "%s: k and v are both NULL", who);
  if (T == 0) return AQ_OK;
  if (!slots) return serve_fail(AQ_ERR_INVALID_ARG, "%s: slots must be non-NULL", who);
  ByteSpan outs[2];
  if (k) {
    if ((st = check_heads(k, k_tok, k_head, hk, D, "k", who)) != AQ_OK) return st;
    if ((st = check_out_heads(k_tok, k_head, T, hk, D, "k", who)) != AQ_OK) return st;
    outs[0] = heads_span(k, k_tok, k_head, T, hk, D);
  }
  if (v) {
    if ((st = check_heads(v, v_tok, v_head, hk, D, "v", who)) != AQ_OK) return st;
    if ((st = check_out_heads(v_tok, v_head, T, hk, D, "v", who)) != AQ_OK) return st;
    outs[1] = heads_span(v, v_tok, v_head, T, hk, D);
  }
  const ByteSpan ins[] = {byte_span(cache->k, 1, 0, kv_cells(cache) * D, kv_elem_bytes(cache)),
                          byte_span(cache->v, 1, 0, kv_cells(cache) * D, kv_elem_bytes(cache)),
                          byte_span(cache->k_scale, 1, 0, kv_cells(cache), 4),
                          byte_span(cache->v_scale, 1, 0, kv_cells(cache), 4), byte_span(slots, 1, 0, T, 8)};
  // k and v as column slices of one [k | v] buffer interleave: only equal token strides show them apart
  bool apart = !byte_overlap(outs[0], outs[1]);
  if (!apart && k_tok == v_tok && k_tok >= k_head * (hk - 1) + D) {
    const int64_t diff = (reinterpret_cast<intptr_t>(v) - reinterpret_cast<intptr_t>(k)) / 2;
    const int64_t col = ((diff % k_tok) + k_tok) % k_tok;
    apart = col >= k_head * (hk - 1) + D && col + v_head * (hk - 1) + D <= k_tok;
  }
  if (!apart) return serve_fail(AQ_ERR_OVERLAP, "%s: k and v overlap", who);
  for (const ByteSpan& o : outs)
    for (const ByteSpan& i : ins)
      if (byte_overlap(o, i)) return serve_fail(AQ_ERR_OVERLAP, "%s: an output overlaps an input", who);
  ServeDev dev;
  if ((st = serve_device(&dev)) != AQ_OK) return st;
  ReadParams p = {};
  p.c[0] = static_cast<const uint8_t*>(cache->k);
  p.c[1] = static_cast<const uint8_t*>(cache->v);
  p.s[0] = cache->k_scale;
  p.s[1] = cache->v_scale;
  p.o[0] = static_cast<uint16_t*>(k);
  p.o[1] = static_cast<uint16_t*>(v);
  p.o_tok[0] = k_tok;
  p.o_tok[1] = v_tok;
  p.o_head[0] = k_head;
  p.o_head[1] = v_head;
  p.slots = slots;
  p.T = T;
  p.n_slots = static_cast<int64_t>(cache->pages) * cache->page_size;
  p.hk = hk;
  p.D = D;
  p.page_shift = log2_of(cache->page_size);
  const int gw = group_width(D);
  const int64_t blocks = (T * hk + 256 / gw - 1) / (256 / gw);
  if (blocks > 0x7fffffffLL) return serve_fail(AQ_ERR_SHAPE, "%s: %lld tokens are too many for one call", who, (long long)T);
  const unsigned grid = static_cast<unsigned>(blocks);
  const cudaStream_t cs = static_cast<cudaStream_t>(stream);
  return serve_launched(cache->type == AQ_KV_E4M3 ? launch_read<true>(p, grid, gw, cs) : launch_read<false>(p, grid, gw, cs), who);
}
