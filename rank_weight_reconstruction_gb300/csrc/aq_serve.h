// aq_serve.h -- what the serving operators (rotary positions, the paged key/value cache, attention
// of drafted tokens, draft verification) share: the device check, the error text, launches with
// programmatic dependent launch, and addressing inside a cache. Not part of the public ABI.
#pragma once

#include <cuda_runtime.h>
#include <stdarg.h>
#include <stdint.h>
#include <stdio.h>

#include "aq.h"
#include "aq_internal.h"
#include "aq_ptx.cuh"

namespace aq {

constexpr int kServeMaxHeadDim = 256;
constexpr float kE4m3Max = 448.0f;
// Smallest scale stored with a quantised vector: its reciprocal stays finite, and a zero vector
// needs no case of its own (codes 0).
constexpr float kKvScaleFloor = 0x1p-100f;

constexpr uint64_t kServeTimeoutNs = 1000ull * 1000 * 1000;   // limit of one in-kernel wait: 1 s

struct ServeDev {
  int index = 0, sms = 0;
  size_t smem_optin = 0;
  int32_t* status = nullptr;   // device status word
};
// Facts of the current device, queried once; refuses any device but sm_103.
aq_status serve_device(ServeDev* out);
// The driver's tensor-map encoder, or NULL.
typedef CUresult (*serve_encode_fn)(CUtensorMap*, CUtensorMapDataType, cuuint32_t, void*, const cuuint64_t*,
                                    const cuuint64_t*, const cuuint32_t*, const cuuint32_t*, CUtensorMapInterleave,
                                    CUtensorMapSwizzle, CUtensorMapL2promotion, CUtensorMapFloatOOBfill);
serve_encode_fn serve_encode();

inline aq_status serve_fail(aq_status st, const char* fmt, ...) {
  char buf[512];
  va_list ap;
  va_start(ap, fmt);
  vsnprintf(buf, sizeof buf, fmt, ap);
  va_end(ap);
  return static_cast<aq_status>(set_last_error(st, buf));
}
inline aq_status serve_launched(cudaError_t e, const char* what) {
  return e == cudaSuccess ? AQ_OK
                          : serve_fail(AQ_ERR_CUDA, "%s: %s (%s)", what, cudaGetErrorName(e), cudaGetErrorString(e));
}
inline bool serve_aligned(const void* p, uintptr_t n) { return (reinterpret_cast<uintptr_t>(p) & (n - 1)) == 0; }

// One launch whose prologue may overlap the tail of the previous kernel in the stream; every
// kernel launched this way calls pdl_wait_prior_grid() before it touches memory, but for the codes and scales
// of NVFP4 weights, which the products read ahead of it (what may write them: aq.h, at the top).
template <typename P>
cudaError_t launch_serve(void (*kernel)(P), const P& p, dim3 grid, int threads, size_t smem, cudaStream_t st,
                         int cluster = 1) {
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = grid;
  cfg.blockDim = dim3(threads);
  cfg.dynamicSmemBytes = smem;
  cfg.stream = st;
  cudaLaunchAttribute at[2] = {};
  at[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  at[0].val.programmaticStreamSerializationAllowed = 1;
  cfg.attrs = at;
  cfg.numAttrs = 1;
  if (cluster > 1) {
    at[1].id = cudaLaunchAttributeClusterDimension;
    at[1].val.clusterDim.x = cluster;
    at[1].val.clusterDim.y = 1;
    at[1].val.clusterDim.z = 1;
    cfg.numAttrs = 2;
  }
  return cudaLaunchKernelEx(&cfg, kernel, p);
}

// Bytes [base, base + n) of a buffer, for overlap checks (strided tensors: their whole extent).
struct ByteSpan {
  uintptr_t base = 0;
  uint64_t bytes = 0;
};
inline ByteSpan byte_span(const void* p, int64_t rows, int64_t stride, int64_t cols, int64_t size) {
  ByteSpan s;
  if (p && rows > 0 && cols > 0) {
    s.base = reinterpret_cast<uintptr_t>(p);
    s.bytes = static_cast<uint64_t>(((rows - 1) * stride + cols) * size);
  }
  return s;
}
inline bool byte_overlap(const ByteSpan& a, const ByteSpan& b) {
  return a.bytes && b.bytes && a.base < b.base + b.bytes && b.base < a.base + a.bytes;
}

// Rows of a strided matrix, in bytes. Equal strides tell column slices of one buffer apart; otherwise their whole extents
// are compared.
struct ByteRows {
  uintptr_t base = 0;
  int64_t rows = 0, stride = 0, bytes = 0;
  ByteRows() = default;
  ByteRows(const void* p, int64_t r, int64_t st, int64_t by) : base(reinterpret_cast<uintptr_t>(p)), rows(p ? r : 0), stride(st), bytes(by) {}
  uintptr_t end() const { return base + static_cast<uintptr_t>((rows - 1) * stride + bytes); }
  bool meets(const ByteRows& b) const {
    if (rows < 1 || bytes < 1 || b.rows < 1 || b.bytes < 1 || end() <= b.base || b.end() <= base) return false;
    if (stride != b.stride || bytes >= stride || b.bytes >= stride) return true;
    const int64_t d = static_cast<int64_t>(b.base - base) % stride, c = d < 0 ? d + stride : d;   // b's first column in this one's rows
    return c < bytes || c + b.bytes > stride;
  }
};

// Checks of an aq_kv_cache that every call taking one makes.
aq_status check_kv_cache(const aq_kv_cache* c, const char* who);
// Bytes of one of its two code arrays.
inline int64_t kv_cells(const aq_kv_cache* c) {
  return static_cast<int64_t>(c->pages) * c->kv_heads * c->page_size;
}
inline int kv_elem_bytes(const aq_kv_cache* c) { return c->type == AQ_KV_BF16 ? 2 : 1; }
aq_status check_rope_spec(const aq_rope_spec* r, int32_t head_dim, const char* who);

// Two fp32 values to a pair of E4M3 codes (nearest, ties to even, saturating); lo in the low byte.
__device__ __forceinline__ uint16_t e4m3x2_from_f32(float lo, float hi) {
  uint16_t r;
  asm("cvt.rn.satfinite.e4m3x2.f32 %0, %1, %2;" : "=h"(r) : "f"(hi), "f"(lo));
  return r;
}
// A pair of E4M3 codes to a pair of halves (exact).
__device__ __forceinline__ uint32_t f16x2_from_e4m3x2(uint16_t c) {
  uint32_t r;
  asm("cvt.rn.f16x2.e4m3x2 %0, %1;" : "=r"(r) : "h"(c));
  return r;
}

}  // namespace aq
