// Declarations shared by the translation units of the entry points in qsa_kv.h.
#pragma once

#include <initializer_list>

#include "qsa_internal.cuh"
#include "qsa_kv.h"

namespace qsa {

constexpr int kErrOrder = 6;  // qsa_kv_append: a request's tokens are not consecutive

// the checks of qsa_dims that all entry points round the cache begin with
qsa_status check_kv_dims(const qsa_dims* d);

inline bool aligned(const void* p, uintptr_t a) { return (reinterpret_cast<uintptr_t>(p) & (a - 1)) == 0; }
inline bool aligned_all(uintptr_t a, std::initializer_list<const void*> ps) {
  for (const void* p : ps)
    if (!aligned(p, a)) return false;
  return true;
}
inline bool check_header(const void* ws, size_t bytes) { return ws && aligned(ws, 256) && bytes >= 256; }
inline qsa_status from_cuda(cudaError_t e) { return e == cudaSuccess ? QSA_OK : QSA_ERR_CUDA; }

// A rotation, or none (turns null).
struct Rope {
  const uint64_t* turns;
  float amplitude;
  int rot_dim, interleaved;
};

// [batch][token][head][dim] BF16 with element strides
struct Strided {
  __nv_bfloat16* p;
  long long batch, token, head;
};

cudaError_t launch_rope(const Rope& rope, int batch, int n_tok, int n_heads, int head_dim, bool inverse,
                        const Strided& x, const int32_t* pos, const Strided& y, cudaStream_t s);
cudaError_t launch_kv_append(const qsa_dims& d, int n_tok, const Rope& rope, const Strided& k, const Strided& v,
                             const Strided& q, const Strided& q_out, const int32_t* pos, const int32_t* page_table,
                             void* k_cache, void* v_cache, const float* k_scale, const float* v_scale, int32_t* err,
                             cudaStream_t s);
cudaError_t launch_kv_gather(const qsa_dims& d, int n_tok, const void* k_cache, const void* v_cache,
                             const float* k_scale, const float* v_scale, const int32_t* page_table,
                             const int32_t* pos, void* k_out, void* v_out, int32_t* err, cudaStream_t s);

// Workspace of qsa_paged_attn behind the header and the ticket counters that
// qsa.h's entry points keep there for the same dims.
struct DenseWs {
  size_t units, parts, total;
};
DenseWs dense_ws(const qsa_dims& d, int num_sms);
// The pages of positions below `len`, for every request (null: none, len 0).
// alone: 1 every request reads them by itself, 0 they are read once for all, -1 by their bytes.
struct Prefix {
  const int32_t* table;
  int len, alone;
};
size_t prefix_ws(const qsa_dims& d, int prefix_len, int num_sms);  // bytes of workspace with a prefix
// short_k: the failure-detection tests (qsa_test_paged_attn_timeout; with a prefix
// that is read once, its kernel's copies: qsa_test_prefix_attn_timeout)
cudaError_t launch_paged_attn(const qsa_dims& d, int window, const void* q, const void* k_cache, const void* v_cache,
                              const float* k_scale, const float* v_scale, const int32_t* page_table,
                              const int32_t* q_pos, void* out, float* lse, void* ws, cudaStream_t s,
                              bool short_k = false, const Prefix& prefix = Prefix{nullptr, 0, -1});

// 16-byte loads and stores of streamed data
__device__ __forceinline__ uint4 ld16(const void* p) { return *reinterpret_cast<const uint4*>(p); }
__device__ __forceinline__ uint2 ld8(const void* p) { return *reinterpret_cast<const uint2*>(p); }

__device__ __forceinline__ float bf_lo(uint32_t w) { return __uint_as_float(w << 16); }
__device__ __forceinline__ float bf_hi(uint32_t w) { return __uint_as_float(w & 0xffff0000u); }
__device__ __forceinline__ uint32_t pack_bf(float lo, float hi) {
  const __nv_bfloat162 h = __floats2bfloat162_rn(lo, hi);
  return *reinterpret_cast<const uint32_t*>(&h);
}

// two FP32 values -> two E4M3 codes (lo in bits 0-7), to nearest even,
// clamped to +-448, NaN kept
__device__ __forceinline__ uint32_t e4m3x2(float lo, float hi) {
  uint16_t r;
  asm("cvt.rn.satfinite.e4m3x2.f32 %0, %1, %2;" : "=h"(r) : "f"(hi), "f"(lo));
  return r;
}
// two E4M3 codes -> two FP16 values (exact)
__device__ __forceinline__ uint32_t e4m3x2_to_h2(uint32_t w) {
  uint32_t r;
  asm("cvt.rn.f16x2.e4m3x2 %0, %1;" : "=r"(r) : "h"((uint16_t)w));
  return r;
}
__device__ __forceinline__ float2 h2_to_f2(uint32_t w) {
  return __half22float2(*reinterpret_cast<const __half2*>(&w));
}

// arithmetic on pairs of FP32 values: one instruction each
__device__ __forceinline__ uint64_t pack2(float2 v) {
  uint64_t r;
  asm("mov.b64 %0, {%1, %2};" : "=l"(r) : "f"(v.x), "f"(v.y));
  return r;
}
__device__ __forceinline__ float2 unpack2(uint64_t v) {
  float2 r;
  asm("mov.b64 {%0, %1}, %2;" : "=f"(r.x), "=f"(r.y) : "l"(v));
  return r;
}
__device__ __forceinline__ float2 add2(float2 a, float2 b) {
  uint64_t r;
  asm("add.rn.f32x2 %0, %1, %2;" : "=l"(r) : "l"(pack2(a)), "l"(pack2(b)));
  return unpack2(r);
}
__device__ __forceinline__ float2 mul2(float2 a, float2 b) {
  uint64_t r;
  asm("mul.rn.f32x2 %0, %1, %2;" : "=l"(r) : "l"(pack2(a)), "l"(pack2(b)));
  return unpack2(r);
}
__device__ __forceinline__ float2 fma2(float2 a, float2 b, float2 c) {
  uint64_t r;
  asm("fma.rn.f32x2 %0, %1, %2, %3;" : "=l"(r) : "l"(pack2(a)), "l"(pack2(b)), "l"(pack2(c)));
  return unpack2(r);
}

}  // namespace qsa
