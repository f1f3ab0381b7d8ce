// Dense attention over the paged cache (decode and verify).
//
//   o = sum_t softmax_t(c q . k_t) v_t   over  max(0, p - window + 1) <= t <= p,
//   lse = ln sum_t exp(c q . k_t)
//
// One warp takes one (query, head) row and one of `splits` equal parts of its
// positions, with a running maximum and sum (exp2 domain, FP32); a second
// kernel joins the parts of a row in order.
#include <algorithm>

#include "qsa_kv_internal.cuh"

namespace qsa {
namespace {

constexpr float kLog2e = 1.4426950408889634f;
constexpr float kLn2 = 0.6931471805599453f;
constexpr float kNegInf = -__builtin_huge_valf();

struct DenseArgs {
  const __nv_bfloat16* q;
  const uint8_t* k_cache;
  const uint8_t* v_cache;
  const float* k_scale;
  const float* v_scale;
  const int32_t* page_table;
  const int32_t* q_pos;
  __nv_bfloat16* out;
  float* lse;
  float* parts;  // [row][splits][2 + D]: maximum, sum, accumulator
  int32_t* err;
  int rows, splits, n_q, n_q_heads, n_kv_heads, page_size, max_pages, num_pages, window;
  float sm_scale;
};

template <int E>
__device__ __forceinline__ void load_vals(const uint8_t* cache, long long at, bool fp8, float (&f)[E]) {
  if (fp8) {
#pragma unroll
    for (int e = 0; e < E; e += 2) {
      const float2 v = h2_to_f2(e4m3x2_to_h2(*reinterpret_cast<const uint16_t*>(cache + at + e)));
      f[e] = v.x;
      f[e + 1] = v.y;
    }
  } else {
#pragma unroll
    for (int e = 0; e < E; e += 2) {
      const uint32_t w = *reinterpret_cast<const uint32_t*>(cache + 2 * (at + e));
      f[e] = bf_lo(w);
      f[e + 1] = bf_hi(w);
    }
  }
}

template <int D, bool FP8>
__global__ void __launch_bounds__(128) dense_part_kernel(const DenseArgs a) {
  constexpr int E = D / 32;
  const int lane = threadIdx.x & 31;
  const long long w = (long long)blockIdx.x * 4 + (threadIdx.x >> 5);
  if (w >= (long long)a.rows * a.splits) return;
  const int row = (int)(w / a.splits), split = (int)(w - (long long)row * a.splits);
  const int rj = row / a.n_q_heads, h = row - rj * a.n_q_heads, r = rj / a.n_q;
  const int g = h / (a.n_q_heads / a.n_kv_heads);
  int p = a.q_pos[rj];
  if (p < -1 || p >= a.max_pages * a.page_size) {
    if (h == 0 && split == 0 && lane == 0) record_error(a.err, kErrQueryPos, r, rj - r * a.n_q, p);
    p = -1;
  }
  const int lo = a.window > 0 ? max(0, p - a.window + 1) : 0;
  const long long n = p + 1 - lo;
  const int t0 = lo + (int)(n * split / a.splits), t1 = lo + (int)(n * (split + 1) / a.splits);
  float q[E], acc[E];
  const __nv_bfloat16* qp = a.q + (long long)row * D + lane * E;
  const float c = a.sm_scale * kLog2e * (FP8 ? a.k_scale[g] : 1.f);
#pragma unroll
  for (int e = 0; e < E; ++e) {
    q[e] = __bfloat162float(qp[e]);
    acc[e] = 0.f;
  }
  float m = kNegInf, l = 0.f;
  for (int t = t0; t < t1; ++t) {
    const int page = a.page_table[(long long)r * a.max_pages + t / a.page_size];
    if ((unsigned)page >= (unsigned)a.num_pages) {
      if (lane == 0) record_error(a.err, kErrPage, r, rj - r * a.n_q, page);
      continue;
    }
    const long long at =
        (((long long)page * a.n_kv_heads + g) * a.page_size + t % a.page_size) * D + lane * E;
    float k[E], v[E];
    load_vals<E>(a.k_cache, at, FP8, k);
    load_vals<E>(a.v_cache, at, FP8, v);
    float s = 0.f;
#pragma unroll
    for (int e = 0; e < E; ++e) s = fmaf(q[e], k[e], s);
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) s += __shfl_xor_sync(0xffffffffu, s, o);
    s *= c;
    const float mn = fmaxf(m, s), mu = mn == kNegInf ? 0.f : mn;
    const float f = exp2f(m - mu), x = exp2f(s - mu);
    l = l * f + x;
#pragma unroll
    for (int e = 0; e < E; ++e) acc[e] = acc[e] * f + x * v[e];
    m = mn;
  }
  float* part = a.parts + w * (2 + D);
  if (lane == 0) {
    part[0] = m;
    part[1] = l;
  }
#pragma unroll
  for (int e = 0; e < E; ++e) part[2 + lane * E + e] = acc[e];
}

template <int D, bool FP8>
__global__ void __launch_bounds__(128) dense_join_kernel(const DenseArgs a) {
  constexpr int E = D / 32;
  const int lane = threadIdx.x & 31;
  const int row = blockIdx.x * 4 + (threadIdx.x >> 5);
  if (row >= a.rows) return;
  const int h = row % a.n_q_heads, g = h / (a.n_q_heads / a.n_kv_heads);
  const float* part = a.parts + (long long)row * a.splits * (2 + D);
  float m = kNegInf, l = 0.f, acc[E];
  for (int s = 0; s < a.splits; ++s) m = fmaxf(m, part[(long long)s * (2 + D)]);
  const float mu = m == kNegInf ? 0.f : m;
#pragma unroll
  for (int e = 0; e < E; ++e) acc[e] = 0.f;
  for (int s = 0; s < a.splits; ++s) {
    const float* ps = part + (long long)s * (2 + D);
    const float f = exp2f(ps[0] - mu);
    if (f == 0.f) continue;
    l += f * ps[1];
#pragma unroll
    for (int e = 0; e < E; ++e) acc[e] += f * ps[2 + lane * E + e];
  }
  const float scale = l > 0.f || l != l ? (FP8 ? a.v_scale[g] : 1.f) / l : 0.f;
  __nv_bfloat16* o = a.out + (long long)row * D + lane * E;
#pragma unroll
  for (int e = 0; e < E; ++e) o[e] = __float2bfloat16_rn(l == 0.f ? 0.f : acc[e] * scale);
  if (a.lse && lane == 0) a.lse[row] = l == 0.f ? kNegInf : (m + log2f(l)) * kLn2;
}

int splits_of(const qsa_dims& d, int num_sms) {
  const long long rows = (long long)d.batch * d.n_q * d.n_q_heads;
  return (int)std::max<long long>(1, std::min<long long>(64, 32LL * num_sms / rows));
}

template <int D, bool FP8>
cudaError_t launch(const DenseArgs& a, cudaStream_t s) {
  const long long warps = (long long)a.rows * a.splits;
  const cudaError_t e =
      launch_k(dense_part_kernel<D, FP8>, dim3((unsigned)((warps + 3) / 4)), dim3(128), 0, s, false, a);
  if (e != cudaSuccess) return e;
  return launch_k(dense_join_kernel<D, FP8>, dim3((unsigned)((a.rows + 3) / 4)), dim3(128), 0, s, false, a);
}

}  // namespace

DenseWs dense_ws(const qsa_dims& d, int num_sms) {
  DenseWs w;
  w.parts = 256 + align_up((size_t)d.batch * d.n_q * d.n_kv_heads * sizeof(int32_t), 256);
  const size_t rows = (size_t)d.batch * d.n_q * d.n_q_heads;
  w.total = align_up(w.parts + rows * splits_of(d, num_sms) * (2 + d.head_dim) * sizeof(float), 256);
  return w;
}

cudaError_t launch_paged_attn(const qsa_dims& d, int window, const void* q, const void* k_cache, const void* v_cache,
                              const float* k_scale, const float* v_scale, const int32_t* page_table,
                              const int32_t* q_pos, void* out, float* lse, void* ws, cudaStream_t s) {
  const int sms = device_sm_count();
  DenseArgs a = {};
  a.q = static_cast<const __nv_bfloat16*>(q);
  a.k_cache = static_cast<const uint8_t*>(k_cache);
  a.v_cache = static_cast<const uint8_t*>(v_cache);
  a.k_scale = k_scale;
  a.v_scale = v_scale;
  a.page_table = page_table;
  a.q_pos = q_pos;
  a.out = static_cast<__nv_bfloat16*>(out);
  a.lse = lse;
  a.parts = reinterpret_cast<float*>(static_cast<uint8_t*>(ws) + dense_ws(d, sms).parts);
  a.err = static_cast<int32_t*>(ws);
  a.rows = d.batch * d.n_q * d.n_q_heads;
  a.splits = splits_of(d, sms);
  a.n_q = d.n_q;
  a.n_q_heads = d.n_q_heads;
  a.n_kv_heads = d.n_kv_heads;
  a.page_size = d.page_size;
  a.max_pages = d.max_pages;
  a.num_pages = d.num_pages;
  a.window = window;
  a.sm_scale = d.sm_scale > 0.f ? d.sm_scale : 1.f / sqrtf((float)d.head_dim);
  const bool fp8 = d.kv_dtype == QSA_KV_FP8_E4M3;
  switch (d.head_dim) {
    case 64: return fp8 ? launch<64, true>(a, s) : launch<64, false>(a, s);
    case 128: return fp8 ? launch<128, true>(a, s) : launch<128, false>(a, s);
    default: return fp8 ? launch<256, true>(a, s) : launch<256, false>(a, s);
  }
}

}  // namespace qsa
