// The attention weight that each cached position gets from the newest tokens:
//   w[t] = decay w[t] + sum_{j, h} exp(c q_jh . k_t - lse_jh).
// A warp takes a position and goes through all query rows.
#include "qsa_serve_internal.cuh"

namespace qsa {
namespace {

constexpr unsigned kFull = 0xffffffffu;

struct WeightArgs {
  const __nv_bfloat16* q;
  const uint8_t* k_cache;
  const float* k_scale;
  const int32_t* page_table;
  const int32_t* q_pos;
  const float* lse;
  float* weight;
  int32_t* err;
  int batch, n_q, hq, hk, head_dim, page_size, max_pages, num_pages;
  float decay, scale;
};

template <bool FP8>
__global__ void __launch_bounds__(128) weight_kernel(const WeightArgs a) {
  const int lane = threadIdx.x & 31, r = blockIdx.y, cap = a.max_pages * a.page_size;
  pdl_wait();
  int most = -1;
  for (int j = 0; j < a.n_q; ++j) {
    const int p = a.q_pos[(long long)r * a.n_q + j];
    if (p >= cap || p < -1) {
      if (blockIdx.x == 0 && threadIdx.x == 0) record_error(a.err, kErrQueryPos, r, j, p);
    } else {
      most = max(most, p);
    }
  }
  for (int t = blockIdx.x * 4 + (threadIdx.x >> 5); t <= most; t += gridDim.x * 4) {
    const int page = a.page_table[(long long)r * a.max_pages + t / a.page_size];
    float sum = 0.f;
    if ((unsigned)page >= (unsigned)a.num_pages) {
      if (lane == 0) record_error(a.err, kErrPage, r, 0, page);
    } else {
      for (int g = 0; g < a.hk; ++g) {
        const long long row = (((long long)page * a.hk + g) * a.page_size + t % a.page_size) * a.head_dim;
        const float c = a.scale * (FP8 ? a.k_scale[g] : 1.f);
        for (int j = 0; j < a.n_q; ++j) {
          const int p = a.q_pos[(long long)r * a.n_q + j];
          if (p < t || p >= cap) continue;
          for (int h = g * (a.hq / a.hk); h < (g + 1) * (a.hq / a.hk); ++h) {
            const long long qrow = ((long long)r * a.n_q + j) * a.hq + h;
            float s = 0.f;
            for (int d = lane; d < a.head_dim; d += 32) {
              const float k = FP8 ? h2_to_f2(e4m3x2_to_h2(a.k_cache[row + d])).x
                                  : __bfloat162float(reinterpret_cast<const __nv_bfloat16*>(a.k_cache)[row + d]);
              s = fmaf(k, __bfloat162float(a.q[qrow * a.head_dim + d]), s);
            }
#pragma unroll
            for (int o = 16; o > 0; o >>= 1) s += __shfl_xor_sync(kFull, s, o);
            const float l = a.lse[qrow];
            if (l > -__builtin_huge_valf() || l != l) sum += expf(s * c - l);
          }
        }
      }
    }
    if (lane == 0) {
      float* w = a.weight + (long long)r * cap + t;
      *w = a.decay == 0.f ? sum : fmaf(a.decay, *w, sum);
    }
  }
}

}  // namespace

cudaError_t launch_kv_weight(const qsa_dims& d, float decay, const void* q, const void* k_cache, const float* k_scale,
                             const int32_t* page_table, const int32_t* q_pos, const float* lse, float* weight,
                             int32_t* err, cudaStream_t s) {
  WeightArgs a = {};
  a.q = static_cast<const __nv_bfloat16*>(q);
  a.k_cache = static_cast<const uint8_t*>(k_cache);
  a.k_scale = k_scale;
  a.page_table = page_table;
  a.q_pos = q_pos;
  a.lse = lse;
  a.weight = weight;
  a.err = err;
  a.batch = d.batch;
  a.n_q = d.n_q;
  a.hq = d.n_q_heads;
  a.hk = d.n_kv_heads;
  a.head_dim = d.head_dim;
  a.page_size = d.page_size;
  a.max_pages = d.max_pages;
  a.num_pages = d.num_pages;
  a.decay = decay;
  a.scale = d.sm_scale > 0.f ? d.sm_scale : 1.f / sqrtf((float)d.head_dim);
  auto kern = d.kv_dtype == QSA_KV_FP8_E4M3 ? weight_kernel<true> : weight_kernel<false>;
  return launch_k(kern, dim3(512, (unsigned)d.batch), dim3(128), 0, s, true, a);
}

}  // namespace qsa
