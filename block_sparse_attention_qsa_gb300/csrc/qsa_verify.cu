// Verification of drafted tokens against the target's probabilities.
//
// Draft j stays while u_j q_j(x_j) < p_j(x_j); at the first one that does not,
// the next token is sampled from max(p - q, 0) by its inverse distribution
// function, else from p behind the last draft:  the lowest y with
//   u S < sum_{v <= y} w(v),   S = sum_v w(v).
// A cluster of CTAs takes a request. Every CTA finds the accepted drafts by
// itself (a lane a draft, the products of two FP32 values exact in 64 bits);
// then each sums the weights of its slice of the vocabulary, a warp a
// contiguous segment; the slices' sums go to every CTA's shared memory, and
// the CTA in whose slice u S falls reads the one segment again that holds it.
// So the row (or two) that is sampled from is read from HBM once.
//
// Weights are summed as integers, multiples of 2^-60: p and q are FP32 values
// of at most 1, so a multiple of 2^-60 is cut off 10^-18 at most, and integer
// sums do not depend on how the row is split: the threshold floor(u S) falls
// between the same two tokens in any order, and both passes agree.
#include "qsa_serve_internal.cuh"

namespace qsa {
namespace {

constexpr unsigned kFull = 0xffffffffu;
constexpr int kThreads = 512, kWarps = kThreads / 32;
constexpr int kMaxCluster = 8;

__device__ __forceinline__ float load(const float* p) { return *p; }
__device__ __forceinline__ float load(const __nv_bfloat16* p) {
  return __uint_as_float((uint32_t)*reinterpret_cast<const uint16_t*>(p) << 16);
}

// a probability in 2^-60ths, cut off; negative and NaN 0, above 1 as 1
__device__ __forceinline__ uint64_t fixed60(float x) {
  const float p = fminf(fmaxf(x, 0.f), 1.f);  // (a NaN becomes 0)
  const uint32_t b = __float_as_uint(p), e = b >> 23;
  const uint64_t m = (uint64_t)((b & 0x7fffffu) | (e ? 0x800000u : 0u)) << 37;  // p = m 2^(e - 127 - 60)
  return m >> min(127u - e, 63u);
}
__device__ __forceinline__ float as_uniform(float u) { return fminf(fmaxf(u, 0.f), 0x1.fffffep-1f); }

__device__ __forceinline__ uint64_t warp_sum(uint64_t x) {
#pragma unroll
  for (int o = 16; o > 0; o >>= 1) x += __shfl_xor_sync(kFull, x, o);
  return x;
}
__device__ __forceinline__ uint64_t warp_inclusive(uint64_t x) {
  const int lane = threadIdx.x & 31;
#pragma unroll
  for (int o = 1; o < 32; o <<= 1) {
    const uint64_t y = __shfl_up_sync(kFull, x, o);
    if (lane >= o) x += y;
  }
  return x;
}
__device__ __forceinline__ void st_peer_u64(uint32_t addr, uint64_t v) {
  asm volatile("st.shared::cluster.u64 [%0], %1;" ::"r"(addr), "l"(v) : "memory");
}

// What is sampled from: a row of the target, less one of the draft's or less a token.
template <typename T>
struct Weights {
  const T* p;
  const T* q;  // null: none
  int token;   // -1: none
  __device__ __forceinline__ uint64_t at(int v) const {
    const uint64_t x = fixed60(load(p + v));
    if (q) {
      const uint64_t y = fixed60(load(q + v));
      return x > y ? x - y : 0;
    }
    return v == token ? 0 : x;
  }
  // sum over first + lane, first + lane + 32, ... below end
  __device__ __forceinline__ uint64_t sum(int first, int end) const {
    uint64_t s = 0;
    for (int v = first + (int)(threadIdx.x & 31); v < end; v += 32) s += at(v);
    return s;
  }
};

template <typename T>
__global__ void __launch_bounds__(kThreads) verify_kernel(const VerifyArgs a) {
  __shared__ uint64_t s_slice[2][kMaxCluster];  // [try][CTA]
  __shared__ uint64_t s_seg[kWarps], s_scan[kWarps];
  __shared__ int s_m, s_end;
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  const int rank = (int)cluster_rank(), ctas = (int)cluster_size(), r = blockIdx.x / ctas;
  const T* target = static_cast<const T*>(a.target) + r * a.target_batch;
  const T* draft = a.draft ? static_cast<const T*>(a.draft) + r * a.draft_batch : nullptr;
  const int32_t* tokens = a.tokens + (long long)r * a.n_draft;
  const float* uniform = a.uniform + (long long)r * (a.n_draft + 1);
  int32_t* out = a.out_tokens + (long long)r * (a.n_draft + 1);
  cluster_arrive_relaxed();  // (waited for before the first store to another CTA)
  pdl_wait();
  if (warp == 0) {
    // m: drafts accepted; end 0: draft m was rejected, 1: there was none, 2: no request
    const int x = lane < a.n_draft ? tokens[lane] : -1;
    const bool valid = (unsigned)x < (unsigned)a.vocab;
    bool ok = false;
    if (valid) {
      const float p = fminf(fmaxf(load(target + lane * a.target_row + x), 0.f), 1.f);
      const float q = draft ? fminf(fmaxf(load(draft + lane * a.draft_row + x), 0.f), 1.f) : 1.f;
      ok = (double)as_uniform(uniform[lane]) * (double)q < (double)p;
    }
    const int m = min(a.n_draft, __ffs(~__ballot_sync(kFull, ok)) - 1);  // (lane 31 is never a draft)
    if (lane == min(m, 31)) {
      const bool none = m == 0 && x == -2;
      s_m = m;
      s_end = none ? 2 : valid ? 0 : 1;
      if (m < a.n_draft && !valid && x != -1 && !none && rank == 0) record_error(a.err, kErrToken, r, m, x);
    }
  }
  __syncthreads();
  const int m = s_m, end = s_end;
  if (rank == 0) {
    if (threadIdx.x < m) out[threadIdx.x] = tokens[threadIdx.x];
    if (threadIdx.x > m && threadIdx.x <= a.n_draft) out[threadIdx.x] = -1;
    if (threadIdx.x == 0) {
      a.accepted[r] = m;
      if (end == 2) out[0] = -1;
    }
  }
  cluster_wait();
  if (end == 2) return;  // (the whole cluster)

  Weights<T> w{target + m * a.target_row, nullptr, -1};
  if (end == 0) {
    if (draft)
      w.q = draft + m * a.draft_row;
    else
      w.token = tokens[m];
  }
  // this CTA's slice and its warps' segments
  const int slice = (a.vocab + ctas - 1) / ctas, s0 = min(rank * slice, a.vocab), s1 = min(s0 + slice, a.vocab);
  const int seg = ((s1 - s0 + kWarps - 1) / kWarps + 31) / 32 * 32;
  const uint64_t u = (uint64_t)((double)as_uniform(uniform[a.n_draft]) * 18446744073709551616.0);
  for (int pass = 0; pass < 2; ++pass) {
    const int g0 = min(s0 + warp * seg, s1);
    const uint64_t mine = warp_sum(w.sum(g0, min(g0 + seg, s1)));
    if (lane == 0) s_seg[warp] = mine;
    __syncthreads();
    if (warp == 0) {
      const uint64_t own = warp_sum(lane < kWarps ? s_seg[lane] : 0);
      if (lane < ctas) st_peer_u64(peer_addr(&s_slice[pass][rank], lane), own);
    }
    cluster_sync();
    uint64_t total = 0, before = 0;
    for (int c = 0; c < ctas; ++c) {
      before += c < rank ? s_slice[pass][c] : 0;
      total += s_slice[pass][c];
    }
    if (total == 0) {  // nothing to sample from: the target's row as it is, if it was not that already
      if (pass == 0 && end == 0) {
        w.q = nullptr;
        w.token = -1;
        continue;
      }
      if (rank == 0 && threadIdx.x == 0) out[m] = -1;
      return;
    }
    const uint64_t t = __umul64hi(total, u);  // floor(u S)
    if (t < before || t - before >= s_slice[pass][rank]) return;  // another CTA's
    // the segment that holds it
    uint64_t rest = t - before;
    int g = 0;
    while (rest >= s_seg[g]) rest -= s_seg[g++];
    const int b0 = s0 + g * seg, n = min(seg, s1 - b0), per = (n + kThreads - 1) / kThreads;
    const int v0 = b0 + min((int)threadIdx.x * per, n), v1 = b0 + min((int)(threadIdx.x + 1) * per, n);
    uint64_t own = 0;
    for (int v = v0; v < v1; ++v) own += w.at(v);
    const uint64_t inc = warp_inclusive(own);
    if (lane == 31) s_scan[warp] = inc;
    __syncthreads();
    uint64_t front = inc - own;
    for (int i = 0; i < warp; ++i) front += s_scan[i];
    if (front <= rest && rest - front < own) {  // one thread
      rest -= front;
      int v = v0;
      for (;; ++v) {
        const uint64_t x = w.at(v);
        if (rest < x) break;
        rest -= x;
      }
      out[m] = v;
    }
    return;
  }
}

}  // namespace

cudaError_t launch_verify(const VerifyArgs& a, bool bf16, cudaStream_t s) {
  // CTAs of a request: enough that few requests use the whole GPU, each with 4,096 tokens or more
  unsigned c = 1;
  while (c < kMaxCluster && (long long)a.batch * c < 2LL * device_sm_count() && a.vocab / (2 * (int)c) >= 4096) c *= 2;
  auto kern = bf16 ? verify_kernel<__nv_bfloat16> : verify_kernel<float>;
  return launch_clusters(kern, dim3((unsigned)a.batch * c), dim3(kThreads), c, s, a);
}

}  // namespace qsa
