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
// The sums are exact, so that they do not depend on how the row is split: the
// threshold floor(u S) falls between the same two tokens in any order, and both
// readings of a segment agree. A weight is p, or p - q where p > q, each rounded
// to a multiple of 2^-54 (what is smaller has no weight). As 64-bit integers these cost the integer pipe 36
// cycles a value and warp, and 256 rows of 150,001 tokens (FP32, sampled drafts)
// 81 us; the conversion instruction to 64 bits was slower still, 158. So they
// are added in FP32 without rounding (see Exact), 11 additions for two values:
// 59 us, where the bytes take 37.5 (16-bit probabilities 53, at odd rows 57, the
// bytes 18.8). Nothing is busy all the time: HBM 52 % (16 bits 28), the additions'
// pipe 43 % of the SMs' busy time (50), issue slots 42 (49). A warp waits half of
// its time for loads, which it issues only behind the additions of those before;
// and 512 CTAs have 304 places, so that an SM has work for 79 % of the time, the
// least busy one for 47. A ring of bulk copies to shared memory in place of the
// loads was slower (92 us), and so were shares for smaller or more CTAs.
#include "qsa_serve_internal.cuh"

namespace qsa {
namespace {

constexpr unsigned kFull = 0xffffffffu;
constexpr int kThreads = 512, kWarps = kThreads / 32;
constexpr int kMaxCluster = 8;
constexpr int kDeep = 8;  // values a thread has on their way, of each row

__device__ __forceinline__ float load(const float* p) { return *p; }
__device__ __forceinline__ float load(const __nv_bfloat16* p) {
  return __uint_as_float((uint32_t)*reinterpret_cast<const uint16_t*>(p) << 16);
}

// Exact sums of values of at most 1 in magnitude, each rounded to a multiple of
// 2^-54. A value is taken apart on three fixed grids: x + M, with M 1.5 2^23 times
// the grid, is rounded to the grid, and what is left is exact again. The parts
// on the grid of 2^-20 add up without rounding to below 2^4, those on 2^-37 (at
// most 2^-21 each) to 2^-13, those on 2^-54 (at most 2^-38) to 2^-30, that is
// for kMost values. The last part's rounding is to nearest, ties to even, and so
// is the whole value's. A probability that is negative or NaN is 0, one above 1
// is 1 (saturated). Where the first sums came near 2^4, which no row of
// probabilities does, the values are added again as integers (full()).
struct Exact {
  static constexpr int kMost = 256;
  static constexpr float kM1 = 1.5f * 0x1p3f, kM2 = 1.5f * 0x1p-14f, kM3 = 1.5f * 0x1p-31f;
  float2 a1, a2, a3;  // less the sums
  __device__ __forceinline__ Exact() : a1(make_float2(0.f, 0.f)), a2(a1), a3(a1) {}
  static __device__ __forceinline__ float2 pair(float x) { return make_float2(x, x); }
  // M - (x + M): less x's part on the grid
  static __device__ __forceinline__ float2 part(float2 x, float m) {
    return fma2(add2(x, pair(m)), pair(-1.f), pair(m));
  }
  __device__ __forceinline__ void add(float2 x) {
    const float2 t1 = part(x, kM1);
    a1 = add2(a1, t1);
    x = add2(x, t1);
    const float2 t2 = part(x, kM2);
    a2 = add2(a2, t2);
    x = add2(x, t2);
    a3 = add2(a3, part(x, kM3));
  }
  // a probability in 2^-54ths: the parts as integers, which are in the sums' last bits
  static __device__ __forceinline__ int64_t of(float x) {
    x = __saturatef(x);
    const float s1 = __fadd_rn(x, kM1);
    x = __fsub_rn(x, __fsub_rn(s1, kM1));
    const float s2 = __fadd_rn(x, kM2);
    x = __fsub_rn(x, __fsub_rn(s2, kM2));
    const float s3 = __fadd_rn(x, kM3);
    return combine(__float_as_int(s1) - __float_as_int(kM1), __float_as_int(s2) - __float_as_int(kM2),
                   __float_as_int(s3) - __float_as_int(kM3));
  }
  static __device__ __forceinline__ int64_t combine(int i1, int i2, int i3) {
    return (int64_t)i1 * (1LL << 34) + (int64_t)i2 * (1LL << 17) + i3;
  }
  // whether a sum on the grid of 2^-20 may have passed 2^4 on its way (a weight's
  // two values are at most 1, so never by more than 1 past its end)
  __device__ __forceinline__ bool full() const { return fminf(a1.x, a1.y) <= -14.f; }
  __device__ __forceinline__ int64_t sum() const {  // in 2^-54ths
    const int i1 = __float2int_rn(a1.x * 0x1p20f) + __float2int_rn(a1.y * 0x1p20f);
    const int i2 = __float2int_rn(a2.x * 0x1p37f) + __float2int_rn(a2.y * 0x1p37f);
    const int i3 = __float2int_rn(a3.x * 0x1p54f) + __float2int_rn(a3.y * 0x1p54f);
    return -combine(i1, i2, i3);
  }
};
// Sums of weights are kept at most kHeavy, 16 in 2^-54ths, so that none of them
// passes 64 bits; a row with that much is no row of probabilities (reported).
constexpr uint64_t kHeavy = 1ULL << 58;
__device__ __forceinline__ uint64_t at_most_heavy(uint64_t x) { return x < kHeavy ? x : kHeavy; }
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
    const float x = load(p + v);
    if (q) {
      const float y = load(q + v);
      return __saturatef(x) > __saturatef(y) ? (uint64_t)(Exact::of(x) - Exact::of(y)) : 0;
    }
    return v == token ? 0 : (uint64_t)Exact::of(x);
  }
  // two weights into a sum
  static __device__ __forceinline__ void add_less(Exact& s, float p0, float q0, float p1, float q1) {
    p0 = __saturatef(p0), q0 = __saturatef(q0), p1 = __saturatef(p1), q1 = __saturatef(q1);
    const bool m0 = p0 > q0, m1 = p1 > q1;
    s.add(make_float2(m0 ? p0 : 0.f, m1 ? p1 : 0.f));
    s.add(make_float2(m0 ? -q0 : 0.f, m1 ? -q1 : 0.f));
  }
  // sum over a lane's share of first .. end - 1, kDeep loads of a row in flight
  __device__ __forceinline__ uint64_t sum(int first, int end) const {
    const int lane = threadIdx.x & 31;
    uint64_t all = 0;
    int v = first + lane;
    bool full = false;
    while (v + 32 * (kDeep - 1) < end) {
      Exact s;
      for (int z = 0; z < Exact::kMost / 2 / kDeep && v + 32 * (kDeep - 1) < end; ++z, v += 32 * kDeep) {
        float x[kDeep], y[kDeep];
#pragma unroll
        for (int i = 0; i < kDeep; ++i) x[i] = load(p + v + 32 * i);
        if (q) {
#pragma unroll
          for (int i = 0; i < kDeep; ++i) y[i] = load(q + v + 32 * i);
#pragma unroll
          for (int i = 0; i < kDeep; i += 2) add_less(s, x[i], y[i], x[i + 1], y[i + 1]);
        } else {
#pragma unroll
          for (int i = 0; i < kDeep; ++i) x[i] = v + 32 * i == token ? 0.f : __saturatef(x[i]);
#pragma unroll
          for (int i = 0; i < kDeep; i += 2) s.add(make_float2(x[i], x[i + 1]));
        }
      }
      all = at_most_heavy(all + (uint64_t)s.sum());
      full |= s.full();
    }
    if (full) {  // all of them again, as integers
      all = 0;
      v = first + lane;
    }
    for (; v < end; v += 32) all = at_most_heavy(all + at(v));
    return all;
  }
  // the same where both rows and `first` are at 16-byte boundaries
  __device__ __forceinline__ uint64_t sum_vec(int first, int end) const {
    constexpr int kVec = 16 / sizeof(T), kStep = 32 * kVec, kLoads = kDeep / 4;
    uint64_t all = 0;
    int v = first + (int)(threadIdx.x & 31) * kVec;
    bool full = false;
    while (v + kStep * (kLoads - 1) + kVec <= end) {
      Exact s;
      for (int z = 0; z < Exact::kMost / 2 / (kVec * kLoads) && v + kStep * (kLoads - 1) + kVec <= end;
           ++z, v += kStep * kLoads) {
        uint4 x[kLoads], y[kLoads];
#pragma unroll
        for (int i = 0; i < kLoads; ++i) x[i] = ld16(p + v + kStep * i);
        if (q) {
#pragma unroll
          for (int i = 0; i < kLoads; ++i) y[i] = ld16(q + v + kStep * i);
#pragma unroll
          for (int i = 0; i < kLoads; ++i)
#pragma unroll
            for (int e = 0; e < kVec; e += 2)
              add_less(s, value(x[i], e), value(y[i], e), value(x[i], e + 1), value(y[i], e + 1));
        } else {
#pragma unroll
          for (int i = 0; i < kLoads; ++i)
#pragma unroll
            for (int e = 0; e < kVec; e += 2) {
              const int at0 = v + kStep * i + e;
              s.add(make_float2(at0 == token ? 0.f : __saturatef(value(x[i], e)),
                                at0 + 1 == token ? 0.f : __saturatef(value(x[i], e + 1))));
            }
        }
      }
      all = at_most_heavy(all + (uint64_t)s.sum());
      full |= s.full();
    }
    if (full) {  // all of them again, as integers
      all = 0;
      v = first + (int)(threadIdx.x & 31) * kVec;
    }
    for (; v < end; v += kStep)
      for (int e = 0; e < kVec && v + e < end; ++e) all = at_most_heavy(all + at(v + e));
    return all;
  }
  static __device__ __forceinline__ float value(const uint4& x, int e) {
    const uint32_t w[4] = {x.x, x.y, x.z, x.w};
    if constexpr (sizeof(T) == 4)
      return __uint_as_float(w[e]);
    else
      return e & 1 ? bf_hi(w[e / 2]) : bf_lo(w[e / 2]);
  }
};

// VEC: all rows are at 16-byte boundaries
template <typename T, bool VEC>
__global__ void __launch_bounds__(kThreads, 2) verify_kernel(const VerifyArgs a) {
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
    // (rows behind the last draft are not looked at: a padded request may have none)
    const int drafts = __ffs(~__ballot_sync(kFull, valid)) - 1;  // (lane 31 is never a draft)
    bool ok = false;
    if (lane < drafts) {
      const float p = fminf(fmaxf(load(target + lane * a.target_row + x), 0.f), 1.f);
      const float q = draft ? fminf(fmaxf(load(draft + lane * a.draft_row + x), 0.f), 1.f) : 1.f;
      ok = (double)as_uniform(uniform[lane]) * (double)q < (double)p;
    }
    const int m = __ffs(~__ballot_sync(kFull, ok)) - 1;
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
    if (threadIdx.x >= m && threadIdx.x <= a.n_draft) out[threadIdx.x] = -1;  // (the next token comes behind a barrier)
    if (threadIdx.x == 0) a.accepted[r] = m;
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
  // (multiples of 256 values, which keeps 16-byte boundaries)
  constexpr int kUnit = 256;
  const int slice = (a.vocab + ctas * kUnit - 1) / (ctas * kUnit) * kUnit;
  const int s0 = min(rank * slice, a.vocab), s1 = min(s0 + slice, a.vocab);
  const int seg = (s1 - s0 + kWarps * kUnit - 1) / (kWarps * kUnit) * kUnit;
  const uint64_t u = (uint64_t)((double)as_uniform(uniform[a.n_draft]) * 18446744073709551616.0);
  for (int pass = 0; pass < 2; ++pass) {
    const int g0 = min(s0 + warp * seg, s1);
    const int g1 = min(g0 + seg, s1);
    const uint64_t mine = at_most_heavy(warp_sum(VEC ? w.sum_vec(g0, g1) : w.sum(g0, g1)));
    if (lane == 0) s_seg[warp] = mine;
    __syncthreads();
    if (warp == 0) {
      const uint64_t own = at_most_heavy(warp_sum(lane < kWarps ? s_seg[lane] : 0));
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
      return;
    }
    if (total >= kHeavy) {
      if (rank == 0 && threadIdx.x == 0) record_error(a.err, kErrHeavy, r, m, 0);
      return;
    }
    const uint64_t t = __umul64hi(total, u);  // floor(u S)
    if (t < before || t - before >= s_slice[pass][rank]) return;  // another CTA's
    // the segment that holds it
    uint64_t rest = t - before;
    int g = 0;
    while (g < kWarps - 1 && rest >= s_seg[g]) rest -= s_seg[g++];
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
      for (; v < v1 - 1; ++v) {
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
  const long long each = bf16 ? 8 : 4;  // values of 16 bytes
  bool vec = aligned_all(16, {a.target, a.draft}) && (a.target_batch | a.target_row) % each == 0;
  if (a.draft) vec = vec && (a.draft_batch | a.draft_row) % each == 0;
  auto kern = bf16 ? (vec ? verify_kernel<__nv_bfloat16, true> : verify_kernel<__nv_bfloat16, false>)
                   : (vec ? verify_kernel<float, true> : verify_kernel<float, false>);
  return launch_clusters(kern, dim3((unsigned)a.batch * c), dim3(kThreads), c, 0, s, a);
}

}  // namespace qsa
