// Eviction from the paged cache by accumulated attention weight.
//
// Of a request's n > keep tokens the first `sinks`, the last `recent` and the
// heaviest between them stay. A cluster of CTAs takes a request, each a slice of
// its positions, and finds the weight of the last one that stays by a radix
// selection on the weight's order-preserving key: counts by the key's first 11
// bits, added up through distributed shared memory; then the keys that share the
// last one's first digit, which are few, go to every CTA, and each finds the
// other two digits by itself. (Where they are many, equal weights for instance,
// all three digits are counted in the cluster.) What stays is then numbered in
// the order of the positions, a warp 32 of them at a time. A barrier of a
// cluster takes about 0.7 us and a digit of the cluster two of them; that and
// the waits for memory, not the weights' bytes, are the time of this kernel:
// 61,201 positions take one request 18.6 us and 32 requests 27 (37 in three
// digits of the cluster; 31 with a contiguous share a thread, and the keys
// gathered one atomic at a time).
//
// A second kernel, chained with programmatic dependent launch, copies K and V of
// the tokens that stay, the bytes of which are the bound for a batch: 32 requests
// from 50,001-61,201 to 16,385 tokens (BF16, 2 KV heads of 128) 160 us, 6.7 TB/s,
// the whole call 187.5.
#include <algorithm>

#include "qsa_serve_internal.cuh"

namespace qsa {
namespace {

constexpr unsigned kFull = 0xffffffffu;
constexpr int kSelThreads = 512, kSelWarps = kSelThreads / 32;
constexpr int kMaxCluster = 8;
constexpr int kBins = 2048;
constexpr unsigned kHeld = 16384;  // weights of a slice that are held in shared memory
constexpr unsigned kCand = 2048;   // keys with the last one's first digit that every CTA can take
constexpr uint32_t kZeroKey = 0x80000000u;  // of a weight of 0
// Positions of a CTA, more or less. (4,200 in slices of 2,112, 1,056 and 528:
// one request 14.2, 13.1 and 12.3 us for the whole call, 32 of them 54.7, 52.9
// and 54.7.)
constexpr int kSlice = 2048;

// Sum over the lanes up to this one.
__device__ __forceinline__ uint32_t warp_inclusive(uint32_t x) {
  const int lane = threadIdx.x & 31;
#pragma unroll
  for (int o = 1; o < 32; o <<= 1) {
    const uint32_t y = __shfl_up_sync(kFull, x, o);
    if (lane >= o) x += y;
  }
  return x;
}
__device__ __forceinline__ void st_peer_u32(uint32_t addr, uint32_t v) {
  asm volatile("st.shared::cluster.u32 [%0], %1;" ::"r"(addr), "r"(v) : "memory");
}
__device__ __forceinline__ void st_peer_u64(uint32_t addr, uint64_t v) {
  asm volatile("st.shared::cluster.u64 [%0], %1;" ::"r"(addr), "l"(v) : "memory");
}

// Sum of x over the threads before this one in the block; `scan` is read behind
// one barrier (the caller has another before it is written again).
__device__ __forceinline__ uint32_t block_before(uint32_t x, uint32_t (&scan)[kSelWarps]) {
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  const uint32_t inc = warp_inclusive(x);
  if (lane == 31) scan[warp] = inc;
  __syncthreads();
  const uint32_t other = lane < warp ? scan[lane] : 0;  // (at most 32 warps)
  return inc - x + __reduce_add_sync(kFull, other);
}

__global__ void __launch_bounds__(kSelThreads) evict_select_kernel(const EvictArgs a) {
  extern __shared__ __align__(16) float s_w[];  // the first a.held weights of the slice
  __shared__ uint32_t s_hist[kBins], s_sum[kBins], s_cand[kCand], s_own[kCand];  // this CTA's counts, the cluster's
  __shared__ uint64_t s_scan[kSelWarps], s_slice[kMaxCluster];
  __shared__ uint32_t s_bin, s_left, s_same, s_at, s_count[kSelWarps];
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
  const int rank = (int)cluster_rank(), ctas = (int)cluster_size(), r = blockIdx.x / ctas;
  auto sync = [&]() {
    if (ctas > 1)
      cluster_sync();
    else
      __syncthreads();
  };
  pdl_wait();
  pdl_trigger();
  // (positions are below 2^31; unsigned, so that a step past the last one is still a number)
  const unsigned cap = (unsigned)(a.max_pages * a.page_size), cap_out = (unsigned)(a.out_pages * a.page_size);
  const unsigned keep = (unsigned)a.keep;
  unsigned n = (unsigned)a.len[r];
  if (n > cap) {
    if (rank == 0 && tid == 0) record_error(a.err, kErrLength, r, 0, (int)n);
    n = 0;
  }
  const float* w = a.weight + (long long)r * cap;
  float* w_out = a.weight_out + (long long)r * cap_out;
  int32_t* kept = a.kept + (long long)r * a.keep;
  const unsigned left = min(n, keep);
  const unsigned first = (unsigned)(rank * kSelThreads + tid), step = (unsigned)(ctas * kSelThreads);
  auto fill = [&]() {  // behind the last one that stays
    for (unsigned i = left + first; i < cap_out; i += step) {
      w_out[i] = 0.f;
      if (i < keep) kept[i] = -1;
    }
  };
  if (n <= keep) {
    fill();
    for (unsigned i = first; i < n; i += step) {
      kept[i] = (int)i;
      w_out[i] = w[i];
    }
    sync();  // every CTA has read len, which new_len may be
    if (rank == 0 && tid == 0) a.new_len[r] = (int)left;
    return;  // (the whole cluster)
  }
  // positions lo .. hi - 1 are chosen from, `need` of them
  const unsigned lo = (unsigned)a.sinks, hi = n - (unsigned)a.recent;
  const unsigned slice = ((n + ctas - 1) / ctas + 3) & ~3u;  // (16-byte boundaries)
  const unsigned s0 = min(rank * slice, n), s1 = min(s0 + slice, n);
  const unsigned held = min(s1 - s0, a.held);
  const unsigned vecs = (reinterpret_cast<uintptr_t>(w + s0) & 15) == 0 ? held / 4 : 0;
#pragma unroll 4
  for (unsigned i = tid; i < vecs; i += kSelThreads)
    reinterpret_cast<uint4*>(s_w)[i] = ld16(reinterpret_cast<const uint4*>(w + s0) + i);
#pragma unroll 8
  for (unsigned i = 4 * vecs + tid; i < held; i += kSelThreads) s_w[i] = w[s0 + i];
  fill();
  auto key_at = [&](unsigned t) { return order_key(t - s0 < held ? s_w[t - s0] : w[t]); };
  uint32_t need = keep - a.sinks - a.recent, prefix = 0, mask = 0;
  if (need > 0) {
    const unsigned c0 = max(s0, lo), c1 = max(c0, min(s1, hi));  // the slice's part of them
    bool gathered = false;
    unsigned cands = 0;
#pragma unroll 1
    for (int d = 0; d < 3; ++d) {
      const int shift = d == 0 ? 21 : d == 1 ? 10 : 0;  // (the last digit has a bit of the second's)
      for (int i = tid; i < kBins; i += kSelThreads) s_hist[i] = 0;
      if (tid == 0) s_at = 0;
      __syncthreads();
      const unsigned from = gathered ? 0 : c0, to = gathered ? cands : c1;
      uint32_t zeros = 0;  // of them there may be many: a warp adds them at once
#pragma unroll 4
      for (unsigned t = from + tid; t < to; t += kSelThreads) {
        const uint32_t k = gathered ? s_cand[t] : key_at(t);
        if ((k & mask) != prefix) continue;
        if (k == kZeroKey)
          ++zeros;
        else
          atomicAdd(&s_hist[(k >> shift) & (kBins - 1)], 1u);
      }
      zeros = __reduce_add_sync(kFull, zeros);
      if ((tid & 31) == 0 && zeros > 0) atomicAdd(&s_hist[(kZeroKey >> shift) & (kBins - 1)], zeros);
      const uint32_t* counts = s_hist;
      if (ctas > 1 && !gathered) {
        // each CTA adds up a part of the bins for all of them
        cluster_sync();
        const int per = kBins / ctas;
        for (int i = tid; i < per; i += kSelThreads) {
          const int bin = rank * per + i;
          uint32_t c = 0;
#pragma unroll
          for (int p = 0; p < kMaxCluster; ++p) c += p < ctas ? ld_peer(peer_addr(&s_hist[bin], p)) : 0;
#pragma unroll
          for (int p = 0; p < kMaxCluster; ++p)
            if (p < ctas) st_peer_u32(peer_addr(&s_sum[bin], p), c);
        }
        cluster_sync();
        counts = s_sum;
      } else {
        __syncthreads();
      }
      // the digit of the last one that stays, from the largest down
      constexpr int kPer = kBins / kSelThreads;
      uint32_t c[kPer];
      uint32_t mine = 0;
#pragma unroll
      for (int i = 0; i < kPer; ++i) {
        c[i] = counts[kBins - 1 - (tid * kPer + i)];
        mine += c[i];
      }
      const uint32_t before = block_before(mine, s_count);
      if (before < need && need <= before + mine) {  // one thread
        uint32_t b = before;
        int i = 0;
        while (b + c[i] < need) b += c[i++];
        s_bin = (uint32_t)(kBins - 1 - (tid * kPer + i));
        s_left = need - b;
        s_same = c[i];
      }
      __syncthreads();
      const uint32_t bin = s_bin;
      prefix |= bin << shift;
      mask |= (uint32_t)(kBins - 1) << shift;
      need = s_left;
      if (ctas > 1 && d == 0 && s_same <= kCand) {
        // the keys with that digit go to every CTA, this one's behind those of the CTAs before it
        uint32_t front = 0;
#pragma unroll
        for (int p = 0; p < kMaxCluster; ++p) front += p < rank ? ld_peer(peer_addr(&s_hist[bin], p)) : 0;
        for (unsigned b0 = c0; b0 < c1; b0 += 32 * kSelThreads) {  // a bit of `hits` each
          const int steps = (int)min(32u, (c1 - b0 + kSelThreads - 1) / kSelThreads);
          uint32_t hits = 0;
#pragma unroll 4
          for (int i = 0; i < steps; ++i) {
            const unsigned t = b0 + i * kSelThreads + tid;
            if (t < c1 && (key_at(t) & mask) == prefix) hits |= 1u << i;
          }
          const uint32_t inc = warp_inclusive(__popc(hits));
          uint32_t at = 0;
          if (lane == 31 && inc > 0) at = atomicAdd(&s_at, inc);
          at = __shfl_sync(kFull, at, 31) + inc - __popc(hits);
          for (; hits; hits &= hits - 1) s_own[at++] = key_at(b0 + (__ffs(hits) - 1) * kSelThreads + tid);
        }
        __syncthreads();
        const uint32_t own = s_at;
        for (uint32_t j = tid; j < own; j += kSelThreads) {
          const uint32_t k = s_own[j];
#pragma unroll
          for (int p = 0; p < kMaxCluster; ++p)
            if (p < ctas) st_peer_u32(peer_addr(&s_cand[front + j], p), k);
        }
        cluster_sync();
        gathered = true;
        cands = s_same;
      }
    }
  } else {
    __syncthreads();
  }
  // Those above the last one's key stay, and the first `need` that equal it.
  const uint32_t last = need > 0 ? prefix : 0xffffffffu;  // (no weight has that key)
  // A warp takes a contiguous part, 32 positions at a time.
  const unsigned part = (s1 - s0 + kSelThreads - 1) / kSelThreads * 32;
  const unsigned t0 = min(s0 + warp * part, s1), t1 = min(t0 + part, s1);
  uint32_t stay = 0, same = 0;
#pragma unroll 4
  for (unsigned t = t0 + lane; t < t1; t += 32) {
    const uint32_t k = key_at(t);
    const bool anyway = t < lo || t >= hi || k > last;
    stay += anyway;
    same += !anyway && k == last;
  }
  stay = __reduce_add_sync(kFull, stay);
  same = __reduce_add_sync(kFull, same);
  if (lane == 0) s_scan[warp] = (uint64_t)same << 32 | stay;
  __syncthreads();
  uint64_t before = 0, all = 0;  // those that equal it << 32 | those that stay anyway
#pragma unroll
  for (int v = 0; v < kSelWarps; ++v) {
    const uint64_t c = s_scan[v];
    before += v < warp ? c : 0;
    all += c;
  }
  if (ctas > 1) {
    if (need == 0) cluster_sync();  // (no other before it: every CTA has started)
    if (tid < ctas) st_peer_u64(peer_addr(&s_slice[rank], tid), all);
    cluster_sync();
    for (int p = 0; p < rank; ++p) before += s_slice[p];
  }
  if (rank == 0 && tid == 0) a.new_len[r] = (int)left;  // (every CTA has read len)
  uint32_t ties = (uint32_t)(before >> 32), at = (uint32_t)before + min(ties, need);
  const uint32_t below = (1u << lane) - 1u;
#pragma unroll 2
  for (unsigned b0 = t0; b0 < t1; b0 += 32) {
    const unsigned t = b0 + lane;
    const bool in = t < t1;
    const float x = !in ? 0.f : t - s0 < held ? s_w[t - s0] : w[t];
    const uint32_t k = order_key(x);
    const bool anyway = in && (t < lo || t >= hi || k > last), equal = in && !anyway && k == last;
    const uint32_t equals = __ballot_sync(kFull, equal);
    const bool stays = anyway || (equal && ties + __popc(equals & below) < need);
    const uint32_t lanes = __ballot_sync(kFull, stays);
    if (stays) {
      const uint32_t to = at + __popc(lanes & below);
      kept[to] = (int)t;
      w_out[to] = x;
    }
    ties += __popc(equals);
    at += __popc(lanes);
  }
}

// K and V of the tokens that stay. A block takes kCopyTok of them, whose rows
// are worked out first, and up to 256 items; an item is 16 bytes of the same
// head of K or V in every token.
constexpr int kCopyTok = 32, kCopyDeep = 4;

__global__ void __launch_bounds__(256) evict_copy_kernel(const EvictArgs a) {
  __shared__ long long s_src[kCopyTok], s_dst[kCopyTok];
  const int tid = threadIdx.x;
  const int per_req = (int)((a.keep + kCopyTok - 1LL) / kCopyTok), r = blockIdx.x / per_req;
  const int i0 = (blockIdx.x - r * per_req) * kCopyTok, n = min(kCopyTok, a.keep - i0);
  const int vecs = a.row_bytes / 16, per = a.hk * vecs, items = 2 * per;
  pdl_wait();
  if (tid < n) {
    const int i = i0 + tid, t = a.kept[(long long)r * a.keep + i];
    long long src = -1, dst = -1;
    if (t >= 0) {
      const int from = a.page_table[(long long)r * a.max_pages + t / a.page_size];
      const int to = a.page_table_out[(long long)r * a.out_pages + i / a.page_size];
      const bool bad_from = (unsigned)from >= (unsigned)a.num_pages, bad_to = (unsigned)to >= (unsigned)a.num_pages;
      if (bad_from || bad_to) {
        if (blockIdx.y == 0) record_error(a.err, kErrPage, r, 0, bad_from ? from : to);
      } else {
        src = ((long long)from * a.hk * a.page_size + t % a.page_size) * a.row_bytes;
        dst = ((long long)to * a.hk * a.page_size + i % a.page_size) * a.row_bytes;
        if (src == dst) src = -1;
      }
    }
    s_src[tid] = src;
    s_dst[tid] = dst;
  }
  const int here = min(256, items - (int)blockIdx.y * 256), lanes = 256 / here;
  const int sub = tid / here, item = (int)blockIdx.y * 256 + tid - sub * here;
  const bool is_v = item >= per;
  const int h = is_v ? item - per : item, g = h / vecs;
  uint8_t* cache = (is_v ? a.v_cache : a.k_cache) + ((long long)g * a.page_size) * a.row_bytes + (h - g * vecs) * 16;
  __syncthreads();
  if (sub >= lanes) return;
  for (int t0 = sub; t0 < n; t0 += kCopyDeep * lanes) {
    uint4 x[kCopyDeep];
#pragma unroll
    for (int u = 0; u < kCopyDeep; ++u) {
      const int t = t0 + u * lanes;
      if (t < n && s_src[t] >= 0) x[u] = ld16(cache + s_src[t]);
    }
#pragma unroll
    for (int u = 0; u < kCopyDeep; ++u) {
      const int t = t0 + u * lanes;
      if (t < n && s_src[t] >= 0) *reinterpret_cast<uint4*>(cache + s_dst[t]) = x[u];
    }
  }
}

}  // namespace

cudaError_t launch_kv_evict(EvictArgs a, cudaStream_t s) {
  // CTAs of a request: few, for their barriers; more only where the slices would be long
  const int cap = a.max_pages * a.page_size;
  unsigned c = 1;
  while (c < kMaxCluster && (long long)a.batch * c < device_sm_count() && cap / (int)c > kSlice) c *= 2;
  a.held = std::min(kHeld, (((unsigned)cap + c - 1) / c + 3) & ~3u);
  static DeviceSlots slots;
  cudaError_t e = slots.raise_smem(evict_select_kernel, kHeld * sizeof(float));
  if (e != cudaSuccess) return e;
  e = launch_clusters(evict_select_kernel, dim3((unsigned)a.batch * c), dim3(kSelThreads), c,
                      a.held * sizeof(float), s, a);
  if (e != cudaSuccess) return e;
  const int vecs = a.row_bytes / 16, items = 2 * a.hk * vecs;
  const long long gx = (long long)a.batch * ((a.keep + kCopyTok - 1LL) / kCopyTok);  // (below 2^31: qsa_kv_evict)
  return launch_k(evict_copy_kernel, dim3((unsigned)gx, (unsigned)((items + 255) / 256)), dim3(256), 0, s, true, a);
}

}  // namespace qsa
