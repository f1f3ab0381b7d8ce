// The attention weight that each cached position gets from the newest tokens:
//   w[t] = decay w[t] + sum_{j, h} exp(c q_jh . k_t - lse_jh).
//
// The first product of the dense attention (qsa_dense_tc.cuh) with a sum in
// place of the second: S^T[position][row] = K Q^T on the tensor cores, K tiles
// of 128 positions by TMA as the cache holds them, the scores in tensor memory,
// a thread a position. With the softmax's sums given, a weight is one
// exponential of a score and a row's constant, and the sum over rows stays in
// the thread: no maxima, no second pass, no atomics, and K is read once.
//
// K's bytes are the bound (2 D a position, head and row against 2 D or D
// bytes), so the work is split by positions: the requests' tiles form one
// stream, cut into equal contiguous shares, one per persistent CTA (Walk in
// qsa_dense.cuh). A CTA goes through its share in runs of up to kRunTiles tiles;
// in a run through the KV heads and blocks of up to 64 query rows, a step each,
// and in a step through the run's tiles, whose sums lie in shared memory until
// the last step. Which thread adds what, and in which order, does not depend on
// the timing: the same call gives the same bits.
//
// E4M3 cache: the codes are the MMA's operand, and a query row is two E4M3
// terms, q = 2^sh (hi + lo / 32), off by at most 2^-22 of the row's largest
// value (see qsa_dense_tc.cuh); the two products are columns of one MMA.
//
// Roles: a copy warp (pages, TMA), a warp that issues the MMAs, a warpgroup that
// stages the query rows of the steps ahead, and two warpgroups for the sums,
// which take a run's even and odd tiles and have two score buffers each.
//
// Measured: 32 requests of 50,004-61,204 tokens, 4 queries, 16 heads over 2 of
// 128, BF16: 142 us, 6.5 TB/s, 0.96 of the measured copy rate (FP32 sums by a
// warp a position, the form before, took 10.7 ms). A request of 1,000 tokens: 6.4
// us, the latency of one tile. Short requests with many KV heads wait for their
// steps one after the other (2 to 3 us each at head dim 256).
#include "qsa_serve_internal.cuh"
#include "qsa_tc.cuh"

namespace qsa {
namespace {

constexpr int kTile = 128;
constexpr int kRows = 64;      // of a step at most
constexpr int kRunTiles = 16;
constexpr int kBadRing = 32;   // page marks of the tiles in flight

struct WeightArgs {
  DenseArgs w;  // the stream of tiles, a unit a request
  const float* lse;
  float* weight;
  int hk, group, blocks;  // blocks of rows of a KV head
  float decay;
};

template <int D_, bool FP8_>
struct Wc {
  static constexpr bool FP8 = FP8_;
  static constexpr int D = D_, EB = FP8 ? 1 : 2, kRowBytes = D * EB;
  static constexpr int kLine = kRowBytes < 128 ? kRowBytes : 128, kLines = kRowBytes / kLine, kChunks = kLine / 16;
  static constexpr int kSlot = kTile * kRowBytes;
  static constexpr int kQRows = FP8 ? 2 * kRows : kRows;  // hi rows, then lo rows
  static constexpr int kQ = kQRows * kRowBytes;
  static constexpr int kAcc = kRunTiles * kTile * 4;
  static constexpr int kStatic = 4096;
  static constexpr int kFixed = 2 * kQ + kAcc + 1024;
  static constexpr int kFit = (kMaxSmem - kStatic - kFixed) / kSlot;
  static constexpr int kSlots = kFit < 12 ? kFit : 12;
  static constexpr int kSmem = kSlots * kSlot + kFixed;
  static constexpr int kThreads = 3 * 128 + 64;
  static constexpr int kCopyWarp = 12, kMmaWarp = 13;
  static constexpr uint32_t kCols = kQRows, kTmem = 4 * kCols;  // four score buffers
  static_assert(kSlots >= 2 && kSlots + 6 < kBadRing, "ring");
  static __device__ __forceinline__ int swizzled(int row, int c) {
    return kLine == 128 ? c ^ (row & 7) : c ^ ((row >> 1) & 3);
  }
};

template <class C>
__global__ void __launch_bounds__(C::kThreads, 1) weight_kernel(const __grid_constant__ CUtensorMap tm_k,
                                                                const WeightArgs a) {
  constexpr bool FP8 = C::FP8;
  constexpr int D = C::D, kLine = C::kLine, kLines = C::kLines, kChunks = C::kChunks;
  constexpr uint64_t kSwizzle = kLine == 128 ? 2 : 4;
  extern __shared__ uint8_t smem_raw[];
  uint8_t* ring = reinterpret_cast<uint8_t*>((reinterpret_cast<uintptr_t>(smem_raw) + 1023) & ~uintptr_t(1023));
  uint8_t* s_q = ring + C::kSlots * C::kSlot;
  float* s_acc = reinterpret_cast<float*>(s_q + 2 * C::kQ);  // [tile of the run][position]
  __shared__ __align__(8) uint64_t slot_full[C::kSlots], slot_empty[C::kSlots];
  __shared__ __align__(8) uint64_t s_full[4], s_empty[4], q_full[2], q_empty[2], fin;
  __shared__ uint32_t s_tmem;
  __shared__ uint32_t s_bad[kBadRing];  // bit i: positions 16 i .. 16 i + 15 of the tile have no page
  __shared__ volatile int s_abort;
  __shared__ long long s_scan[C::kThreads / 32];
  __shared__ Share s_share;
  __shared__ __align__(16) float s_scale[2][kRows], s_less[2][kRows];  // of a row: factor and - lse, exp2 domain
  __shared__ __align__(16) int s_end[2][kRows];                        // one past the last position it sees
  __shared__ int s_all[2];                                             // positions that all rows of the step see
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
  const DenseArgs& w = a.w;
  if (tid == 0) {
    s_abort = 0;
    for (int s = 0; s < C::kSlots; ++s) {
      mbar_init(smem_u32(&slot_full[s]), 1);
      mbar_init(smem_u32(&slot_empty[s]), 1);
    }
    for (int b = 0; b < 4; ++b) {
      mbar_init(smem_u32(&s_full[b]), 1);
      mbar_init(smem_u32(&s_empty[b]), 128);
    }
    for (int b = 0; b < 2; ++b) {
      mbar_init(smem_u32(&q_full[b]), 128);
      // (One arrival a warp of the sums and the tensor cores'. The 32 of a warp are
      // counted at once: where the sums run on past a wait that was given up and the
      // last commit never comes, 256 + 1 of them would take the count below zero.)
      mbar_init(smem_u32(&q_empty[b]), 8 + 1);
    }
    mbar_init(smem_u32(&fin), 1);
    asm volatile("fence.mbarrier_init.release.cluster;" ::: "memory");
  }
  if (warp == C::kMmaWarp) {
    asm volatile("tcgen05.alloc.cta_group::1.sync.aligned.shared::cta.b32 [%0], %1;" ::"r"(smem_u32(&s_tmem)),
                 "r"(C::kTmem)
                 : "memory");
    asm volatile("tcgen05.relinquish_alloc_permit.cta_group::1.sync.aligned;" ::: "memory");
  }
  tc_before();
  pdl_wait();
  Walk<kTile> at;
  const bool work = find_start<kTile, C::kThreads>(w, s_scan, s_share, at);  // (with a barrier behind the allocation)
  tc_after();
  const uint32_t tmem = s_tmem;
  auto free_tmem = [&]() {
    asm volatile("tcgen05.dealloc.cta_group::1.sync.aligned.b32 %0, %1;" ::"r"(tmem), "r"(C::kTmem) : "memory");
  };
  if (!work) {
    if (warp == C::kMmaWarp) free_tmem();
    return;
  }
  auto wait = [&](uint64_t* bar, uint32_t parity) { return mbar_wait(bar, parity, &s_abort, w.err); };
  const int steps = a.hk * a.blocks, rows_all = w.n_q * a.group;
  auto rows_of = [&](int x) { return min(kRows, rows_all - x % a.blocks * kRows); };

  if (warp == C::kCopyWarp) {
    // ---- copies of K tiles ----
    PageFeed<kTile> feed(w);
    const int line = lane >> (7 - feed.box_shift);  // this lane's line of a tile; at most 32 copies
    const uint32_t dst = (uint32_t)(line * (kTile * kLine) + (feed.my_box << feed.box_shift) * kLine);
    int slot = 0, it = 0;
    uint32_t phase = 0;
    bool ok = true;
    do {
      Walk<kTile> run = at;
      for (int left = at.n; left > 0 && ok; left -= run.n, run.t += run.n) {
        run.n = min(kRunTiles, left);
        for (int x = 0; x < steps && ok; ++x) {
          const int g = x / a.blocks;
          feed.start(w, run);
          for (int k = 0; k < run.n; ++k, ++it) {
            const int page = feed.of_tile(w, run, k);
            const uint32_t bad = feed.bad_groups(page);
            if (!__all_sync(kFull, wait(&slot_empty[slot], phase ^ 1u))) {
              ok = false;
              break;
            }
            const uint32_t bar = smem_u32(&slot_full[slot]);
            if (lane == 0) {
              s_bad[it % kBadRing] = bad;
              mbar_expect_tx(bar, C::kSlot);
            }
            __syncwarp();
            if (line < kLines)
              tma_load_4d(smem_u32(ring + slot * C::kSlot) + dst, &tm_k, line * (kLine / C::EB), feed.slot_of(w, k), g,
                          page < 0 ? w.num_pages : page /* outside: zeros */, bar);
            if (++slot == C::kSlots) {
              slot = 0;
              phase ^= 1u;
            }
          }
        }
      }
    } while (ok && at.next(w, s_share));
    if (s_abort) {  // copies in flight land before the CTA leaves (bounded)
      for (int i = 0; i < C::kSlots; ++i) {
        const uint32_t par = i < slot ? phase : phase ^ 1u;
        const long long start = clock64();
        while (!mbar_try_wait(smem_u32(&slot_full[i]), par) && clock64() - start < kWaitCycles / 64) {
        }
      }
    }
  } else if (warp == C::kMmaWarp) {
    // ---- S^T = K Q^T (the whole warp walks the loop, one elected thread issues) ----
    const bool one = elect_one();
    constexpr int kSteps = C::kRowBytes / 32, kPerLine = kLine / 32;  // 32 bytes of a row each
    int slot = 0, st = 0;
    int even = 0, odd = 0;  // tiles of each warpgroup
    uint32_t phase = 0;
    bool ok = true;
    do {
      int n = 0;
      for (int left = at.n; left > 0 && ok; left -= n) {
        n = min(kRunTiles, left);
        for (int x = 0; x < steps && ok; ++x, ++st) {
          const int cols = (rows_of(x) + 15) / 16 * 16 * (FP8 ? 2 : 1), buf = st & 1;
          const uint32_t idesc = instr_desc(FP8 ? 0u : kTypeBf16, false, false, cols, kTile);
          const uint64_t dq = smem_desc(smem_u32(s_q + buf * C::kQ), 16, 8 * kLine, kSwizzle);
          ok = __all_sync(kFull, wait(&q_full[buf], (uint32_t)(st >> 1) & 1u));
          for (int k = 0; k < n && ok; ++k) {
            const int done = (k & 1) ? odd : even, b = (k & 1) * 2 + (done & 1);
            ok = __all_sync(kFull, wait(&slot_full[slot], phase) &&
                                       (done < 2 || wait(&s_empty[b], (uint32_t)((done - 2) >> 1) & 1u)));
            if (!ok) break;
            tc_after();
            const uint64_t dk = smem_desc(smem_u32(ring + slot * C::kSlot), 16, 8 * kLine, kSwizzle);
#pragma unroll
            for (int ks = 0; ks < kSteps; ++ks) {
              // (addresses are in units of 16 bytes)
              const uint32_t ln = (uint32_t)(ks / kPerLine), in = (uint32_t)(ks % kPerLine) * 2u;
              if (one)
                mma_tc<FP8>(tmem + (uint32_t)b * C::kCols, dk + (ln * (kTile * kLine / 16) + in),
                            dq + (ln * (C::kQRows * kLine / 16) + in), idesc, ks > 0);
            }
            if (one) {
              commit_tc(&s_full[b]);
              commit_tc(&slot_empty[slot]);
              if (k == n - 1) commit_tc(&q_empty[buf]);
            }
            __syncwarp();
            (k & 1) ? ++odd : ++even;
            if (++slot == C::kSlots) {
              slot = 0;
              phase ^= 1u;
            }
          }
        }
      }
    } while (ok && at.next(w, s_share));
    // the tensor cores are done before the CTA gives its memory back
    if (one) commit_tc(&fin);
    const long long start = clock64();
    while (!mbar_try_wait(smem_u32(&fin), 0) && clock64() - start < 2 * kWaitCycles) {
    }
    __syncwarp();
  } else if (warp >= 8) {
    // ---- query rows of the steps ahead ----
    const int t = tid - 256;
    int st = 0;
    do {
      int n = 0;
      for (int left = at.n; left > 0; left -= n) {
        n = min(kRunTiles, left);
        for (int x = 0; x < steps; ++x, ++st) {
          const int buf = st & 1, g = x / a.blocks, first = x % a.blocks * kRows, rows = rows_of(x);
          const int pad = (rows + 15) / 16 * 16;
          // (Given up: on without meaning, to the same barriers. What one thread sees of
          // a wait that ran out its neighbour may not: no loop here may end by it.)
          if (st >= 2) wait(&q_empty[buf], (uint32_t)((st - 2) >> 1) & 1u);
          __syncwarp();
          const float base = w.sm_scale * kLog2e * (FP8 ? w.k_scale[g] : 1.f);
          uint8_t* dst = s_q + buf * C::kQ;
          constexpr int kLanes = D / 8, kPass = 128 / kLanes;  // 8 components a lane
          for (int r = t / kLanes; r < pad; r += kPass) {      // (whole groups of kLanes lanes)
            const int c = t % kLanes;
            uint4 v = make_uint4(0, 0, 0, 0);
            if (r < rows) {
              const int i = first + r, j = i / a.group, h = g * a.group + (i - j * a.group);
              v = ld16(w.q + (((size_t)at.r * w.n_q + j) * w.n_q_heads + h) * D + c * 8);
            }
            if constexpr (FP8) {
              uint32_t big = 0;  // magnitudes of BF16 values order like their bit patterns
              const uint32_t wd[4] = {v.x, v.y, v.z, v.w};
#pragma unroll
              for (int e = 0; e < 4; ++e) big = max(big, max((wd[e] << 16) & 0x7fff0000u, wd[e] & 0x7fff0000u));
              const uint32_t group = kLanes == 32 ? kFull : ((1u << (kLanes % 32)) - 1u) << (lane / kLanes * kLanes);
#pragma unroll
              for (int o = 1; o < kLanes; o <<= 1) big = max(big, __shfl_xor_sync(group, big, o));
              // 2^-sh brings the row's largest value into [2^7, 2^8)
              const int sh = big == 0 ? 0 : min(126, max(-126, (int)(big >> 23) - 127 - 7));
              // (a row with an infinity or NaN: every component NaN, as its scores are)
              const float down = big >= 0x7f800000u ? __uint_as_float(0x7fffffffu) : pow2(-sh);
              uint32_t hi[4], lo[4];
#pragma unroll
              for (int e = 0; e < 4; ++e) {
                const float p = bf_lo(wd[e]) * down, q = bf_hi(wd[e]) * down;
                hi[e] = e4m3x2(p, q);
                const float2 f = h2_to_f2(e4m3x2_to_h2(hi[e]));
                lo[e] = e4m3x2((p - f.x) * 32.f, (q - f.y) * 32.f);
              }
              const int chunk = c >> 1, lr = pad + r;
              uint8_t* at_line = dst + chunk / kChunks * (C::kQRows * kLine) + (c & 1) * 8;
              *reinterpret_cast<uint2*>(at_line + r * kLine + (C::swizzled(r, chunk % kChunks) << 4)) =
                  make_uint2(hi[0] | (hi[1] << 16), hi[2] | (hi[3] << 16));
              *reinterpret_cast<uint2*>(at_line + lr * kLine + (C::swizzled(lr, chunk % kChunks) << 4)) =
                  make_uint2(lo[0] | (lo[1] << 16), lo[2] | (lo[3] << 16));
              if (c == 0) s_scale[buf][r] = base * pow2(sh);
            } else {
              *reinterpret_cast<uint4*>(dst + c / kChunks * (C::kQRows * kLine) + r * kLine +
                                        (C::swizzled(r, c % kChunks) << 4)) = v;
              if (c == 0) s_scale[buf][r] = base;
            }
          }
          int end = 0x7fffffff;
          if (t < kRows) {
            float less = 0.f;
            if (t < rows) {
              const int i = first + t, j = i / a.group, h = g * a.group + (i - j * a.group);
              const size_t row = (size_t)at.r * w.n_q + j;
              const int p = w.q_pos[row];
              const float l = a.lse[row * w.n_q_heads + h];
              end = valid_pos(w, p) && l != kNegInf ? p + 1 : 0;
              less = -l * kLog2e;
            }
            s_less[buf][t] = less;
            s_end[buf][t] = t < rows ? end : 0;
          }
          if (warp < 10) {  // the first 64 threads: the least of the ends
#pragma unroll
            for (int o = 16; o > 0; o >>= 1) end = min(end, __shfl_xor_sync(kFull, end, o));
          }
          if (t == 0) s_all[buf] = 0x7fffffff;
          asm volatile("bar.sync 1, 128;" ::: "memory");
          if (warp < 10 && lane == 0) atomicMin(&s_all[buf], end);
          async_fence();
          mbar_arrive(smem_u32(&q_full[buf]));
        }
      }
    } while (at.next(w, s_share));
  } else {
    // ---- sums ----
    const int wg = warp >> 2, t = tid & 127;
    const uint32_t lane_base = (uint32_t)((warp & 3) * 32) << 16;
    int st = 0, it = 0, done = 0;
    do {
      float* weight = a.weight + (size_t)at.r * capacity(w);
      int n = 0;
      for (int left = at.n, t0 = at.t; left > 0; left -= n, t0 += n) {
        n = min(kRunTiles, left);
        for (int x = 0; x < steps; ++x, ++st) {
          const int buf = st & 1, rows = rows_of(x), pad = (rows + 15) / 16 * 16;
          wait(&q_full[buf], (uint32_t)(st >> 1) & 1u);
          const int all = s_all[buf];
          for (int k = wg; k < n; k += 2, ++done) {
            const int p0 = (t0 + k) * kTile, p = p0 + t, b = wg * 2 + (done & 1);
            const bool last = x == steps - 1, mine = p < at.g.hi;
            float old = 0.f;
            if (last && mine && a.decay != 0.f) old = weight[p];
            wait(&s_full[b], (uint32_t)(done >> 1) & 1u);  // (given up: on without meaning, to the same barriers)
            __syncwarp();
            tc_after();
            const uint32_t bad = *reinterpret_cast<volatile uint32_t*>(&s_bad[(it + k) % kBadRing]);
            const uint32_t addr = tmem + lane_base + (uint32_t)b * C::kCols;
            const bool edge = all - p0 < kTile;  // a row does not see the whole tile
            float2 sum = make_float2(0.f, 0.f);
            for (int r0 = 0; r0 < rows; r0 += 16) {
              uint32_t v[16];
              Tmem<16>::load(addr + r0, v);
              float2 y[8];
              if constexpr (FP8) {
                uint32_t u[16];
                Tmem<16>::load(addr + pad + r0, u);
                tc_wait_ld();
#pragma unroll
                for (int i = 0; i < 8; ++i) {
                  const float2 s = fma2(make_float2(__uint_as_float(u[2 * i]), __uint_as_float(u[2 * i + 1])),
                                        make_float2(0.03125f, 0.03125f),
                                        make_float2(__uint_as_float(v[2 * i]), __uint_as_float(v[2 * i + 1])));
                  y[i] = fma2(s, *reinterpret_cast<const float2*>(&s_scale[buf][r0 + 2 * i]),
                              *reinterpret_cast<const float2*>(&s_less[buf][r0 + 2 * i]));
                }
              } else {
                const float2 sc = make_float2(s_scale[buf][0], s_scale[buf][0]);
                tc_wait_ld();
#pragma unroll
                for (int i = 0; i < 8; ++i)
                  y[i] = fma2(make_float2(__uint_as_float(v[2 * i]), __uint_as_float(v[2 * i + 1])), sc,
                              *reinterpret_cast<const float2*>(&s_less[buf][r0 + 2 * i]));
              }
              if (edge || r0 + 16 > rows) {
#pragma unroll
                for (int i = 0; i < 8; ++i) {
                  const int2 end = *reinterpret_cast<const int2*>(&s_end[buf][r0 + 2 * i]);
                  y[i].x = p < end.x ? exp2_sfu(y[i].x) : 0.f;
                  y[i].y = p < end.y ? exp2_sfu(y[i].y) : 0.f;
                }
              } else {
#pragma unroll
                for (int i = 0; i < 8; ++i) y[i] = make_float2(exp2_sfu(y[i].x), exp2_sfu(y[i].y));
              }
#pragma unroll
              for (int i = 0; i < 8; ++i) sum = add2(sum, y[i]);
            }
            tc_before();
            mbar_arrive(smem_u32(&s_empty[b]));
            float acc = sum.x + sum.y;
            if ((bad >> (t >> 4)) & 1u) acc = 0.f;
            if (x > 0) acc += s_acc[k * kTile + t];
            if (!last)
              s_acc[k * kTile + t] = acc;
            else if (mine)
              weight[p] = a.decay == 0.f ? acc : fmaf(a.decay, old, acc);
          }
          it += n;
          __syncwarp();
          if (lane == 0) mbar_arrive(smem_u32(&q_empty[buf]));
        }
      }
    } while (at.next(w, s_share));
  }
  tc_before();
  __syncthreads();
  tc_after();
  if (warp == C::kMmaWarp) free_tmem();
}

template <int D, bool FP8>
cudaError_t launch(const qsa_dims& d, const WeightArgs& a, const void* k_cache, bool short_k, cudaStream_t s) {
  using C = Wc<D, FP8>;
  alignas(64) CUtensorMap tk;
  if (!make_cache_map(&tk, d, k_cache, kTile, C::kLine, short_k)) return cudaErrorInvalidValue;
  static DeviceSlots slots;
  const cudaError_t e = slots.raise_smem(weight_kernel<C>, C::kSmem);
  if (e != cudaSuccess) return e;
  return launch_k(weight_kernel<C>, dim3(a.w.grid), dim3(C::kThreads), C::kSmem, s, true, tk, a);
}

}  // namespace

cudaError_t launch_kv_weight(const qsa_dims& d, float decay, const void* q, const void* k_cache, const float* k_scale,
                             const int32_t* page_table, const int32_t* q_pos, const float* lse, float* weight,
                             int32_t* err, cudaStream_t s, bool short_k) {
  WeightArgs a = {};
  DenseArgs& w = a.w;
  w.q = static_cast<const __nv_bfloat16*>(q);
  w.k_scale = k_scale;
  w.page_table = page_table;
  w.q_pos = q_pos;
  w.err = err;
  w.batch = d.batch;
  w.n_q = d.n_q;
  w.n_q_heads = d.n_q_heads;
  w.n_kv_heads = w.row_blocks = 1;  // a unit a request
  w.page_size = d.page_size;
  while ((1 << w.page_shift) < d.page_size) ++w.page_shift;
  w.max_pages = d.max_pages;
  w.num_pages = d.num_pages;
  w.grid = device_sm_count();
  w.sm_scale = d.sm_scale > 0.f ? d.sm_scale : 1.f / sqrtf((float)d.head_dim);
  a.lse = lse;
  a.weight = weight;
  a.hk = d.n_kv_heads;
  a.group = d.n_q_heads / d.n_kv_heads;
  a.blocks = (d.n_q * a.group + kRows - 1) / kRows;
  a.decay = decay;
  const bool fp8 = d.kv_dtype == QSA_KV_FP8_E4M3;
  switch (d.head_dim) {
    case 64: return fp8 ? launch<64, true>(d, a, k_cache, short_k, s) : launch<64, false>(d, a, k_cache, short_k, s);
    case 128: return fp8 ? launch<128, true>(d, a, k_cache, short_k, s) : launch<128, false>(d, a, k_cache, short_k, s);
    default: return fp8 ? launch<256, true>(d, a, k_cache, short_k, s) : launch<256, false>(d, a, k_cache, short_k, s);
  }
}

}  // namespace qsa
