// Dense attention over a prefix that all requests of a batch share.
//
// A request's own positions are worked on as in qsa_dense_tc.cuh, whose kernel
// reads K and V once a request. The prefix is read once for all: its rows are
// the queries of the whole batch, batch x n_q x group of a KV head, and with
// hundreds of them the two products are bound by the tensor cores, no longer by
// HBM (4 D flops a row and position against 4 D or 2 D bytes a position). So
// this kernel has the rows on the MMA's 128 rows (M), two such row tiles a CTA:
//   S[row][position] = Q K^T     (both from shared memory, S in tensor memory)
//   O[row][d]       += P V       (P in tensor memory, where S was)
// One thread owns one row of S and O (a TMEM lane): maxima, references and sums
// of a row's softmax need no other thread. The two row tiles take turns on the
// tensor cores: while one's softmax runs, the other's products do.
//
// The reference of a row: weights are 2^(s - mu), where mu only has to keep the
// largest weight between 1 and 2^8. It starts 6 below the row's first maximum
// and moves when a score passes mu + 8, which after a row's first tiles hardly
// happens; then O is rescaled in tensor memory by the row's thread.
//
// An E4M3 cache is widened to FP16 on its way (exactly: a code has 4 significant
// bits), by a warpgroup between the copies' buffers and the products'; with 256
// rows a CTA that is a small part of a tile's work, and both products then have
// FP16's 11 bits. Q is FP16 too: its row is scaled by a power of two so that its
// largest value is in [2^14, 2^15); BF16's 8 bits fit but below 2^-14, so a
// component is off by at most 2^-25, that is 2^-39 of the row's largest.
//
// A unit is a KV head and a group of row tiles; the prefix's tiles of every
// unit are cut into the same number of equal parts, one CTA each, chosen on the
// host so that the last wave of CTAs is full (plan). A CTA leaves (reference,
// sum, acc) of its rows in the workspace; a last kernel joins them with the
// pieces of the requests' own positions, in the order of the positions.
//
// The chain: own positions, prefix, joint, each launched while the one before
// runs out. The prefix kernel reads nothing that the first writes, so it does
// not wait for it before its work, only before its end.
#pragma once

#include "qsa_serve_internal.cuh"
#include "qsa_tc.cuh"

namespace qsa {

constexpr int kPrefixRows = 128;  // of a row tile

struct PrefixArgs {
  DenseArgs a;
  float* parts;    // [KV head][row tile][split] pieces: m[128], l[128], acc[128][D]
  int rows;        // of a KV head
  int row_tiles;   // of a KV head
  int units;       // KV heads x groups of row tiles
  int splits, tiles;
  int own_rows;    // of a unit of the requests' own positions
};

cudaError_t launch_prefix_64(const qsa_dims& d, const PrefixArgs& a, const void* k, const void* v, cudaStream_t s);
cudaError_t launch_prefix_128(const qsa_dims& d, const PrefixArgs& a, const void* k, const void* v, cudaStream_t s);
cudaError_t launch_prefix_256(const qsa_dims& d, const PrefixArgs& a, const void* k, const void* v, cudaStream_t s);

namespace {

// D: head dim, NT: row tiles of a CTA
template <int D_, bool FP8_, int NT_>
struct Pc {
  static constexpr bool FP8 = FP8_;
  static constexpr int D = D_, NT = NT_;
  static constexpr int T = D > 128 ? 64 : 128;  // positions of a tile (tensor memory: two S, NT O)
  static constexpr int kLines = D / 64;         // 128-byte lines of a row in 16 bits
  static constexpr int kSlot = T * D * 2;       // K or V of a tile
  static constexpr int kQ = 128 * D * 2;        // a row tile's Q
  static constexpr int kStage = T * D;          // E4M3 codes of K or V of a tile
  static constexpr int kStageLine = D < 128 ? D : 128, kStageLines = D / kStageLine;
  static constexpr int kStatic = 2048;
  static constexpr int kRoom = kMaxSmem - kStatic - 1024 - NT * kQ;
  static constexpr int kSlots = FP8 ? 4 : (kRoom / kSlot < 8 ? kRoom / kSlot : 8);
  static constexpr int kStages = FP8 ? ((kRoom - 4 * kSlot) / kStage < 8 ? (kRoom - 4 * kSlot) / kStage : 8) : 1;
  static constexpr int kUsed = NT * kQ + kSlots * kSlot + (FP8 ? kStages * kStage : 0);
  static constexpr int kOutPitch = D + 4;       // floats of a row on its way out
  static constexpr int kOut = NT * 128 * kOutPitch * 4;
  static constexpr int kSmem = (kUsed > kOut ? kUsed : kOut) + 1024;
  static constexpr int kSoft = NT * 128;        // softmax threads
  static constexpr int kWiden = FP8 ? 128 : 0;  // threads that widen
  static constexpr int kThreads = kSoft + kWiden + 64;
  static constexpr int kCopyWarp = (kSoft + kWiden) / 32, kMmaWarp = kCopyWarp + 1;
  static constexpr uint32_t kO = 2 * T;
  static constexpr uint32_t kNeed = 2 * T + NT * D;
  static constexpr uint32_t kTmem = kNeed <= 256 ? 256 : 512;
  static constexpr int kPieceFloats = kPrefixRows * (D + 2);
  static_assert(kSlots >= 4 && kStages >= 1 && kNeed <= 512 && kSmem + kStatic <= kMaxSmem, "memory");
};
constexpr int kBadTiles = 16;      // page marks of the tiles in flight
constexpr float kBelow = 6.f, kMost = 8.f;
constexpr float kNone = __builtin_huge_valf();  // the reference of a row that has seen nothing
constexpr float kHuge = 16777216.f;  // from a reference of this size on, a product less it is not fused (see less())

template <bool FP8>
__device__ __forceinline__ uint32_t pack16(float lo, float hi) {
  if constexpr (FP8) {
    const __half2 h = __floats2half2_rn(lo, hi);
    return *reinterpret_cast<const uint32_t*>(&h);
  } else {
    return pack_bf(lo, hi);
  }
}

template <class C>
__global__ void __launch_bounds__(C::kThreads, 1) prefix_kernel(const __grid_constant__ CUtensorMap tm_k,
                                                                const __grid_constant__ CUtensorMap tm_v,
                                                                const PrefixArgs pa) {
  constexpr bool FP8 = C::FP8;
  constexpr int D = C::D, T = C::T, NT = C::NT, kLines = C::kLines;
  const DenseArgs& a = pa.a;
  extern __shared__ uint8_t smem_raw[];
  uint8_t* ring = reinterpret_cast<uint8_t*>((reinterpret_cast<uintptr_t>(smem_raw) + 1023) & ~uintptr_t(1023));
  uint8_t* s_q = ring + C::kSlots * C::kSlot;
  uint8_t* stage = s_q + NT * C::kQ;
  __shared__ __align__(8) uint64_t slot_full[C::kSlots], slot_empty[C::kSlots];
  __shared__ __align__(8) uint64_t stage_full[C::kStages], stage_empty[C::kStages];
  __shared__ __align__(8) uint64_t s_full[2], p_full[2], pv_done[2], q_full, fin;
  __shared__ uint32_t s_tmem;
  __shared__ uint32_t s_bad[kBadTiles];  // bit i: positions 16 i .. 16 i + 15 of the tile have no page
  __shared__ volatile int s_abort;
  __shared__ float s_scale[C::kSoft];    // E4M3: a row's softmax scale
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;

  // the CTA's unit and its part of the prefix (CTAs of one part are neighbours: they read the same K and V)
  const int split = blockIdx.x / pa.units, unit = blockIdx.x - split * pa.units;
  const int groups = (pa.row_tiles + NT - 1) / NT, g = unit / groups, rt0 = (unit - g * groups) * NT;
  const int t0 = (int)((long long)split * pa.tiles / pa.splits);
  const int n = (int)((long long)(split + 1) * pa.tiles / pa.splits) - t0;

  if (tid == 0) {
    s_abort = 0;
    for (int s = 0; s < C::kSlots; ++s) {
      mbar_init(smem_u32(&slot_full[s]), FP8 ? 128 : 1);
      mbar_init(smem_u32(&slot_empty[s]), 1);
    }
    for (int s = 0; s < C::kStages; ++s) {
      mbar_init(smem_u32(&stage_full[s]), 1);
      mbar_init(smem_u32(&stage_empty[s]), 128);
    }
    for (int b = 0; b < 2; ++b) {
      mbar_init(smem_u32(&s_full[b]), 1);
      mbar_init(smem_u32(&p_full[b]), 128);
      mbar_init(smem_u32(&pv_done[b]), 1);
    }
    mbar_init(smem_u32(&q_full), C::kSoft);
    mbar_init(smem_u32(&fin), 1);
    asm volatile("fence.mbarrier_init.release.cluster;" ::: "memory");
  }
  if (warp == C::kMmaWarp) {
    asm volatile("tcgen05.alloc.cta_group::1.sync.aligned.shared::cta.b32 [%0], %1;" ::"r"(smem_u32(&s_tmem)),
                 "r"(C::kTmem)
                 : "memory");
    asm volatile("tcgen05.relinquish_alloc_permit.cta_group::1.sync.aligned;" ::: "memory");
  }
  // (The kernel in front, the own positions', was launched by the same call;
  // its CTAs let this one start behind their own wait, so all that this kernel
  // reads is older, and what it writes is read by nothing that still runs.)
  pdl_trigger();
  tc_before();
  __syncthreads();
  tc_after();
  const uint32_t tmem = s_tmem;
  auto wait = [&](uint64_t* bar, uint32_t parity) { return mbar_wait(bar, parity, &s_abort, a.err); };

  if (warp == C::kCopyWarp) {
    // ---- copies: K then V of each tile ----
    Walk<T> at{};
    at.t = t0;
    at.n = n;
    at.r = 0;
    at.g = Range{0, a.prefix_len};
    PageFeed<T> feed(a);
    feed.start(a, at);
    constexpr int kLine = FP8 ? C::kStageLine : 128, kCopyLines = FP8 ? C::kStageLines : kLines;
    constexpr int kRing = FP8 ? C::kStages : C::kSlots, kBytes = FP8 ? C::kStage : C::kSlot;
    uint8_t* base = FP8 ? stage : ring;
    uint64_t* full = FP8 ? stage_full : slot_full;
    uint64_t* empty = FP8 ? stage_empty : slot_empty;
    const int line = lane / feed.boxes;  // this lane's line of a K or V tile; at most 32 copies
    const uint32_t dst = (uint32_t)(line * (T * kLine) + (feed.my_box << feed.box_shift) * kLine);
    int slot = 0;
    uint32_t phase = 0;
    bool ok = true;
    for (int i = 0; i < n && ok; ++i) {
      const int page = feed.of_tile(a, at, i);
      const uint32_t bad = feed.bad_groups(page);
#pragma unroll
      for (int v = 0; v < 2; ++v) {
        if (!__all_sync(kFull, wait(&empty[slot], phase ^ 1u))) {
          ok = false;
          break;
        }
        const uint32_t bar = smem_u32(&full[slot]);
        if (lane == 0) {
          if (v == 0) s_bad[i % kBadTiles] = bad;
          mbar_expect_tx(bar, kBytes);
        }
        __syncwarp();
        if (line < kCopyLines)
          tma_load_4d(smem_u32(base + slot * kBytes) + dst, v ? &tm_v : &tm_k, line * (FP8 ? kLine : kLine / 2),
                      feed.slot_of(a, i), g, page < 0 ? a.num_pages : page /* outside: zeros */, bar);
        if (++slot == kRing) {
          slot = 0;
          phase ^= 1u;
        }
      }
    }
    if (s_abort) {  // copies in flight land before the CTA leaves (bounded)
      for (int s = 0; s < kRing; ++s) {
        const uint32_t par = s < slot ? phase : phase ^ 1u;
        const long long start = clock64();
        while (!mbar_try_wait(smem_u32(&full[s]), par) && clock64() - start < kWaitCycles / 64) {
        }
      }
    }
  } else if (warp == C::kMmaWarp) {
    // ---- both products (the whole warp walks the loop, one elected thread issues) ----
    // Step u is row tile u % NT of tile u / NT; S and P of it are in buffer u % 2.
    const bool one = elect_one();
    constexpr uint32_t kTypes = FP8 ? 0u : kTypeBf16;
    constexpr uint32_t kDescS = instr_desc(kTypes, false, false, T, 128);
    constexpr uint32_t kDescO = instr_desc(kTypes, false, true, D, 128);
    const int steps = NT * n;
    bool ok = __all_sync(kFull, wait(&q_full, 0));
    auto slot_ready = [&](int q) { return wait(&slot_full[q % C::kSlots], (uint32_t)(q / C::kSlots) & 1u); };
    auto score = [&](int u) {
      const int x = u % NT, i = u / NT, q = 2 * i, slot = q % C::kSlots;
      if (x == 0) ok = __all_sync(kFull, slot_ready(q));
      // P of step u - 2, which S of this one overwrites, has been read
      if (u >= 2) ok = __all_sync(kFull, ok && wait(&pv_done[u & 1], (uint32_t)((u - 2) >> 1) & 1u));
      if (!ok) return;
      tc_after();
      const uint64_t dq = smem_desc(smem_u32(s_q + x * C::kQ), 16, 1024, 2);
      const uint64_t dk = smem_desc(smem_u32(ring + slot * C::kSlot), 16, 1024, 2);
#pragma unroll
      for (int ks = 0; ks < D / 16; ++ks) {
        // (addresses are in units of 16 bytes)
        const uint32_t ln = (uint32_t)(ks / 4), in = (uint32_t)(ks % 4) * 2u;
        if (one)
          mma_tc<false>(tmem + (uint32_t)((u & 1) * T), dq + (ln * (128 * 128 / 16) + in), dk + (ln * (T * 128 / 16) + in),
                        kDescS, ks > 0);
      }
      if (one) {
        commit_tc(&s_full[u & 1]);
        if (x == NT - 1) commit_tc(&slot_empty[slot]);
      }
      __syncwarp();
    };
    if (ok) score(0);
    if (ok && steps > 1) score(1);
    for (int u = 0; u < steps && ok; ++u) {
      const int x = u % NT, i = u / NT, q = 2 * i + 1, slot = q % C::kSlots;
      ok = __all_sync(kFull, wait(&p_full[u & 1], (uint32_t)(u >> 1) & 1u) && (x > 0 || slot_ready(q)));
      if (!ok) break;
      tc_after();
      // V: positions as k; its columns are lines of 64 (leading offset: a line)
      const uint64_t dv = smem_desc(smem_u32(ring + slot * C::kSlot), kLines > 1 ? T * 128 : 0, 1024, 2);
#pragma unroll
      for (int ks = 0; ks < T / 16; ++ks)
        if (one)
          mma_ts(tmem + C::kO + (uint32_t)(x * D), tmem + (uint32_t)((u & 1) * T + ks * 8), dv + (uint32_t)(ks * 128), kDescO,
                 i > 0 || ks > 0);
      if (one) {
        commit_tc(&pv_done[u & 1]);
        if (x == NT - 1) commit_tc(&slot_empty[slot]);
      }
      __syncwarp();
      if (u + 2 < steps) score(u + 2);
    }
    // the tensor cores are done before the CTA gives its memory back
    if (one) commit_tc(&fin);
    const long long start = clock64();
    while (!mbar_try_wait(smem_u32(&fin), 0) && clock64() - start < 2 * kWaitCycles) {
    }
    __syncwarp();
  } else if (FP8 && tid >= C::kSoft) {
    // ---- E4M3 codes to FP16 tiles ----
    const int w = warp - C::kSoft / 32;
    // Eight lanes take the four 16-byte chunks of a line's half at rows r and
    // r + 4, and write the two chunks of each in opposite orders: no two in one
    // bank group.
    const int c4 = lane & 3, r8 = ((lane >> 3) & 3) + (lane & 4), flip = (lane >> 2) & 1;
    constexpr int kChunks8 = C::kStageLine / 16;
    int st = 0, slot = 0;
    uint32_t st_phase = 0, phase = 0;
    for (int q = 0; q < 2 * n; ++q) {
      wait(&stage_full[st], st_phase);
      wait(&slot_empty[slot], phase ^ 1u);  // (given up: on without meaning, to the end)
      const uint8_t* src = stage + st * C::kStage;
      uint8_t* dst = ring + slot * C::kSlot;
#pragma unroll 4
      for (int z = w; z < T / 8 * kLines; z += 4) {
        const int r = z / kLines * 8 + r8, ln = z % kLines, c = ln * 4 + c4;  // 16 codes: chunk c of the row
        const int sw = kChunks8 == 8 ? (c % 8) ^ (r & 7) : (c % 4) ^ ((r >> 1) & 3);
        const uint4 x = *reinterpret_cast<const uint4*>(src + c / kChunks8 * (T * C::kStageLine) + r * C::kStageLine + sw * 16);
        const uint4 lo = make_uint4(e4m3x2_to_h2(x.x), e4m3x2_to_h2(x.x >> 16), e4m3x2_to_h2(x.y), e4m3x2_to_h2(x.y >> 16));
        const uint4 hi = make_uint4(e4m3x2_to_h2(x.z), e4m3x2_to_h2(x.z >> 16), e4m3x2_to_h2(x.w), e4m3x2_to_h2(x.w >> 16));
        uint8_t* row = dst + ln * (T * 128) + r * 128;
        *reinterpret_cast<uint4*>(row + (((2 * c4 + flip) ^ (r & 7)) << 4)) = flip ? hi : lo;
        *reinterpret_cast<uint4*>(row + (((2 * c4 + 1 - flip) ^ (r & 7)) << 4)) = flip ? lo : hi;
      }
      mbar_arrive(smem_u32(&stage_empty[st]));
      async_fence();
      mbar_arrive(smem_u32(&slot_full[slot]));
      if (++st == C::kStages) {
        st = 0;
        st_phase ^= 1u;
      }
      if (++slot == C::kSlots) {
        slot = 0;
        phase ^= 1u;
      }
    }
  } else {
    // ---- softmax: a row a thread ----
    const int x = NT == 2 ? warp >> 2 : 0, t = tid & 127, rt = rt0 + x;
    const uint32_t lane_base = (uint32_t)((warp & 3) * 32) << 16;
    const float base_scale = a.sm_scale * kLog2e * (FP8 ? fabsf(a.k_scale[g]) : 1.f);
    {
      constexpr int kLanes = D / 8, kPass = 128 / kLanes;  // 8 components a lane
      uint8_t* dst = s_q + x * C::kQ;
#pragma unroll 4
      for (int r = t / kLanes; r < 128; r += kPass) {
        const int c = t % kLanes, row = rt * 128 + r;
        uint4 v = make_uint4(0, 0, 0, 0);
        if (row < pa.rows) {
          const int rj = row / a.group, h = g * a.group + (row - rj * a.group);
          v = ld16(a.q + ((size_t)rj * a.n_q_heads + h) * D + c * 8);
        }
        if constexpr (FP8) {
          uint32_t big = 0;  // magnitudes of BF16 values order like their bit patterns
          uint32_t wd[4] = {v.x, v.y, v.z, v.w};
#pragma unroll
          for (int e = 0; e < 4; ++e) big = max(big, max((wd[e] << 16) & 0x7fff0000u, wd[e] & 0x7fff0000u));
#pragma unroll
          for (int o = 1; o < kLanes; o <<= 1) big = max(big, __shfl_xor_sync(kFull, big, o));
          // 2^-sh brings the row's largest value into [2^14, 2^15)
          const int sh = big == 0 ? 0 : min(126, max(-126, (int)(big >> 23) - 127 - 14));
          // (a row with an infinity or NaN: every component NaN, as its scores
          // are; a negative scale of K goes into Q, so that a larger product is
          // a larger score)
          const float down = big >= 0x7f800000u ? __uint_as_float(0x7fffffffu) : a.k_scale[g] < 0.f ? -pow2(-sh) : pow2(-sh);
#pragma unroll
          for (int e = 0; e < 4; ++e) wd[e] = pack16<true>(bf_lo(wd[e]) * down, bf_hi(wd[e]) * down);
          v = make_uint4(wd[0], wd[1], wd[2], wd[3]);
          if (c == 0) s_scale[x * 128 + r] = base_scale * pow2(sh);
        }
        *reinterpret_cast<uint4*>(dst + c / 8 * (128 * 128) + r * 128 + (((c % 8) ^ (r & 7)) << 4)) = v;
      }
      async_fence();
      mbar_arrive(smem_u32(&q_full));
    }
    if constexpr (FP8) {  // (a row's scale is written by another thread of its warpgroup)
      asm volatile("bar.sync %0, 128;" ::"r"(1 + x) : "memory");
    }
    const float sc = FP8 ? s_scale[x * 128 + t] : base_scale;
    float mu = kNone;
    float2 l = make_float2(0.f, 0.f);
    for (int i = 0; i < n; ++i) {
      const int u = NT * i + x, b = u & 1;
      wait(&s_full[b], (uint32_t)(u >> 1) & 1u);  // (given up: on without meaning, to the end)
      __syncwarp();
      tc_after();
      const uint32_t bad = *reinterpret_cast<volatile uint32_t*>(&s_bad[i % kBadTiles]);
      const uint32_t addr = tmem + lane_base + (uint32_t)(b * T);
      // The largest product first, half of the columns at a time; the first
      // half's stay in registers.
      uint32_t v[64];
      float top = kNegInf;
      auto load64 = [&](int c0) {
        uint32_t h[32];
        Tmem<32>::load(addr + c0, h);
#pragma unroll
        for (int e = 0; e < 32; ++e) v[e] = h[e];
        Tmem<32>::load(addr + c0 + 32, h);
#pragma unroll
        for (int e = 0; e < 32; ++e) v[32 + e] = h[e];
        tc_wait_ld();
      };
      if (bad == 0) {
#pragma unroll
        for (int c0 = T - 64; c0 >= 0; c0 -= 64) {
          load64(c0);
#pragma unroll
          for (int e = 0; e < 64; e += 2) top = max3(top, __uint_as_float(v[e]), __uint_as_float(v[e + 1]));
        }
      } else {
#pragma unroll 1
        for (int c0 = 0; c0 < T; c0 += 16) {
          if ((bad >> (c0 >> 4)) & 1u) continue;
          uint32_t h[16];
          Tmem<16>::load(addr + c0, h);
          tc_wait_ld();
#pragma unroll
          for (int e = 0; e < 16; ++e) top = fmaxf(top, __uint_as_float(h[e]));
        }
      }
      top *= sc;
      const bool none = mu == kNone;
      const float up = none ? (top > kNegInf ? kMost + 1.f : 0.f) : top - mu;
      if (__any_sync(kFull, up > kMost)) {
        float f = 1.f;
        if (up > kMost) {
          const float to = top == kNone ? 0.f : top - kBelow;  // (an infinite score: its row is NaN)
          if (!none) f = exp2_sfu(mu - to);
          mu = to;
        }
        l = mul2(l, both(f));
        if (i > 0) {  // what O holds so far
          const int before = u - NT;
          wait(&pv_done[before & 1], (uint32_t)(before >> 1) & 1u);
          __syncwarp();
          tc_after();
#pragma unroll 1
          for (int c0 = 0; c0 < D; c0 += 16) {
            uint32_t o[16];
            Tmem<16>::load(tmem + lane_base + C::kO + (uint32_t)(x * D + c0), o);
            tc_wait_ld();
#pragma unroll
            for (int e = 0; e < 16; ++e) o[e] = __float_as_uint(__uint_as_float(o[e]) * f);
            Tmem<16>::store(tmem + lane_base + C::kO + (uint32_t)(x * D + c0), o);
          }
          tc_wait_st();
        }
      }
      const float nmu = mu == kNone ? 0.f : -mu;
      if (bad == 0 && !__any_sync(kFull, fabsf(nmu) >= kHuge)) {
        float2 sum[2] = {make_float2(0.f, 0.f), make_float2(0.f, 0.f)};
#pragma unroll
        for (int c0 = 0; c0 < T; c0 += 64) {
          if (c0 > 0) load64(c0);
          uint32_t p[32];
#pragma unroll
          for (int e = 0; e < 64; e += 2) {
            float2 y = fma2(pair(v + e), both(sc), both(nmu));
            y = make_float2(exp2_sfu(y.x), exp2_sfu(y.y));
            sum[(e >> 1) & 1] = add2(sum[(e >> 1) & 1], y);
            p[e / 2] = pack16<FP8>(y.x, y.y);
          }
          Tmem<32>::store(addr + (uint32_t)(c0 / 2), p);
        }
        l = add2(l, add2(sum[0], sum[1]));
      } else {
        // positions without a page, or references so large that a fused product's rounding would show
#pragma unroll 1
        for (int c0 = 0; c0 < T; c0 += 16) {
          uint32_t h[16], p[8];
          Tmem<16>::load(addr + c0, h);
          tc_wait_ld();
          const bool gone = (bad >> (c0 >> 4)) & 1u;
#pragma unroll
          for (int e = 0; e < 16; e += 2) {
            float2 y = less(pair(h + e), both(sc), both(a.one), both(nmu));
            y = gone ? make_float2(0.f, 0.f) : make_float2(exp2_sfu(y.x), exp2_sfu(y.y));
            l = add2(l, y);
            p[e / 2] = pack16<FP8>(y.x, y.y);
          }
          Tmem<8>::store(addr + (uint32_t)(c0 / 2), p);
          tc_wait_st();
        }
      }
      tc_wait_st();
      tc_before();
      mbar_arrive(smem_u32(&p_full[b]));
    }

    // ---- the piece: through shared memory, which nothing uses any more, so that rows leave whole ----
    // (not pv_done of the last step: the other row tile's phases are not followed
    // here, and a parity does not tell the last but one from the one before it)
    wait(&fin, 0);
    __syncwarp();
    tc_after();
    const float sum = l.x + l.y;
    const int row0 = rt * 128 + (warp & 3) * 32, live = min(32, pa.rows - row0);  // rows of this warp
    float* piece = pa.parts + ((size_t)(g * pa.row_tiles + rt) * pa.splits + split) * C::kPieceFloats;
    float* out = reinterpret_cast<float*>(ring) + (size_t)(x * 128 + (warp & 3) * 32) * C::kOutPitch;
#pragma unroll 1
    for (int c0 = 0; c0 < D; c0 += 32) {
      uint32_t o[32];
      Tmem<32>::load(tmem + lane_base + C::kO + (uint32_t)(x * D + c0), o);
      tc_wait_ld();
#pragma unroll
      for (int e = 0; e < 32; e += 4)
        *reinterpret_cast<uint4*>(out + lane * C::kOutPitch + c0 + e) = make_uint4(o[e], o[e + 1], o[e + 2], o[e + 3]);
    }
    __syncwarp();
    if (lane < live) {
      piece[t] = sum == 0.f ? kNegInf : mu;
      piece[128 + t] = sum;
    }
    constexpr int kVecs = D / 4;  // of a row
    float* dst = piece + 256 + (size_t)((warp & 3) * 32) * D;
    for (int z = lane; z < live * kVecs; z += 32) {
      const int r = z / kVecs, c = z % kVecs;
      *reinterpret_cast<uint4*>(dst + r * D + c * 4) = *reinterpret_cast<const uint4*>(out + r * C::kOutPitch + c * 4);
    }
  }
  tc_before();
  __syncthreads();
  tc_after();
  if (warp == C::kMmaWarp)
    asm volatile("tcgen05.dealloc.cta_group::1.sync.aligned.b32 %0, %1;" ::"r"(tmem), "r"(C::kTmem) : "memory");
  pdl_wait();  // this kernel's end stands for the own positions' too
}

// Joins the pieces of a row: the prefix's parts, then those of the request's own
// positions (as in dense_join_kernel). WARPS warps a row, the pieces dealt to
// them; WARPS 1: a block of kJoinRows rows.
template <int D, bool FP8, int WARPS>
__global__ void __launch_bounds__(WARPS > 1 ? 32 * WARPS : 32 * kJoinRows) prefix_join_kernel(const PrefixArgs pa) {
  constexpr int E = D / 32, kBatch = 8, TILE = 128;
  const DenseArgs& a = pa.a;
  __shared__ float s_m[WARPS], s_l[WARPS], s_acc[WARPS > 1 ? WARPS : 1][WARPS > 1 ? D : 1];
  const int lane = threadIdx.x & 31, warp = WARPS > 1 ? threadIdx.x >> 5 : 0;
  const int orow = WARPS > 1 ? blockIdx.x : blockIdx.x * kJoinRows + (threadIdx.x >> 5);
  if (WARPS == 1 && orow >= a.batch * a.n_q * a.n_q_heads) return;
  const int rj = orow / a.n_q_heads, h = orow - rj * a.n_q_heads, r = rj / a.n_q, j = rj - r * a.n_q;
  const int g = h / a.group, hg = h - g * a.group;
  const int i = j * a.group + hg, rb = i / pa.own_rows, own_row = i - rb * pa.own_rows;
  const int units = a.n_kv_heads * a.row_blocks, x = g * a.row_blocks + rb;
  // the request's own positions
  int c0 = 0, c1 = -1, first_slot = 0;  // pieces of CTAs c0 .. c1
  bool whole = false;
  auto unpack = [&](long long desc) {
    whole = desc == kUnitWhole;
    if (desc >= 0) {
      c0 = (int)(desc & 0xffffff);
      c1 = (int)((desc >> 24) & 0xffffff);
      first_slot = (int)(desc >> 48);
    }
  };
  if (a.batch <= kJoinScan) {
    long long all = 0, below = 0;
    for (int q = lane; q < a.batch; q += 32) {
      const long long t = load_of(range_of(a, q).tiles(TILE));
      all += t;
      below += q < r ? t : 0;
    }
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) {
      all += __shfl_xor_sync(kFull, all, o);
      below += __shfl_xor_sync(kFull, below, o);
    }
    const int tiles = range_of(a, r).tiles(TILE);
    if (tiles > 0) {
      Split sp;
      sp.init(a, all);
      const long long u = sp.slots(below) * units + (long long)x * (sp.seg + tiles);
      const int f = sp.first_cta(u), e = sp.last_cta(u, tiles);
      unpack(f == e ? kUnitWhole : unit_pieces(f, e, sp.piece_slot(u, f)));
    }
  }
  int p[kMaxNq];
#pragma unroll
  for (int q = 0; q < kMaxNq; ++q) p[q] = q < a.n_q ? a.q_pos[(size_t)r * a.n_q + q] : -1;
  const int mine = a.q_pos[(size_t)r * a.n_q + j];
  const int pre = sees_prefix(a, p) && valid_pos(a, mine) ? pa.splits : 0;
  const float vscale = FP8 ? a.v_scale[g] : 1.f;
  pdl_wait();
  if (a.batch > kJoinScan) unpack(a.unit_desc[(long long)r * units + x]);
  const int row = rj * a.group + hg, rt = row / kPrefixRows, pre_row = row % kPrefixRows;
  const float* pre_parts = pa.parts + (size_t)(g * pa.row_tiles + rt) * pa.splits * (kPrefixRows * (D + 2));
  const int own = whole ? 1 : c1 - c0 + 1, own_piece = pa.own_rows * (D + 2);
  float m = kNegInf, l = 0.f, acc[E];
#pragma unroll
  for (int e = 0; e < E; ++e) acc[e] = 0.f;
  for (int z = warp; z < pre + own; z += WARPS * kBatch) {
    float pm[kBatch], pl[kBatch], px[kBatch][E];
#pragma unroll
    for (int b = 0; b < kBatch; ++b) {
      const int y = z + b * WARPS;
      pm[b] = kNegInf;
      pl[b] = 0.f;
#pragma unroll
      for (int e = 0; e < E; ++e) px[b][e] = 0.f;
      if (y < pre + own) {
        const float* q;
        int rows, at;
        if (y < pre) {
          q = pre_parts + (size_t)y * (kPrefixRows * (D + 2));
          rows = kPrefixRows;
          at = pre_row;
        } else {
          const int c = c0 + y - pre;
          q = whole ? a.whole + ((size_t)r * units + x) * own_piece
                    : a.parts + ((size_t)c * 2 + (c == c0 ? first_slot : 0)) * own_piece;
          rows = pa.own_rows;
          at = own_row;
        }
        pm[b] = q[at];
        pl[b] = q[rows + at];
#pragma unroll
        for (int e = 0; e < E; ++e) px[b][e] = q[2 * rows + at * D + e * 32 + lane];
      }
    }
    float mn = m;
#pragma unroll
    for (int b = 0; b < kBatch; ++b) mn = fmaxf(mn, pm[b]);
    const float mu = mn == kNegInf ? 0.f : mn, f = exp2_sfu(m - mu);
    m = mn;
    l *= f;
#pragma unroll
    for (int e = 0; e < E; ++e) acc[e] *= f;
#pragma unroll
    for (int b = 0; b < kBatch; ++b) {
      const float w = exp2_sfu(pm[b] - mu);
      l = fmaf(pl[b], w, l);
      // (a row without weights has no meaning in its acc)
#pragma unroll
      for (int e = 0; e < E; ++e) acc[e] = pm[b] == kNegInf ? acc[e] : fmaf(px[b][e], w, acc[e]);
    }
  }
  if constexpr (WARPS > 1) {
    if (lane == 0) {
      s_m[warp] = m;
      s_l[warp] = l;
    }
#pragma unroll
    for (int e = 0; e < E; ++e) s_acc[warp][e * 32 + lane] = acc[e];
    __syncthreads();
    if (warp > 0) return;
    float big = kNegInf;
#pragma unroll
    for (int u = 0; u < WARPS; ++u) big = fmaxf(big, s_m[u]);
    const float mu = big == kNegInf ? 0.f : big;
    l = 0.f;
#pragma unroll
    for (int e = 0; e < E; ++e) acc[e] = 0.f;
#pragma unroll
    for (int u = 0; u < WARPS; ++u) {
      const float f = exp2_sfu(s_m[u] - mu);
      l += s_l[u] * f;
#pragma unroll
      for (int e = 0; e < E; ++e) acc[e] += s_acc[u][e * 32 + lane] * f;
    }
    m = big;
  }
  const float inv = vscale / l;
#pragma unroll
  for (int e = 0; e < E; ++e)
    a.out[(size_t)orow * D + e * 32 + lane] = __float2bfloat16_rn(l == 0.f ? 0.f : acc[e] * inv);
  if (a.lse && lane == 0) a.lse[orow] = l == 0.f ? kNegInf : (m + log2f(l)) * kLn2;
}

template <int D, bool FP8, int NT>
cudaError_t launch_prefix(const qsa_dims& d, const PrefixArgs& a, const void* k, const void* v, cudaStream_t s) {
  using C = Pc<D, FP8, NT>;
  alignas(64) CUtensorMap tk, tv;
  constexpr int kLine = FP8 ? C::kStageLine : 128;
  if (!make_cache_map(&tk, d, k, C::T, kLine, false) || !make_cache_map(&tv, d, v, C::T, kLine, false))
    return cudaErrorInvalidValue;
  static DeviceSlots slots;
  cudaError_t e = slots.raise_smem(prefix_kernel<C>, C::kSmem);
  if (e != cudaSuccess) return e;
  e = launch_k(prefix_kernel<C>, dim3((unsigned)a.units * a.splits), dim3(C::kThreads), C::kSmem, s, true, tk, tv, a);
  if (e != cudaSuccess) return e;
  // 4 warps a row where rows are few; with a warp a row their loads fill the GPU
  const unsigned rows = (unsigned)(a.a.batch * a.a.n_q * a.a.n_q_heads);
  if (rows < 8u * a.a.grid)
    return launch_k(prefix_join_kernel<D, FP8, 4>, dim3(rows), dim3(128), 0, s, true, a);
  return launch_k(prefix_join_kernel<D, FP8, 1>, dim3((rows + kJoinRows - 1) / kJoinRows), dim3(32 * kJoinRows), 0, s, true,
                  a);
}

}  // namespace
}  // namespace qsa
