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
// of a row's softmax need no other thread. Each row tile has a warp that issues
// its products, and the two take turns (P V, then the next S), so that one's
// products run while the other's softmax does: left to themselves both fell
// into step, softmax beside softmax and products behind products (a tile pair
// of 128 positions took 3,650 cycles; in turns 2,830, where the tensor cores'
// own time is 2,110), and one warp issuing for both lost as much, for what it
// does next waits until its MMAs have left the queue. Products with 64
// positions a step were slower (4,800): an MMA with Q from shared memory takes
// 66 cycles with 64 columns as with 128.
//
// The reference of a row: weights are 2^(s - mu), where mu only has to keep them
// in range. It starts 6 below the row's first tile's maximum, so that no maximum
// is needed before the exponentials of the tiles behind it; it moves when a
// weight has passed kMost (O is then rescaled in tensor memory by the row's
// thread before the next tile), and at once where there is no room left
// (kLimit).
//
// An E4M3 cache is widened to FP16 on its way (exactly: a code has 4 significant
// bits), by a warpgroup between the copies' buffers and the products'; with 256
// rows a CTA that is a small part of a tile's work, and both products then have
// FP16's 11 bits. Q is FP16 too: its row is scaled by a power of two so that its
// largest value is in [2^14, 2^15); BF16's 8 bits fit but below 2^-14, so a
// component is off by at most 2^-25, that is 2^-39 of the row's largest.
//
// A unit is a KV head and a group of row tiles; the prefix's tiles of every
// unit are cut into the same number of equal parts, one CTA each. A CTA leaves
// (reference, sum, acc) of its rows in the workspace; a last kernel joins them
// with the pieces of the requests' own positions, in the order of the positions.
//
// The chain: own positions, prefix, joint, each launched while the one before
// runs. The prefix kernel reads nothing that the first writes, so it does not
// wait for it before its work, only before its end; and the first one leaves it
// SMs of its own (shared_plan in qsa_dense.cuh).
//
// Measured: 32 requests x 4 queries x 16 heads (2 KV heads of 128) over 50,048
// shared and 4 to 6,401 own tokens, BF16: 66 us for the whole call, of which this
// kernel has 57 on two thirds of the SMs (tensor cores busy 39 % of the time of
// all, 53 % of its own SMs', HBM 11 %); E4M3 72. Both products at the measured
// BF16 rate on all SMs: 29.6. What is between: the SMs that the own positions'
// kernel has, 10 us of beginnings, ends and the join, the wait of the tensor
// cores for softmax in each tile.
#pragma once

#include "qsa_serve_internal.cuh"
#include "qsa_tc.cuh"

namespace qsa {

constexpr int kPrefixRows = 128;  // of a row tile

struct PrefixArgs {
  SharedArgs a;
  int32_t* n_parts;  // the parts of this call, from the kernel
  float* parts;    // [KV head][row tile][part] pieces: m[128], l[128], acc[128][D]
  int rows;        // of a KV head
  int row_tiles;   // of a KV head
  int units;       // KV heads x groups of row tiles
  int most;        // parts at most: the grid's
  int room;        // parts there is room for
  int own_rows;    // of a unit of the requests' own positions
};

// short_k: the failure-detection test (qsa_test_prefix_attn_timeout)
cudaError_t launch_prefix_64(const qsa_dims& d, const PrefixArgs& a, const void* k, const void* v, bool short_k,
                             cudaStream_t s);
cudaError_t launch_prefix_128(const qsa_dims& d, const PrefixArgs& a, const void* k, const void* v, bool short_k,
                              cudaStream_t s);
cudaError_t launch_prefix_256(const qsa_dims& d, const PrefixArgs& a, const void* k, const void* v, bool short_k,
                              cudaStream_t s);

namespace {

// D: head dim, NT: row tiles of a CTA
template <int D_, bool FP8_, int NT_>
struct Pc {
  static constexpr bool FP8 = FP8_;
  static constexpr int D = D_, NT = NT_;
  static constexpr int T = D > 128 ? 64 : 128;  // positions of a tile of K or V in shared memory
  static constexpr int kLines = D / 64;         // 128-byte lines of a row in 16 bits
  static constexpr int kSlot = T * D * 2;       // K or V of a tile
  static constexpr int kQ = 128 * D * 2;        // a row tile's Q
  static constexpr int kStage = T * D;          // E4M3 codes of K or V of a tile
  static constexpr int kStageLine = D < 128 ? D : 128, kStageLines = D / kStageLine;
  static constexpr int kStatic = 2048;
  static constexpr int kRoom = kMaxSmem - kStatic - 1024 - NT * kQ;
  // E4M3: what the products read is there soon after the copies have landed, so
  // the room is for copies on their way (four tiles of codes and three of FP16 at
  // head dim 128: 84 us at batch 32, two and four 93)
  static constexpr int kFit = kRoom / kSlot < 8 ? kRoom / kSlot : 8;
  static constexpr int kSlots = FP8 ? (kFit < 8 ? 3 : 4) : kFit;
  static constexpr int kLeft = (kRoom - kSlots * kSlot) / kStage;
  static constexpr int kStages = FP8 ? (kLeft < 8 ? kLeft : 8) : 1;
  static constexpr int kUsed = NT * kQ + kSlots * kSlot + (FP8 ? kStages * kStage : 0);
  static constexpr int kOutPitch = D + 4;       // floats of a row on its way out
  static constexpr int kOut = NT * 128 * kOutPitch * 4;
  static constexpr int kSmem = (kUsed > kOut ? kUsed : kOut) + 1024;
  static constexpr int kSoft = NT * 128;        // softmax threads
  static constexpr int kWiden = FP8 ? 128 : 0;  // threads that widen
  static constexpr int kThreads = kSoft + kWiden + 128;
  static constexpr int kCopyWarp = (kSoft + kWiden) / 32, kMmaWarp = kCopyWarp + 1;
  // Registers: a softmax thread holds a row of S. A launch of 256, 384 or 512
  // threads has 255, 168 or 128 a thread, of which the other warpgroups give
  // some up; the sums stay the launch's.
  static constexpr int kRegs = kThreads == 256 ? 255 : kThreads == 384 ? 168 : 128;
  static constexpr int kSoftRegs = kThreads == 512 ? 184 : FP8 ? 232 : 216;
  static constexpr int kOtherRegs = kThreads == 512 ? 72 : FP8 ? 136 : 72;
  static constexpr bool kSplit = kThreads > 256;
  static_assert(!kSplit || NT * kSoftRegs + (kThreads / 128 - NT) * kOtherRegs <= kThreads / 128 * kRegs, "registers");
  // query rows on their way: kLanes threads a row, 16 bytes each, kPass rows a pass
  static constexpr int kLanes = D / 8, kPass = 128 / kLanes, kPasses = 128 / kPass;
  static __device__ __forceinline__ int q_at(int x, int r, int c) {  // byte of 16-byte chunk c of row r of row tile x
    return x * kQ + c / 8 * (128 * 128) + r * 128 + (((c % 8) ^ (r & 7)) << 4);
  }
  static constexpr uint32_t kO = 2 * T;         // tensor memory: two S buffers (P where S was), then O
  static constexpr uint32_t kNeed = kO + NT * D;
  static constexpr uint32_t kTmem = kNeed <= 256 ? 256 : 512;
  // log2 of a weight that moves its row's reference before the next tile, and of
  // one that there is no room for: FP16 ends at 2^16; with BF16 the sums keep
  // room for V. (With 2^8, as in qsa_dense_tc.cuh, where the rows of a warp are
  // fewer and their tiles more, half of the warps' tiles began with a move.)
  static constexpr float kMost = FP8 ? 13.f : 20.f, kLimit = FP8 ? 15.f : 24.f;
  static constexpr int kPieceFloats = kPrefixRows * (D + 2);
  static_assert(kSlots >= 3 && kStages >= 1 && kNeed <= 512 && kSmem + kStatic <= kMaxSmem, "memory");
};
constexpr int kBadTiles = 16;  // page marks of the tiles in flight
constexpr float kBelow = 6.f;  // log2 of a row's first largest weight
constexpr float kNone = __builtin_huge_valf();  // the reference of a row that has seen nothing
constexpr float kHuge = 16777216.f;  // from a reference of this size on, a product less it is not fused (see less())

template <int N>
__device__ __forceinline__ void more_regs() {
  asm volatile("setmaxnreg.inc.sync.aligned.u32 %0;" ::"n"(N));
}
template <int N>
__device__ __forceinline__ void fewer_regs() {
  asm volatile("setmaxnreg.dec.sync.aligned.u32 %0;" ::"n"(N));
}
template <bool FP8>
__device__ __forceinline__ uint32_t pack16(float lo, float hi) {
  if constexpr (FP8) {
    const __half2 h = __floats2half2_rn(lo, hi);
    return *reinterpret_cast<const uint32_t*>(&h);
  } else {
    return pack_bf(lo, hi);
  }
}

// Parts of the prefix in this call (a whole warp).
__device__ __forceinline__ int prefix_parts(const SharedArgs& a) {
  if (a.batch > kJoinScan) return a.cost.parts;
  int tiles = 0, some = 0;  // of the requests' own positions, a unit of each
  for (int q = threadIdx.x & 31; q < a.batch; q += 32) {
    const int t = min(range_of(a, q).tiles(128), 1 << 20);  // (no sum past 2^28)
    tiles += t;
    some += t > 0;
  }
  const long long units = a.n_kv_heads * a.row_blocks;
  return shared_plan(a, __reduce_add_sync(kFull, tiles) * units, __reduce_add_sync(kFull, some) * units).parts;
}

template <class C>
__global__ void __launch_bounds__(C::kThreads, 1) prefix_kernel(const __grid_constant__ CUtensorMap tm_k,
                                                                const __grid_constant__ CUtensorMap tm_v,
                                                                const PrefixArgs pa) {
  constexpr bool FP8 = C::FP8;
  constexpr int D = C::D, T = C::T, NT = C::NT, kLines = C::kLines;
  const SharedArgs& a = pa.a;
  extern __shared__ uint8_t smem_raw[];
  uint8_t* ring = reinterpret_cast<uint8_t*>((reinterpret_cast<uintptr_t>(smem_raw) + 1023) & ~uintptr_t(1023));
  uint8_t* s_q = ring + C::kSlots * C::kSlot;
  uint8_t* stage = s_q + NT * C::kQ;
  __shared__ __align__(8) uint64_t slot_full[C::kSlots], slot_empty[C::kSlots];
  __shared__ __align__(8) uint64_t stage_full[C::kStages], stage_empty[C::kStages];
  __shared__ __align__(8) uint64_t s_full[2], pv_half[2], pv_done[2], q_full, turn[2], fin[2];
  __shared__ __align__(8) uint64_t p_full[2][2];  // [half][buffer]
  __shared__ uint32_t s_tmem;
  __shared__ int s_parts;
  __shared__ uint32_t s_bad[kBadTiles];  // bit i: positions 16 i .. 16 i + 15 of the tile have no page
  __shared__ volatile int s_abort;
  __shared__ float s_scale[C::kSoft];    // E4M3: a row's softmax scale
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;

  // the CTA's unit and its part of the prefix (CTAs of one part are neighbours: they read the same K and V)
  const int split = blockIdx.x / pa.units, unit = blockIdx.x - split * pa.units;
  const int groups = (pa.row_tiles + NT - 1) / NT, g = unit / groups, rt0 = (unit - g * groups) * NT;
  if (tid < C::kSoft) {
    // the query rows on their way, before anything that has to be waited for
    const int x = tid >> 7, t = tid & 127, c = t % C::kLanes;
    const int step_j = C::kPass / a.group, step_h = C::kPass - step_j * a.group;
    int row = (rt0 + x) * 128 + t / C::kLanes, rj = row / a.group, hg = row - rj * a.group;
#pragma unroll 4
    for (int z = 0; z < C::kPasses; ++z) {
      const bool live = row < pa.rows;  // (behind the last: zeros)
      const void* src = live ? a.q + ((size_t)rj * a.n_q_heads + g * a.group + hg) * D + c * 8 : a.q;
      asm volatile("cp.async.cg.shared.global [%0], [%1], 16, %2;" ::"r"(
                       smem_u32(s_q + C::q_at(x, z * C::kPass + t / C::kLanes, c))),
                   "l"(src), "r"(live ? 16 : 0)
                   : "memory");
      row += C::kPass;
      rj += step_j;
      hg += step_h;
      if (hg >= a.group) {
        hg -= a.group;
        ++rj;
      }
    }
  }
  if (tid == 0) {
    s_abort = 0;
    for (int s = 0; s < C::kSlots; ++s) {
      mbar_init(smem_u32(&slot_full[s]), FP8 ? 128 : 1);
      mbar_init(smem_u32(&slot_empty[s]), NT);
    }
    for (int s = 0; s < C::kStages; ++s) {
      mbar_init(smem_u32(&stage_full[s]), 1);
      mbar_init(smem_u32(&stage_empty[s]), 128);
    }
    for (int b = 0; b < 2; ++b) {
      mbar_init(smem_u32(&s_full[b]), 1);
      mbar_init(smem_u32(&p_full[0][b]), 128);
      mbar_init(smem_u32(&p_full[1][b]), 128);
      mbar_init(smem_u32(&pv_half[b]), 1);
      mbar_init(smem_u32(&turn[b]), 1);
      mbar_init(smem_u32(&fin[b]), 1);
      mbar_init(smem_u32(&pv_done[b]), 1);
    }
    mbar_init(smem_u32(&q_full), C::kSoft);
    asm volatile("fence.mbarrier_init.release.cluster;" ::: "memory");
  }
  if (warp == C::kMmaWarp) {
    asm volatile("tcgen05.alloc.cta_group::1.sync.aligned.shared::cta.b32 [%0], %1;" ::"r"(smem_u32(&s_tmem)),
                 "r"(C::kTmem)
                 : "memory");
    asm volatile("tcgen05.relinquish_alloc_permit.cta_group::1.sync.aligned;" ::: "memory");
  }
  if (warp == C::kCopyWarp) {
    const int parts = prefix_parts(a);
    if (lane == 0) s_parts = parts;
    if (lane == 0 && blockIdx.x == 0) *pa.n_parts = parts;
  }
  // (The kernel in front, the own positions', was launched by the same call;
  // its CTAs let this one start behind their own wait, so all that this kernel
  // reads is older, and what it writes is read by nothing that still runs.)
  pdl_trigger();
  tc_before();
  __syncthreads();
  tc_after();
  const uint32_t tmem = s_tmem;
  const int parts = s_parts;
  const bool spare = split >= parts;  // (part 0 always has CTAs: the kernel's end is theirs)
  const int t0 = (int)((long long)split * a.cost.tiles / parts);
  const int n = spare ? 0 : (int)((long long)(split + 1) * a.cost.tiles / parts) - t0;
  auto wait = [&](uint64_t* bar, uint32_t parity) { return mbar_wait(bar, parity, &s_abort, a.err); };

  if (spare) {
    asm volatile("cp.async.wait_all;" ::: "memory");
  } else if (tid >= C::kSoft + C::kWiden) {
    if constexpr (C::kSplit) fewer_regs<C::kOtherRegs>();  // (a whole warpgroup, two warps of which have no work)
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
    } else if (warp < C::kMmaWarp + NT) {
      // ---- both products of a row tile (a warp each; the whole warp walks the loop, one elected thread issues) ----
      // With one row tile S of tile i + 1 is computed before P of tile i is there
      // (two buffers); with two, the other row tile's products fill that time.
      const bool one = elect_one();
      constexpr uint32_t kTypes = FP8 ? 0u : kTypeBf16;
      constexpr uint32_t kDescS = instr_desc(kTypes, false, false, T, 128);
      constexpr uint32_t kDescO = instr_desc(kTypes, false, true, D, 128);
      const int x = warp - C::kMmaWarp;
      bool ok = wait(&q_full, 0);
      auto slot_ready = [&](int q) { return wait(&slot_full[q % C::kSlots], (uint32_t)(q / C::kSlots) & 1u); };
      auto buffer = [&](int i) { return NT == 2 ? x : i & 1; };
      auto phase = [&](int i) { return (uint32_t)(NT == 2 ? i : i >> 1) & 1u; };
      auto score = [&](int i) {
        const int slot = 2 * i % C::kSlots, b = buffer(i);
        ok = ok && slot_ready(2 * i);
        // P of the step before in this buffer, which S overwrites, has been read
        constexpr int kBack = NT == 2 ? 1 : 2;
        if (i >= kBack) ok = ok && wait(&pv_done[b], phase(i - kBack));
        ok = __all_sync(kFull, ok);
        if (!ok) return;
        tc_after();
        // (passed on before S is issued: behind its MMAs the arrival would wait for them)
        if (NT == 2 && i > 0 && one) mbar_arrive(smem_u32(&turn[x ^ 1]));
        const uint64_t dq = smem_desc(smem_u32(s_q + x * C::kQ), 16, 1024, 2);
        const uint64_t dk = smem_desc(smem_u32(ring + slot * C::kSlot), 16, 1024, 2);
#pragma unroll
        for (int ks = 0; ks < D / 16; ++ks) {
          // (addresses are in units of 16 bytes)
          const uint32_t ln = (uint32_t)(ks / 4), in = (uint32_t)(ks % 4) * 2u;
          if (one)
            mma_tc<false>(tmem + (uint32_t)(b * T), dq + (ln * (128 * 128 / 16) + in), dk + (ln * (T * 128 / 16) + in),
                          kDescS, ks > 0);
        }
        if (one) {
          commit_tc(&s_full[b]);
          commit_tc(&slot_empty[slot]);
        }
        __syncwarp();
      };
      score(0);
      if (NT == 1 && n > 1 && ok) score(1);
      for (int i = 0; i < n && ok; ++i) {
        const int q = 2 * i + 1, slot = q % C::kSlots, b = buffer(i);
        // V: positions as k; its columns are lines of 64 (leading offset: a line)
        const uint64_t dv = smem_desc(smem_u32(ring + slot * C::kSlot), kLines > 1 ? T * 128 : 0, 1024, 2);
        ok = slot_ready(q);
#pragma unroll
        for (int h = 0; h < 2; ++h) {  // half of the positions as soon as their weights are there
          ok = __all_sync(kFull, ok && wait(&p_full[h][b], phase(i)));
          // the row tiles take turns
          if (NT == 2 && h == 0 && i + x > 0) ok = __all_sync(kFull, ok && wait(&turn[x], (uint32_t)(i - 1 + x) & 1u));
          if (!ok) break;
          tc_after();
#pragma unroll
          for (int ks = h * (T / 32); ks < (h + 1) * (T / 32); ++ks)
            if (one)
              mma_ts(tmem + C::kO + (uint32_t)(x * D), tmem + (uint32_t)(b * T + ks * 8), dv + (uint32_t)(ks * 128),
                     kDescO, i > 0 || ks > 0);
          if (one && h == 0) commit_tc(&pv_half[b]);
        }
        if (!ok) break;
        if (one) {
          commit_tc(&pv_done[b]);
          commit_tc(&slot_empty[slot]);
        }
        __syncwarp();
        if (i + (NT == 2 ? 1 : 2) < n)
          score(i + (NT == 2 ? 1 : 2));
        else if (NT == 2 && one)
          mbar_arrive(smem_u32(&turn[x ^ 1]));
      }
      // the tensor cores are done before the CTA gives its memory back
      if (one) commit_tc(&fin[x]);
      const long long start = clock64();
      while (!mbar_try_wait(smem_u32(&fin[x]), 0) && clock64() - start < 2 * kWaitCycles) {
      }
      __syncwarp();
    }
  } else if (FP8 && tid >= C::kSoft) {
    // ---- E4M3 codes to FP16 tiles ----
    if constexpr (C::kSplit) fewer_regs<C::kOtherRegs>();
    const int w = warp - C::kSoft / 32;
    // Eight lanes take the four 16-byte chunks of a line's half at rows r and
    // r + 4, and write the two chunks of each in opposite orders: no two in one
    // bank group.
    const int c4 = lane & 3, r8 = ((lane >> 3) & 3) + (lane & 4), flip = (lane >> 2) & 1;
    constexpr int kChunks8 = C::kStageLine / 16;
    int st = 0, slot = 0;
    uint32_t st_phase = 0, phase = 0;
    for (int q = 0; q < 2 * n; ++q) {
      // (Given up: nothing is waited for here any more but the kernel's end. An
      // arrival for a copy that has not landed would let the next one be announced
      // at a barrier whose phase is not over, and its count fall below zero.)
      if (!__all_sync(kFull, wait(&stage_full[st], st_phase) && wait(&slot_empty[slot], phase ^ 1u))) break;
      const uint8_t* src = stage + st * C::kStage;
      uint8_t* dst = ring + slot * C::kSlot;
#pragma unroll 4
      for (int z = w; z < T / 8 * kLines; z += 4) {
        const int r = z / kLines * 8 + r8, ln = z % kLines, c = ln * 4 + c4;  // 16 codes: chunk c of the row
        const int sw = kChunks8 == 8 ? (c % 8) ^ (r & 7) : (c % 4) ^ ((r >> 1) & 3);
        const uint8_t* from = src + c / kChunks8 * (T * C::kStageLine) + r * C::kStageLine + sw * 16;
        const uint4 x = *reinterpret_cast<const uint4*>(from);
        auto widen = [](uint32_t u, uint32_t v) {
          return make_uint4(e4m3x2_to_h2(u), e4m3x2_to_h2(u >> 16), e4m3x2_to_h2(v), e4m3x2_to_h2(v >> 16));
        };
        const uint4 lo = widen(x.x, x.y), hi = widen(x.z, x.w);
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
    if constexpr (C::kSplit) more_regs<C::kSoftRegs>();
    const int x = NT == 2 ? warp >> 2 : 0, t = tid & 127, rt = rt0 + x;
    const uint32_t lane_base = (uint32_t)((warp & 3) * 32) << 16;
    const float base_scale = a.sm_scale * kLog2e * (FP8 ? fabsf(a.k_scale[g]) : 1.f);
    asm volatile("cp.async.wait_all;" ::: "memory");
    if constexpr (FP8) {  // in place: a thread's own 16 bytes of kDeep rows at a time, the rows' shuffles side by side
      const float sign = a.k_scale[g] < 0.f ? -1.f : 1.f;
      constexpr int kDeep = 4;  // (16: its code, read once, took 1.5 us longer)
#pragma unroll 1
      for (int z0 = 0; z0 < C::kPasses; z0 += kDeep) {
        uint4 w[kDeep];
        uint32_t bigs[kDeep];
#pragma unroll
        for (int z = 0; z < kDeep; ++z) {
          w[z] = *reinterpret_cast<const uint4*>(s_q + C::q_at(x, (z0 + z) * C::kPass + t / C::kLanes, t % C::kLanes));
          const uint32_t wd[4] = {w[z].x, w[z].y, w[z].z, w[z].w};
          bigs[z] = 0;  // magnitudes of BF16 values order like their bit patterns
#pragma unroll
          for (int e = 0; e < 4; ++e) bigs[z] = max(bigs[z], max((wd[e] << 16) & 0x7fff0000u, wd[e] & 0x7fff0000u));
        }
#pragma unroll
        for (int o = 1; o < C::kLanes; o <<= 1)
#pragma unroll
          for (int z = 0; z < kDeep; ++z) bigs[z] = max(bigs[z], __shfl_xor_sync(kFull, bigs[z], o));
#pragma unroll
        for (int z = 0; z < kDeep; ++z) {
          const int r = (z0 + z) * C::kPass + t / C::kLanes, c = t % C::kLanes;
          const uint32_t big = bigs[z];
          uint32_t wd[4] = {w[z].x, w[z].y, w[z].z, w[z].w};
          // 2^-sh brings the row's largest value into [2^14, 2^15)
          const int sh = big == 0 ? 0 : min(126, max(-126, (int)(big >> 23) - 127 - 14));
          // (a row with an infinity or NaN: every component NaN, as its scores
          // are; a negative scale of K goes into Q, so that a larger product is
          // a larger score)
          const float down = big >= 0x7f800000u ? __uint_as_float(0x7fffffffu) : sign * pow2(-sh);
#pragma unroll
          for (int e = 0; e < 4; ++e) wd[e] = pack16<true>(bf_lo(wd[e]) * down, bf_hi(wd[e]) * down);
          *reinterpret_cast<uint4*>(s_q + C::q_at(x, r, c)) = make_uint4(wd[0], wd[1], wd[2], wd[3]);
          if (c == 0) s_scale[x * 128 + r] = base_scale * pow2(sh);
        }
      }
    }
    async_fence();
    mbar_arrive(smem_u32(&q_full));
    if constexpr (FP8) {  // (a row's scale is written by another thread of its warpgroup)
      asm volatile("bar.sync %0, 128;" ::"r"(1 + x) : "memory");
    }
    float sc = FP8 ? s_scale[x * 128 + t] : base_scale;
    // (every score is about 0 then; a product with an absent position's -inf is no NaN)
    if (FP8 && sc == 0.f) sc = 0x1p-126f;
    float mu = kNone, pending = 0.f;  // pending: how far the tile before went past the reference
    float2 l = make_float2(0.f, 0.f);
    const uint32_t o_addr = tmem + lane_base + C::kO + (uint32_t)(x * D);
    // The reference moves to `to`: the sum and, where it holds anything, O follow.
    // `bar` is the products of P so far.
    auto move_to = [&](float to, bool any, uint64_t* bar, uint32_t parity) {
      const float f = mu == kNone ? 1.f : exp2_sfu(mu - to);
      mu = to;
      l = mul2(l, both(f));
      if (!any) return;
      wait(bar, parity);
      __syncwarp();
      tc_after();
#pragma unroll 1
      for (int c0 = 0; c0 < D; c0 += 16) {
        uint32_t o[16];
        Tmem<16>::load(o_addr + c0, o);
        tc_wait_ld();
#pragma unroll
        for (int e = 0; e < 16; ++e) o[e] = __float_as_uint(__uint_as_float(o[e]) * f);
        Tmem<16>::store(o_addr + c0, o);
      }
      tc_wait_st();
    };
    for (int i = 0; i < n; ++i) {
      const int b = NT == 2 ? x : i & 1;
      const uint32_t phase = (uint32_t)(NT == 2 ? i : i >> 1) & 1u;
      // the products of the tile before: its buffer, its phase
      uint64_t* before = &pv_done[NT == 2 ? x : (i - 1) & 1];
      const uint32_t before_phase = (uint32_t)(NT == 2 ? i - 1 : (i - 1) >> 1) & 1u;
      wait(&s_full[b], phase);  // (given up: on without meaning, to the end)
      __syncwarp();
      tc_after();
      const uint32_t bad = *reinterpret_cast<volatile uint32_t*>(&s_bad[i % kBadTiles]);
      const uint32_t addr = tmem + lane_base + (uint32_t)(b * T);
      // 32 columns at a time, the next ones on their way
      constexpr int kParts = T / 32;
      uint32_t v[2][32];
      Tmem<32>::load(addr, v[0]);
      if (i == 0) {  // the first maximum
        float top = kNegInf;
#pragma unroll
        for (int k = 0; k < kParts; ++k) {
          tc_wait_ld(v[k & 1]);
          Tmem<32>::load(addr + (uint32_t)((k + 1) % kParts * 32), v[(k + 1) & 1]);
#pragma unroll
          for (int e = 0; e < 32; ++e)
            if (!((bad >> (2 * k + (e >> 4))) & 1u)) top = fmaxf(top, __uint_as_float(v[k & 1][e]));
        }
        top *= sc;
        if (top > kNegInf && top < kNone) mu = top - kBelow;
      } else if (__any_sync(kFull, pending > C::kMost)) {
        move_to(pending > C::kMost ? mu + (pending - kBelow) : mu, true, before, before_phase);
      }
      pending = 0.f;
#pragma unroll
      for (int h = 0; h < 2; ++h) {
        const float nmu = mu == kNone ? 0.f : -mu;
        float2 sum[2] = {make_float2(0.f, 0.f), make_float2(0.f, 0.f)};
        float tops[2] = {kNegInf, kNegInf};
        uint32_t p[T / 4];
#pragma unroll
        for (int k = h * (kParts / 2); k < (h + 1) * (kParts / 2); ++k) {
          uint32_t(&w)[32] = v[k & 1];
          tc_wait_ld(w);
          if (k + 1 < kParts) Tmem<32>::load(addr + (uint32_t)((k + 1) * 32), v[(k + 1) & 1]);
          if (((bad >> (2 * k)) & 3u) != 0) {  // positions without a page
#pragma unroll
            for (int e = 0; e < 32; ++e)
              if ((bad >> (2 * k + (e >> 4))) & 1u) w[e] = __float_as_uint(kNegInf);
          }
#pragma unroll
          for (int e = 0; e < 32; e += 2) {
            float2 y = fma2(pair(w + e), both(sc), both(nmu));
            tops[(e >> 1) & 1] = max3(tops[(e >> 1) & 1], y.x, y.y);
            y = make_float2(exp2_sfu(y.x), exp2_sfu(y.y));
            sum[(e >> 1) & 1] = add2(sum[(e >> 1) & 1], y);
            p[(k - h * (kParts / 2)) * 16 + e / 2] = pack16<FP8>(y.x, y.y);
          }
        }
        const float top = fmaxf(tops[0], tops[1]);
        if (!__any_sync(kFull, top > C::kLimit || mu == kNone || fabsf(mu) >= kHuge)) {
          pending = fmaxf(pending, top);
          l = add2(l, add2(sum[0], sum[1]));
          Tmem<T / 4>::store(addr + (uint32_t)(h * (T / 4)), p);
        } else {
          // A weight with no room left, a row that has seen nothing yet, or a
          // reference so large that a fused product's rounding would show: again
          // from tensor memory, maximum first, and with the product rounded.
          float big = kNegInf;
#pragma unroll 1
          for (int c0 = h * (T / 2); c0 < (h + 1) * (T / 2); c0 += 16) {
            uint32_t s16[16];
            Tmem<16>::load(addr + c0, s16);
            tc_wait_ld();
            if ((bad >> (c0 >> 4)) & 1u) continue;
#pragma unroll
            for (int e = 0; e < 16; ++e) big = fmaxf(big, __uint_as_float(s16[e]));
          }
          big *= sc;
          const bool up = mu == kNone ? big > kNegInf : big - mu > C::kMost;
          const float to = !up ? mu : big == kNone ? 0.f : big - kBelow;  // (an infinite score: its row is NaN)
          if (h == 0)
            move_to(to, i > 0, before, before_phase);
          else
            move_to(to, true, &pv_half[b], phase);
          const float less_mu = mu == kNone ? 0.f : -mu;
#pragma unroll 1
          for (int c0 = h * (T / 2); c0 < (h + 1) * (T / 2); c0 += 16) {
            uint32_t s16[16], q[8];
            Tmem<16>::load(addr + c0, s16);
            tc_wait_ld();
            const bool gone = (bad >> (c0 >> 4)) & 1u;
#pragma unroll
            for (int e = 0; e < 16; e += 2) {
              float2 y = less(pair(s16 + e), both(sc), both(a.one), both(less_mu));
              y = gone ? make_float2(0.f, 0.f) : make_float2(exp2_sfu(y.x), exp2_sfu(y.y));
              l = add2(l, y);
              q[e / 2] = pack16<FP8>(y.x, y.y);
            }
            Tmem<8>::store(addr + (uint32_t)(c0 / 2), q);
            tc_wait_st();
          }
        }
        tc_wait_st();
        tc_before();
        mbar_arrive(smem_u32(&p_full[h][b]));
      }
    }

    // ---- the piece: through shared memory, which nothing uses any more, so that rows leave whole ----
    // (the other row tile's products may still read it: both warps' ends)
#pragma unroll
    for (int z = 0; z < NT; ++z) wait(&fin[z], 0);
    __syncwarp();
    tc_after();
    const float sum = l.x + l.y;
    const int row0 = rt * 128 + (warp & 3) * 32, live = min(32, pa.rows - row0);  // rows of this warp
    float* piece = pa.parts + ((size_t)(g * pa.row_tiles + rt) * pa.room + split) * C::kPieceFloats;
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
    async_fence();
    __syncwarp();
    if (lane < live) {  // a row each, by bulk copies
      float* dst = piece + 256 + (size_t)((warp & 3) * 32 + lane) * D;
      asm volatile("cp.async.bulk.global.shared::cta.bulk_group [%0], [%1], %2;" ::"l"(dst),
                   "r"(smem_u32(out + lane * C::kOutPitch)), "n"(D * 4)
                   : "memory");
    }
    asm volatile("cp.async.bulk.commit_group;\n\tcp.async.bulk.wait_group 0;" ::: "memory");
  }
  tc_before();
  __syncthreads();
  tc_after();
  if (warp == C::kMmaWarp)
    asm volatile("tcgen05.dealloc.cta_group::1.sync.aligned.b32 %0, %1;" ::"r"(tmem), "r"(C::kTmem) : "memory");
  if (!spare) pdl_wait();  // this kernel's end stands for the own positions' too
}

// Joins the pieces of a row: the prefix's parts, then those of the request's own
// positions (as in dense_join_kernel). WARPS warps a row, the pieces dealt to
// them; WARPS 1: a block of kJoinRows rows.
template <int D, bool FP8, int WARPS>
__global__ void __launch_bounds__(WARPS > 1 ? 32 * WARPS : 32 * kJoinRows) prefix_join_kernel(const PrefixArgs pa) {
  // (pieces on their way: 12 for a warp a row, 8 where 4 share one; 8 for a warp
  // 1.2 us slower at 2,048 rows, 12 for 4 warps 2 us at 1,024)
  constexpr int E = D / 32, kBatch = WARPS > 1 ? 8 : 12, TILE = 128;
  const SharedArgs& a = pa.a;
  __shared__ float s_m[WARPS], s_l[WARPS], s_acc[WARPS > 1 ? WARPS : 1][WARPS > 1 ? D : 1];
  const int lane = threadIdx.x & 31, warp = WARPS > 1 ? threadIdx.x >> 5 : 0;
  const int orow = WARPS > 1 ? blockIdx.x : blockIdx.x * kJoinRows + (threadIdx.x >> 5);
  if (WARPS == 1 && orow >= a.batch * a.n_q * a.n_q_heads) return;
  const int rj = orow / a.n_q_heads, h = orow - rj * a.n_q_heads, r = rj / a.n_q, j = rj - r * a.n_q;
  const int g = h / a.group, hg = h - g * a.group;
  const int i = j * a.group + hg, rb = i / pa.own_rows, own_row = i - rb * pa.own_rows;
  const int units = a.n_kv_heads * a.row_blocks, x = g * a.row_blocks + rb;
  int p[kMaxNq];
#pragma unroll
  for (int q = 0; q < kMaxNq; ++q) p[q] = q < a.n_q ? a.q_pos[(size_t)r * a.n_q + q] : -1;
  const int mine = a.q_pos[(size_t)r * a.n_q + j];
  const bool sees = sees_prefix(a, p) && valid_pos(a, mine), has_own = range_of(a, r).tiles(TILE) > 0;
  const float vscale = FP8 ? a.v_scale[g] : 1.f;
  pdl_wait();
  // The pieces: both kernels leave word of them. (Worked out here from q_pos, as
  // dense_join_kernel does, they took every block 3 us where rows are many: 64
  // requests x 16 heads 10.5 us from the prefix kernel's end to this one's.)
  // (Bounded, so that a workspace that was overwritten leads to no read outside it.)
  const int pre = sees ? max(0, min(*pa.n_parts, pa.room)) : 0;
  int c0 = 0, c1 = -1, first_slot = 0;  // pieces of CTAs c0 .. c1
  bool whole = false;
  if (has_own) {
    const long long desc = a.unit_desc[(long long)r * units + x];
    whole = desc == kUnitWhole;
    if (desc >= 0) {
      c0 = (int)(desc & 0xffffff);
      c1 = min((int)((desc >> 24) & 0xffffff), a.grid - 1);
      first_slot = (int)(desc >> 48) & 1;
    }
  }
  const int row = rj * a.group + hg, rt = row / kPrefixRows, pre_row = row % kPrefixRows;
  const float* pre_parts = pa.parts + (size_t)(g * pa.row_tiles + rt) * pa.room * (kPrefixRows * (D + 2));
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
cudaError_t launch_prefix(const qsa_dims& d, const PrefixArgs& a, const void* k, const void* v, bool short_k,
                          cudaStream_t s) {
  using C = Pc<D, FP8, NT>;
  alignas(64) CUtensorMap tk, tv;
  constexpr int kLine = FP8 ? C::kStageLine : 128;
  if (!make_cache_map(&tk, d, k, C::T, kLine, short_k) || !make_cache_map(&tv, d, v, C::T, kLine, false))
    return cudaErrorInvalidValue;
  static DeviceSlots slots, regs;
  cudaError_t e = slots.raise_smem(prefix_kernel<C>, C::kSmem);
  if (e != cudaSuccess) return e;
  if (C::kSplit) {  // the warpgroups' shares are of what the launch has
    const int n = regs.get([] {
      cudaFuncAttributes at;
      return cudaFuncGetAttributes(&at, prefix_kernel<C>) == cudaSuccess ? at.numRegs : 0;
    });
    if (n != C::kRegs) return cudaErrorInvalidKernelImage;
  }
  e = launch_k(prefix_kernel<C>, dim3((unsigned)a.units * a.most), dim3(C::kThreads), C::kSmem, s, true, tk, tv, a);
  if (e != cudaSuccess) return e;
  // 4 warps a row where rows are few; else a warp a row (2,048 rows of 20 to 25
  // pieces: 4 warps each made the whole call 1.8 us slower, 2 no faster)
  const unsigned rows = (unsigned)(a.a.batch * a.a.n_q * a.a.n_q_heads);
  if (rows < 8u * a.a.grid)
    return launch_k(prefix_join_kernel<D, FP8, 4>, dim3(rows), dim3(128), 0, s, true, a);
  return launch_k(prefix_join_kernel<D, FP8, 1>, dim3((rows + kJoinRows - 1) / kJoinRows), dim3(32 * kJoinRows), 0, s,
                  true, a);
}

}  // namespace
}  // namespace qsa
