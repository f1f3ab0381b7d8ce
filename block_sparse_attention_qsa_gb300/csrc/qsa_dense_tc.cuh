// Dense attention on the fifth-generation tensor cores.
//
// The mathematics, the stream of tiles and its split are in qsa_dense.cuh.
// This kernel takes tiles of 128 positions, and computes both products
// transposed, so that the long dimension fills the MMA's 128 rows (M) and the
// few query rows are its columns (N):
//   S^T[position][row] = K Q^T      (A = K, as the cache holds it; B = Q)
//   O^T[d][row]       += V^T P^T    (A = V read along its other dimension:
//                                    tcgen05 takes it from the same TMA tile)
// with S^T and O^T in tensor memory. A softmax thread owns one position (one
// TMEM lane) and all 8, 16 or 32 rows of its warpgroup, so there are no
// shuffles, every row's arithmetic is independent of the others', and at the
// end of a unit a thread owns one component d of every row: no joint of the
// warps is left, the pieces go out as they are. K and V never pass through
// registers. (Head dim 64: the MMA's upper 64 rows repeat the lower ones; 256:
// two MMAs, two components a thread.)
//
// Before it the same loop ran on mma.sync, fragments by ldmatrix and E4M3
// widened in registers, and was bound by its warps' issue and latency: batch
// 32, about 55,600 tokens, 4 verify queries x 16 heads over 2 KV heads of 128:
// 318 us with a BF16 cache and 290 with E4M3, where the bytes take 273 and 136;
// this kernel takes 267 and 149.
//
// E4M3 cache: the MMA's operands are E4M3 as well, so the cache's codes are
// used as they are, and Q and P become two E4M3 terms each, x = hi + lo / 32,
// as 32 + 32 columns. A code has 4 significant bits, so the two together have
// 8, as many as BF16. Q: its row is scaled by a power of two so that its
// largest value is in [2^7, 2^8); lo / 32 ends in steps of 2^-14, so a component
// is off by at most 2^-15, that is 2^-22 of the row's largest value. P: a
// weight from 2^-6 on (the row's largest is 2^6 to 2^8) is off by at most 2^-8
// of itself, as it is in BF16. Below that its steps are of 2^-14, and a long
// tail of weights of that size and less would be lost, or counted double, all
// in the same direction: 61,204 equal keys 14.6 nats below one other gave 0.973
// for 1, a million 0.69. So lo is rounded up or down by the position's place in
// an equidistributed sequence (see `dither`) in proportion to what is cut off:
// each such weight is off by less than 2^-14 with mean zero. The errors of a
// tail of sum S then have a variance of at most 2^-14 S, which is at most 2^-11
// (one standard deviation) of the row's sum, S + 2^6 or more, however many
// positions there are.
//
// The reference of a row: weights are 2^(s - mu), where mu only has to keep
// the largest weight between 1 and 2^8 (E4M3 ends at 448): it starts 6 below
// the row's first maximum and moves when a score passes mu + 8, which after a
// row's first tiles hardly happens. Moving it rescales O in tensor memory.
//
// Roles: a copy warp (pages, TMA: K and V tiles in a ring of slots), a warp
// that issues the MMAs of S and one for those of PV (issuing a tile's takes
// each 500 to 700 cycles, about half of the time that HBM takes for an E4M3
// tile; one warp for both was the loop's bound), and one or two warpgroups of
// softmax. S and P are double-buffered, so the tensor cores and the copies run
// ahead of the softmax.
//
// Masks. A tile in which a row does not see every position is an edge tile.
// There the thread that owns a position that no row sees zeroes its V row in
// shared memory, and a V row that only some rows see and that is not finite is
// taken out of the MMA and added in FP32 to those rows. (Positions without a
// page: the copies fill zeros, and their scores become -inf.)
#pragma once

#include "qsa_tc.cuh"

namespace qsa {
namespace {

constexpr int kTileTc = 128;
constexpr float kRefBelow = 6.f;  // log2 of a row's first largest weight
constexpr float kRefMost = 8.f;   // log2 of a weight that moves the reference
constexpr float kNoRef = __builtin_huge_valf();  // the reference of a row that has seen nothing (its scores are less 0)
constexpr int kBadRing = 16;      // page marks of the tiles in flight
constexpr int kRun = 256;         // tiles of a run: O in tensor memory holds no more (a power of two)

// D: head dim, RC: rows of a softmax warpgroup (8, 16 or 32), WGS: softmax
// warpgroups, BLK: blocks of up to 32 rows, each one set of MMA columns
template <int D_, bool FP8_, int RC_, int WGS_>
struct Tc {
  static constexpr bool FP8 = FP8_;
  static constexpr int D = D_, RC = RC_, WGS = WGS_, EB = FP8 ? 1 : 2;
  static constexpr int kRows = RC * WGS, BLK = kRows > 32 ? kRows / 32 : 1;
  static constexpr int kRowBytes = D * EB;
  static constexpr int kLine = kRowBytes < 128 ? kRowBytes : 128;  // bytes of a TMA box's row
  static constexpr int kLines = kRowBytes / kLine, kChunks = kLine / 16;
  static constexpr int kSlot = kTileTc * kRowBytes;  // K or V of a tile
  static constexpr int N = FP8 ? 64 : 32;            // MMA columns of a block (those past its rows idle)
  static constexpr int MB = D > 128 ? D / 128 : 1;   // blocks of 128 output components
  static constexpr int kQ = N * kRowBytes;           // a block's Q
  static constexpr int kP = kTileTc * 64;            // a block's P: 64 bytes a position
  // Q of the next unit is staged ahead, but for rows of 512 bytes, where its
  // buffer would cost the third slot
  static constexpr int kQBufs = kRowBytes > 256 ? 1 : 2;
  static constexpr int kFixed = BLK * (kQBufs * kQ + 2 * kP) + 1024;
  static constexpr int kStatic = BLK == 1 ? (FP8 ? 2560 : 2048) : 4608;  // barriers and tables
  static constexpr int kFit = (kMaxSmem - kStatic - kFixed) / kSlot;
  static constexpr int kSlots = kFit < 24 ? kFit : 24;
  // K and V have a ring each: every phase of a slot's barriers is then met by
  // the same warps (a parity says nothing about a phase two ahead). V, which
  // stays until its PV is done, has the odd slot.
  static constexpr int kNK = kSlots / 2, kNV = kSlots - kNK;
  static constexpr int kSmem = kSlots * kSlot + kFixed;
  static constexpr int kThreads = 128 * WGS + 96;
  static constexpr int kCopyWarp = 4 * WGS, kSWarp = kCopyWarp + 1, kPvWarp = kCopyWarp + 2;
  static constexpr uint32_t kO = 2 * BLK * N;        // TMEM: two S buffers, then O
  static constexpr uint32_t kNeed = (2 + MB) * BLK * N;
  static constexpr uint32_t kTmem = kNeed <= 128 ? 128 : kNeed <= 256 ? 256 : 512;
  static constexpr int kPieceFloats = kRows * (D + 2);
  static_assert(kSlots >= 3 && kNV + 2 < kBadRing && kNeed <= 512, "ring, tensor memory");
  // where 16-byte chunk c of a line is in row `row` (the TMA and MMA swizzle)
  static __device__ __forceinline__ int swizzled(int row, int c) {
    return kLine == 128 ? c ^ (row & 7) : c ^ ((row >> 1) & 3);
  }
  // byte offset of byte `b` of row `row` in a slot
  static __device__ __forceinline__ int at_byte(int row, int b) {
    return b / kLine * (kTileTc * kLine) + row * kLine + (swizzled(row, b % kLine / 16) << 4) + b % 16;
  }
};

template <class C>
__host__ __device__ constexpr uint32_t mma_desc(bool mn_major) {
  return instr_desc(C::FP8 ? 0u : kTypeBf16, mn_major, mn_major, C::N, kTileTc);
}

// barriers of one softmax warpgroup (id 1 + wg) or of all of them (id 3)
__device__ __forceinline__ void group_sync(int id, int threads) {
  asm volatile("bar.sync %0, %1;" ::"r"(id), "r"(threads) : "memory");
}
__device__ __forceinline__ bool group_any(int id, int threads, bool x) {
  uint32_t r;
  asm volatile(
      "{\n\t.reg .pred p, q;\n\tsetp.ne.u32 p, %3, 0;\n\tbarrier.cta.red.or.pred q, %1, %2, p;\n\tselp.u32 %0, 1, 0, "
      "q;\n\t}"
      : "=r"(r)
      : "r"(id), "r"(threads), "r"((uint32_t)x)
      : "memory");
  return r != 0;
}

// Reduces v[i] over the warp's lanes for every i < RC; the result for i is in
// v[0] of the lanes with lane % RC == i. Halving: at each step a lane hands
// the half of its values that it gives up to its partner.
template <int RC, class Op>
__device__ __forceinline__ float reduce_rows(float (&v)[RC], Op op) {
  const int lane = threadIdx.x & 31;
#pragma unroll
  for (int o = 16; o >= RC; o >>= 1)
#pragma unroll
    for (int i = 0; i < RC; ++i) v[i] = op(v[i], __shfl_xor_sync(kFull, v[i], o));
#pragma unroll
  for (int o = RC / 2; o > 0; o >>= 1) {
    const bool up = (lane & o) != 0;
#pragma unroll
    for (int i = 0; i < o; ++i) {
      const float give = up ? v[i] : v[i + o], keep = up ? v[i + o] : v[i];
      v[i] = op(keep, __shfl_xor_sync(kFull, give, o));
    }
  }
  return v[0];
}

// What is added to lo of a position's weights before it is rounded to E4M3, whose
// steps are of 2^-9 there: between -2^-10 and 2^-10 (exclusive: a weight of 0
// stays 0), equidistributed over any run of positions (multiples of the golden
// ratio, modulo 1). It depends on the position alone: the same call gives the
// same bits.
__device__ __forceinline__ float dither(int p) {
  return (float)(((int)((uint32_t)p * 0x9e3779b9u) >> 8) | 1) * 0x1p-33f;
}
template <class C, class A>
__global__ void __launch_bounds__(C::kThreads, 1) dense_tc_kernel(const __grid_constant__ CUtensorMap tm_k,
                                                                  const __grid_constant__ CUtensorMap tm_v,
                                                                  const A a) {
  constexpr bool FP8 = C::FP8;
  constexpr int RC = C::RC, WGS = C::WGS, BLK = C::BLK, N = C::N, kTile = kTileTc, D = C::D, MB = C::MB;
  constexpr int kLine = C::kLine, kLines = C::kLines, kChunks = C::kChunks;
  constexpr uint64_t kSwizzle = kLine == 128 ? 2 : 4;
  extern __shared__ uint8_t smem_raw[];
  uint8_t* ring = reinterpret_cast<uint8_t*>((reinterpret_cast<uintptr_t>(smem_raw) + 1023) & ~uintptr_t(1023));
  uint8_t* s_q = ring + C::kSlots * C::kSlot;   // [buffer][block]
  uint8_t* s_p = s_q + C::kQBufs * BLK * C::kQ; // [buffer][block]
  __shared__ __align__(8) uint64_t slot_full[C::kSlots], slot_empty[C::kSlots];  // K's, then V's
  __shared__ __align__(8) uint64_t s_full[2], p_full[2], pv_done[2], q_full[2], fin;
  __shared__ uint32_t s_tmem;
  __shared__ uint32_t s_bad[kBadRing];  // bit i: positions 16 i .. 16 i + 15 of the tile have no page
  __shared__ int s_keep;                // a run's first PV adds to what O holds
  __shared__ volatile int s_abort;
  __shared__ long long s_scan[C::kThreads / 32];
  __shared__ Share s_share;
  __shared__ int2 s_rng[2][C::kRows];   // [buffer][row]: positions the row sees, first and one past the last
  __shared__ int2 s_all[2];             // positions that all rows of the unit see
  __shared__ __align__(16) float s_scale[2][FP8 ? C::kRows : 1];  // softmax scale of a row (BF16: of all)
  __shared__ int s_out[2][C::kRows];    // [buffer][row]: its row of q and out, -1: none
  __shared__ float s_red[WGS][4][RC];
  __shared__ __align__(16) float s_mu[WGS][RC], s_nmu[WGS][RC];
  __shared__ uint32_t s_odd[WGS][4];    // positions whose V is not finite
  __shared__ uint32_t s_see[WGS];
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
  const int units = a.n_kv_heads * a.row_blocks;

  if (tid == 0) {
    s_abort = 0;
    for (int s = 0; s < C::kSlots; ++s) {
      mbar_init(smem_u32(&slot_full[s]), 1);
      mbar_init(smem_u32(&slot_empty[s]), 1);
    }
    for (int b = 0; b < 2; ++b) {
      mbar_init(smem_u32(&s_full[b]), 1);
      mbar_init(smem_u32(&p_full[b]), 128 * WGS);
      mbar_init(smem_u32(&pv_done[b]), 1);
      mbar_init(smem_u32(&q_full[b]), 128 * WGS);
    }
    mbar_init(smem_u32(&fin), 2);
    asm volatile("fence.mbarrier_init.release.cluster;" ::: "memory");
  }
  if (warp == C::kPvWarp) {
    asm volatile("tcgen05.alloc.cta_group::1.sync.aligned.shared::cta.b32 [%0], %1;" ::"r"(smem_u32(&s_tmem)),
                 "r"(C::kTmem)
                 : "memory");
    asm volatile("tcgen05.relinquish_alloc_permit.cta_group::1.sync.aligned;" ::: "memory");
  }
  tc_before();
  pdl_wait();     // positions, queries and the cache may come from the kernel before
  pdl_trigger();  // the joining kernel may be set up; it waits for this one's end
  Walk<kTile> at;
  const bool work = find_start<kTile, C::kThreads>(a, s_scan, s_share, at);  // (with a barrier behind the allocation)
  tc_after();
  auto free_tmem = [&]() {
    asm volatile("tcgen05.dealloc.cta_group::1.sync.aligned.b32 %0, %1;" ::"r"(s_tmem), "r"(C::kTmem) : "memory");
  };
  if (!work) {
    if (warp == C::kPvWarp) free_tmem();
    return;
  }
  auto wait = [&](uint64_t* bar, uint32_t parity) { return mbar_wait(bar, parity, &s_abort, a.err); };
  const uint32_t tmem = s_tmem;

  if (warp == C::kCopyWarp) {
    // ---- copies: K then V of each tile ----
    PageFeed<kTile> feed(a);
    const int line = lane >> (7 - feed.box_shift);  // this lane's line of a K or V tile; at most 32 copies
    const uint32_t dst = (uint32_t)(line * (kTile * kLine) + (feed.my_box << feed.box_shift) * kLine);
    int slot[2] = {0, 0}, it = 0;
    uint32_t phase[2] = {0, 0};
    bool ok = true;
    do {
      const int g = at.x / a.row_blocks;
      feed.start(a, at);
      for (int k = 0; k < at.n && ok; ++k, ++it) {
        const int page = feed.of_tile(a, at, k);
        const uint32_t bad = feed.bad_groups(page);
        const int first = feed.slot_of(a, k), at_page = page < 0 ? a.num_pages : page /* outside: zeros */;
#pragma unroll
        for (int v = 0; v < 2; ++v) {
          const int i = (v ? C::kNK : 0) + slot[v];
          if (!__all_sync(kFull, wait(&slot_empty[i], phase[v] ^ 1u))) {
            ok = false;
            break;
          }
          const uint32_t bar = smem_u32(&slot_full[i]);
          if (lane == 0) {
            if (v == 0) s_bad[it % kBadRing] = bad;
            mbar_expect_tx(bar, C::kSlot);
          }
          __syncwarp();
          if (line < kLines)
            tma_load_4d(smem_u32(ring + i * C::kSlot) + dst, v ? &tm_v : &tm_k, line * (kLine / C::EB), first, g,
                        at_page, bar);
          if (++slot[v] == (v ? C::kNV : C::kNK)) {
            slot[v] = 0;
            phase[v] ^= 1u;
          }
        }
      }
    } while (ok && at.next(a, s_share));
    if (s_abort) {  // copies in flight land before the CTA leaves (bounded)
      for (int i = 0; i < C::kSlots; ++i) {
        const int v = i >= C::kNK ? 1 : 0;
        const uint32_t par = i - (v ? C::kNK : 0) < slot[v] ? phase[v] : phase[v] ^ 1u;
        const long long start = clock64();
        while (!mbar_try_wait(smem_u32(&slot_full[i]), par) && clock64() - start < kWaitCycles / 64) {
        }
      }
    }
  } else if (warp == C::kSWarp) {
    // ---- S^T = K Q^T ----
    // (the whole warp walks the loop, one elected thread issues: descriptors
    // then stay in uniform registers, which is what the instructions take)
    {
      const bool one = elect_one();
      constexpr uint32_t kIdesc = mma_desc<C>(false);
      constexpr int kSteps = C::kRowBytes / 32, kPerLine = kLine / 32;  // 32 bytes of a row each
      int it = 0, seg = 0;
      bool ok = true;
      do {
        const int buf = seg % C::kQBufs;
        ok = __all_sync(kFull, wait(&q_full[buf], (uint32_t)(seg / C::kQBufs) & 1u));
        for (int k = 0; k < at.n && ok; ++k, ++it) {
          const int slot = it % C::kNK;
          ok = __all_sync(kFull, wait(&slot_full[slot], (uint32_t)(it / C::kNK) & 1u) &&
                                     (it < 2 || wait(&p_full[it & 1], (uint32_t)((it - 2) >> 1) & 1u)));  // S was read
          if (!ok) break;
          tc_after();
          const uint64_t dk = smem_desc(smem_u32(ring + slot * C::kSlot), 16, 8 * kLine, kSwizzle);
#pragma unroll
          for (int b = 0; b < BLK; ++b) {
            const uint64_t dq = smem_desc(smem_u32(s_q + (buf * BLK + b) * C::kQ), 16, 8 * kLine, kSwizzle);
#pragma unroll
            for (int ks = 0; ks < kSteps; ++ks) {
              // (addresses are in units of 16 bytes)
              const uint32_t line = (uint32_t)(ks / kPerLine), step = (uint32_t)(ks % kPerLine) * 2u;
              if (one)
                mma_tc<FP8>(tmem + (uint32_t)(((it & 1) * BLK + b) * N), dk + (line * (kTile * kLine / 16) + step),
                            dq + (line * (N * kLine / 16) + step), kIdesc, ks > 0);
            }
          }
          if (one) {
            commit_tc(&s_full[it & 1]);
            commit_tc(&slot_empty[slot]);
          }
          __syncwarp();
        }
        ++seg;
      } while (ok && at.next(a, s_share));
      if (one) commit_tc(&fin);
    }
    __syncwarp();
  } else if (warp == C::kPvWarp) {
    // ---- O^T += V^T P^T ----
    {
      const bool one = elect_one();
      constexpr uint32_t kIdesc = mma_desc<C>(true);
      constexpr int kSteps = kTile / (FP8 ? 32 : 16), kPos = kTile / kSteps;  // positions of an MMA
      int it = 0;
      bool ok = true;
      do {
        for (int k = 0; k < at.n && ok; ++k, ++it) {
          const int slot = C::kNK + it % C::kNV;
          ok = __all_sync(kFull, wait(&p_full[it & 1], (uint32_t)(it >> 1) & 1u) &&
                                     wait(&slot_full[slot], (uint32_t)(it / C::kNV) & 1u));
          if (!ok) break;
          tc_after();
          const bool fresh = k % kRun == 0 && *reinterpret_cast<volatile int*>(&s_keep) == 0;
          // A: positions as k. Its 128 rows are components: one line of 128,
          // or two of 64 (leading offset: a line), or one of 64 twice (leading
          // offset 0; the upper half of O is then a copy)
          constexpr int kPer = kLine / C::EB;  // components of a line
          const uint64_t dv = smem_desc(smem_u32(ring + slot * C::kSlot), D >= 128 && kPer == 64 ? kTile * kLine : 0,
                                        8 * kLine, kSwizzle);
#pragma unroll
          for (int b = 0; b < BLK; ++b) {
            // B: positions as k, 64-byte rows
            const uint64_t dp = smem_desc(smem_u32(s_p + ((it & 1) * BLK + b) * C::kP), 512, 512, 4);
#pragma unroll
            for (int mb = 0; mb < MB; ++mb)
#pragma unroll
              for (int ks = 0; ks < kSteps; ++ks)
                if (one)
                  mma_tc<FP8>(tmem + C::kO + (uint32_t)((mb * BLK + b) * N),
                              dv + (uint32_t)((mb * (128 / kPer) * kTile * kLine + ks * kPos * kLine) / 16),
                              dp + (uint32_t)(ks * kPos * 4), kIdesc, !(fresh && ks == 0));
          }
          if (one) {
            commit_tc(&pv_done[it & 1]);
            commit_tc(&slot_empty[slot]);
          }
          __syncwarp();
        }
      } while (ok && at.next(a, s_share));
      // the tensor cores are done before the CTA gives its memory back
      if (one) commit_tc(&fin);
      const long long start = clock64();
      while (!mbar_try_wait(smem_u32(&fin), 0) && clock64() - start < 2 * kWaitCycles) {
      }
    }
    __syncwarp();
  } else {
    // ---- softmax ----
    const int wg = warp >> 2, quarter = warp & 3, t = tid & 127;
    const uint32_t lane_base = (uint32_t)(quarter * 32) << 16;
    // the warpgroup's rows: row_off .. + RC - 1 of the unit, columns col .. of block blk
    const int row_off = wg * RC, blk = row_off / 32, col = row_off % 32;
    const uint32_t o_addr = tmem + lane_base + C::kO + (uint32_t)(blk * N + col);

    // the rows of the unit at `u` into Q buffer `buf`, with what is known of them
    auto stage_q = [&](const Walk<kTile>& u, int buf) {
      const int g = u.x / a.row_blocks, rb = u.x - g * a.row_blocks;
      const int rows = min(C::kRows, a.n_q * a.group - rb * C::kRows);
      const float base_scale = a.sm_scale * kLog2e * (FP8 ? a.k_scale[g] : 1.f);
      uint8_t* dst = s_q + (buf * BLK + blk) * C::kQ + col * kLine;
      constexpr int kLanes = D / 8, kPass = 128 / kLanes;  // 8 components a lane
#pragma unroll
      for (int z = 0; z < (RC + kPass - 1) / kPass; ++z) {
        const int r = t / kLanes + kPass * z, c = t % kLanes;
        if (r >= RC) break;  // (a whole warp)
        uint4 v = make_uint4(0, 0, 0, 0);
        if (row_off + r < rows) {
          const int i = rb * C::kRows + row_off + r, j = i / a.group, h = g * a.group + (i - j * a.group);
          v = ld16(a.q + (((size_t)u.r * a.n_q + j) * a.n_q_heads + h) * D + c * 8);
        }
        if constexpr (FP8) {
          uint32_t big = 0;  // magnitudes of BF16 values order like their bit patterns
          const uint32_t wd[4] = {v.x, v.y, v.z, v.w};
#pragma unroll
          for (int e = 0; e < 4; ++e) big = max(big, max((wd[e] << 16) & 0x7fff0000u, wd[e] & 0x7fff0000u));
#pragma unroll
          for (int o = 1; o < kLanes; o <<= 1) big = max(big, __shfl_xor_sync(kFull, big, o));
          // 2^-sh brings the row's largest value into [2^7, 2^8)
          const int sh = big == 0 ? 0 : min(126, max(-126, (int)(big >> 23) - 127 - 7));
          // (a row with an infinity or NaN: every component NaN, as its scores are)
          const float down = big >= 0x7f800000u ? __uint_as_float(0x7fffffffu) : pow2(-sh);
          uint32_t hi[4], lo[4];
#pragma unroll
          for (int e = 0; e < 4; ++e) {
            const float x = bf_lo(wd[e]) * down, y = bf_hi(wd[e]) * down;
            hi[e] = e4m3x2(x, y);
            const float2 f = h2_to_f2(e4m3x2_to_h2(hi[e]));
            lo[e] = e4m3x2((x - f.x) * 32.f, (y - f.y) * 32.f);
          }
          const int chunk = c >> 1;
          uint8_t* d8 = dst + chunk / kChunks * (N * kLine) + r * kLine +
                        (C::swizzled(col + r, chunk % kChunks) << 4) + (c & 1) * 8;
          *reinterpret_cast<uint2*>(d8) = make_uint2(hi[0] | (hi[1] << 16), hi[2] | (hi[3] << 16));
          *reinterpret_cast<uint2*>(d8 + 32 * kLine) = make_uint2(lo[0] | (lo[1] << 16), lo[2] | (lo[3] << 16));
          if (c == 0) s_scale[buf][row_off + r] = base_scale * pow2(sh);
        } else {
          *reinterpret_cast<uint4*>(dst + c / kChunks * (N * kLine) + r * kLine +
                                    (C::swizzled(col + r, c % kChunks) << 4)) = v;
          if (tid == 0) s_scale[buf][0] = base_scale;
        }
      }
      if (t < RC) {
        int2 rg = make_int2(0, 0);
        int o = -1;
        if (row_off + t < rows) {
          const int i = rb * C::kRows + row_off + t, j = i / a.group, h = g * a.group + (i - j * a.group);
          const int p = a.q_pos[(size_t)u.r * a.n_q + j];
          if (valid_pos(a, p)) rg = make_int2(first_seen(a, u.g, p), p + 1);
          o = (u.r * a.n_q + j) * a.n_q_heads + h;
        }
        s_rng[buf][row_off + t] = rg;
        s_out[buf][row_off + t] = o;
      }
      if (tid == 0) {
        int2 all = make_int2(0, 0x7fffffff);
        for (int j = rb * C::kRows / a.group; j <= (rb * C::kRows + rows - 1) / a.group; ++j) {
          const int p = a.q_pos[(size_t)u.r * a.n_q + j];
          all.x = max(all.x, valid_pos(a, p) ? first_seen(a, u.g, p) : 0);
          all.y = min(all.y, valid_pos(a, p) ? p + 1 : 0);
        }
        s_all[buf] = all;
      }
      async_fence();
      mbar_arrive(smem_u32(&q_full[buf]));
    };

    // A segment goes by in runs of kRun tiles, whose O and sums are added up in
    // FP32 where the segment's piece is (or would be, for a unit that is whole).
    // The tensor cores add to an accumulator by cutting off, not by rounding: one
    // that grows steadily loses about half of its last bit at each step (8 a tile
    // with BF16, 4 with E4M3): 0.4 % over 1,000,000 positions in one CTA, 2 % over
    // 4,000,000. A run loses at most 2^-12, and a thread's part of a row's sum has
    // no more than kRun terms.
    stage_q(at, 0);
    int it = 0, seg = 0;
    bool last;
    do {  // (at.t, at.n: what is left of the segment)
      const int n = min(kRun, at.n), buf = seg % C::kQBufs;
      if (at.t == at.start(s_share)) {
        if constexpr (C::kQBufs == 1) {
          if (seg > 0) stage_q(at, 0);
        } else {
          Walk<kTile> following = at;
          if (following.next(a, s_share)) stage_q(following, buf ^ 1);  // (the rows of the unit before are done with)
        }
        if (t < RC) {
          s_mu[wg][t] = kNoRef;
          s_nmu[wg][t] = 0.f;
        }
        if constexpr (WGS == 1)
          group_sync(1 + wg, 128);  // the tables of this unit
        else
          group_sync(3, 128 * WGS);
      }
      const int2 all = s_all[buf];
      float l[RC];
      const float sc = FP8 ? 0.f : s_scale[buf][0];
#pragma unroll
      for (int r = 0; r < RC; ++r) l[r] = 0.f;
      bool fresh = true;  // a row has no reference yet (asked anew in each run)
      for (int k = 0; k < n; ++k, ++it) {
        const bool ok = wait(&s_full[it & 1], (uint32_t)(it >> 1) & 1u);
        (void)ok;  // given up: the loop runs on without meaning, to the same barriers
        __syncwarp();
        tc_after();
        const uint32_t s_addr = tmem + lane_base + (uint32_t)(((it & 1) * BLK + blk) * N + col);
        const int p0 = (at.g.lo / kTile + at.t + k) * kTile, p = p0 + t;
        const uint32_t bad = *reinterpret_cast<volatile uint32_t*>(&s_bad[it % kBadRing]);
        const bool edge = p0 < all.x || all.y - p0 < kTile;
        const bool paged = !((bad >> (t >> 4)) & 1u);
        float y[RC];
        // Scores (exp2 domain) less the rows' references. (16 rows at a time, and
        // the references from shared memory: with more in registers 64 rows of an
        // E4M3 cache spilled, 155 us for 120.)
        constexpr int kPart = RC < 16 ? RC : 16;
#pragma unroll
        for (int r0 = 0; r0 < RC; r0 += kPart) {
          uint32_t v[kPart];
          Tmem<kPart>::load(s_addr + r0, v);
          if constexpr (FP8) {
            uint32_t u[kPart];
            Tmem<kPart>::load(s_addr + 32 + r0, u);
            tc_wait_ld();
#pragma unroll
            for (int r = 0; r < kPart; r += 2) {
              const float2 x = less(fma2(pair(u + r), both(0.03125f), pair(v + r)),
                                    pair(&s_scale[buf][row_off + r0 + r]), both(a.one), pair(&s_nmu[wg][r0 + r]));
              y[r0 + r] = x.x;
              y[r0 + r + 1] = x.y;
            }
          } else {
            tc_wait_ld();
#pragma unroll
            for (int r = 0; r < kPart; r += 2) {
              const float2 x = less(pair(v + r), both(sc), both(a.one), pair(&s_nmu[wg][r0 + r]));
              y[r0 + r] = x.x;
              y[r0 + r + 1] = x.y;
            }
          }
        }
        if (edge || bad != 0) {
#pragma unroll
          for (int r = 0; r < RC; ++r) {
            const int2 rg = s_rng[buf][row_off + r];
            if (p < rg.x || p >= rg.y || !paged) y[r] = kNegInf;
          }
        }
        // Where a score passes its reference by too much, and as long as a row of
        // the unit has seen nothing yet, the references move to the maxima; scores
        // and sums follow by the difference. (The warps' vote is 3 of the 149 us of
        // batch 32 with E4M3. Voting through an mbarrier with the exponentials
        // before its wait was slower, 152, and so was a second pass over the scores
        // in place of the difference, for the length of its code.)
        bool move = fresh;
        if (fresh) {
          if (k > 0) group_sync(1 + wg, 128);  // (s_red has been read)
        } else {
          float top = kNegInf;
#pragma unroll
          for (int r = 0; r < RC; r += 2) top = max3(top, y[r], y[r + 1]);
          move = group_any(1 + wg, 128, top > kRefMost);
        }
        if (move) {
          {
            float top = 0.f;
#pragma unroll
            for (int r = 0; r < RC; ++r) {
              const float x = warp_max(y[r]);
              if (lane == r) top = x;
            }
            if (lane < RC) s_red[wg][quarter][lane] = top;
          }
          group_sync(1 + wg, 128);
          bool unseen = false;
          if (t < RC) {
            const float top = fmaxf(fmaxf(s_red[wg][0][t], s_red[wg][1][t]), fmaxf(s_red[wg][2][t], s_red[wg][3][t]));
            const float from = s_mu[wg][t];
            const bool none = from == kNoRef;
            // by how much the row's reference moves
            const float by = none ? (top > kNegInf ? top - kRefBelow : 0.f) : top > kRefMost ? top - kRefBelow : 0.f;
            s_red[wg][0][t] = none ? 1.f : exp2_sfu(-by);  // the row's factor
            s_red[wg][1][t] = by;
            if (!none || top > kNegInf) {
              const float to = (none ? 0.f : from) + by;
              s_mu[wg][t] = to;
              s_nmu[wg][t] = to == kNoRef ? 0.f : -to;
            }
            const int2 rg = s_rng[buf][row_off + t];
            unseen = none && !(top > kNegInf) && rg.x < rg.y;
          }
          fresh = group_any(1 + wg, 128, unseen);
#pragma unroll
          for (int r = 0; r < RC; ++r) {
            y[r] -= s_red[wg][1][r];
            l[r] *= s_red[wg][0][r];
          }
          if (k > 0) {  // what O holds so far
            wait(&pv_done[(it - 1) & 1], (uint32_t)((it - 1) >> 1) & 1u);
            __syncwarp();
            tc_after();
#pragma unroll 1
            for (int part = 0; part < MB * (FP8 ? 2 : 1); ++part) {
              const uint32_t addr = o_addr + (uint32_t)(FP8 ? (part >> 1) * (BLK * N) + (part & 1) * 32 : part * (BLK * N));
              uint32_t o[RC];
              Tmem<RC>::load(addr, o);
              tc_wait_ld();
#pragma unroll
              for (int r = 0; r < RC; ++r) o[r] = __float_as_uint(__uint_as_float(o[r]) * s_red[wg][0][r]);
              Tmem<RC>::store(addr, o);
            }
            tc_wait_st();
          }
        }
#pragma unroll
        for (int r = 0; r < RC; r += 2) {
          y[r] = exp2_sfu(y[r]);
          y[r + 1] = exp2_sfu(y[r + 1]);
          const float2 x = add2(pair(l + r), pair(y + r));
          l[r] = x.x;
          l[r + 1] = x.y;
        }
        if (k == 0 && tid == 0) s_keep = 0;
        if (edge) {
          const int vs = C::kNK + it % C::kNV;
          wait(&slot_full[vs], (uint32_t)(it / C::kNV) & 1u);
          uint8_t* vrow = ring + vs * C::kSlot;
          auto zero_row = [&]() {
#pragma unroll 1
            for (int c = 0; c < C::kRowBytes / 16; ++c)
              *reinterpret_cast<uint4*>(vrow + c / kChunks * (kTile * kLine) + t * kLine + (c % kChunks << 4)) =
                  make_uint4(0, 0, 0, 0);
          };
          bool odd = false;
          if (p < at.g.lo || p >= at.g.hi) {
            zero_row();
          } else if (p < all.x || p >= all.y) {  // (what every row sees cannot reach a row that does not)
#pragma unroll 1
            for (int c = 0; c < C::kRowBytes / 16; ++c) {
              const uint4 x = *reinterpret_cast<const uint4*>(vrow + c / kChunks * (kTile * kLine) + t * kLine +
                                                              ((c + lane) % kChunks << 4));
              const uint32_t wd[4] = {x.x, x.y, x.z, x.w};
#pragma unroll
              for (int e = 0; e < 4; ++e) {
                if constexpr (FP8)
                  odd |= (((wd[e] & 0x7f7f7f7fu) + 0x01010101u) & 0x80808080u) != 0;
                else
                  odd |= (wd[e] & 0x7f80u) == 0x7f80u || (wd[e] & 0x7f800000u) == 0x7f800000u;
              }
            }
          }
          if (group_any(3, 128 * WGS, odd)) {
            // these rows go to O by hand (FP32), where they are seen, and leave the MMA
            const uint32_t mask = __ballot_sync(kFull, odd);
            if (lane == 0) s_odd[wg][quarter] = mask;
            if (k > 0) wait(&pv_done[(it - 1) & 1], (uint32_t)((it - 1) >> 1) & 1u);
            __syncwarp();
            tc_after();
            group_sync(1 + wg, 128);
#pragma unroll 1
            for (int mb = 0; mb < MB; ++mb) {
              const uint32_t addr = o_addr + (uint32_t)(mb * (BLK * N));
              const int comp = D < 128 ? t % D : mb * 128 + t;
              uint32_t o[RC];
#pragma unroll
              for (int r = 0; r < RC; ++r) o[r] = 0;
              if (k > 0) {
                Tmem<RC>::load(addr, o);
                tc_wait_ld();
              } else if (FP8) {
                Tmem<RC>::store(addr + 32, o);
              }
#pragma unroll 1
              for (int u = 0; u < kTile; ++u) {
                if (!((s_odd[wg][u >> 5] >> (u & 31)) & 1u)) continue;
                if (t == u) {
                  uint32_t see = 0;
#pragma unroll
                  for (int r = 0; r < RC; ++r) {
                    const int2 rg = s_rng[buf][row_off + r];
                    if (p >= rg.x && p < rg.y) see |= 1u << r;
                    s_red[wg][0][r] = y[r];
                  }
                  s_see[wg] = see;
                }
                group_sync(1 + wg, 128);
                const uint8_t* at_v = vrow + C::at_byte(u, comp * C::EB);
                const float v = FP8 ? h2_to_f2(e4m3x2_to_h2(*at_v)).x
                                    : __uint_as_float((uint32_t)*reinterpret_cast<const uint16_t*>(at_v) << 16);
#pragma unroll
                for (int r = 0; r < RC; ++r)
                  if ((s_see[wg] >> r) & 1u) o[r] = __float_as_uint(fmaf(s_red[wg][0][r], v, __uint_as_float(o[r])));
                group_sync(1 + wg, 128);
              }
              Tmem<RC>::store(addr, o);
              tc_wait_st();
            }
            group_sync(3, 128 * WGS);  // every warpgroup has read the rows
            if (odd) {
              zero_row();
#pragma unroll
              for (int r = 0; r < RC; ++r) y[r] = 0.f;
            }
            if (k == 0 && tid == 0) s_keep = 1;
          }
        }
        // P of the tile before last has been read
        if (it >= 2) wait(&pv_done[it & 1], (uint32_t)((it - 2) >> 1) & 1u);
        uint8_t* prow = s_p + ((it & 1) * BLK + blk) * C::kP + t * 64;
        const int x4 = (t >> 1) & 3;
        if constexpr (FP8) {
          const float dith = dither(p);
          uint32_t hi[RC / 2], lo[RC / 2];
#pragma unroll
          for (int r = 0; r < RC; r += 2) {
            hi[r / 2] = e4m3x2(y[r], y[r + 1]);
            const float2 f = h2_to_f2(e4m3x2_to_h2(hi[r / 2]));
            const float2 x = fma2(add2(pair(y + r), make_float2(-f.x, -f.y)), both(32.f), both(dith));
            lo[r / 2] = e4m3x2(x.x, x.y);
          }
          const int c0 = col / 16;  // a 16-byte chunk has 16 rows: hi in chunks 0 and 1, lo in 2 and 3
          if constexpr (RC == 8) {
            *reinterpret_cast<uint2*>(prow + ((c0 ^ x4) << 4)) = make_uint2(hi[0] | (hi[1] << 16), hi[2] | (hi[3] << 16));
            *reinterpret_cast<uint2*>(prow + (((2 + c0) ^ x4) << 4)) =
                make_uint2(lo[0] | (lo[1] << 16), lo[2] | (lo[3] << 16));
          } else {
#pragma unroll
            for (int c = 0; c < RC / 16; ++c) {
              const uint32_t* h = hi + 8 * c;
              const uint32_t* g = lo + 8 * c;
              *reinterpret_cast<uint4*>(prow + (((c0 + c) ^ x4) << 4)) = make_uint4(
                  h[0] | (h[1] << 16), h[2] | (h[3] << 16), h[4] | (h[5] << 16), h[6] | (h[7] << 16));
              *reinterpret_cast<uint4*>(prow + (((2 + c0 + c) ^ x4) << 4)) = make_uint4(
                  g[0] | (g[1] << 16), g[2] | (g[3] << 16), g[4] | (g[5] << 16), g[6] | (g[7] << 16));
            }
          }
        } else {
          const int c0 = col / 8;
#pragma unroll
          for (int c = 0; c < RC / 8; ++c)
            *reinterpret_cast<uint4*>(prow + (((c0 + c) ^ x4) << 4)) =
                make_uint4(pack_bf(y[8 * c], y[8 * c + 1]), pack_bf(y[8 * c + 2], y[8 * c + 3]),
                           pack_bf(y[8 * c + 4], y[8 * c + 5]), pack_bf(y[8 * c + 6], y[8 * c + 7]));
        }
        async_fence();
        tc_before();
        mbar_arrive(smem_u32(&p_full[it & 1]));
      }

      // ---- the run's end: component t of every row ----
      const int g = at.x / a.row_blocks;
      last = n == at.n;
      const int start = at.start(s_share);
      const bool whole = start == 0 && at.t + at.n == at.tiles, more = at.t > start;
      bool apart = false;  // with a shared prefix a whole unit is a piece too
      if constexpr (A::kShared) apart = a.shared_len > 0;
      const bool done = whole && last && !apart;
      const int pslot = seg == 0 ? 0 : 1;  // a CTA's first segment has its slot 0, a later one (its last) slot 1
      if ((apart || a.batch > kJoinScan) && tid == 0 && start == 0 && last)
        a.unit_desc[(long long)at.r * units + at.x] =
            whole ? kUnitWhole : unit_pieces(blockIdx.x, s_share.split.last_cta(at.unit, at.tiles), pslot);
      const float part = reduce_rows<RC>(l, [](float c, float d) { return c + d; });
      // (behind this wait every warp has arrived with the last tile's P, so
      // none still reads s_red as that tile's factors)
      wait(&pv_done[(it - 1) & 1], (uint32_t)((it - 1) >> 1) & 1u);
      __syncwarp();
      tc_after();
      if (lane < RC) s_red[wg][quarter][lane] = part;
      group_sync(1 + wg, 128);
      float* piece = a.parts + ((size_t)blockIdx.x * 2 + pslot) * C::kPieceFloats;
      if constexpr (A::kShared) {
        if (whole && apart) piece = a.whole + ((size_t)at.r * units + at.x) * C::kPieceFloats;
      }
      if (t < RC) {  // a row's sum, its factors, and lse
        float sum = (s_red[wg][0][t] + s_red[wg][1][t]) + (s_red[wg][2][t] + s_red[wg][3][t]);
        const float ref = s_mu[wg][t];
        const int orow = s_out[buf][row_off + t];
        if (more) {  // the runs before, to the reference of now (which every row has that had weights)
          const float before = piece[C::kRows + row_off + t];
          const float f = before == 0.f ? 0.f : exp2_sfu(piece[row_off + t] - ref);
          sum = fmaf(before, f, sum);
          s_red[wg][1][t] = f;
        }
        if (!done) {
          piece[row_off + t] = sum == 0.f ? kNegInf : ref;
          piece[C::kRows + row_off + t] = sum;
        } else {
          s_red[wg][0][t] = sum == 0.f ? 0.f : (FP8 ? a.v_scale[g] : 1.f) / sum;
          if (a.lse && orow >= 0) a.lse[orow] = sum == 0.f ? kNegInf : (ref + log2f(sum)) * kLn2;
        }
      }
      if (done || more) group_sync(1 + wg, 128);
      constexpr int kPart = RC < 16 ? RC : 16;  // rows at a time
#pragma unroll 1
      for (int i = 0; i < MB * (RC / kPart); ++i) {
        const int mb = i / (RC / kPart), r0 = i % (RC / kPart) * kPart;
        const uint32_t addr = o_addr + (uint32_t)(mb * (BLK * N) + r0);
        uint32_t o[kPart];
        Tmem<kPart>::load(addr, o);
        if constexpr (FP8) {
          uint32_t u[kPart];
          Tmem<kPart>::load(addr + 32, u);
          tc_wait_ld();
#pragma unroll
          for (int r = 0; r < kPart; ++r)
            o[r] = __float_as_uint(fmaf(__uint_as_float(u[r]), 0.03125f, __uint_as_float(o[r])));
        } else {
          tc_wait_ld();
        }
        const int comp = mb * 128 + t;
        if (D < 128 && t >= D) continue;  // (a copy; no more barriers here)
        float* dst = piece + 2 * C::kRows + (row_off + r0) * D + comp;
        if (more) {
#pragma unroll
          for (int r = 0; r < kPart; ++r)
            o[r] = __float_as_uint(fmaf(dst[r * D], s_red[wg][1][r0 + r], __uint_as_float(o[r])));
        }
        if (!done) {
#pragma unroll
          for (int r = 0; r < kPart; ++r) dst[r * D] = __uint_as_float(o[r]);  // (rows that are none: of no meaning)
        } else {
#pragma unroll
          for (int r = 0; r < kPart; ++r) {
            const int orow = s_out[buf][row_off + r0 + r];
            // a row that sees nothing (factor 0) is zero whatever O holds
            const float f = s_red[wg][0][r0 + r];
            if (orow >= 0)
              a.out[(size_t)orow * D + comp] = __float2bfloat16_rn(f == 0.f ? 0.f : __uint_as_float(o[r]) * f);
          }
        }
      }
      tc_before();
      group_sync(1 + wg, 128);  // no warp still reads this unit's tables
      at.t += n;
      at.n -= n;
      if (last) ++seg;
    } while (!last || at.next(a, s_share));
  }
  tc_before();
  __syncthreads();
  tc_after();
  if (warp == C::kPvWarp) free_tmem();
}

template <int D, bool FP8, int RC, int WGS, class A>
cudaError_t launch_tc(const qsa_dims& d, A a, const void* k_cache, const void* v_cache, bool short_k,
                      cudaStream_t s) {
  using C = Tc<D, FP8, RC, WGS>;
  alignas(64) CUtensorMap tk, tv;
  if (!make_cache_map(&tk, d, k_cache, kTileTc, C::kLine, short_k) ||
      !make_cache_map(&tv, d, v_cache, kTileTc, C::kLine, false))
    return cudaErrorInvalidValue;
  static DeviceSlots slots;
  cudaError_t e = slots.raise_smem(dense_tc_kernel<C, A>, C::kSmem);
  if (e != cudaSuccess) return e;
  a.row_blocks = (a.n_q * a.group + C::kRows - 1) / C::kRows;
  e = launch_k(dense_tc_kernel<C, A>, dim3(a.grid), dim3(C::kThreads), C::kSmem, s, true, tk, tv, a);
  if (e != cudaSuccess) return e;
  if constexpr (A::kShared) {
    if (a.shared_len > 0) return cudaSuccess;  // (joined with the prefix's pieces)
  }
  return launch_join<D, C::kRows, FP8, kTileTc>(a, s);
}

template <int D, bool FP8, class A>
cudaError_t launch_tc(int rows, const qsa_dims& d, const A& a, const void* k, const void* v, bool short_k,
                      cudaStream_t s) {
  switch (rows) {
    case 8: return launch_tc<D, FP8, 8, 1>(d, a, k, v, short_k, s);
    case 16: return launch_tc<D, FP8, 16, 1>(d, a, k, v, short_k, s);
    case 32: return launch_tc<D, FP8, 16, 2>(d, a, k, v, short_k, s);
    default:
      if constexpr (D * (FP8 ? 1 : 2) <= 256) return launch_tc<D, FP8, 32, 2>(d, a, k, v, short_k, s);
  }
  return cudaErrorInvalidValue;  // (not reached: unit_rows)
}

}  // namespace
}  // namespace qsa
