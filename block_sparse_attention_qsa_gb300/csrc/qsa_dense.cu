// Dense attention over the paged cache (decode and verify).
//
//   o = sum_t softmax_t(c q . k_t) v_t   over  max(0, p - window + 1) <= t <= p,
//   lse = ln sum_t exp(c q . k_t)
//
// One pass over K and V with the running maximum and sum of a softmax (FP32,
// exp2 domain). All n_q x group query rows that share a KV head are worked on
// together, so K and V are read once: 4 D flops a row and position against
// 4 D (BF16) or 2 D (E4M3) bytes, which is far below the card's ratio for up
// to 32 rows. HBM is the bound, and the design follows from it:
//
//  * Split. A unit is one (request, KV head, block of rows); the units' tiles
//    of 64 positions form one stream that is cut into equal contiguous shares,
//    one per persistent CTA, so no SM waits for a long request. The lengths
//    are on the device, so every CTA works the stream out from q_pos itself
//    (one block scan). A unit that ends up in several CTAs leaves (max, sum,
//    acc) pieces in the workspace, which a second kernel, chained with
//    programmatic dependent launch, joins in order (no atomics: the same bits
//    on every call).
//  * Feeding. One warp looks the pages up (32 boxes ahead) and issues the TMA
//    copies of whole tiles, swizzled, into a ring of as many stages as shared
//    memory holds (about 160 KB in flight on every SM, several times what
//    HBM's latency needs), across unit borders.
//  * Eight warps compute: 16 positions of a tile each (four slices, two tiles
//    at a time; with more rows than two MMA tiles hold, the two groups of four
//    warps take half of the rows each instead), S = Q K^T and O += P V with
//    mma.sync m16n8k16. These contractions have 8 to 64 rows and are a few
//    per cent of the tensor pipe; tcgen05's 128-row tiles would be mostly
//    padding and need P back through tensor memory. Each warp has its own
//    running maximum, so warps meet only at the end of a unit.
//  * E4M3 codes are widened to FP16 in registers (exact). K: a 32-bit word of
//    an ldmatrix row holds 4 consecutive codes of a position, taken as
//    components 2c, 2c+1, 2c+8, 2c+9 of the MMA's k dimension, an order that Q
//    is stored in too. V: a transposed ldmatrix word holds two adjacent
//    components of two positions; one byte permute sorts them by component.
//    The BF16 query is scaled per row by a power of two into FP16's range
//    (exact) and the factor goes into the row's softmax scale.
//  * P is rounded to BF16 (FP16 for an E4M3 cache) as the MMA's operand: an
//    error of 2^-9 a weight, random in sign, below the output's own rounding.
//    The sum keeps the unrounded weights.
//
// What is masked never arrives: scores of masked positions are replaced, not
// added to; V of positions that no row of the unit sees is zeroed in
// registers; and where a tile holds a position that only some rows see and
// its V is not finite (0 x NaN would reach the other rows), that tile's PV is
// done row by row on the FP32 pipe.
//
// Every wait is bounded by a clock limit (kind 5, see the abort flag).
#include "qsa_dense.cuh"

namespace qsa {
namespace {

constexpr int kStaticSmem = 768;   // barriers and the like
constexpr int kSlice = 16;         // positions of an MMA
constexpr float kSlack = 8.f;      // a row's reference may trail its maximum by a factor 2^8
constexpr int kComputeWarps = 8;
constexpr int kWarps = kComputeWarps + 4;  // and the copy warp's warpgroup, whose other warps leave at once
constexpr int kThreads = 32 * kWarps;
// The compute warps' accumulators want more registers than 384 threads can be
// launched with (168): the copy warpgroup hands most of its own over.
// 232 x 256 + 40 x 128 = 168 x 384.
constexpr int kComputeRegs = 216, kCopyRegs = 72;
static_assert(kComputeRegs * 32 * kComputeWarps + kCopyRegs * 128 <= 168 * kThreads, "register split");
template <int D_, bool FP8_, int MT_, int RG_>
struct Cfg {
  static constexpr int D = D_, MT = MT_, RG = RG_;
  static constexpr bool FP8 = FP8_;
  static constexpr int kGroupRows = 16 * MT;         // rows of a warp
  static constexpr int kRows = kGroupRows * RG;      // rows of a unit
  static constexpr int kRowBytes = D * (FP8 ? 1 : 2);
  // positions of a tile, four warps' steps: 16 each, or 32 where rows are
  // short and the registers allow it
  static constexpr int kTile = kRowBytes <= 128 && D * MT <= 128 ? 128 : 64;
  static constexpr int kTileShift = kTile == 128 ? 7 : 6;
  static constexpr int NS = kTile / (4 * kSlice);
  static constexpr int kLine = kRowBytes < 128 ? kRowBytes : 128;  // bytes of a TMA box's row
  static constexpr int kLines = kRowBytes / kLine;
  static constexpr int kHalf = kTile * kRowBytes;    // K (or V) of a tile
  static constexpr int kStage = 2 * kHalf;
  static constexpr int kQPitch = D * 2 + 16;         // bytes, conflict-free for ldmatrix
  static constexpr int kQBytes = kRows * kQPitch;
  // slab of the units' joint: 16 columns of every warp's accumulators (BF16
  // rows padded against bank conflicts of the 8-byte stores)
  static constexpr int kSlabPitch = FP8 ? 16 : 20;
  static constexpr int kSlabBytes = kComputeWarps * kGroupRows * kSlabPitch * 4;
  static constexpr int kFixed = kQBytes + kSlabBytes + 2 * kComputeWarps * kGroupRows * 4 + kRows * 4 + 1024;
  static constexpr int kFit = (kMaxSmem - kStaticSmem - kFixed) / kStage;
  // With every other tile for a group of warps (RG 1) the number of stages is
  // even: a stage then always belongs to the same group, which so meets every
  // phase of its barrier (a parity says nothing about a phase two ahead).
  static constexpr int kStages = kFit >= 12 ? 12 : RG == 1 ? kFit & ~1 : kFit;
  static constexpr int kSmem = kStages * kStage + kFixed;
  static constexpr int kPieceFloats = kRows * (D + 2);  // m, l, acc of a piece
  static constexpr bool kQInRegs = D * MT <= 128;
  static_assert(kStages >= 2 && kSlabBytes >= kComputeWarps * kGroupRows * kSlice * 4, "shared memory");
};

__device__ __forceinline__ void compute_sync() {  // the compute warps only
  asm volatile("bar.sync 1, %0;" ::"n"(32 * kComputeWarps) : "memory");
}
__device__ __forceinline__ void ldsm4(uint32_t addr, uint32_t (&r)[4]) {
  asm volatile("ldmatrix.sync.aligned.m8n8.x4.shared.b16 {%0,%1,%2,%3}, [%4];"
               : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3])
               : "r"(addr)
               : "memory");
}
__device__ __forceinline__ void ldsm4t(uint32_t addr, uint32_t (&r)[4]) {
  asm volatile("ldmatrix.sync.aligned.m8n8.x4.trans.shared.b16 {%0,%1,%2,%3}, [%4];"
               : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3])
               : "r"(addr)
               : "memory");
}
template <bool F16>
__device__ __forceinline__ void mma(float (&d)[4], const uint32_t (&a)[4], uint32_t b0, uint32_t b1) {
  if constexpr (F16) {
    asm volatile(
        "mma.sync.aligned.m16n8k16.row.col.f32.f16.f16.f32 {%0,%1,%2,%3}, {%4,%5,%6,%7}, {%8,%9}, {%0,%1,%2,%3};"
        : "+f"(d[0]), "+f"(d[1]), "+f"(d[2]), "+f"(d[3])
        : "r"(a[0]), "r"(a[1]), "r"(a[2]), "r"(a[3]), "r"(b0), "r"(b1));
  } else {
    asm volatile(
        "mma.sync.aligned.m16n8k16.row.col.f32.bf16.bf16.f32 {%0,%1,%2,%3}, {%4,%5,%6,%7}, {%8,%9}, {%0,%1,%2,%3};"
        : "+f"(d[0]), "+f"(d[1]), "+f"(d[2]), "+f"(d[3])
        : "r"(a[0]), "r"(a[1]), "r"(a[2]), "r"(a[3]), "r"(b0), "r"(b1));
  }
}
template <bool F16>
__device__ __forceinline__ uint32_t pack2(float lo, float hi) {
  if constexpr (F16) {
    const __half2 h = __floats2half2_rn(lo, hi);
    return *reinterpret_cast<const uint32_t*>(&h);
  } else {
    return pack_bf(lo, hi);
  }
}
// address of 16-byte chunk `chunk` of row `row` (a position) of a staged K or V
// tile, as the TMA swizzle lays it out
template <class C>
__device__ __forceinline__ uint32_t chunk_at(uint32_t base, int row, int chunk) {
  if constexpr (C::kLine == 128)
    return base + (uint32_t)((chunk >> 3) * (C::kTile * 128) + row * 128 + (((chunk & 7) ^ (row & 7)) << 4));
  else
    return base + (uint32_t)(row * 64 + (((chunk & 3) ^ ((row >> 1) & 3)) << 4));
}

template <class C>
__global__ void __launch_bounds__(kThreads, 1) dense_kernel(const __grid_constant__ CUtensorMap tm_k,
                                                            const __grid_constant__ CUtensorMap tm_v,
                                                            const DenseArgs a) {
  constexpr int D = C::D, MT = C::MT, RG = C::RG;
  constexpr bool FP8 = C::FP8;
  constexpr int kTile = C::kTile, NS = C::NS;
  extern __shared__ uint8_t smem_raw[];
  uint8_t* smem = reinterpret_cast<uint8_t*>((reinterpret_cast<uintptr_t>(smem_raw) + 1023) & ~uintptr_t(1023));
  uint8_t* ring = smem;
  uint8_t* s_q = ring + C::kStages * C::kStage;
  float* slab = reinterpret_cast<float*>(s_q + C::kQBytes);
  float* s_m = slab + C::kSlabBytes / 4;                      // [warp][group row]
  float* s_l = s_m + kComputeWarps * C::kGroupRows;
  float* s_qs = s_l + kComputeWarps * C::kGroupRows;          // [row] softmax scale (exp2 domain)
  __shared__ __align__(8) uint64_t full_bar[C::kStages], empty_bar[C::kStages];
  __shared__ uint32_t s_bad[C::kStages];  // bit s: slice s of the staged tile has no page
  __shared__ long long s_scan[kWarps];
  __shared__ Share s_share;
  __shared__ volatile int s_abort;
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
  const int units = a.n_kv_heads * a.row_blocks;  // of a request

  if (tid == 0) {
    s_abort = 0;
    for (int s = 0; s < C::kStages; ++s) {
      mbar_init(smem_u32(&full_bar[s]), 1);
      mbar_init(smem_u32(&empty_bar[s]), RG == 1 ? 4 : 8);
    }
    asm volatile("fence.mbarrier_init.release.cluster;" ::: "memory");
  }
  pdl_wait();     // positions, queries and the cache may come from the kernel before
  pdl_trigger();  // the joining kernel may be set up; it waits for this one's end

  Walk<kTile> at;
  if (!find_start<kTile, kThreads>(a, s_scan, s_share, at)) return;
  auto wait = [&](uint64_t* bar, uint32_t parity) { return mbar_wait(bar, parity, &s_abort, a.err); };

  if (warp >= kComputeWarps) {
    // ---- the copy warp ----
    asm volatile("setmaxnreg.dec.sync.aligned.u32 %0;" ::"n"(kCopyRegs));
    if (warp > kComputeWarps) return;
    PageFeed<kTile> feed(a);
    const int box_bytes = C::kLine << feed.box_shift, line_ops = feed.boxes * C::kLines;
    int stage = 0;
    uint32_t phase = 0;
    bool ok = true;
    do {
      const int g = at.x / a.row_blocks;
      feed.start(a, at);
      for (int k = 0; k < at.n && ok; ++k) {
        const int page = feed.of_tile(a, at, k);
        const uint32_t bad = feed.bad_groups(page);  // (a box holds whole sub-slices)
        ok = __all_sync(kFull, wait(&empty_bar[stage], phase ^ 1u));
        if (!ok) break;
        const uint32_t bar = smem_u32(&full_bar[stage]);
        if (lane == 0) {
          s_bad[stage] = bad;
          mbar_expect_tx(bar, C::kStage);
        }
        __syncwarp();
        const int slot = feed.slot_of(a, k);
        const uint32_t base = smem_u32(ring + stage * C::kStage);
        for (int i = lane; i < 2 * line_ops; i += 32) {  // (32 is a multiple of boxes: lane i's box is my_box)
          const bool v = i >= line_ops;
          const int line = (v ? i - line_ops : i) >> (C::kTileShift - feed.box_shift);
          tma_load_4d(base + (uint32_t)((v ? C::kHalf : 0) + line * (kTile * C::kLine) + feed.my_box * box_bytes),
                      v ? &tm_v : &tm_k, line * (C::kLine / (FP8 ? 1 : 2)), slot, g,
                      page < 0 ? a.num_pages : page /* outside: zeros */, bar);
        }
        if (++stage == C::kStages) {
          stage = 0;
          phase ^= 1u;
        }
      }
    } while (ok && at.next(a, s_share));
    if (s_abort) {
      // copies in flight land before the CTA leaves: the last kStages issued
      // (bounded; a stage whose phase already completed answers at once)
      for (int s = 0; s < C::kStages; ++s) {
        const uint32_t par = s < stage ? phase : phase ^ 1u;
        const long long start = clock64();
        while (!mbar_try_wait(smem_u32(&full_bar[s]), par) && clock64() - start < kWaitCycles / 64) {
        }
      }
    }
    return;
  }

  // ---- the compute warps ----
  asm volatile("setmaxnreg.inc.sync.aligned.u32 %0;" ::"n"(kComputeRegs));
  const int slice = warp & 3, grp = warp >> 2;  // grp: every other tile (RG 1) or half of the rows (RG 2)
  const int gq = lane >> 2, c4 = lane & 3;
  const int row_base = RG == 2 ? grp * C::kGroupRows : 0;
  const uint32_t q_addr = smem_u32(s_q) + (uint32_t)((row_base + (lane & 15)) * C::kQPitch + (lane >> 4) * 16);
  long long it = 0;  // tiles of this CTA so far
  int pslot = 0;     // a CTA's first segment has its slot 0, a later one (its last) slot 1
  do {
    const int n = at.n;
    const int g = at.x / a.row_blocks, rb = at.x - g * a.row_blocks;
    const int rows = min(C::kRows, a.n_q * a.group - rb * C::kRows);  // of this unit
    const float vscale = FP8 ? a.v_scale[g] : 1.f;

    // the unit's query rows into shared memory
    {
      constexpr int kLanes = D / 8;  // lanes of a row, 16 bytes each
      const float base_scale = a.sm_scale * kLog2e * (FP8 ? a.k_scale[g] : 1.f);
      for (int row = tid / kLanes; row < C::kRows; row += 32 * kComputeWarps / kLanes) {
        const int c = tid % kLanes;
        uint4 v = make_uint4(0, 0, 0, 0);
        if (row < rows) {
          const int i = rb * C::kRows + row, j = i / a.group, h = g * a.group + (i - j * a.group);
          v = ld16(a.q + (((size_t)at.r * a.n_q + j) * a.n_q_heads + h) * D + c * 8);
        }
        uint8_t* dst = s_q + row * C::kQPitch;
        if constexpr (FP8) {
          // magnitudes of BF16 values order like their bit patterns
          uint32_t big = 0;
          const uint32_t wd[4] = {v.x, v.y, v.z, v.w};
#pragma unroll
          for (int e = 0; e < 4; ++e) big = max(big, max((wd[e] << 16) & 0x7fff0000u, wd[e] & 0x7fff0000u));
#pragma unroll
          for (int o = 1; o < kLanes; o <<= 1) big = max(big, __shfl_xor_sync(kFull, big, o));
          // 2^-sh brings the row's largest value into [2^14, 2^15)
          const int sh = big == 0 ? 0 : min(126, max(-126, (int)(big >> 23) - 127 - 14));
          const float down = pow2(-sh);
          uint32_t h2[4];
#pragma unroll
          for (int e = 0; e < 4; ++e) h2[e] = pack2<true>(bf_lo(wd[e]) * down, bf_hi(wd[e]) * down);
          // components 8c + 0..7 of k step c / 2: words 4x..4x+3 of K go to k
          // slots 2x, 2x+1 and 2x+8, 2x+9
          const int x = (c & 1) * 2;
          uint32_t* d32 = reinterpret_cast<uint32_t*>(dst + (c >> 1) * 32);
          d32[x] = h2[0];
          d32[x + 4] = h2[1];
          d32[x + 1] = h2[2];
          d32[x + 5] = h2[3];
          if (c == 0) s_qs[row] = base_scale * pow2(sh);
        } else {
          *reinterpret_cast<uint4*>(dst + c * 16) = v;
          if (c == 0) s_qs[row] = base_scale;
        }
      }
    }
    // positions that the lane's rows see, and that all rows of the unit see
    int lo[2 * MT], hi[2 * MT];
#pragma unroll
    for (int k = 0; k < 2 * MT; ++k) {
      const int row = row_base + 8 * k + gq;
      lo[k] = hi[k] = 0;
      if (row < rows) {
        const int p = a.q_pos[(size_t)at.r * a.n_q + (rb * C::kRows + row) / a.group];
        if (valid_pos(a, p)) {
          lo[k] = low_of(a, p);
          hi[k] = p + 1;
        }
      }
    }
    int all_lo = 0, all_hi = 0x7fffffff;
    {
      const int j0 = rb * C::kRows / a.group, j1 = (rb * C::kRows + rows - 1) / a.group;
      for (int j = j0; j <= j1; ++j) {
        const int p = a.q_pos[(size_t)at.r * a.n_q + j];
        all_lo = max(all_lo, valid_pos(a, p) ? low_of(a, p) : 0);
        all_hi = min(all_hi, valid_pos(a, p) ? p + 1 : 0);
      }
    }
    compute_sync();

    float scale[2 * MT];
#pragma unroll
    for (int k = 0; k < 2 * MT; ++k) scale[k] = s_qs[row_base + 8 * k + gq];
    uint32_t qr[C::kQInRegs ? MT * D / 16 : 1][4];
    if constexpr (C::kQInRegs) {
#pragma unroll
      for (int mt = 0; mt < MT; ++mt)
#pragma unroll
        for (int ks = 0; ks < D / 16; ++ks)
          ldsm4(q_addr + (uint32_t)(mt * 16 * C::kQPitch + ks * 32), qr[mt * (D / 16) + ks]);
    }
    float m[2 * MT], l[2 * MT], o[MT][D / 8][4];
#pragma unroll
    for (int k = 0; k < 2 * MT; ++k) {
      m[k] = kNegInf;
      l[k] = 0.f;
    }
#pragma unroll
    for (int mt = 0; mt < MT; ++mt)
#pragma unroll
      for (int i = 0; i < D / 8; ++i)
#pragma unroll
        for (int e = 0; e < 4; ++e) o[mt][i][e] = 0.f;

    for (int k = 0; k < n; ++k, ++it) {
      if (RG == 1 && (int)(it & 1) != grp) continue;
      const int stage = (int)(it % C::kStages);
      if (!wait(&full_bar[stage], (uint32_t)(it / C::kStages) & 1u)) continue;
      const int row0 = slice * (NS * kSlice);  // this warp's positions within the tile
      const int p0 = (at.g.lo / kTile + at.t + k) * kTile + row0;
      // sub-slices without a page are masked
      const uint32_t bad = (s_bad[stage] >> (slice * NS)) & ((1u << NS) - 1u);
      if (bad != (1u << NS) - 1u && p0 < at.g.hi && p0 + NS * kSlice > at.g.lo) {
        const uint32_t kb = smem_u32(ring + stage * C::kStage), vb = kb + C::kHalf;
        const int r8 = lane & 7, q8 = lane >> 3;  // ldmatrix: this lane's row of matrix q8
        // ---- S = Q K^T: 16 x MT rows, 16 x NS positions ----
        float s[NS][MT][2][4];
#pragma unroll
        for (int ns = 0; ns < NS; ++ns)
#pragma unroll
          for (int mt = 0; mt < MT; ++mt)
#pragma unroll
            for (int i = 0; i < 2; ++i)
#pragma unroll
              for (int e = 0; e < 4; ++e) s[ns][mt][i][e] = 0.f;
#pragma unroll
        for (int ks = 0; ks < D / 16; ks += FP8 ? 2 : 1) {
          uint32_t kr[NS][4];
#pragma unroll
          for (int ns = 0; ns < NS; ++ns) {
            const int row = row0 + ns * kSlice + r8;
            if constexpr (FP8) {
              // matrices: positions 0-7 and 8-15 of k step ks, then of ks + 1
              ldsm4(chunk_at<C>(kb, row + (q8 & 1) * 8, ks + (q8 >> 1)), kr[ns]);
            } else {
              // matrices: the two 8-component halves for positions 0-7, then 8-15
              ldsm4(chunk_at<C>(kb, row + (q8 >> 1) * 8, 2 * ks + (q8 & 1)), kr[ns]);
            }
          }
#pragma unroll
          for (int u = 0; u < (FP8 ? 2 : 1); ++u) {
            uint32_t b[NS][2][2];
#pragma unroll
            for (int ns = 0; ns < NS; ++ns) {
              if constexpr (FP8) {
                widen4(kr[ns][2 * u], b[ns][0][0], b[ns][0][1]);
                widen4(kr[ns][2 * u + 1], b[ns][1][0], b[ns][1][1]);
              } else {
                b[ns][0][0] = kr[ns][0], b[ns][0][1] = kr[ns][1], b[ns][1][0] = kr[ns][2], b[ns][1][1] = kr[ns][3];
              }
            }
#pragma unroll
            for (int mt = 0; mt < MT; ++mt) {
              uint32_t qa[4];
              if constexpr (!C::kQInRegs) ldsm4(q_addr + (uint32_t)(mt * 16 * C::kQPitch + (ks + u) * 32), qa);
              const uint32_t(&qf)[4] = C::kQInRegs ? qr[C::kQInRegs ? mt * (D / 16) + ks + u : 0] : qa;
#pragma unroll
              for (int ns = 0; ns < NS; ++ns) {
                mma<FP8>(s[ns][mt][0], qf, b[ns][0][0], b[ns][0][1]);
                mma<FP8>(s[ns][mt][1], qf, b[ns][1][0], b[ns][1][1]);
              }
            }
          }
        }
        // ---- softmax ----
        // lane's values: s[ns][mt][i][2 half + e] is row 16 mt + 8 half + gq,
        // position p0 + 16 ns + 8 i + 2 c4 + e
        const bool edge = p0 < all_lo || p0 + NS * kSlice > all_hi || bad != 0;
        bool grew = false;  // some score is more than 2^kSlack above its row's reference
#pragma unroll
        for (int ns = 0; ns < NS; ++ns)
#pragma unroll
          for (int mt = 0; mt < MT; ++mt)
#pragma unroll
            for (int i = 0; i < 2; ++i)
#pragma unroll
              for (int e = 0; e < 4; ++e) {
                const int kk = 2 * mt + (e >> 1);
                float& x = s[ns][mt][i][e];
                x *= scale[kk];
                if (edge) {
                  const int p = p0 + kSlice * ns + 8 * i + 2 * c4 + (e & 1);
                  if (p < lo[kk] || p >= hi[kk] || ((bad >> ns) & 1u)) x = kNegInf;
                }
                grew |= x > m[kk] + kSlack;
              }
        // The reference m of a row (which its weights are relative to) only
        // has to keep the weights in range, so it moves when a score passes it
        // by 2^8, not with every new maximum: of 16 or 32 rows one has a new
        // maximum in most early steps, and moving costs D / 2 products a lane
        // and row pair. (From -infinity it moves with the first position.)
        if (__any_sync(kFull, grew)) {
#pragma unroll
          for (int kk = 0; kk < 2 * MT; ++kk) {
            const int mt = kk >> 1, e = 2 * (kk & 1);
            float x = m[kk];
#pragma unroll
            for (int ns = 0; ns < NS; ++ns)
              x = fmaxf(x, fmaxf(fmaxf(s[ns][mt][0][e], s[ns][mt][0][e + 1]), fmaxf(s[ns][mt][1][e], s[ns][mt][1][e + 1])));
            x = fmaxf(x, __shfl_xor_sync(kFull, x, 1));
            x = fmaxf(x, __shfl_xor_sync(kFull, x, 2));
            const float f = exp2_sfu(m[kk] - (x == kNegInf ? 0.f : x));
            m[kk] = x;
            l[kk] *= f;
#pragma unroll
            for (int i = 0; i < D / 8; ++i) {
              o[mt][i][e] *= f;
              o[mt][i][e + 1] *= f;
            }
          }
        }
#pragma unroll
        for (int kk = 0; kk < 2 * MT; ++kk) {
          const int mt = kk >> 1, e = 2 * (kk & 1);
          const float mu = m[kk] == kNegInf ? 0.f : m[kk];
#pragma unroll
          for (int ns = 0; ns < NS; ++ns)
#pragma unroll
            for (int i = 0; i < 2; ++i) {
              s[ns][mt][i][e] = exp2_sfu(s[ns][mt][i][e] - mu);
              s[ns][mt][i][e + 1] = exp2_sfu(s[ns][mt][i][e + 1] - mu);
              l[kk] += s[ns][mt][i][e] + s[ns][mt][i][e + 1];
            }
        }
        // ---- O += P V ----
        // V words: BF16: positions 2 c4, 2 c4 + 1 (+ 8) of one component;
        // E4M3 (after the permute): those positions of two components
        uint32_t keep[NS][2];
        bool by_row = false;
        if (edge) {
#pragma unroll
          for (int ns = 0; ns < NS; ++ns)
#pragma unroll
            for (int i = 0; i < 2; ++i) {
              const int p = p0 + ns * kSlice + 8 * i + 2 * c4;
              const bool ok0 = p >= at.g.lo && p < at.g.hi, ok1 = p + 1 >= at.g.lo && p + 1 < at.g.hi;
              keep[ns][i] = FP8 ? (ok0 ? 0x00ff00ffu : 0u) | (ok1 ? 0xff00ff00u : 0u)
                                : (ok0 ? 0x0000ffffu : 0u) | (ok1 ? 0xffff0000u : 0u);
            }
          bool odd = false;  // some V that is seen is not finite
#pragma unroll
          for (int ns = 0; ns < NS; ++ns)
#pragma unroll 4
            for (int i = 0; i < C::kRowBytes / 16; i += 2) {
              uint32_t vr[4];
              ldsm4t(chunk_at<C>(vb, row0 + ns * kSlice + (q8 & 1) * 8 + r8, i + (q8 >> 1)), vr);
#pragma unroll
              for (int e = 0; e < 4; ++e) {
                if constexpr (FP8) {
                  const uint32_t x = __byte_perm(vr[e], 0, 0x3120) & keep[ns][e & 1] & 0x7f7f7f7fu;
                  odd |= ((x + 0x01010101u) & 0x80808080u) != 0;
                } else {
                  const uint32_t x = vr[e] & keep[ns][e & 1];
                  odd |= (x & 0x7f80u) == 0x7f80u || (x & 0x7f800000u) == 0x7f800000u;
                }
              }
            }
          by_row = __any_sync(kFull, odd);
        }
        if (!by_row) {
          uint32_t pa[NS][MT][4];
#pragma unroll
          for (int ns = 0; ns < NS; ++ns)
#pragma unroll
            for (int mt = 0; mt < MT; ++mt) {
              pa[ns][mt][0] = pack2<FP8>(s[ns][mt][0][0], s[ns][mt][0][1]);
              pa[ns][mt][1] = pack2<FP8>(s[ns][mt][0][2], s[ns][mt][0][3]);
              pa[ns][mt][2] = pack2<FP8>(s[ns][mt][1][0], s[ns][mt][1][1]);
              pa[ns][mt][3] = pack2<FP8>(s[ns][mt][1][2], s[ns][mt][1][3]);
            }
#pragma unroll
          for (int i = 0; i < C::kRowBytes / 16; i += 2) {
#pragma unroll
            for (int ns = 0; ns < NS; ++ns) {
              uint32_t vr[4];  // positions 0-7 and 8-15 of chunk i, then of chunk i + 1
              ldsm4t(chunk_at<C>(vb, row0 + ns * kSlice + (q8 & 1) * 8 + r8, i + (q8 >> 1)), vr);
#pragma unroll
              for (int u = 0; u < 2; ++u) {
                if constexpr (FP8) {
                  uint32_t ev[2], od[2];  // even and odd components of the chunk's 16
#pragma unroll
                  for (int e = 0; e < 2; ++e) {
                    uint32_t x = __byte_perm(vr[2 * u + e], 0, 0x3120);
                    if (edge) x &= keep[ns][e];
                    widen4(x, ev[e], od[e]);
                  }
#pragma unroll
                  for (int mt = 0; mt < MT; ++mt) {
                    mma<true>(o[mt][2 * (i + u)], pa[ns][mt], ev[0], ev[1]);
                    mma<true>(o[mt][2 * (i + u) + 1], pa[ns][mt], od[0], od[1]);
                  }
                } else {
                  if (edge) {
                    vr[2 * u] &= keep[ns][0];
                    vr[2 * u + 1] &= keep[ns][1];
                  }
#pragma unroll
                  for (int mt = 0; mt < MT; ++mt) mma<false>(o[mt][i + u], pa[ns][mt], vr[2 * u], vr[2 * u + 1]);
                }
              }
            }
          }
        } else {
          float* pw = slab + warp * C::kGroupRows * kSlice;  // this warp's P of one sub-slice, [row][position]
#pragma unroll
          for (int ns = 0; ns < NS; ++ns) {
#pragma unroll
            for (int mt = 0; mt < MT; ++mt)
#pragma unroll
              for (int i = 0; i < 2; ++i)
#pragma unroll
                for (int e = 0; e < 4; ++e)
                  pw[(16 * mt + 8 * (e >> 1) + gq) * kSlice + 8 * i + 2 * c4 + (e & 1)] = s[ns][mt][i][e];
            __syncwarp();
#pragma unroll 1
            for (int t = 0; t < kSlice; ++t) {
              const int p = p0 + ns * kSlice + t, row = row0 + ns * kSlice + t;
              float pv[2 * MT];
              bool see[2 * MT];
#pragma unroll
              for (int kk = 0; kk < 2 * MT; ++kk) {
                see[kk] = p >= lo[kk] && p < hi[kk];
                pv[kk] = pw[(8 * kk + gq) * kSlice + t];
              }
#pragma unroll
              for (int i = 0; i < D / 8; i += FP8 ? 2 : 1) {
                // the lane's components of tile i (BF16: 8 i + 2 c4 + 0, 1) or
                // of tiles i, i + 1 (E4M3: 8 i + 4 c4 + 0..3, even ones in tile i)
                const int comp = FP8 ? 8 * i + 4 * c4 : 8 * i + 2 * c4;
                const int byte = comp * (FP8 ? 1 : 2);
                uint32_t word;
                asm volatile("ld.shared.u32 %0, [%1];"
                             : "=r"(word)
                             : "r"(chunk_at<C>(vb, row, byte >> 4) + (uint32_t)(byte & 15)));
                float v[4];
                if constexpr (FP8) {
                  uint32_t x, y;
                  widen4(word, x, y);
                  const float2 f0 = h2_to_f2(x), f1 = h2_to_f2(y);
                  v[0] = f0.x, v[1] = f0.y, v[2] = f1.x, v[3] = f1.y;
                } else {
                  v[0] = bf_lo(word), v[1] = bf_hi(word);
                }
#pragma unroll
                for (int kk = 0; kk < 2 * MT; ++kk) {
                  if (!see[kk]) continue;
                  float(&acc)[4] = o[kk >> 1][i];
                  const int e = 2 * (kk & 1);
                  if constexpr (FP8) {
                    float(&odd)[4] = o[kk >> 1][i + 1];
                    acc[e] = fmaf(pv[kk], v[0], acc[e]);
                    odd[e] = fmaf(pv[kk], v[1], odd[e]);
                    acc[e + 1] = fmaf(pv[kk], v[2], acc[e + 1]);
                    odd[e + 1] = fmaf(pv[kk], v[3], odd[e + 1]);
                  } else {
                    acc[e] = fmaf(pv[kk], v[0], acc[e]);
                    acc[e + 1] = fmaf(pv[kk], v[1], acc[e + 1]);
                  }
                }
              }
            }
            __syncwarp();
          }
        }
      }
      __syncwarp();
      if (lane == 0) mbar_arrive(smem_u32(&empty_bar[stage]));
    }

    // ---- the segment's end: join the warps ----
    const bool whole = n == at.tiles;
    const long long unit = (long long)at.r * units + at.x;
    if (a.batch > kJoinScan && tid == 0 && at.t == 0)
      a.unit_desc[unit] = whole ? kUnitWhole : unit_pieces(blockIdx.x, s_share.split.last_cta(at.unit, at.tiles), pslot);
    float* piece = a.parts + ((size_t)blockIdx.x * 2 + pslot) * C::kPieceFloats;
    const int wrow = warp * C::kGroupRows;
#pragma unroll
    for (int kk = 0; kk < 2 * MT; ++kk) {
      l[kk] += __shfl_xor_sync(kFull, l[kk], 1);
      l[kk] += __shfl_xor_sync(kFull, l[kk], 2);
      if (c4 == 0) {
        s_m[wrow + 8 * kk + gq] = m[kk];
        s_l[wrow + 8 * kk + gq] = l[kk];
      }
    }
    compute_sync();
    constexpr int kJoin = RG == 1 ? 8 : 4;  // warps that hold a row
    const int j0 = RG == 1 ? 0 : 4 * grp;
#pragma unroll
    for (int kk = 0; kk < 2 * MT; ++kk) {
      float big = kNegInf;
#pragma unroll
      for (int u = 0; u < kJoin; ++u) big = fmaxf(big, s_m[(j0 + u) * C::kGroupRows + 8 * kk + gq]);
      const float f = exp2_sfu(m[kk] - (big == kNegInf ? 0.f : big));
#pragma unroll
      for (int i = 0; i < D / 8; ++i) {
        o[kk >> 1][i][2 * (kk & 1)] *= f;
        o[kk >> 1][i][2 * (kk & 1) + 1] *= f;
      }
    }
    // each thread adds up column col of rows row0, row0 + 16, ..
    const int col = tid & 15, row0 = tid >> 4;
    constexpr int kSteps = C::kRows / 16;
    float big_r[kSteps], sum_r[kSteps];
#pragma unroll
    for (int z = 0; z < kSteps; ++z) {
      const int row = row0 + 16 * z, u0 = row / C::kGroupRows * 4, gr = row % C::kGroupRows;
      big_r[z] = kNegInf;
      sum_r[z] = 0.f;
#pragma unroll
      for (int u = 0; u < kJoin; ++u) big_r[z] = fmaxf(big_r[z], s_m[(u0 + u) * C::kGroupRows + gr]);
      const float mu = big_r[z] == kNegInf ? 0.f : big_r[z];
#pragma unroll
      for (int u = 0; u < kJoin; ++u)
        sum_r[z] += s_l[(u0 + u) * C::kGroupRows + gr] * exp2_sfu(s_m[(u0 + u) * C::kGroupRows + gr] - mu);
    }
#pragma unroll
    for (int ch = 0; ch < D / 16; ++ch) {
#pragma unroll
      for (int kk = 0; kk < 2 * MT; ++kk) {
        float* dst = slab + (wrow + 8 * kk + gq) * C::kSlabPitch;
        const int mt = kk >> 1, e = 2 * (kk & 1);
        if constexpr (FP8) {
          *reinterpret_cast<float4*>(dst + 4 * c4) =
              make_float4(o[mt][2 * ch][e], o[mt][2 * ch + 1][e], o[mt][2 * ch][e + 1], o[mt][2 * ch + 1][e + 1]);
        } else {
          *reinterpret_cast<float2*>(dst + 2 * c4) = make_float2(o[mt][2 * ch][e], o[mt][2 * ch][e + 1]);
          *reinterpret_cast<float2*>(dst + 8 + 2 * c4) = make_float2(o[mt][2 * ch + 1][e], o[mt][2 * ch + 1][e + 1]);
        }
      }
      compute_sync();
#pragma unroll
      for (int z = 0; z < kSteps; ++z) {
        const int row = row0 + 16 * z, u0 = row / C::kGroupRows * 4, gr = row % C::kGroupRows;
        float acc = 0.f;
#pragma unroll
        for (int u = 0; u < kJoin; ++u) acc += slab[((u0 + u) * C::kGroupRows + gr) * C::kSlabPitch + col];
        if (row < rows) {
          if (whole) {
            const int i = rb * C::kRows + row, j = i / a.group, h = g * a.group + (i - j * a.group);
            const size_t orow = ((size_t)at.r * a.n_q + j) * a.n_q_heads + h;
            const float v = sum_r[z] == 0.f ? 0.f : acc / sum_r[z] * vscale;
            a.out[orow * D + ch * 16 + col] = __float2bfloat16_rn(v);
            if (a.lse && ch == 0 && col == 0)
              a.lse[orow] = sum_r[z] == 0.f ? kNegInf : (big_r[z] + log2f(sum_r[z])) * kLn2;
          } else {
            piece[2 * C::kRows + row * D + ch * 16 + col] = acc;
            if (ch == 0 && col == 0) {
              piece[row] = big_r[z];
              piece[C::kRows + row] = sum_r[z];
            }
          }
        }
      }
      compute_sync();
    }
    pslot = 1;
  } while (at.next(a, s_share));
}

// ---------------------------------------------------------------------------
// host
// ---------------------------------------------------------------------------
// Rows of a unit: two MMA row tiles a warp (one for head dim 256, whose
// accumulators fill the registers), and twice that when the two warp groups
// take half of the rows each; more rows than that become several units that
// each read K and V.
struct Shape {
  int mt, rg;
  int rows() const { return 16 * mt * rg; }
};
Shape shape_of(const qsa_dims& d) {
  const int rows = d.n_q * (d.n_q_heads / d.n_kv_heads);
  const int mt = rows <= 16 || d.head_dim == 256 ? 1 : 2;
  return {mt, rows > 16 * mt ? 2 : 1};
}

template <class C>
cudaError_t launch(const qsa_dims& d, DenseArgs a, const void* k_cache, const void* v_cache, cudaStream_t s) {
  alignas(64) CUtensorMap tk, tv;
  if (!make_cache_map(&tk, d, k_cache, C::kTile, C::kLine) || !make_cache_map(&tv, d, v_cache, C::kTile, C::kLine))
    return cudaErrorInvalidValue;
  static DeviceSlots slots;
  cudaError_t e = slots.raise_smem(dense_kernel<C>, C::kSmem);
  if (e != cudaSuccess) return e;
  a.row_blocks = (a.n_q * a.group + C::kRows - 1) / C::kRows;
  e = launch_k(dense_kernel<C>, dim3(a.grid), dim3(kThreads), C::kSmem, s, true, tk, tv, a);
  if (e != cudaSuccess) return e;
  return launch_join<C::D, C::kRows, C::FP8, C::kTile>(a, s);
}

template <int D, bool FP8>
cudaError_t launch(const Shape& sh, const qsa_dims& d, const DenseArgs& a, const void* k, const void* v,
                   cudaStream_t s) {
  if constexpr (D == 256) {
    return sh.rg == 1 ? launch<Cfg<D, FP8, 1, 1>>(d, a, k, v, s) : launch<Cfg<D, FP8, 1, 2>>(d, a, k, v, s);
  } else {
    if (sh.mt == 1) return launch<Cfg<D, FP8, 1, 1>>(d, a, k, v, s);
    return sh.rg == 1 ? launch<Cfg<D, FP8, 2, 1>>(d, a, k, v, s) : launch<Cfg<D, FP8, 2, 2>>(d, a, k, v, s);
  }
}

// rows of a unit of these dims
int unit_rows(const qsa_dims& d) { return d.head_dim == 128 ? dense_tc_rows(d) : shape_of(d).rows(); }

}  // namespace

EncodeTiled encode_tiled() {
  static EncodeTiled fn = [] {
    void* p = nullptr;
    cudaDriverEntryPointQueryResult q;
    if (cudaGetDriverEntryPointByVersion("cuTensorMapEncodeTiled", &p, 12000, cudaEnableDefault, &q) != cudaSuccess ||
        q != cudaDriverEntryPointSuccess)
      p = nullptr;
    return reinterpret_cast<EncodeTiled>(p);
  }();
  return fn;
}

DenseWs dense_ws(const qsa_dims& d, int num_sms) {
  DenseWs w;
  const int rows = d.n_q * (d.n_q_heads / d.n_kv_heads), per = unit_rows(d);
  const size_t units = (size_t)d.batch * d.n_kv_heads * ((rows + per - 1) / per);
  w.units = 256 + align_up((size_t)d.batch * d.n_q * d.n_kv_heads * sizeof(int32_t), 256);
  w.parts = align_up(w.units + units * sizeof(long long), 256);
  w.total = align_up(w.parts + (size_t)num_sms * 2 * per * (d.head_dim + 2) * sizeof(float), 256);
  return w;
}

cudaError_t launch_paged_attn(const qsa_dims& d, int window, const void* q, const void* k_cache, const void* v_cache,
                              const float* k_scale, const float* v_scale, const int32_t* page_table,
                              const int32_t* q_pos, void* out, float* lse, void* ws, cudaStream_t s) {
  const int sms = device_sm_count();
  const DenseWs w = dense_ws(d, sms);
  uint8_t* base = static_cast<uint8_t*>(ws);
  DenseArgs a = {};
  a.q = static_cast<const __nv_bfloat16*>(q);
  a.k_scale = k_scale;
  a.v_scale = v_scale;
  a.page_table = page_table;
  a.q_pos = q_pos;
  a.out = static_cast<__nv_bfloat16*>(out);
  a.lse = lse;
  a.unit_desc = reinterpret_cast<long long*>(base + w.units);
  a.parts = reinterpret_cast<float*>(base + w.parts);
  a.err = static_cast<int32_t*>(ws);
  a.batch = d.batch;
  a.n_q = d.n_q;
  a.n_q_heads = d.n_q_heads;
  a.n_kv_heads = d.n_kv_heads;
  a.group = d.n_q_heads / d.n_kv_heads;
  a.page_size = d.page_size;
  while ((1 << a.page_shift) < d.page_size) ++a.page_shift;
  a.max_pages = d.max_pages;
  a.num_pages = d.num_pages;
  a.window = window;
  a.grid = sms;
  a.sm_scale = d.sm_scale > 0.f ? d.sm_scale : 1.f / sqrtf((float)d.head_dim);
  if (d.head_dim == 128) return launch_dense_tc(d, a, k_cache, v_cache, s);
  const Shape sh = shape_of(d);
  const bool fp8 = d.kv_dtype == QSA_KV_FP8_E4M3;
  if (d.head_dim == 64)
    return fp8 ? launch<64, true>(sh, d, a, k_cache, v_cache, s) : launch<64, false>(sh, d, a, k_cache, v_cache, s);
  return fp8 ? launch<256, true>(sh, d, a, k_cache, v_cache, s) : launch<256, false>(sh, d, a, k_cache, v_cache, s);
}

}  // namespace qsa
