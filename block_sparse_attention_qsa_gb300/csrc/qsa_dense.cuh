// Dense attention over the paged cache (decode and verify): the stream of
// tiles and its split, and the kernel that joins the pieces. The kernel that
// makes them is in qsa_dense_tc.cuh.
//
//   o = sum_t softmax_t(c q . k_t) v_t   over  max(0, p - window + 1) <= t <= p,
//   lse = ln sum_t exp(c q . k_t)
//
// One pass over K and V with the running sum of a softmax (FP32, exp2 domain).
// All n_q x group query rows that share a KV head are worked on together, so K
// and V are read once: 4 D flops a row and position against 4 D (BF16) or 2 D
// (E4M3) bytes, for up to 32 rows a tenth or less of the tensor cores' rate at
// HBM's. HBM is the bound, and so the work is split by bytes: a unit is one
// (request, KV head, block of rows), and the units' tiles of 128 positions form
// one stream that is cut into equal contiguous shares, one per persistent CTA,
// so that no SM waits for a long request. The lengths are on the device; every
// CTA works the stream out from q_pos by itself. A unit that ends up in several
// CTAs leaves (reference, sum, acc) pieces in the workspace, which a second
// kernel, chained with programmatic dependent launch, joins in the order of
// the positions: no atomics, the same bits on every call. (One CTA joining the
// pieces of its unit was not tried: the 76 pieces of a unit of 32 rows are 1.2
// MB, 10 us for one SM, against 3 for the second kernel.)
#pragma once

#include <cuda.h>

#include <algorithm>

#include "qsa_kv_internal.cuh"

namespace qsa {

constexpr float kLog2e = 1.4426950408889634f;
constexpr float kLn2 = 0.6931471805599453f;
constexpr float kNegInf = -__builtin_huge_valf();
constexpr unsigned kFull = 0xffffffffu;
constexpr int kMaxSmem = 232448;  // 227 KB a CTA
constexpr long long kWaitCycles = 1LL << 31;  // bound of every wait: about one second

// What the host knows of the two kernels that share the GPU when a prefix is read
// once (shared_plan): CTAs of a part of the prefix, its tiles, the fewest and
// most parts, and the parts if the kernels run one after the other; what a tile
// and a unit of the own positions take a CTA, a tile HBM, a tile of the prefix a
// CTA, and a CTA's beginning and end in either kernel (ns).
struct SharedCost {
  int units, tiles, least, most, parts;
  unsigned own_ns, unit_ns, own_hbm_ns, part_ns, own_begin_ns, part_begin_ns;
};

struct DenseArgs {
  const __nv_bfloat16* q;
  const float* k_scale;
  const float* v_scale;
  const int32_t* page_table;
  const int32_t* q_pos;
  __nv_bfloat16* out;
  float* lse;
  long long* unit_desc;  // where each unit's pieces are (see unit_* below); null: the stream has no pieces
  float* parts;          // [grid][2] pieces: m[rows], l[rows], acc[rows][D]
  int32_t* err;
  int batch, n_q, n_q_heads, n_kv_heads, group, row_blocks;
  int page_size, page_shift, max_pages, num_pages, window, grid;
  float sm_scale;
  float one;  // 1
  static constexpr bool kShared = false;
};
// With a prefix that all requests share. (Kernels of their own: what the prefix
// adds made the others 1 to 6 % slower, one request of 50,004 tokens 18.4 us ->
// 19.5.)
struct SharedArgs : DenseArgs {
  const int32_t* prefix_table;  // the pages of positions below prefix_len
  float* whole;                 // [unit] the pieces of units that are one CTA's
  int prefix_len;               // whole pages
  int shared_len;  // prefix_len, or 0: every request is worked on by itself, its prefix too
  SharedCost cost;
  static constexpr bool kShared = true;
};

// Unit descriptors: written whole, without positions, or the pieces of CTAs
// first .. last (the first CTA's in its slot `slot`, the others' in slot 0).
constexpr long long kUnitWhole = -1, kUnitEmpty = -2;
__device__ __forceinline__ long long unit_pieces(int first, int last, int slot) {
  return (long long)first | ((long long)last << 24) | ((long long)slot << 48);
}

// ---------------------------------------------------------------------------
// instructions
// ---------------------------------------------------------------------------
__device__ __forceinline__ uint32_t smem_u32(const void* p) { return (uint32_t)__cvta_generic_to_shared(p); }
__device__ __forceinline__ void mbar_init(uint32_t bar, uint32_t count) {
  asm volatile("mbarrier.init.shared::cta.b64 [%0], %1;" ::"r"(bar), "r"(count) : "memory");
}
__device__ __forceinline__ void mbar_expect_tx(uint32_t bar, uint32_t bytes) {
  asm volatile("mbarrier.arrive.expect_tx.shared::cta.b64 _, [%0], %1;" ::"r"(bar), "r"(bytes) : "memory");
}
__device__ __forceinline__ void mbar_arrive(uint32_t bar) {
  asm volatile("mbarrier.arrive.shared::cta.b64 _, [%0];" ::"r"(bar) : "memory");
}
__device__ __forceinline__ bool mbar_try_wait(uint32_t bar, uint32_t parity) {
  uint32_t ok;
  asm volatile(
      "{\n\t.reg .pred p;\n\tmbarrier.try_wait.parity.shared::cta.b64 p, [%1], %2;\n\tselp.u32 %0, 1, 0, p;\n\t}"
      : "=r"(ok)
      : "r"(bar), "r"(parity)
      : "memory");
  return ok != 0;
}
// Bounded wait for a phase of a barrier. The first wait that runs out records
// the timeout and sets the CTA's abort flag; the others then give up too.
__device__ __forceinline__ bool mbar_wait(uint64_t* bar, uint32_t parity, volatile int* abort, int32_t* err) {
  const uint32_t b = smem_u32(bar);
  if (mbar_try_wait(b, parity)) return true;
  const long long start = clock64();
  while (!mbar_try_wait(b, parity)) {
    if (*abort) return false;
    if (clock64() - start > kWaitCycles) {
      *abort = 1;
      record_error(err, kErrTimeout, 0, 0, (int)threadIdx.x);
      return false;
    }
  }
  return true;
}
__device__ __forceinline__ void tma_load_4d(uint32_t dst, const CUtensorMap* map, int x, int y, int z, int w,
                                            uint32_t bar) {
  asm volatile(
      "cp.async.bulk.tensor.4d.shared::cluster.global.mbarrier::complete_tx::bytes [%0], [%1, {%2, %3, %4, %5}], "
      "[%6];" ::"r"(dst),
      "l"(reinterpret_cast<uint64_t>(map)), "r"(x), "r"(y), "r"(z), "r"(w), "r"(bar)
      : "memory");
}
// 2^x on the special-function unit (relative error about 2^-22, 2^-inf = 0)
__device__ __forceinline__ float exp2_sfu(float x) {
  float y;
  asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
  return y;
}
__device__ __forceinline__ float pow2(int s) { return __uint_as_float((uint32_t)(127 + s) << 23); }

// ---------------------------------------------------------------------------
// the stream of tiles
// ---------------------------------------------------------------------------
// Positions lo .. hi - 1 that any query of request r sees (hi = 0: none).
struct Range {
  int lo, hi;
  __device__ __forceinline__ int tiles(int tile) const { return hi > 0 ? (hi - 1) / tile + 1 - lo / tile : 0; }
};
__device__ __forceinline__ int capacity(const DenseArgs& a) { return a.max_pages * a.page_size; }
__device__ __forceinline__ bool valid_pos(const DenseArgs& a, int p) { return p >= 0 && p < capacity(a); }
__device__ __forceinline__ int low_of(const DenseArgs& a, int p) {
  return a.window > 0 && p >= a.window ? p - a.window + 1 : 0;
}
// Whether every query of a request at positions p sees the whole prefix. If so,
// the prefix is left to the kernel that takes it for all requests
// (qsa_prefix.cuh), and the request's unit is what lies behind it; else the
// request is worked on by itself, from position 0. (No window in either case.)
__device__ __forceinline__ bool sees_prefix(const SharedArgs& a, const int (&p)[kMaxNq]) {
  bool all = true;
#pragma unroll
  for (int j = 0; j < kMaxNq; ++j) all &= !valid_pos(a, p[j]) || p[j] >= a.shared_len - 1;
  return all;
}
template <class A>
__device__ __forceinline__ Range range_of(const A& a, int r) {
  int p[kMaxNq];
#pragma unroll
  for (int j = 0; j < kMaxNq; ++j) p[j] = j < a.n_q ? a.q_pos[(size_t)r * a.n_q + j] : -1;
  Range g{0x7fffffff, 0};
#pragma unroll
  for (int j = 0; j < kMaxNq; ++j) {
    if (!valid_pos(a, p[j])) continue;
    g.lo = min(g.lo, low_of(a, p[j]));
    g.hi = max(g.hi, p[j] + 1);
  }
  if constexpr (A::kShared) {
    if (a.shared_len > 0 && sees_prefix(a, p)) g.lo = a.shared_len;
  }
  return g.hi > g.lo ? g : Range{0, 0};
}

// The first position that a query at p sees, in a unit whose positions are g.
template <class A>
__device__ __forceinline__ int first_seen(const A& a, const Range& g, int p) {
  if constexpr (A::kShared) {
    if (a.shared_len > 0) return g.lo;
  }
  return low_of(a, p);
}

// With more requests than this the main kernel writes unit descriptors; with
// fewer the joining kernel works them out itself while it waits.
constexpr int kJoinScan = 256;

// quotient of non-negative numbers; most streams fit the 32-bit division
__device__ __forceinline__ long long quot(long long x, long long y) {
  return ((x | y) >> 32) == 0 ? (long long)((uint32_t)x / (uint32_t)y) : x / y;
}

// The stream, in slots: a unit of T > 0 tiles takes `seg` + T slots. The first
// `seg` hold no tile; they stand for what beginning a unit costs its CTA (query
// rows, first maximum, the end of the unit before), so that equal shares of
// slots are about equal work. Without them, one request of 50,000 tokens (2
// units on 152 SMs) waited 5 of 18 us for the one CTA that had the end of one
// unit and the beginning of the other (measured from 0 to 5 tiles: 3 is best or
// within 2 % of it at every size). Where there is no more than a tile a CTA, no
// CTA begins two units, and seg is 0. The slots are cut into `ctas` shares, the
// first `rem` of them one slot longer than `q`.
constexpr int kSegCost = 3;

// Tiles (bits 0-39) and units that have any (40-63) of some requests, for one
// unit of each.
__device__ __forceinline__ long long load_of(int tiles) { return tiles > 0 ? (1LL << 40) + tiles : 0; }

// How the GPU is divided when a prefix is read once: `own` CTAs for the requests'
// own positions, and the prefix in `parts` parts, a CTA each a unit. The first
// kernel is bound by HBM and the second by the tensor cores, so the two run side
// by side on SMs of their own where that ends earlier than one after the other,
// each on all. The host does not know the lengths; every CTA of either kernel
// comes to the same division from q_pos. (A whole warp; tiles and units: of the
// own positions of all requests. More than kJoinScan requests: one after the
// other, which takes no pass over q_pos and leaves the first kernel all SMs. Each
// way, 1 query over 50,048 shared and 1 to 200 own tokens: 512 requests, BF16 209
// us one after the other and 225 side by side, E4M3 251 and 260; 1,024, 381 and
// 413, 461 and 490; 257, 120 and 124, 141 and 135.)
struct SharedPlan {
  int own, parts;
};
__device__ __forceinline__ SharedPlan shared_plan(const SharedArgs& a, long long tiles, long long units) {
  const SharedCost& c = a.cost;
  if (a.batch > kJoinScan) return SharedPlan{a.grid, c.parts};
  const unsigned own = (unsigned)min(tiles, 1LL << 18), lane = threadIdx.x & 31;  // (products below 2^32)
  const unsigned work = own * c.own_ns + (unsigned)min(units, 1LL << 18) * c.unit_ns;
  auto own_time = [&](unsigned ctas) { return own == 0 ? 0u : c.own_begin_ns + max(work / ctas, own * c.own_hbm_ns); };
  auto part_time = [&](unsigned parts) { return c.part_begin_ns + (c.tiles + parts - 1) / parts * c.part_ns; };
  // (time << 8 | parts), or parts 255: one after the other
  const unsigned long long waves = ((unsigned long long)c.units * c.parts + a.grid - 1) / a.grid;
  unsigned long long best = (own_time(a.grid) + waves * part_time(c.parts)) << 8 | 255u;
  for (unsigned p = c.least + lane; p <= (unsigned)c.most && p * c.units < (unsigned)a.grid; p += 32)
    best = min(best, (unsigned long long)max(own_time(a.grid - p * c.units), part_time(p)) << 8 | p);
#pragma unroll
  for (int o = 16; o > 0; o >>= 1) best = min(best, __shfl_xor_sync(kFull, best, o));
  const int parts = (int)(best & 255u);
  return parts == 255 ? SharedPlan{a.grid, c.parts} : SharedPlan{a.grid - parts * c.units, parts};
}

struct Split {
  long long q;
  int ctas, rem, seg;
  __device__ __forceinline__ long long slots(long long load) const {
    return (load & ((1LL << 40) - 1)) + (load >> 40) * seg;
  }
  template <class A>
  __device__ __forceinline__ void init(const A& a, long long load) {
    const int units = a.n_kv_heads * a.row_blocks;
    const long long tiles = (load & ((1LL << 40) - 1)) * units;
    int grid = a.grid;
    if constexpr (A::kShared) {
      if (a.shared_len > 0) grid = shared_plan(a, tiles, (load >> 40) * units).own;
    }
    seg = tiles > grid ? kSegCost : 0;
    const long long all = slots(load) * units;
    // shares of kSegCost + 1 slots, or one less where that does not divide: such
    // a one may hold no tile (Walk::cut)
    static_assert(((kSegCost + 1) & kSegCost) == 0, "a division by a power of two");
    const long long most = seg ? (all + kSegCost) / (kSegCost + 1) : all;
    ctas = (int)min((long long)grid, most);
    q = ctas > 0 ? quot(all, ctas) : 0;
    rem = (int)(all - q * ctas);
  }
  __device__ __forceinline__ long long begin(int c) const { return c * q + min(c, rem); }
  __device__ __forceinline__ int of_slot(long long w) const {
    const long long wide = rem * (q + 1);
    return (int)(w < wide ? quot(w, q + 1) : rem + quot(w - wide, q));
  }
  // the CTAs with tiles of a unit of `tiles` tiles whose slots begin at `unit`
  __device__ __forceinline__ int first_cta(long long unit) const { return of_slot(unit + seg); }
  __device__ __forceinline__ int last_cta(long long unit, int tiles) const { return of_slot(unit + seg + tiles - 1); }
  // where the first of them has the unit's piece: in its slot 0 if the unit is
  // its first, else in its slot 1 (the unit is then its last)
  __device__ __forceinline__ int piece_slot(long long unit, int cta) const { return begin(cta) < unit ? 1 : 0; }
};

// What find_start leaves in shared memory: the split and the CTA's share of the
// stream, slots w0 .. w1 - 1.
struct Share {
  Split split;
  long long w0, w1, first;
  int first_r;
};

// A CTA's way through its share: segments, each the tiles t .. t + n - 1 of
// unit x = 0 .. n_kv_heads * row_blocks - 1 of request r (`tiles` in all, its
// slots beginning at `unit`).
template <int TILE>
struct Walk {
  long long unit;
  int r, x, t, n, tiles;
  Range g;
  __device__ __forceinline__ int start(const Share& sh) const {  // the share's first tile of this unit
    const long long first = unit + sh.split.seg, w0 = sh.w0;
    return w0 > first ? (int)(w0 - first) : 0;
  }
  __device__ __forceinline__ bool cut(const Share& sh) {  // the share's tiles of this unit
    t = start(sh);
    n = (int)min((long long)tiles, sh.w1 - (unit + sh.split.seg)) - t;
    return n > 0;
  }
  // (A whole warp. The next request that has positions is looked for 32 at a
  // time, a lane each: one after the other, 262,144 empty ones between two took
  // 86 ms, and at 2^22 the roles that meanwhile wait for one another came near
  // the limit of their waits.)
  template <class A>
  __device__ __forceinline__ bool next(const A& a, const Share& sh) {
    unit += sh.split.seg + tiles;
    if (unit + sh.split.seg >= sh.w1) return false;
    if (++x == a.n_kv_heads * a.row_blocks) {
      x = 0;
      uint32_t found;
      Range mine;
      for (++r;; r += 32) {
        if (r >= a.batch) return false;
        const int own = r + (int)(threadIdx.x & 31);
        mine = own < a.batch ? range_of(a, own) : Range{0, 0};
        found = __ballot_sync(kFull, mine.hi > 0);
        if (found) break;
      }
      const int src = __ffs(found) - 1;
      r += src;
      g.lo = __shfl_sync(kFull, mine.lo, src);
      g.hi = __shfl_sync(kFull, mine.hi, src);
      tiles = g.tiles(TILE);
    }
    return cut(sh);
  }
};

// Positions that are none are reported once, by block 0.
__device__ __forceinline__ void report_positions(const DenseArgs& a, int r) {
  for (int j = 0; j < a.n_q; ++j) {
    const int p = a.q_pos[(size_t)r * a.n_q + j];
    if (p != -1 && !valid_pos(a, p)) record_error(a.err, kErrQueryPos, r, j, p);
  }
}

// Every thread of the block: works the stream out from q_pos and finds the
// CTA's share and its first segment. False: nothing to do. It ends with the
// block's only barrier (up to 32 requests: every warp works it all out by
// itself, a lane a request), or has several (each thread sums the tiles of a
// contiguous run of requests, one block scan; units without a tile are marked).
template <int TILE, int THREADS, class A>
__device__ __forceinline__ bool find_start(const A& a, long long (&scan)[THREADS / 32], Share& sh,
                                           Walk<TILE>& at) {
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
  const int units = a.n_kv_heads * a.row_blocks;  // of a request
  if (a.batch <= 32) {
    Range g{0, 0};
    if (lane < a.batch) g = range_of(a, lane);
    const int tiles = g.tiles(TILE);
    const long long mine = load_of(tiles);
    long long inc = mine;
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
      const long long v = __shfl_up_sync(kFull, inc, o);
      if (lane >= o) inc += v;
    }
    Split sp;
    sp.init(a, __shfl_sync(kFull, inc, 31));
    const bool work = (int)blockIdx.x < sp.ctas;
    const long long w0 = sp.begin(blockIdx.x), unit = sp.slots(inc - mine) * units;
    const uint32_t in = __ballot_sync(kFull, unit <= w0 && w0 < unit + sp.slots(mine) * units);
    const int src = in ? __ffs(in) - 1 : 0;  // the request that w0 is in
    at.r = src;
    at.g.lo = __shfl_sync(kFull, g.lo, src);
    at.g.hi = __shfl_sync(kFull, g.hi, src);
    at.tiles = __shfl_sync(kFull, tiles, src);
    at.unit = __shfl_sync(kFull, unit, src);
    if (tid == 0) {
      sh.split = sp;
      sh.w0 = w0;
      sh.w1 = sp.begin(blockIdx.x + 1);
    }
    if (blockIdx.x == 0 && warp == 0 && lane < a.batch) report_positions(a, lane);
    if (work) {
      at.x = (int)quot(w0 - at.unit, sp.seg + at.tiles);
      at.unit += (long long)at.x * (sp.seg + at.tiles);
    }
    __syncthreads();
    return work && at.cut(sh);
  }
  const int per = (a.batch + THREADS - 1) / THREADS;
  const int r0 = min(tid * per, a.batch), r1 = min(r0 + per, a.batch);
  long long mine = 0;
  for (int r = r0; r < r1; ++r) mine += load_of(range_of(a, r).tiles(TILE));
  long long inc = mine;
#pragma unroll
  for (int o = 1; o < 32; o <<= 1) {
    const long long v = __shfl_up_sync(kFull, inc, o);
    if (lane >= o) inc += v;
  }
  if (lane == 31) scan[warp] = inc;
  __syncthreads();
  long long before = inc - mine, total = 0;
#pragma unroll
  for (int w = 0; w < THREADS / 32; ++w) {
    const long long v = scan[w];
    if (w < warp) before += v;
    total += v;
  }
  Split sp;
  sp.init(a, total);
  if (blockIdx.x == 0) {
    for (int r = r0; r < r1; ++r) {
      report_positions(a, r);
      if (a.unit_desc && a.batch > kJoinScan && range_of(a, r).tiles(TILE) == 0)
        for (int x = 0; x < units; ++x) a.unit_desc[(long long)r * units + x] = kUnitEmpty;
    }
  }
  if ((int)blockIdx.x >= sp.ctas) return false;
  const long long w0 = sp.begin(blockIdx.x);
  // one thread: w0 is in one of its requests
  if (sp.slots(before) * units <= w0 && w0 < sp.slots(before + mine) * units) {
    sh.split = sp;
    sh.w0 = w0;
    sh.w1 = sp.begin(blockIdx.x + 1);
    long long b = before;
    for (int r = r0; r < r1; ++r) {
      const long long t = load_of(range_of(a, r).tiles(TILE));
      if (w0 < sp.slots(b + t) * units) {
        sh.first_r = r;
        sh.first = sp.slots(b) * units;
        break;
      }
      b += t;
    }
  }
  __syncthreads();
  at.r = sh.first_r;
  at.g = range_of(a, at.r);
  at.tiles = at.g.tiles(TILE);
  at.unit = sh.first;
  at.x = (int)quot(w0 - at.unit, sp.seg + at.tiles);
  at.unit += (long long)at.x * (sp.seg + at.tiles);
  return at.cut(sh);
}

// The pages of a segment's boxes (box = the positions that one TMA copy takes,
// all in one page), looked up by a whole warp 32 boxes ahead. A box that no
// query sees has none (and is not looked up: its entry may mean nothing).
// Everything is a power of two: the copy warp feeds the SM alone, and integer
// divisions here were most of what a tile cost it.
template <int TILE>
struct PageFeed {
  int box_shift, boxes;  // log2 of a box's positions; boxes of a tile
  int my_box;            // this lane's box of a tile (lane % boxes)
  int cur, nxt, first_box, n_boxes;
  __device__ __forceinline__ explicit PageFeed(const DenseArgs& a) {
    constexpr int kTileShift = TILE == 128 ? 7 : 6;
    static_assert(TILE == 1 << kTileShift, "tile");
    box_shift = min(kTileShift, a.page_shift);
    boxes = TILE >> box_shift;
    my_box = (int)(threadIdx.x & 31) & (boxes - 1);
  }
  template <class A>
  __device__ __forceinline__ int page_of(const A& a, const Walk<TILE>& at, int i) const {
    const unsigned p = (unsigned)(first_box + i) << box_shift;  // (a box that is seen starts below 2^31)
    if (i >= n_boxes || p >= (unsigned)at.g.hi || p + (1u << box_shift) <= (unsigned)at.g.lo) return -1;
    const int32_t* table = a.page_table + (size_t)at.r * a.max_pages;
    int r = at.r;
    if constexpr (A::kShared) {
      if (p < (unsigned)a.prefix_len) {
        table = a.prefix_table;
        r = -1;
      }
    }
    const int page = table[p >> a.page_shift];
    if ((unsigned)page < (unsigned)a.num_pages) return page;
    record_error(a.err, kErrPage, r, 0, page);
    return -1;
  }
  template <class A>
  __device__ __forceinline__ void start(const A& a, const Walk<TILE>& at) {
    first_box = (at.g.lo / TILE + at.t) * boxes;
    n_boxes = at.n * boxes;
    cur = page_of(a, at, threadIdx.x & 31);
    nxt = page_of(a, at, 32 + (threadIdx.x & 31));
  }
  // page of this lane's box of the segment's tile k
  template <class A>
  __device__ __forceinline__ int of_tile(const A& a, const Walk<TILE>& at, int k) {
    const int b0 = k * boxes;
    if (b0 > 0 && (b0 & 31) == 0) {
      cur = nxt;
      nxt = page_of(a, at, b0 + 32 + (int)(threadIdx.x & 31));
    }
    return __shfl_sync(kFull, cur, (b0 & 31) + my_box);
  }
  // its first position's slot in the page
  __device__ __forceinline__ int slot_of(const DenseArgs& a, int k) const {
    return (int)(((unsigned)(first_box + k * boxes + my_box) << box_shift) & (unsigned)(a.page_size - 1));
  }
  // bit i: positions 16 i .. 16 i + 15 of the tile have no page (this lane's box: `page`)
  __device__ __forceinline__ uint32_t bad_groups(int page) const {
    const uint32_t bad_boxes = __ballot_sync(kFull, page < 0);  // bit i (i < boxes): box i
    const int group = (int)(threadIdx.x & 31) & (TILE / 16 - 1);
    return __ballot_sync(kFull, (bad_boxes >> ((group * 16) >> box_shift)) & 1u) & ((1u << (TILE / 16)) - 1u);
  }
};

// ---------------------------------------------------------------------------
// joining split units
// ---------------------------------------------------------------------------
// Joins the pieces of split units and writes the rows of requests without
// positions. WARPS warps a row, the pieces dealt to them (WARPS 1: a block of
// kJoinRows rows), every warp's loads (kBatch pieces) issued before their
// maxima are looked at. Which pieces a row has follows from q_pos alone. With
// up to kJoinScan requests that is worked out before the wait for the main
// kernel (q_pos is older than that kernel's trigger, which its CTAs give after
// their own wait), so that behind the wait there is one round of loads and the
// store.
constexpr int kJoinRows = 8;

template <int D, int ROWS, bool FP8, int TILE, int WARPS>
__global__ void __launch_bounds__(WARPS > 1 ? 32 * WARPS : 32 * kJoinRows) dense_join_kernel(const DenseArgs a) {
  constexpr int E = D / 32, kPiece = ROWS * (D + 2), kBatch = 10;
  __shared__ float s_m[WARPS], s_l[WARPS], s_acc[WARPS > 1 ? WARPS : 1][WARPS > 1 ? D : 1];
  __shared__ long long s_sum[2][WARPS];
  const int lane = threadIdx.x & 31, warp = WARPS > 1 ? threadIdx.x >> 5 : 0;
  const int orow = WARPS > 1 ? blockIdx.x : blockIdx.x * kJoinRows + (threadIdx.x >> 5);
  if (WARPS == 1 && orow >= a.batch * a.n_q * a.n_q_heads) return;
  const int rj = orow / a.n_q_heads, h = orow - rj * a.n_q_heads, r = rj / a.n_q, j = rj - r * a.n_q;
  const int g = h / a.group, i = j * a.group + (h - g * a.group);
  const int rb = i / ROWS, row = i - rb * ROWS, units = a.n_kv_heads * a.row_blocks;
  const float vscale = FP8 ? a.v_scale[g] : 1.f;
  long long desc;
  if (a.batch <= kJoinScan) {
    long long all = 0, below = 0;
    for (int q = warp * 32 + lane; q < a.batch; q += 32 * WARPS) {
      const long long t = load_of(range_of(a, q).tiles(TILE));
      all += t;
      below += q < r ? t : 0;
    }
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) {
      all += __shfl_xor_sync(kFull, all, o);
      below += __shfl_xor_sync(kFull, below, o);
    }
    if constexpr (WARPS > 1) {
      if (lane == 0) {
        s_sum[0][warp] = all;
        s_sum[1][warp] = below;
      }
      __syncthreads();
      all = below = 0;
#pragma unroll
      for (int w = 0; w < WARPS; ++w) {
        all += s_sum[0][w];
        below += s_sum[1][w];
      }
    }
    const int tiles = range_of(a, r).tiles(TILE);
    desc = kUnitEmpty;
    if (tiles > 0) {
      Split sp;
      sp.init(a, all);
      const long long unit = sp.slots(below) * units + (long long)(g * a.row_blocks + rb) * (sp.seg + tiles);
      const int c0 = sp.first_cta(unit), c1 = sp.last_cta(unit, tiles);
      desc = c0 == c1 ? kUnitWhole : unit_pieces(c0, c1, sp.piece_slot(unit, c0));
    }
    // (also where there is nothing to join: this kernel ends behind the main one)
    pdl_wait();
    if (desc == kUnitWhole) return;  // its CTA writes the row
  } else {
    pdl_wait();
    desc = a.unit_desc[(long long)r * units + g * a.row_blocks + rb];
    if (desc == kUnitWhole) return;
  }
  float m = kNegInf, l = 0.f, acc[E];
#pragma unroll
  for (int e = 0; e < E; ++e) acc[e] = 0.f;
  if (desc != kUnitEmpty) {
    const int c0 = (int)(desc & 0xffffff), c1 = (int)((desc >> 24) & 0xffffff), slot = (int)(desc >> 48);
    for (int c = c0 + warp; c <= c1; c += WARPS * kBatch) {
      float pm[kBatch], pl[kBatch], pa[kBatch][E];
#pragma unroll
      for (int b = 0; b < kBatch; ++b) {
        const int cc = c + b * WARPS;
        pm[b] = kNegInf;
        pl[b] = 0.f;
#pragma unroll
        for (int e = 0; e < E; ++e) pa[b][e] = 0.f;
        if (cc <= c1) {
          const float* p = a.parts + ((size_t)cc * 2 + (cc == c0 ? slot : 0)) * kPiece;
          pm[b] = p[row];
          pl[b] = p[ROWS + row];
#pragma unroll
          for (int e = 0; e < E; ++e) pa[b][e] = p[2 * ROWS + row * D + e * 32 + lane];
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
        const float x = exp2_sfu(pm[b] - mu);
        l = fmaf(pl[b], x, l);
#pragma unroll
        for (int e = 0; e < E; ++e) acc[e] = fmaf(pa[b][e], x, acc[e]);
      }
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

// ---------------------------------------------------------------------------
// host
// ---------------------------------------------------------------------------
using EncodeTiled = CUresult (*)(CUtensorMap*, CUtensorMapDataType, cuuint32_t, void*, const cuuint64_t*,
                                 const cuuint64_t*, const cuuint32_t*, const cuuint32_t*, CUtensorMapInterleave,
                                 CUtensorMapSwizzle, CUtensorMapL2promotion, CUtensorMapFloatOOBfill);
EncodeTiled encode_tiled();  // cuTensorMapEncodeTiled through the runtime, or null

// the cache [num_pages][n_kv_heads][page_size][head_dim] with boxes of one
// page's (or `tile`) positions of one head, `line` (64 or 128) bytes of a row
// wide; short_box: of half as many positions (qsa_test_paged_attn_timeout)
inline bool make_cache_map(CUtensorMap* map, const qsa_dims& d, const void* cache, int tile, int line,
                           bool short_box) {
  const EncodeTiled enc = encode_tiled();
  if (!enc) return false;
  const int eb = d.kv_dtype == QSA_KV_FP8_E4M3 ? 1 : 2;
  const cuuint64_t dims[4] = {(cuuint64_t)d.head_dim, (cuuint64_t)d.page_size, (cuuint64_t)d.n_kv_heads,
                              (cuuint64_t)d.num_pages};
  const cuuint64_t row = (cuuint64_t)d.head_dim * eb;
  const cuuint64_t strides[3] = {row, row * d.page_size, row * d.page_size * d.n_kv_heads};
  const int rows = std::min(tile, d.page_size) / (short_box ? 2 : 1);
  const cuuint32_t box[4] = {(cuuint32_t)(line / eb), (cuuint32_t)rows, 1, 1};
  const cuuint32_t estr[4] = {1, 1, 1, 1};
  return enc(map, eb == 1 ? CU_TENSOR_MAP_DATA_TYPE_UINT8 : CU_TENSOR_MAP_DATA_TYPE_BFLOAT16, 4,
             const_cast<void*>(cache), dims, strides, box, estr, CU_TENSOR_MAP_INTERLEAVE_NONE,
             line == 128 ? CU_TENSOR_MAP_SWIZZLE_128B : CU_TENSOR_MAP_SWIZZLE_64B, CU_TENSOR_MAP_L2_PROMOTION_L2_256B,
             CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) == CUDA_SUCCESS;
}

// The joining kernel: units that are cut into many pieces (few units on many
// SMs) get 16 warps a row, whose one round of loads takes up to 160 pieces;
// many rows one each (4,096 rows of two or three pieces: 4 warps a row made
// the whole call 10 us slower); else 4. The odd long request among short ones
// takes more rounds.
template <int D, int ROWS, bool FP8, int TILE>
cudaError_t launch_join(const DenseArgs& a, cudaStream_t s) {
  const unsigned rows = (unsigned)(a.batch * a.n_q * a.n_q_heads);
  const long long units = (long long)a.batch * a.n_kv_heads * a.row_blocks;
  if (a.grid > 24 * units)
    return launch_k(dense_join_kernel<D, ROWS, FP8, TILE, 16>, dim3(rows), dim3(512), 0, s, true, a);
  if (rows < 8u * a.grid)
    return launch_k(dense_join_kernel<D, ROWS, FP8, TILE, 4>, dim3(rows), dim3(128), 0, s, true, a);
  return launch_k(dense_join_kernel<D, ROWS, FP8, TILE, 1>, dim3((rows + kJoinRows - 1) / kJoinRows),
                  dim3(32 * kJoinRows), 0, s, true, a);
}

// the kernels by head dim (qsa_dense_64.cu, _128.cu, _256.cu; with a shared
// prefix qsa_shared_64.cu, _128.cu, _256.cu); rows: of a unit; short_k: K's
// copies bring half of what the kernel waits for
cudaError_t launch_dense_64(int rows, const qsa_dims& d, const DenseArgs& a, const void* k_cache, const void* v_cache,
                            bool short_k, cudaStream_t s);
cudaError_t launch_dense_128(int rows, const qsa_dims& d, const DenseArgs& a, const void* k_cache, const void* v_cache,
                             bool short_k, cudaStream_t s);
cudaError_t launch_dense_256(int rows, const qsa_dims& d, const DenseArgs& a, const void* k_cache, const void* v_cache,
                             bool short_k, cudaStream_t s);
cudaError_t launch_dense_64(int rows, const qsa_dims& d, const SharedArgs& a, const void* k_cache, const void* v_cache,
                            bool short_k, cudaStream_t s);
cudaError_t launch_dense_128(int rows, const qsa_dims& d, const SharedArgs& a, const void* k_cache, const void* v_cache,
                             bool short_k, cudaStream_t s);
cudaError_t launch_dense_256(int rows, const qsa_dims& d, const SharedArgs& a, const void* k_cache, const void* v_cache,
                             bool short_k, cudaStream_t s);

}  // namespace qsa
