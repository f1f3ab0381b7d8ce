// Rotary positions, writing the paged cache and reading it back.
//
// Rotation. Token j at position t turns the pair (a, b) by t w_i:
//   y_a = A (x_a cos - x_b sin),  y_b = A (x_b cos + x_a sin).
// The angle is taken in turns as a 64-bit binary fraction: t (an integer)
// times the pair's frequency (times 2^64) in wrapping integer arithmetic drops
// whole turns exactly, so positions of millions cost no accuracy and no
// 64-bit floating point; the remainder, a signed fraction of a turn, goes to
// sincospi in FP32.
//
// Cache write. BF16: the rotated key rounded once. E4M3: x / scale[head] in
// FP32, then to nearest even with clamping. The rotated key is not rounded to
// BF16 in between.
//
// All of it is streaming: each input is read once and each output written
// once, with nothing to reuse but the R / 2 (cos, sin) of a token, which all
// its heads share. Three kernels:
//
//  * wide_kernel, where rows can be read 16 bytes at a time and the rotated
//    part is a multiple of 16 components: a warp takes a token. It works out
//    the token's (cos, sin) once (each lane one to four of them), and a lane
//    keeps the 8 that its components need in registers for all heads: an item
//    is 2 x 8 components that hold 8 whole pairs, D / 16 of them a head, and a
//    pass of the warp covers 32 / (D / 16) heads. Loads of five passes are in
//    flight at a time, the first ones while the angles are worked out. No
//    block barrier: an earlier layout (a block per four tokens, one item a
//    thread, the table of angles shared through a barrier) was bound by the
//    warps' waiting for one another, 76 us for 2 x 16,385 tokens of 16 + 2 + 2
//    heads of 128 into an E4M3 cache. This one takes 56 (46 at HBM's copy
//    rate), bound by issue and latency: with rotation and division on single
//    values, the division the compiler's, it took 62. Six blocks an SM, or four
//    passes deep, are slower there (61 to 62) and the same elsewhere.
//  * row_kernel, where rows can be read 16 bytes at a time but the halves of the
//    rotated part are not multiples of 8 components. A warp takes a token here
//    too: rows go through shared memory 16 bytes at a time, in which a lane
//    finds its pairs (lane, lane + 32, ...) of every head at any offset, without
//    bank conflicts, and keeps their (cos, sin) in registers. 8,192 tokens of 16
//    heads of 128, 90 components rotated: 15 us (10 at HBM's copy rate; the
//    pair kernel 35); appends of 16 + 2 + 2 heads 19 us into BF16 and 24 into
//    E4M3 (45 and 48). For multiples of 16 the wide kernel is the faster one: 19
//    for 24 into E4M3, 56 for 72 at 2 x 16,385 tokens, 42 for 45 in the rotation
//    of 32,768 alone. Chunks of two vectors a lane: with five, 32 tokens took
//    3.3 to 4.3 us in place of 2.6 to 3.5, and long inputs the same.
//  * pair_kernel for the rest: one pair a thread.
//
// All kernels here are launched with programmatic dependent launch and wait at
// their start for what is before them in the stream; none lets its own
// successor start early.
#include <algorithm>

#include "qsa_kv_internal.cuh"

namespace qsa {
namespace {

constexpr int kMaxHalf = 128;  // pairs of a head at most

struct TokenArgs {
  Rope rope;
  float sign;
  Strided q, q_out, k, v;
  int hq, hk;  // heads: hq of q, then hk of k, then hk of v
  int n_tok, head_dim;
  long long tokens;  // batch * n_tok
  const int32_t* pos;
  // cache write
  const int32_t* page_table;
  uint8_t* k_cache;
  uint8_t* v_cache;
  const float* k_scale;
  const float* v_scale;
  int32_t* err;
  int max_pages, num_pages, page_size, fp8;
};

// (cos, sin) of `pos` times a frequency in turns (times 2^64)
__device__ __forceinline__ float2 cos_sin(int pos, uint64_t turns) {
  const long long frac = (long long)((uint64_t)(long long)pos * turns);  // a signed fraction of a turn, times 2^64
  float s, c;
  sincospif((float)frac * 1.0842021724855044e-19f /* 2^-63: half turns */, &s, &c);
  return make_float2(c, s);
}

__device__ __forceinline__ void rotate(float& xa, float& xb, float2 cs) {
  const float a = xa, b = xb;
  xa = a * cs.x - b * cs.y;
  xb = b * cs.x + a * cs.y;
}

// The token's checks: its cache row for KV head 0 (-1: K and V are not
// written), and whether it is there, in order and within the page table.
__device__ __forceinline__ bool check_token(const TokenArgs& a, int tok, int r, int j, bool report, long long& row) {
  row = -1;
  const int p = a.pos[tok];
  if (a.hk == 0) return p >= 0;  // rotation only
  if (p == -1) return false;
  const int first = a.pos[(long long)r * a.n_tok];
  if (p < 0 || p >= a.max_pages * a.page_size) {
    if (report) record_error(a.err, kErrQueryPos, r, j, p);
    return false;
  }
  if (p != (long long)first + j) {
    if (report) record_error(a.err, kErrOrder, r, j, p);
    return false;
  }
  const int page = a.page_table[(long long)r * a.max_pages + p / a.page_size];
  if ((unsigned)page < (unsigned)a.num_pages)
    row = ((long long)page * a.hk * a.page_size + p % a.page_size) * a.head_dim;
  else if (report)
    record_error(a.err, kErrPage, r, j, page);
  return true;
}

// ---------------------------------------------------------------------------
// 16 bytes at a time
// ---------------------------------------------------------------------------
constexpr int kWideWarps = 4, kWideDeep = 5;

// An item's 16 components as 8 pairs (a[e], b[e]): with IL neighbours of a
// vector, else the same component of the two vectors.
template <bool IL>
__device__ __forceinline__ void unpack(const uint4& x0, const uint4& x1, float (&a)[8], float (&b)[8]) {
  const uint32_t w[8] = {x0.x, x0.y, x0.z, x0.w, x1.x, x1.y, x1.z, x1.w};
#pragma unroll
  for (int e = 0; e < 8; ++e) {
    if constexpr (IL) {
      a[e] = bf_lo(w[e]);
      b[e] = bf_hi(w[e]);
    } else {
      float(&f)[8] = e < 4 ? a : b;
      f[2 * e % 8] = bf_lo(w[e]);
      f[2 * e % 8 + 1] = bf_hi(w[e]);
    }
  }
}
// the two components that are in word e (two of BF16, half a one of codes)
template <bool IL>
__device__ __forceinline__ float2 of_word(const float (&a)[8], const float (&b)[8], int e) {
  if constexpr (IL) return make_float2(a[e], b[e]);
  const float(&f)[8] = e < 4 ? a : b;
  return make_float2(f[2 * e % 8], f[2 * e % 8 + 1]);
}
template <bool IL>
__device__ __forceinline__ uint4 pack(const float (&a)[8], const float (&b)[8], int e0) {
  uint32_t w[4];
#pragma unroll
  for (int e = 0; e < 4; ++e) {
    const float2 f = of_word<IL>(a, b, e0 + e);
    w[e] = pack_bf(f.x, f.y);
  }
  return make_uint4(w[0], w[1], w[2], w[3]);
}
template <bool IL>
__device__ __forceinline__ uint2 codes(const float (&a)[8], const float (&b)[8], int e0) {
  uint32_t c[4];
#pragma unroll
  for (int e = 0; e < 4; ++e) {
    const float2 f = of_word<IL>(a, b, e0 + e);
    c[e] = e4m3x2(f.x, f.y);
  }
  return make_uint2(c[0] | (c[1] << 16), c[2] | (c[3] << 16));
}
// |x| or |y|, whichever is less (NaN if one is), with the product's sign
__device__ __forceinline__ float min_signed(float x, float y) {
  float r;
  asm("min.NaN.xorsign.abs.f32 %0, %1, %2;" : "=f"(r) : "f"(x), "f"(y));
  return r;
}
// f[i] / scale. For a scale of usual size: a quotient by the scale's reciprocal
// and one step with its exact remainder (Markstein, "Computation of elementary
// functions on the IBM RISC System/6000 processor", 1990), on pairs. What the
// step adds is right to 2^-23 of itself, so the result is the division's, but
// where the quotient is within 2^-46 of the middle of two FP32 values. Values
// that are clamped to 448 anyway are cut at 512 scales first, so that nothing
// overflows. The scale's sign goes to the value, and remainder and reciprocal are
// negated: a zero then keeps its sign.
struct Divisor {
  float scale, size, nr, cut;
  bool usual;
  __device__ __forceinline__ explicit Divisor(float s) : scale(s), size(fabsf(s)) {
    usual = size >= 0x1p-60f && size <= 0x1p60f;
    nr = -1.f / size;
    cut = -512.f * s;
  }
  // lane `from`'s
  __device__ __forceinline__ Divisor(const Divisor& d, int from) {
    scale = __shfl_sync(0xffffffffu, d.scale, from);
    nr = __shfl_sync(0xffffffffu, d.nr, from);
    size = fabsf(scale);
    cut = -512.f * scale;
    usual = size >= 0x1p-60f && size <= 0x1p60f;
  }
  __device__ __forceinline__ float2 quick(float2 x) const {
    const float2 nx = make_float2(min_signed(x.x, cut), min_signed(x.y, cut)), s2 = make_float2(size, size);
    const float2 r2 = make_float2(nr, nr), q = mul2(nx, r2);
    return fma2(fma2(q, s2, nx), r2, q);
  }
  __device__ __forceinline__ void operator()(float (&f)[8]) const {
    if (usual) {
#pragma unroll
      for (int i = 0; i < 8; i += 2) {
        const float2 y = quick(make_float2(f[i], f[i + 1]));
        f[i] = y.x;
        f[i + 1] = y.y;
      }
    } else {
#pragma unroll 1
      for (int i = 0; i < 4; ++i) {  // (rotated through: an index that is not constant would put f in memory)
        const float x = f[0] / scale, y = f[1] / scale;
#pragma unroll
        for (int e = 0; e < 6; ++e) f[e] = f[e + 2];
        f[6] = x;
        f[7] = y;
      }
    }
  }
};

// grid (ceil(tokens / kWideWarps), parts of the passes); PER = head_dim / 16
template <int PER, bool IL, bool FP8>
__global__ void __launch_bounds__(32 * kWideWarps, 5) wide_kernel(const TokenArgs a) {
  constexpr int kHeads = 32 / PER, D = 16 * PER;  // heads of a pass
  __shared__ __align__(16) float s_cs[kWideWarps][2][kMaxHalf];  // cosines, sines
  pdl_wait();
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  const int tok = (int)blockIdx.x * kWideWarps + warp;  // (below 2^31)
  if (tok >= a.tokens) return;
  const int r = (int)((unsigned)tok / (unsigned)a.n_tok), j = tok - r * a.n_tok;
  const int i = lane % PER, sub = lane / PER;  // this lane's item of a head, its head within a pass
  const int half = a.rope.rot_dim >> 1;
  const bool in_rot = i < (a.rope.rot_dim >> 4);
  const int heads = a.hq + 2 * a.hk;
  const int passes = (heads + kHeads - 1) / kHeads, per_part = (passes + gridDim.y - 1) / gridDim.y;
  const int p0 = blockIdx.y * per_part, p1 = min(passes, p0 + per_part);
  const __nv_bfloat16* q = a.q.p + r * a.q.batch + j * a.q.token;
  const __nv_bfloat16* k = a.k.p + r * a.k.batch + j * a.k.token;
  const __nv_bfloat16* v = a.v.p + r * a.v.batch + j * a.v.token;
  // an item's two vectors: of a rotated part the two that hold whole pairs
  const int split = IL || !in_rot ? i * 16 : i * 8, other = IL || !in_rot ? 8 : half;
  uint4 x0[kWideDeep], x1[kWideDeep];
  auto load = [&](int p) {
#pragma unroll
    for (int u = 0; u < kWideDeep; ++u) {
      const int h = (p + u) * kHeads + sub;
      if (p + u < p1 && h < heads) {
        const __nv_bfloat16* src = h < a.hq             ? q + h * a.q.head + split
                                   : h < a.hq + a.hk ? k + (h - a.hq) * a.k.head + split
                                                     : v + (h - a.hq - a.hk) * a.v.head + i * 16;
        x0[u] = ld16(src);
        x1[u] = ld16(src + (h < a.hq + a.hk ? other : 8));
      }
    }
  };
  load(p0);
  long long row;
  const bool live = check_token(a, tok, r, j, lane == 0 && blockIdx.y == 0, row);
  float cosv[8], sinv[8];
  if (half > 0) {
    const int pos = a.pos[tok];
    for (int f = lane; f < half; f += 32) {
      const float2 c = cos_sin(pos, a.rope.turns[f]);
      s_cs[warp][0][f] = c.x * a.rope.amplitude;
      s_cs[warp][1][f] = c.y * a.rope.amplitude * a.sign;
    }
    __syncwarp();
    if (in_rot) {
#pragma unroll
      for (int e = 0; e < 8; e += 4) {
        const float4 c = *reinterpret_cast<const float4*>(&s_cs[warp][0][i * 8 + e]);
        const float4 s = *reinterpret_cast<const float4*>(&s_cs[warp][1][i * 8 + e]);
        cosv[e] = c.x, cosv[e + 1] = c.y, cosv[e + 2] = c.z, cosv[e + 3] = c.w;
        sinv[e] = s.x, sinv[e + 1] = s.y, sinv[e + 2] = s.z, sinv[e + 3] = s.w;
      }
    }
  }
  if (!live) return;
  __nv_bfloat16* qo = a.q_out.p + r * a.q_out.batch + j * a.q_out.token;
  for (int p = p0; p < p1; p += kWideDeep) {
    if (p > p0) load(p);
#pragma unroll
    for (int u = 0; u < kWideDeep; ++u) {
      const int h = (p + u) * kHeads + sub;
      if (p + u >= p1 || h >= heads) continue;
      const bool is_v = h >= a.hq + a.hk;
      float xa[8], xb[8];
      unpack<IL>(x0[u], x1[u], xa, xb);
      if (in_rot && !is_v) {
#pragma unroll
        for (int e = 0; e < 8; e += 2) {
          const float2 c = make_float2(cosv[e], cosv[e + 1]), s = make_float2(sinv[e], sinv[e + 1]);
          const float2 va = make_float2(xa[e], xa[e + 1]), vb = make_float2(xb[e], xb[e + 1]);
          const float2 ya = fma2(va, c, mul2(vb, make_float2(-s.x, -s.y))), yb = fma2(vb, c, mul2(va, s));
          xa[e] = ya.x, xa[e + 1] = ya.y;
          xb[e] = yb.x, xb[e + 1] = yb.y;
        }
      }
      if (h < a.hq) {
        __nv_bfloat16* dst = qo + h * a.q_out.head + split;
        *reinterpret_cast<uint4*>(dst) = pack<IL>(xa, xb, 0);
        *reinterpret_cast<uint4*>(dst + other) = pack<IL>(xa, xb, 4);
      } else if (row >= 0) {
        const int g = is_v ? h - a.hq - a.hk : h - a.hq;
        const int o0 = is_v ? i * 16 : split, o1 = o0 + (is_v ? 8 : other);
        const long long at = row + (long long)g * a.page_size * D;
        uint8_t* cache = is_v ? a.v_cache : a.k_cache;
        if constexpr (FP8) {
          const Divisor by(is_v ? a.v_scale[g] : a.k_scale[g]);
          by(xa);
          by(xb);
          *reinterpret_cast<uint2*>(cache + at + o0) = codes<IL>(xa, xb, 0);
          *reinterpret_cast<uint2*>(cache + at + o1) = codes<IL>(xa, xb, 4);
        } else {
          __nv_bfloat16* dst = reinterpret_cast<__nv_bfloat16*>(cache) + at;
          *reinterpret_cast<uint4*>(dst + o0) = pack<IL>(xa, xb, 0);
          *reinterpret_cast<uint4*>(dst + o1) = pack<IL>(xa, xb, 4);
        }
      }
    }
  }
}

// ---------------------------------------------------------------------------
// 16 bytes at a time, pairs from shared memory
// ---------------------------------------------------------------------------
constexpr int kRowWarps = 4, kRowDeep = 2;

// grid (ceil(tokens / kRowWarps), parts of the chunks)
template <int D, bool IL, bool FP8>
__global__ void __launch_bounds__(32 * kRowWarps) row_kernel(const TokenArgs a) {
  constexpr int kVecs = D / 8, kHeads = kRowDeep * 32 / kVecs, kPairs = D / 64;  // vectors of a head, heads of a chunk
  constexpr int kGroup = D == 64 ? 4 : D == 128 ? 2 : 1;  // heads at a time: four pairs a lane
  static_assert(kHeads % kGroup == 0, "groups do not cross chunks");
  __shared__ __align__(16) __nv_bfloat16 s_rows[kRowWarps][kHeads * D];
  __shared__ __align__(16) uint8_t s_codes[FP8 ? kRowWarps : 1][FP8 ? kHeads * D : 16];
  pdl_wait();
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  const int tok = (int)blockIdx.x * kRowWarps + warp;  // (below 2^31)
  if (tok >= a.tokens) return;
  const int r = (int)((unsigned)tok / (unsigned)a.n_tok), j = tok - r * a.n_tok;
  const int half = a.rope.rot_dim >> 1, heads = a.hq + 2 * a.hk;
  const int chunks = (heads + kHeads - 1) / kHeads, per_part = (chunks + gridDim.y - 1) / gridDim.y;
  const int c0 = blockIdx.y * per_part, c1 = min(chunks, c0 + per_part);
  const __nv_bfloat16* q = a.q.p + r * a.q.batch + j * a.q.token;
  const __nv_bfloat16* k = a.k.p + r * a.k.batch + j * a.k.token;
  const __nv_bfloat16* v = a.v.p + r * a.v.batch + j * a.v.token;
  uint4 x[kRowDeep];
  auto load = [&](int c) {
#pragma unroll
    for (int u = 0; u < kRowDeep; ++u) {
      const int h = c * kHeads + (u * 32 + lane) / kVecs;
      if (h < heads)
        x[u] = ld16((h < a.hq             ? q + h * a.q.head
                     : h < a.hq + a.hk ? k + (h - a.hq) * a.k.head
                                       : v + (h - a.hq - a.hk) * a.v.head) +
                    lane % kVecs * 8);
    }
  };
  if (c0 < c1) load(c0);
  long long row;
  const bool live = check_token(a, tok, r, j, lane == 0 && blockIdx.y == 0, row);
  if (!live) return;
  // this lane's pairs: cosine and sine, and where their components are (two
  // neighbours where they are not rotated)
  float2 cs[kPairs];
  int at_a[kPairs], at_b[kPairs];
#pragma unroll
  for (int i = 0; i < kPairs; ++i) {
    const int e = lane + 32 * i;
    const bool turn = e < half;
    cs[i] = make_float2(1.f, 0.f);
    if (turn) {
      const float2 c = cos_sin(a.pos[tok], a.rope.turns[e]);
      cs[i] = make_float2(c.x * a.rope.amplitude, c.y * a.rope.amplitude * a.sign);
    }
    at_a[i] = !IL && turn ? e : 2 * e;
    at_b[i] = !IL && turn ? half + e : 2 * e + 1;
  }
  __nv_bfloat16* rows = s_rows[warp];
  uint8_t* codes = s_codes[FP8 ? warp : 0];
  __nv_bfloat16* qo = a.q_out.p + r * a.q_out.batch + j * a.q_out.token;
  for (int c = c0; c < c1; ++c) {
    const int h0 = c * kHeads, n = min(kHeads, heads - h0);
#pragma unroll
    for (int u = 0; u < kRowDeep; ++u) *reinterpret_cast<uint4*>(rows + (u * 32 + lane) * 8) = x[u];
    __syncwarp();
    if (c + 1 < c1) load(c + 1);
    // scales: lane g has head g's of the chunk
    Divisor mine(1.f);
    if (FP8 && lane < n && h0 + lane >= a.hq) {
      const int h = h0 + lane - a.hq;
      mine = Divisor(h < a.hk ? a.k_scale[h] : a.v_scale[h - a.hk]);
    }
    // heads that are rotated and stay BF16, some at a time
    const int turned = max(0, min(n, a.hq + (FP8 ? 0 : a.hk) - h0));
    for (int g = 0; g < turned; g += kGroup) {
      float fa[4], fb[4];
#pragma unroll
      for (int u = 0; u < kGroup * kPairs; ++u) {
        const __nv_bfloat16* x0 = rows + (g + u / kPairs) * D;
        if (lane + 32 * (u % kPairs) < half) {
          fa[u] = __bfloat162float(x0[at_a[u % kPairs]]);
          fb[u] = __bfloat162float(x0[at_b[u % kPairs]]);
        }
      }
#pragma unroll
      for (int u = 0; u < kGroup * kPairs; ++u) {
        __nv_bfloat16* x0 = rows + (g + u / kPairs) * D;
        if (lane + 32 * (u % kPairs) < half && g + u / kPairs < turned) {
          rotate(fa[u], fb[u], cs[u % kPairs]);
          x0[at_a[u % kPairs]] = __float2bfloat16_rn(fa[u]);
          x0[at_b[u % kPairs]] = __float2bfloat16_rn(fb[u]);
        }
      }
    }
    if constexpr (FP8) {
      for (int g = turned; g < n; ++g) {  // heads that become codes
        const Divisor by(mine, g);
        const bool is_k = h0 + g < a.hq + a.hk;
#pragma unroll
        for (int i = 0; i < kPairs; ++i) {
          const int oa = is_k ? at_a[i] : 2 * (lane + 32 * i), ob = is_k ? at_b[i] : oa + 1;
          float2 f = make_float2(__bfloat162float(rows[g * D + oa]), __bfloat162float(rows[g * D + ob]));
          if (is_k && lane + 32 * i < half) rotate(f.x, f.y, cs[i]);
          f = by.usual ? by.quick(f) : make_float2(f.x / by.scale, f.y / by.scale);
          const uint32_t w = e4m3x2(f.x, f.y);
          codes[g * D + oa] = (uint8_t)w;
          codes[g * D + ob] = (uint8_t)(w >> 8);
        }
      }
    }
    __syncwarp();
#pragma unroll
    for (int u = 0; u < kRowDeep; ++u) {
      const int h = h0 + (u * 32 + lane) / kVecs, at = lane % kVecs * 8;
      if (h >= heads) continue;
      const uint4 y = *reinterpret_cast<const uint4*>(rows + (u * 32 + lane) * 8);
      if (h < a.hq) {
        *reinterpret_cast<uint4*>(qo + h * a.q_out.head + at) = y;
      } else if (!FP8 && row >= 0) {
        const bool is_v = h >= a.hq + a.hk;
        const int g = is_v ? h - a.hq - a.hk : h - a.hq;
        __nv_bfloat16* cache = reinterpret_cast<__nv_bfloat16*>(is_v ? a.v_cache : a.k_cache);
        *reinterpret_cast<uint4*>(cache + row + (long long)g * a.page_size * D + at) = y;
      }
    }
    if (FP8 && row >= 0) {
      for (int w = lane; w < n * (D / 16); w += 32) {
        const int h = h0 + w / (D / 16);
        if (h < a.hq) continue;
        const bool is_v = h >= a.hq + a.hk;
        const int g = is_v ? h - a.hq - a.hk : h - a.hq;
        uint8_t* cache = is_v ? a.v_cache : a.k_cache;
        *reinterpret_cast<uint4*>(cache + row + (long long)g * a.page_size * D + w % (D / 16) * 16) =
            *reinterpret_cast<const uint4*>(codes + w * 16);
      }
    }
    __syncwarp();
  }
}

// ---------------------------------------------------------------------------
// one pair (or two components that are not rotated) a thread
// ---------------------------------------------------------------------------
constexpr int kPairTok = 4, kPairThreads = 256;

// grid (ceil(tokens / kPairTok), ceil(pairs of a token / kPairThreads)): a
// thread keeps its pair for kPairTok tokens; the tokens' angles are shared
__global__ void __launch_bounds__(kPairThreads) pair_kernel(const TokenArgs a) {
  __shared__ float2 s_cs[kPairTok][kMaxHalf];
  __shared__ long long s_row[kPairTok];
  __shared__ int s_live[kPairTok];
  pdl_wait();
  const int tid = threadIdx.x;
  const int tok0 = (int)blockIdx.x * kPairTok;
  const int half = a.rope.rot_dim >> 1, per_head = a.head_dim / 2;
  const int item = blockIdx.y * kPairThreads + tid;
  const int head = item / per_head, i = item - head * per_head;
  const bool mine = head < a.hq + 2 * a.hk;
  const int seg = head < a.hq ? 0 : head < a.hq + a.hk ? 1 : 2;  // q, k, v
  const int g = seg == 0 ? head : seg == 1 ? head - a.hq : head - a.hq - a.hk;
  const bool turn = seg < 2 && i < half;
  const bool apart = turn && !a.rope.interleaved;
  const int o0 = apart ? i : 2 * i, o1 = apart ? half + i : o0 + 1;
  const Strided& in = seg == 0 ? a.q : seg == 1 ? a.k : a.v;
  const int rb = (int)((unsigned)tok0 / (unsigned)a.n_tok), jb = tok0 - rb * a.n_tok;
  __nv_bfloat16 x0[kPairTok], x1[kPairTok];
  int r = rb, j = jb;
#pragma unroll
  for (int t = 0; t < kPairTok; ++t) {
    if (mine && tok0 + t < a.tokens) {
      const __nv_bfloat16* p = in.p + r * in.batch + j * in.token + g * in.head;
      x0[t] = p[o0];
      x1[t] = p[o1];
    }
    if (++j == a.n_tok) {
      j = 0;
      ++r;
    }
  }
  if (tid < kPairTok && tok0 + tid < a.tokens) {
    const int tok = tok0 + tid, tr = (int)((unsigned)tok / (unsigned)a.n_tok);
    s_live[tid] = check_token(a, tok, tr, tok - tr * a.n_tok, blockIdx.y == 0, s_row[tid]);
  }
  for (int e = tid; e < kPairTok * half; e += kPairThreads) {
    const int t = e / half, f = e - t * half;
    if (tok0 + t < a.tokens) {
      const float2 c = cos_sin(a.pos[tok0 + t], a.rope.turns[f]);
      s_cs[t][f] = make_float2(c.x * a.rope.amplitude, c.y * a.rope.amplitude * a.sign);
    }
  }
  __syncthreads();
  if (!mine) return;
  const float scale = seg == 0 || !a.fp8 ? 1.f : seg == 1 ? a.k_scale[g] : a.v_scale[g];
  r = rb, j = jb;
#pragma unroll
  for (int t = 0; t < kPairTok; ++t) {
    if (tok0 + t < a.tokens && s_live[t]) {
      float f0 = __bfloat162float(x0[t]), f1 = __bfloat162float(x1[t]);
      if (turn) rotate(f0, f1, s_cs[t][i]);
      if (seg == 0) {
        __nv_bfloat16* p = a.q_out.p + r * a.q_out.batch + j * a.q_out.token + g * a.q_out.head;
        p[o0] = __float2bfloat16_rn(f0);
        p[o1] = __float2bfloat16_rn(f1);
      } else if (s_row[t] >= 0) {
        uint8_t* cache = seg == 1 ? a.k_cache : a.v_cache;
        const long long at = s_row[t] + (long long)g * a.page_size * a.head_dim;
        if (a.fp8) {
          cache[at + o0] = (uint8_t)e4m3x2(f0 / scale, 0.f);
          cache[at + o1] = (uint8_t)e4m3x2(f1 / scale, 0.f);
        } else {
          __nv_bfloat16* p = reinterpret_cast<__nv_bfloat16*>(cache) + at;
          p[o0] = __float2bfloat16_rn(f0);
          p[o1] = __float2bfloat16_rn(f1);
        }
      }
    }
    if (++j == a.n_tok) {
      j = 0;
      ++r;
    }
  }
}

// whether 16-byte vectors of 8 components can be used on t
bool vec8(const Strided& t) {
  return t.p == nullptr || ((reinterpret_cast<uintptr_t>(t.p) & 15u) == 0 && t.batch % 8 == 0 && t.token % 8 == 0 &&
                            t.head % 8 == 0);
}

template <int PER, bool FP8>
cudaError_t launch_wide(const TokenArgs& a, cudaStream_t s) {
  const int passes = (a.hq + 2 * a.hk + 32 / PER - 1) / (32 / PER);
  const unsigned gx = (unsigned)((a.tokens + kWideWarps - 1) / kWideWarps);
  // few tokens: their passes are dealt to several warps, which each work out
  // the angles (32 tokens of 20 heads of 128: 5 parts)
  const unsigned gy = (unsigned)std::max<long long>(1, std::min<long long>(passes, 2LL * device_sm_count() / gx));
  return a.rope.interleaved ? launch_k(wide_kernel<PER, true, FP8>, dim3(gx, gy), dim3(32 * kWideWarps), 0, s, true, a)
                            : launch_k(wide_kernel<PER, false, FP8>, dim3(gx, gy), dim3(32 * kWideWarps), 0, s, true, a);
}
template <bool FP8>
cudaError_t launch_wide(const TokenArgs& a, cudaStream_t s) {
  return a.head_dim == 64    ? launch_wide<4, FP8>(a, s)
         : a.head_dim == 128 ? launch_wide<8, FP8>(a, s)
                             : launch_wide<16, FP8>(a, s);
}

template <int D, bool FP8>
cudaError_t launch_row(const TokenArgs& a, cudaStream_t s) {
  const int heads = kRowDeep * 32 / (D / 8), chunks = (a.hq + 2 * a.hk + heads - 1) / heads;
  const unsigned gx = (unsigned)((a.tokens + kRowWarps - 1) / kRowWarps);
  const unsigned gy = (unsigned)std::max<long long>(1, std::min<long long>(chunks, 2LL * device_sm_count() / gx));
  return a.rope.interleaved ? launch_k(row_kernel<D, true, FP8>, dim3(gx, gy), dim3(32 * kRowWarps), 0, s, true, a)
                            : launch_k(row_kernel<D, false, FP8>, dim3(gx, gy), dim3(32 * kRowWarps), 0, s, true, a);
}
template <bool FP8>
cudaError_t launch_row(const TokenArgs& a, cudaStream_t s) {
  return a.head_dim == 64    ? launch_row<64, FP8>(a, s)
         : a.head_dim == 128 ? launch_row<128, FP8>(a, s)
                             : launch_row<256, FP8>(a, s);
}

cudaError_t launch_tokens(const TokenArgs& a, cudaStream_t s) {
  if (vec8(a.q) && vec8(a.q_out) && vec8(a.k) && vec8(a.v)) {
    if (a.rope.rot_dim % 16 == 0) return a.fp8 ? launch_wide<true>(a, s) : launch_wide<false>(a, s);
    return a.fp8 ? launch_row<true>(a, s) : launch_row<false>(a, s);
  }
  const int pairs = (a.hq + 2 * a.hk) * (a.head_dim / 2);
  const dim3 grid((unsigned)((a.tokens + kPairTok - 1) / kPairTok),
                  (unsigned)((pairs + kPairThreads - 1) / kPairThreads));
  return launch_k(pair_kernel, grid, dim3(kPairThreads), 0, s, true, a);
}

// Reading back. A block takes kGatherTok tokens, whose cache rows are worked
// out first, and up to 256 items; an item is the same 8 components of the same
// head of K or V in every token, so a thread decodes its item once and only
// adds up offsets, with the loads of kGatherDeep tokens in flight. E4M3 codes
// are widened (exactly, through FP16) and scaled in FP32, one rounding to BF16.
// 50,001 tokens of 2 heads of 128, BF16: 19 us (15 at HBM's copy rate; twice as
// many 34 for 31): the chain of look-ups at its start and its last blocks.
constexpr int kGatherTok = 32, kGatherDeep = 4;

struct GatherArgs {
  const uint8_t* k_cache;
  const uint8_t* v_cache;
  const float* k_scale;
  const float* v_scale;
  const int32_t* page_table;
  const int32_t* pos;
  __nv_bfloat16* k_out;
  __nv_bfloat16* v_out;
  int32_t* err;
  long long tokens;
  int n_tok, hk, head_dim, max_pages, num_pages, page_size;
};

// grid (ceil(tokens / kGatherTok), ceil(items / 256))
template <bool FP8>
__global__ void __launch_bounds__(256) gather_kernel(const GatherArgs a) {
  __shared__ long long s_row[kGatherTok];
  pdl_wait();
  const int tid = threadIdx.x;
  const long long tok0 = (long long)blockIdx.x * kGatherTok;
  const int n = (int)min((long long)kGatherTok, a.tokens - tok0);
  if (tid < n) {
    const long long tok = tok0 + tid;
    const int p = a.pos[tok];
    const bool report = blockIdx.y == 0;
    long long row = -1;
    if (p != -1) {
      const int r = (int)((unsigned)tok / (unsigned)a.n_tok), j = (int)tok - r * a.n_tok;
      if (p < 0 || p >= a.max_pages * a.page_size) {
        if (report) record_error(a.err, kErrQueryPos, r, j, p);
      } else {
        const int page = a.page_table[(long long)r * a.max_pages + p / a.page_size];
        if ((unsigned)page < (unsigned)a.num_pages)
          row = ((long long)page * a.hk * a.page_size + p % a.page_size) * a.head_dim;
        else if (report)
          record_error(a.err, kErrPage, r, j, page);
      }
    }
    s_row[tid] = row;
  }
  const int vecs = a.head_dim / 8, per = a.hk * vecs, items = 2 * per;  // items of a token
  const int here = min(256, items - (int)blockIdx.y * 256);             // of them in this block
  const int lanes = 256 / here;                                         // tokens at a time
  const int sub = tid / here, item = (int)blockIdx.y * 256 + tid - sub * here;
  const bool is_v = item >= per;
  const int h = is_v ? item - per : item, g = h / vecs;
  const uint8_t* cache = is_v ? a.v_cache : a.k_cache;
  const long long off = ((long long)g * a.page_size) * a.head_dim + (h - g * vecs) * 8;
  const float s = !FP8 ? 1.f : is_v ? a.v_scale[g] : a.k_scale[g];
  __nv_bfloat16* out = (is_v ? a.v_out : a.k_out) + tok0 * a.hk * a.head_dim + h * 8;
  __syncthreads();
  if (sub >= lanes) return;
  for (int t0 = sub; t0 < n; t0 += kGatherDeep * lanes) {
    uint4 w[kGatherDeep];
#pragma unroll
    for (int u = 0; u < kGatherDeep; ++u) {
      const int t = t0 + u * lanes;
      if (t < n && s_row[t] >= 0) {
        if constexpr (FP8) {
          const uint2 c = ld8(cache + s_row[t] + off);
          w[u].x = c.x;
          w[u].y = c.y;
        } else {
          w[u] = ld16(cache + 2 * (s_row[t] + off));
        }
      }
    }
#pragma unroll
    for (int u = 0; u < kGatherDeep; ++u) {
      const int t = t0 + u * lanes;
      if (t >= n || s_row[t] < 0) continue;
      if constexpr (FP8) {
        const float2 f0 = h2_to_f2(e4m3x2_to_h2(w[u].x)), f1 = h2_to_f2(e4m3x2_to_h2(w[u].x >> 16));
        const float2 f2 = h2_to_f2(e4m3x2_to_h2(w[u].y)), f3 = h2_to_f2(e4m3x2_to_h2(w[u].y >> 16));
        w[u] = make_uint4(pack_bf(f0.x * s, f0.y * s), pack_bf(f1.x * s, f1.y * s), pack_bf(f2.x * s, f2.y * s),
                          pack_bf(f3.x * s, f3.y * s));
      }
      *reinterpret_cast<uint4*>(out + (long long)t * a.hk * a.head_dim) = w[u];
    }
  }
}

}  // namespace

cudaError_t launch_rope(const Rope& rope, int batch, int n_tok, int n_heads, int head_dim, bool inverse,
                        const Strided& x, const int32_t* pos, const Strided& y, cudaStream_t s) {
  TokenArgs a = {};
  a.rope = rope;
  a.sign = inverse ? -1.f : 1.f;
  a.q = x;
  a.q_out = y;
  a.hq = n_heads;
  a.n_tok = n_tok;
  a.head_dim = head_dim;
  a.tokens = (long long)batch * n_tok;
  a.pos = pos;
  return launch_tokens(a, s);
}

cudaError_t launch_kv_append(const qsa_dims& d, int n_tok, const Rope& rope, const Strided& k, const Strided& v,
                             const Strided& q, const Strided& q_out, const int32_t* pos, const int32_t* page_table,
                             void* k_cache, void* v_cache, const float* k_scale, const float* v_scale, int32_t* err,
                             cudaStream_t s) {
  TokenArgs a = {};
  a.rope = rope;
  a.sign = 1.f;
  a.q = q;
  a.q_out = q_out;
  a.k = k;
  a.v = v;
  a.hq = q.p ? d.n_q_heads : 0;
  a.hk = d.n_kv_heads;
  a.n_tok = n_tok;
  a.head_dim = d.head_dim;
  a.tokens = (long long)d.batch * n_tok;
  a.pos = pos;
  a.page_table = page_table;
  a.k_cache = static_cast<uint8_t*>(k_cache);
  a.v_cache = static_cast<uint8_t*>(v_cache);
  a.k_scale = k_scale;
  a.v_scale = v_scale;
  a.err = err;
  a.max_pages = d.max_pages;
  a.num_pages = d.num_pages;
  a.page_size = d.page_size;
  a.fp8 = d.kv_dtype == QSA_KV_FP8_E4M3;
  return launch_tokens(a, s);
}

cudaError_t launch_kv_gather(const qsa_dims& d, int n_tok, const void* k_cache, const void* v_cache,
                             const float* k_scale, const float* v_scale, const int32_t* page_table,
                             const int32_t* pos, void* k_out, void* v_out, int32_t* err, cudaStream_t s) {
  GatherArgs a = {};
  a.k_cache = static_cast<const uint8_t*>(k_cache);
  a.v_cache = static_cast<const uint8_t*>(v_cache);
  a.k_scale = k_scale;
  a.v_scale = v_scale;
  a.page_table = page_table;
  a.pos = pos;
  a.k_out = static_cast<__nv_bfloat16*>(k_out);
  a.v_out = static_cast<__nv_bfloat16*>(v_out);
  a.err = err;
  a.tokens = (long long)d.batch * n_tok;
  a.n_tok = n_tok;
  a.hk = d.n_kv_heads;
  a.head_dim = d.head_dim;
  a.max_pages = d.max_pages;
  a.num_pages = d.num_pages;
  a.page_size = d.page_size;
  const unsigned gx = (unsigned)((a.tokens + kGatherTok - 1) / kGatherTok);
  const unsigned gy = (unsigned)((2 * a.hk * (a.head_dim / 8) + 255) / 256);
  auto kern = d.kv_dtype == QSA_KV_FP8_E4M3 ? gather_kernel<true> : gather_kernel<false>;
  return launch_k(kern, dim3(gx, gy), dim3(256), 0, s, true, a);
}

}  // namespace qsa
