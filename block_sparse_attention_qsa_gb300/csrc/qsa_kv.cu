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
// Cache write. BF16: the rotated key rounded once. E4M3: x / scale[head] (an
// FP32 division, correctly rounded), then to nearest even with clamping. The
// rotated key is not rounded to BF16 in between.
//
// All of it is streaming: each input is read once and each output written
// once, with nothing to reuse but the R / 2 (cos, sin) of a token, which all
// its heads share. So the layout is made for that: a block takes kTok tokens
// and up to kItems items; an item is the same 2 x W components of the same
// head in every token (W = 8: two 16-byte vectors that hold 8 whole pairs; W =
// 1: one pair, for row starts, strides or rotated parts that are not multiples
// of 16 bytes or 16 components). A thread decodes its item once, issues the
// loads of all its tokens before anything else, and meets the block's table of
// (cos, sin), worked out while the loads are in flight, at one barrier.
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

template <int W>
struct Vec;
template <>
struct Vec<8> {
  uint4 w;
  __device__ __forceinline__ void load(const __nv_bfloat16* p) { w = ld16(p); }
  __device__ __forceinline__ void get(float (&f)[8]) const {
    f[0] = bf_lo(w.x), f[1] = bf_hi(w.x), f[2] = bf_lo(w.y), f[3] = bf_hi(w.y);
    f[4] = bf_lo(w.z), f[5] = bf_hi(w.z), f[6] = bf_lo(w.w), f[7] = bf_hi(w.w);
  }
  static __device__ __forceinline__ void store_bf(__nv_bfloat16* p, const float (&f)[8]) {
    *reinterpret_cast<uint4*>(p) =
        make_uint4(pack_bf(f[0], f[1]), pack_bf(f[2], f[3]), pack_bf(f[4], f[5]), pack_bf(f[6], f[7]));
  }
  static __device__ __forceinline__ void store_e4m3(uint8_t* p, const float (&f)[8], float scale) {
    uint32_t c[4];
#pragma unroll
    for (int i = 0; i < 4; ++i) c[i] = e4m3x2(f[2 * i] / scale, f[2 * i + 1] / scale);
    *reinterpret_cast<uint2*>(p) = make_uint2(c[0] | (c[1] << 16), c[2] | (c[3] << 16));
  }
};
template <>
struct Vec<1> {
  __nv_bfloat16 w;
  __device__ __forceinline__ void load(const __nv_bfloat16* p) { w = *p; }
  __device__ __forceinline__ void get(float (&f)[1]) const { f[0] = __bfloat162float(w); }
  static __device__ __forceinline__ void store_bf(__nv_bfloat16* p, const float (&f)[1]) {
    *p = __float2bfloat16_rn(f[0]);
  }
  static __device__ __forceinline__ void store_e4m3(uint8_t* p, const float (&f)[1], float scale) {
    *p = (uint8_t)e4m3x2(f[0] / scale, 0.f);
  }
};

// grid (ceil(tokens / TOK), ceil(items / kItems)), kItems threads
constexpr int kItems = 256;

template <int W, int TOK>
__global__ void __launch_bounds__(kItems) token_kernel(const TokenArgs a) {
  __shared__ float2 s_cs[TOK][kMaxHalf];
  __shared__ long long s_row[TOK];  // cache row of KV head 0; -1: K and V are not written
  __shared__ int s_live[TOK];       // the token is there and in order
  const int tid = threadIdx.x;
  const long long tok0 = (long long)blockIdx.x * TOK;
  const int half = a.rope.rot_dim >> 1;
  const int per_head = a.head_dim / (2 * W);  // items of a head
  const int item = blockIdx.y * kItems + tid;
  const int head = item / per_head, i = item - head * per_head;
  const int heads = a.hq + 2 * a.hk;
  const bool mine = head < heads;
  const int seg = head < a.hq ? 0 : head < a.hq + a.hk ? 1 : 2;  // q, k, v
  const int g = seg == 0 ? head : seg == 1 ? head - a.hq : head - a.hq - a.hk;
  const bool turn = seg < 2 && i < a.rope.rot_dim / (2 * W);
  // the item's two vectors: 8 whole pairs of a rotated part, else 2 W consecutive components
  const bool split = turn && !a.rope.interleaved;
  const int o0 = split ? i * W : i * 2 * W, o1 = split ? half + i * W : o0 + W;
  const Strided& in = seg == 0 ? a.q : seg == 1 ? a.k : a.v;

  Vec<W> x0[TOK], x1[TOK];
#pragma unroll
  for (int t = 0; t < TOK; ++t) {
    const long long tok = tok0 + t;
    if (mine && tok < a.tokens) {
      const long long r = tok / a.n_tok, j = tok - r * a.n_tok;
      const __nv_bfloat16* p = in.p + r * in.batch + j * in.token + g * in.head;
      x0[t].load(p + o0);
      x1[t].load(p + o1);
    }
  }
  // the tokens' checks and cache rows
  if (tid < TOK) {
    const long long tok = tok0 + tid;
    long long row = -1;
    int live = 0;
    if (tok < a.tokens) {
      const int p = a.pos[tok];
      live = p >= 0;
      if (a.hk > 0 && p != -1) {
        const int r = (int)(tok / a.n_tok), j = (int)(tok - (long long)r * a.n_tok);
        const bool report = blockIdx.y == 0;
        if (p < 0 || p >= a.max_pages * a.page_size) {
          live = 0;
          if (report) record_error(a.err, kErrQueryPos, r, j, p);
        } else if (p != (long long)a.pos[(long long)r * a.n_tok] + j) {
          live = 0;
          if (report) record_error(a.err, kErrOrder, r, j, p);
        } else {
          const int page = a.page_table[(long long)r * a.max_pages + p / a.page_size];
          if ((unsigned)page < (unsigned)a.num_pages)
            row = (long long)page * a.hk * a.page_size + p % a.page_size;
          else if (report)
            record_error(a.err, kErrPage, r, j, page);
        }
      }
    }
    s_row[tid] = row;
    s_live[tid] = live;
  }
  for (int e = tid; e < TOK * half; e += kItems) {
    const int t = e / half, f = e - t * half;
    if (tok0 + t < a.tokens) {
      const float2 cs = cos_sin(a.pos[tok0 + t], a.rope.turns[f]);
      s_cs[t][f] = make_float2(cs.x * a.rope.amplitude, cs.y * a.rope.amplitude * a.sign);
    }
  }
  __syncthreads();
  if (!mine) return;

  const float scale = seg == 0 || !a.fp8 ? 1.f : seg == 1 ? a.k_scale[g] : a.v_scale[g];
#pragma unroll
  for (int t = 0; t < TOK; ++t) {
    const long long tok = tok0 + t;
    if (tok >= a.tokens || !s_live[t]) continue;
    float f0[W], f1[W];
    x0[t].get(f0);
    x1[t].get(f1);
    if (turn) {
      if (W > 1 && a.rope.interleaved) {
#pragma unroll
        for (int e = 0; e + 1 < W; e += 2) {
          const float2 u = s_cs[t][i * W + e / 2], w = s_cs[t][i * W + W / 2 + e / 2];
          const float a0 = f0[e], b0 = f0[e + 1], a1 = f1[e], b1 = f1[e + 1];
          f0[e] = a0 * u.x - b0 * u.y;
          f0[e + 1] = b0 * u.x + a0 * u.y;
          f1[e] = a1 * w.x - b1 * w.y;
          f1[e + 1] = b1 * w.x + a1 * w.y;
        }
      } else {
#pragma unroll
        for (int e = 0; e < W; ++e) {
          const float2 u = s_cs[t][i * W + e];
          const float xa = f0[e], xb = f1[e];
          f0[e] = xa * u.x - xb * u.y;
          f1[e] = xb * u.x + xa * u.y;
        }
      }
    }
    if (seg == 0) {
      const long long r = tok / a.n_tok, j = tok - r * a.n_tok;
      __nv_bfloat16* p = a.q_out.p + r * a.q_out.batch + j * a.q_out.token + g * a.q_out.head;
      Vec<W>::store_bf(p + o0, f0);
      Vec<W>::store_bf(p + o1, f1);
    } else if (s_row[t] >= 0) {
      uint8_t* cache = seg == 1 ? a.k_cache : a.v_cache;
      const long long at = (s_row[t] + (long long)g * a.page_size) * a.head_dim;
      if (a.fp8) {
        Vec<W>::store_e4m3(cache + at + o0, f0, scale);
        Vec<W>::store_e4m3(cache + at + o1, f1, scale);
      } else {
        __nv_bfloat16* p = reinterpret_cast<__nv_bfloat16*>(cache) + at;
        Vec<W>::store_bf(p + o0, f0);
        Vec<W>::store_bf(p + o1, f1);
      }
    }
  }
}

// whether 16-byte vectors of 8 components can be used on t
bool vec8(const Strided& t) {
  return t.p == nullptr || ((reinterpret_cast<uintptr_t>(t.p) & 15u) == 0 && t.batch % 8 == 0 && t.token % 8 == 0 &&
                            t.head % 8 == 0);
}

template <int W>
cudaError_t launch_tokens(const TokenArgs& a, cudaStream_t s) {
  const int items = (a.hq + 2 * a.hk) * (a.head_dim / (2 * W));
  const unsigned gy = (unsigned)((items + kItems - 1) / kItems);
  constexpr int kTok = 4;
  if (a.tokens * gy <= 4 * device_sm_count())
    return launch_k(token_kernel<W, 1>, dim3((unsigned)a.tokens, gy), dim3(kItems), 0, s, false, a);
  const long long gx = (a.tokens + kTok - 1) / kTok;
  return launch_k(token_kernel<W, kTok>, dim3((unsigned)gx, gy), dim3(kItems), 0, s, false, a);
}

cudaError_t launch_tokens(const TokenArgs& a, cudaStream_t s) {
  const bool wide = a.rope.rot_dim % 16 == 0 && vec8(a.q) && vec8(a.q_out) && vec8(a.k) && vec8(a.v);
  return wide ? launch_tokens<8>(a, s) : launch_tokens<1>(a, s);
}

// Reading back. A block takes kGatherTok tokens: their cache rows are worked
// out first, then the 8-component vectors of all heads of K and V are copied,
// kGatherTok * 2 * heads * head_dim / 8 of them, E4M3 codes widened (exactly,
// through FP16) and scaled in FP32, one rounding to BF16.
constexpr int kGatherTok = 32;

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

template <bool FP8>
__global__ void __launch_bounds__(256) gather_kernel(const GatherArgs a) {
  __shared__ long long s_row[kGatherTok];
  const int tid = threadIdx.x;
  const long long tok0 = (long long)blockIdx.x * kGatherTok;
  const int n = (int)min((long long)kGatherTok, a.tokens - tok0);
  if (tid < n) {
    const long long tok = tok0 + tid;
    const int p = a.pos[tok];
    long long row = -1;
    if (p != -1) {
      const int r = (int)(tok / a.n_tok), j = (int)(tok - (long long)r * a.n_tok);
      if (p < 0 || p >= a.max_pages * a.page_size) {
        record_error(a.err, kErrQueryPos, r, j, p);
      } else {
        const int page = a.page_table[(long long)r * a.max_pages + p / a.page_size];
        if ((unsigned)page < (unsigned)a.num_pages)
          row = (long long)page * a.hk * a.page_size + p % a.page_size;
        else
          record_error(a.err, kErrPage, r, j, page);
      }
    }
    s_row[tid] = row;
  }
  __syncthreads();
  const int vecs = a.head_dim / 8, per_tok = a.hk * vecs;  // of K or of V
  const int total = n * per_tok;
#pragma unroll 4
  for (int e = tid; e < 2 * total; e += 256) {
    const bool is_v = e >= total;
    const int f = is_v ? e - total : e;
    const int t = f / per_tok, h = f - t * per_tok, g = h / vecs, c = h - g * vecs;
    const long long row = s_row[t];
    if (row < 0) continue;
    const long long at = (row + (long long)g * a.page_size) * a.head_dim + c * 8;
    const uint8_t* cache = is_v ? a.v_cache : a.k_cache;
    uint4 w;
    if constexpr (FP8) {
      const float s = is_v ? a.v_scale[g] : a.k_scale[g];
      const uint2 u = ld8(cache + at);
      const float2 f0 = h2_to_f2(e4m3x2_to_h2(u.x)), f1 = h2_to_f2(e4m3x2_to_h2(u.x >> 16));
      const float2 f2 = h2_to_f2(e4m3x2_to_h2(u.y)), f3 = h2_to_f2(e4m3x2_to_h2(u.y >> 16));
      w = make_uint4(pack_bf(f0.x * s, f0.y * s), pack_bf(f1.x * s, f1.y * s), pack_bf(f2.x * s, f2.y * s),
                     pack_bf(f3.x * s, f3.y * s));
    } else {
      w = ld16(cache + 2 * at);
    }
    __nv_bfloat16* out = (is_v ? a.v_out : a.k_out) + (tok0 + t) * a.hk * a.head_dim;
    *reinterpret_cast<uint4*>(out + h * 8) = w;
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
  const unsigned grid = (unsigned)((a.tokens + kGatherTok - 1) / kGatherTok);
  auto kern = d.kv_dtype == QSA_KV_FP8_E4M3 ? gather_kernel<true> : gather_kernel<false>;
  return launch_k(kern, dim3(grid), dim3(256), 0, s, false, a);
}

}  // namespace qsa
