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

__device__ __forceinline__ void rotate(float& xa, float& xb, float2 cs) {
  const float a = xa, b = xb;
  xa = a * cs.x - b * cs.y;
  xb = b * cs.x + a * cs.y;
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
  // (cos, sin) of a token's pairs. W = 8: the 16-byte unit of pairs 8 i + 2 u,
  // 8 i + 2 u + 1 is at [u][i], so that items i = 0, 1, .. of a warp read
  // consecutive units; W = 1: in order
  __shared__ __align__(16) float2 s_cs[TOK][kMaxHalf];
  __shared__ long long s_row[TOK];  // cache row of KV head 0; -1: K and V are not written
  __shared__ int s_live[TOK];       // the token is there and in order
  const int tid = threadIdx.x;
  const long long tok0 = (long long)blockIdx.x * TOK;  // (below 2^31)
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

  // (request, token) of the block's first token; the others follow by counting
  const int rb = (int)((unsigned)tok0 / (unsigned)a.n_tok), jb = (int)tok0 - rb * a.n_tok;
  Vec<W> x0[TOK], x1[TOK];
  {
    int r = rb, j = jb;
#pragma unroll
    for (int t = 0; t < TOK; ++t) {
      if (mine && tok0 + t < a.tokens) {
        const __nv_bfloat16* p = in.p + r * in.batch + j * in.token + g * in.head;
        x0[t].load(p + o0);
        x1[t].load(p + o1);
      }
      if (++j == a.n_tok) {
        j = 0;
        ++r;
      }
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
        const int r = (int)((unsigned)tok / (unsigned)a.n_tok), j = (int)tok - r * a.n_tok;
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
      const int at = W == 1 ? f : (((f >> 1) & 3) * (half >> 3) + (f >> 3)) * 2 + (f & 1);
      s_cs[t][at] = make_float2(cs.x * a.rope.amplitude, cs.y * a.rope.amplitude * a.sign);
    }
  }
  __syncthreads();
  if (!mine) return;

  const float scale = seg == 0 || !a.fp8 ? 1.f : seg == 1 ? a.k_scale[g] : a.v_scale[g];
  int rn = rb, jn = jb;
#pragma unroll
  for (int t = 0; t < TOK; ++t) {
    const int r = rn, j = jn;
    if (++jn == a.n_tok) {
      jn = 0;
      ++rn;
    }
    if (tok0 + t >= a.tokens || !s_live[t]) continue;
    float f0[W], f1[W];
    x0[t].get(f0);
    x1[t].get(f1);
    if (turn) {
      if constexpr (W == 1) {
        rotate(f0[0], f1[0], s_cs[t][i]);
      } else {
        const float4* cs = reinterpret_cast<const float4*>(s_cs[t]) + i;
        const int step = half >> 3;
#pragma unroll
        for (int u = 0; u < 4; ++u) {
          const float4 w = cs[u * step];
          const float2 c0 = make_float2(w.x, w.y), c1 = make_float2(w.z, w.w);
          if (a.rope.interleaved) {  // pairs 8 i + 2 u, + 1: adjacent components of the first or second vector
            float(&f)[W] = u < 2 ? f0 : f1;
            rotate(f[4 * u % W], f[4 * u % W + 1], c0);
            rotate(f[4 * u % W + 2], f[4 * u % W + 3], c1);
          } else {
            rotate(f0[2 * u], f1[2 * u], c0);
            rotate(f0[2 * u + 1], f1[2 * u + 1], c1);
          }
        }
      }
    }
    if (seg == 0) {
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

// Reading back. A block takes kGatherTok tokens, whose cache rows are worked
// out first, and up to 256 items; an item is the same 8 components of the same
// head of K or V in every token, so a thread decodes its item once and only
// adds up offsets, with the loads of kGatherDeep tokens in flight. E4M3 codes
// are widened (exactly, through FP16) and scaled in FP32, one rounding to BF16.
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
  return launch_k(kern, dim3(gx, gy), dim3(256), 0, s, false, a);
}

}  // namespace qsa
