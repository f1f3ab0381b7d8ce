#include "qsa_prefix.cuh"

namespace qsa {

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

// Rows of a unit: a softmax thread's work grows with its warpgroup's rows, so
// the smallest of 8, 16, 32 (two warpgroups of 16) and 64 (two of 32) that
// holds them; more rows are several units, which each read K and V. Rows of
// 512 bytes leave no shared memory for 64.
static int unit_rows(const qsa_dims& d) {
  const int rows = d.n_q * (d.n_q_heads / d.n_kv_heads);
  const bool wide = d.head_dim == 256 && d.kv_dtype == QSA_KV_BF16;
  return rows <= 8 ? 8 : rows <= 16 ? 16 : rows <= 32 || wide ? 32 : 64;
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

template <class A>
static cudaError_t launch_dense(int rows, const qsa_dims& d, const A& a, const void* k_cache, const void* v_cache,
                                bool short_k, cudaStream_t s) {
  switch (d.head_dim) {
    case 64: return launch_dense_64(rows, d, a, k_cache, v_cache, short_k, s);
    case 128: return launch_dense_128(rows, d, a, k_cache, v_cache, short_k, s);
    default: return launch_dense_256(rows, d, a, k_cache, v_cache, short_k, s);
  }
}

// The prefix's work: units, and the parts that its tiles are cut into, of at
// most kMaxPart tiles each (an accumulator in tensor memory holds no more, see
// kRun in qsa_dense_tc.cuh).
constexpr int kMaxPart = 256, kWaves = 3;
struct PrefixPlan {
  int rows, row_tiles, units, tiles;
  int least, splits, most;  // parts: at least, one kernel after the other, at most
  int room;                 // what a workspace has room for
};
static PrefixPlan prefix_plan(const qsa_dims& d, int prefix_len, int sms) {
  PrefixPlan p;
  p.rows = d.batch * d.n_q * (d.n_q_heads / d.n_kv_heads);
  p.row_tiles = (p.rows + kPrefixRows - 1) / kPrefixRows;
  const int at_once = d.head_dim == 256 || p.row_tiles == 1 ? 1 : 2;  // row tiles of a CTA
  p.units = d.n_kv_heads * ((p.row_tiles + at_once - 1) / at_once);
  const int tile = d.head_dim == 256 ? 64 : 128;
  p.tiles = (prefix_len + tile - 1) / tile;
  p.least = std::max(1, (p.tiles + kMaxPart - 1) / kMaxPart);
  // Parts for 1 to kWaves full waves of CTAs; a CTA's time is its tiles and
  // about as much as 4 for its beginning and its piece.
  p.splits = p.least;
  long long best = 1LL << 62;
  for (int k = 1; k <= kWaves; ++k) {
    const int s = std::min(p.tiles, std::max(p.least, k * sms / p.units));
    const long long waves = ((long long)p.units * s + sms - 1) / sms;
    const long long cost = waves * ((p.tiles + s - 1) / s + 4);
    if (cost < best) {
      best = cost;
      p.splits = s;
    }
  }
  p.most = std::max(p.splits, std::min(p.tiles, (sms - 1) / p.units));
  // (never less for a longer prefix: a workspace serves shorter ones too)
  p.room = std::max(p.least, std::min(p.tiles, std::max(1, kWaves * sms / p.units)));
  return p;
}

// Whether every request reads the prefix by itself: where its tiles are few, the
// two kernels of a shared one cost more than they save. (Read once and by each,
// BF16, head dim 128: 32 requests x 1 query over 1,024 tokens 15.9 and 12.1 us,
// over 4,096, 860 KB an SM, 19.3 and 18.9; 8 x 4 over 8,192, 430 KB, 21.1 and 17.9,
// over 16,384, 860 KB, 23.6 and 23.0; 16 x 1 over 50,048 27 and 65. A tile of less
// than 32 KB takes as long: 6 x 1, E4M3, head dim 64, over 58,368, 23 and 28.)
constexpr long long kAloneBytes = 640 * 1024, kAloneTile = 32 * 1024;  // an SM; a tile, at least
static bool alone(const qsa_dims& d, int prefix_len, int rows, int sms) {
  const int all = d.n_q * (d.n_q_heads / d.n_kv_heads), eb = d.kv_dtype == QSA_KV_FP8_E4M3 ? 1 : 2;
  const long long reads = (long long)d.batch * d.n_kv_heads * ((all + rows - 1) / rows);
  const long long tile = std::max(kAloneTile, 256LL * d.head_dim * eb);
  return d.batch == 1 || reads * ((prefix_len + 127) / 128) * tile <= kAloneBytes * sms;
}

struct PrefixWs {
  size_t count, whole, parts, total;
};
static PrefixWs prefix_ws_layout(const qsa_dims& d, int prefix_len, int sms) {
  PrefixWs w;
  const int rows = d.n_q * (d.n_q_heads / d.n_kv_heads), per = unit_rows(d);
  const size_t units = (size_t)d.batch * d.n_kv_heads * ((rows + per - 1) / per);
  const size_t row = (d.head_dim + 2) * sizeof(float);
  w.count = dense_ws(d, sms).total;
  w.whole = w.count + 256;
  w.parts = align_up(w.whole + units * per * row, 256);
  const PrefixPlan p = prefix_plan(d, prefix_len, sms);
  w.total = align_up(w.parts + (size_t)d.n_kv_heads * p.row_tiles * p.room * kPrefixRows * row, 256);
  return w;
}
size_t prefix_ws(const qsa_dims& d, int prefix_len, int num_sms) {
  return prefix_len > 0 ? prefix_ws_layout(d, prefix_len, num_sms).total : dense_ws(d, num_sms).total;
}

static cudaError_t launch_with_prefix(const qsa_dims& d, SharedArgs a, int rows, uint8_t* ws, const void* k_cache,
                                      const void* v_cache, bool short_k, cudaStream_t s) {
  const PrefixWs w = prefix_ws_layout(d, a.prefix_len, a.grid);
  const PrefixPlan plan = prefix_plan(d, a.prefix_len, a.grid);
  a.whole = reinterpret_cast<float*>(ws + w.whole);
  a.row_blocks = (a.n_q * a.group + rows - 1) / rows;
  // What things take, measured (head dim 128): a tile of the own positions 1.25 us
  // a CTA for 64 KB on 40 SMs, and not much less for 32 KB; beginning a unit of
  // one tile, of which a CTA has several, 5 to 6 us; a tile of the prefix, two row
  // tiles, 1.5 us with a BF16 cache and 2.3 with E4M3. A CTA's beginning and end
  // take the first kernel 9 us, the second 15. (Without the units, 32 requests of
  // 4 to 60 own tokens over 50,048 had 8 SMs for them: 73 us, now 55.)
  const int eb = d.kv_dtype == QSA_KV_FP8_E4M3 ? 1 : 2, bytes = 256 * d.head_dim * eb;
  SharedCost& c = a.cost;
  c.units = plan.units;
  c.tiles = plan.tiles;
  c.least = plan.least;
  c.most = std::min(plan.most, 254);
  c.parts = plan.splits;
  c.own_ns = std::max(bytes / 52, 1000);
  c.unit_ns = 5000;
  c.own_hbm_ns = bytes / 6800;
  c.part_ns = (d.head_dim == 64 ? 1000 : 1500) * (eb == 1 ? 3 : 2) / 2;
  c.own_begin_ns = 9000;
  c.part_begin_ns = 15000;
  cudaError_t e = launch_dense(rows, d, a, k_cache, v_cache, false, s);
  if (e != cudaSuccess) return e;
  PrefixArgs p = {};
  p.a = a;
  p.n_parts = reinterpret_cast<int32_t*>(ws + w.count);
  p.parts = reinterpret_cast<float*>(ws + w.parts);
  p.rows = plan.rows;
  p.row_tiles = plan.row_tiles;
  p.units = plan.units;
  p.room = plan.room;
  p.most = plan.most;
  p.own_rows = rows;
  switch (d.head_dim) {
    case 64: return launch_prefix_64(d, p, k_cache, v_cache, short_k, s);
    case 128: return launch_prefix_128(d, p, k_cache, v_cache, short_k, s);
    default: return launch_prefix_256(d, p, k_cache, v_cache, short_k, s);
  }
}

// Own positions, prefix (if there is one), joint.
cudaError_t launch_paged_attn(const qsa_dims& d, int window, const void* q, const void* k_cache, const void* v_cache,
                              const float* k_scale, const float* v_scale, const int32_t* page_table,
                              const int32_t* q_pos, void* out, float* lse, void* ws, cudaStream_t s, bool short_k,
                              const Prefix& prefix) {
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
  a.one = 1.f;
  const int rows = unit_rows(d);
  if (prefix.len == 0) return launch_dense(rows, d, a, k_cache, v_cache, short_k, s);
  SharedArgs x = {};
  static_cast<DenseArgs&>(x) = a;
  x.prefix_table = prefix.table;
  x.prefix_len = prefix.len;
  if (prefix.alone < 0 ? alone(d, prefix.len, rows, sms) : prefix.alone)
    return launch_dense(rows, d, x, k_cache, v_cache, short_k, s);
  x.shared_len = prefix.len;
  return launch_with_prefix(d, x, rows, base, k_cache, v_cache, short_k, s);
}

}  // namespace qsa
