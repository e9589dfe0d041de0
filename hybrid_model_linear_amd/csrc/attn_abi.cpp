// C-ABI entry points of the softmax-attention operators: host-side validation, then the
// launches.  Declarations and the contract are in include/gdn.h.
#include "../../include/gdn.h"

#include <hip/hip_runtime.h>

#include <cmath>

#include "attn_launch.h"

namespace {

bool aligned(const void* p, uintptr_t bytes) { return reinterpret_cast<uintptr_t>(p) % bytes == 0; }

constexpr int64_t kMaxStride = 1 << 22;     // a 64-row tile's byte offsets stay in 32 bits
constexpr int64_t kMaxGrid = (1 << 24) - 1;   // workgroups of 256 threads: a launch has fewer than 2^32 in a dimension
constexpr int32_t kMaxWindow = 1 << 30;     // distances are shorter; a window added to one stays in 32 bits

int page_log2(int32_t page) { return page == 16 ? 4 : page == 32 ? 5 : page == 64 ? 6 : page == 128 ? 7 : -1; }

// The cache and block table of a call; `track`: pos and weight are required.
int check_cache(const gdn_kv_cache& c, int32_t N, const int32_t* table, int64_t table_stride, int32_t table_width,
                bool track, gdn::CacheRef& r) {
  if (c.d != 64 && c.d != 128 && c.d != 256) return GDN_E_UNSUPPORTED;
  if (page_log2(c.page) < 0) return GDN_E_UNSUPPORTED;
  if (c.H_kv <= 0 || c.H_kv > 65535 || c.num_pages <= 0) return GDN_E_SHAPE;
  if (table_width <= 0 || table_stride < table_width || (int64_t)table_width * c.page > INT32_MAX - 4096) return GDN_E_SHAPE;
  if (!c.k || !c.v || !c.k_scale || !c.v_scale || (N > 0 && !table) || (track && (!c.pos || !c.weight))) return GDN_E_NULL;
  if (!aligned(c.k, 16) || !aligned(c.v, 16) || !aligned(c.pos, 16) || !aligned(c.weight, 16) || !aligned(c.k_scale, 4) ||
      !aligned(c.v_scale, 4) || !aligned(table, 4))
    return GDN_E_SHAPE;
  r.k = static_cast<uint8_t*>(c.k);
  r.v = static_cast<uint8_t*>(c.v);
  r.k_scale = c.k_scale;
  r.v_scale = c.v_scale;
  r.pos = c.pos;
  r.weight = c.weight;
  r.num_pages = c.num_pages;
  r.page_log2 = page_log2(c.page);
  r.H_kv = c.H_kv;
  r.d = c.d;
  r.table = table;
  r.table_stride = table_stride;
  r.table_width = table_width;
  return GDN_OK;
}

// bf16 rows [*, heads, d] read or written 16 bytes at a time
bool rows_ok(const void* p, int64_t stride, int64_t heads, int64_t d) {
  return aligned(p, 16) && stride >= heads * d && stride % 8 == 0 && stride <= kMaxStride;
}

bool overlap(const void* a, int64_t a_bytes, const void* b, int64_t b_bytes) {
  const uintptr_t x = reinterpret_cast<uintptr_t>(a), y = reinterpret_cast<uintptr_t>(b);
  return a && b && x < y + (uintptr_t)b_bytes && y < x + (uintptr_t)a_bytes;
}
int64_t rows_bytes(int64_t rows, int64_t stride, int64_t width) { return rows > 0 ? ((rows - 1) * stride + width) * 2 : 0; }

int check_scores(float scale, float softcap, int32_t window) {
  if (!std::isfinite(scale) || !std::isfinite(softcap) || softcap < 0.f || window < 0) return GDN_E_SHAPE;
  // the tanh is off by softcap 2^-22 (2^-9 at most here, below the weights' rounding), and its
  // argument's factor has to be a number
  if (softcap > 8192.f || (softcap > 0.f && !std::isfinite(scale / softcap * 4.f))) return GDN_E_UNSUPPORTED;
  return GDN_OK;
}

// Descriptor of a decode call; *need receives its workspace bytes.
int plan_decode(const gdn_attn_decode_args* a, gdn::AttnDecodeLaunch& p, int64_t& need) {
  need = 0;
  if (!a) return GDN_E_NULL;
  if (a->in_dtype != GDN_BF16 || a->out_dtype != GDN_BF16) return GDN_E_DTYPE;
  if (a->N < 0 || a->N > 65535 || a->H <= 0 || a->max_kvlen < 0) return GDN_E_SHAPE;
  int st = check_cache(a->cache, a->N, a->block_table, a->table_stride, a->table_width, false, p.c);
  if (st != GDN_OK) return st;
  if (a->H % p.c.H_kv != 0) return GDN_E_SHAPE;
  st = check_scores(a->scale, a->softcap, a->window);
  if (st != GDN_OK) return st;
  if (a->accumulate && !a->cache.weight) return GDN_E_NULL;
  if (a->N > 0 && (!a->q || !a->out || !a->kv_len)) return GDN_E_NULL;
  if (!rows_ok(a->q, a->q_stride, a->H, p.c.d) || !rows_ok(a->out, a->out_stride, a->H, p.c.d)) return GDN_E_SHAPE;
  if (overlap(a->out, rows_bytes(a->N, a->out_stride, (int64_t)a->H * p.c.d), a->q,
              rows_bytes(a->N, a->q_stride, (int64_t)a->H * p.c.d)))
    return GDN_E_SHAPE;
  p.N = a->N;
  p.H = a->H;
  p.q = static_cast<const gdn::u16*>(a->q);
  p.q_stride = a->q_stride;
  p.out = static_cast<gdn::u16*>(a->out);
  p.out_stride = a->out_stride;
  p.kv_len = a->kv_len;
  p.q_pos = a->q_pos;
  p.slopes = a->slopes;
  p.window = a->window < kMaxWindow ? a->window : kMaxWindow;
  p.scale = a->scale;
  p.softcap = a->softcap;
  p.accumulate = a->accumulate != 0;
  if (a->N == 0) return GDN_OK;
  int64_t rows = (int64_t)a->table_width * a->cache.page;
  p.score_cap = (rows + 63) / 64 * 64;
  if (a->max_kvlen > 0 && a->max_kvlen < rows) rows = a->max_kvlen;
  if (a->window > 0 && !a->cache.pos && a->window < rows) rows = a->window;
  gdn::plan_attn_decode(p, rows, gdn::current_device_cus());
  if ((int64_t)p.splits * ((a->H / p.c.H_kv + 15) / 16) * p.c.H_kv * a->N > kMaxGrid) return GDN_E_UNSUPPORTED;
  if (p.accumulate && a->H + (p.score_cap / 1024 + 2) * p.c.H_kv > kMaxGrid) return GDN_E_UNSUPPORTED;   // (the join: 1024 rows each)
  const int64_t heads = (int64_t)a->N * a->H;
  auto part = [&](int64_t floats) {
    const int64_t at = need;
    need += (floats * 4 + 255) / 256 * 256;
    return reinterpret_cast<float*>(reinterpret_cast<uintptr_t>(a->workspace) + at);
  };
  if (p.splits > 1) p.part_o = part(heads * p.splits * p.c.d);
  if (p.splits > 1 || p.accumulate) p.part_ml = part(heads * p.splits * 2);
  if (p.accumulate) p.scores = part(heads * p.score_cap);
  return GDN_OK;
}

// Descriptor of an extend call; need receives the workspace bytes with which its keys are split.
int plan_extend(const gdn_attn_extend_args* a, gdn::AttnExtendLaunch& p, int64_t& need) {
  need = 0;
  if (!a) return GDN_E_NULL;
  if (a->in_dtype != GDN_BF16 || a->out_dtype != GDN_BF16) return GDN_E_DTYPE;
  if (a->d != 64 && a->d != 128 && a->d != 256) return GDN_E_UNSUPPORTED;
  if (a->N < 0 || a->T < 0 || a->T > INT32_MAX || a->H_kv <= 0 || a->H <= 0 || a->H % a->H_kv != 0 || a->max_cached < 0)
    return GDN_E_SHAPE;
  int st = check_scores(a->scale, a->softcap, a->window);
  if (st != GDN_OK) return st;
  if (a->cache.k) {
    st = check_cache(a->cache, a->N, a->block_table, a->table_stride, a->table_width, false, p.c);
    if (st != GDN_OK) return st;
    if (p.c.d != a->d || p.c.H_kv != a->H_kv) return GDN_E_SHAPE;
    if (a->doc) return GDN_E_UNSUPPORTED;
    if (a->N > 0 && !a->cache_len) return GDN_E_NULL;
  } else if (a->cache_len || a->block_table) {
    return GDN_E_NULL;
  }
  if (a->T > 0 && (!a->q || !a->k || !a->v || !a->out)) return GDN_E_NULL;
  if (a->N > 0 && !a->cu_seqlens) return GDN_E_NULL;
  if (!rows_ok(a->q, a->q_stride, a->H, a->d) || !rows_ok(a->k, a->k_stride, a->H_kv, a->d) ||
      !rows_ok(a->v, a->v_stride, a->H_kv, a->d) || !rows_ok(a->out, a->out_stride, a->H, a->d))
    return GDN_E_SHAPE;
  const int64_t out_bytes = rows_bytes(a->T, a->out_stride, (int64_t)a->H * a->d);
  if (overlap(a->out, out_bytes, a->q, rows_bytes(a->T, a->q_stride, (int64_t)a->H * a->d)) ||
      overlap(a->out, out_bytes, a->k, rows_bytes(a->T, a->k_stride, (int64_t)a->H_kv * a->d)) ||
      overlap(a->out, out_bytes, a->v, rows_bytes(a->T, a->v_stride, (int64_t)a->H_kv * a->d)))
    return GDN_E_SHAPE;
  if (a->N == 0 || a->T == 0) return GDN_OK;
  const int64_t rows = a->T * (a->H / a->H_kv);          // (token, head of a group) rows: 32-bit in the kernel
  if (rows > INT32_MAX - 1024 || (rows / 128 + a->N) * a->H_kv > kMaxGrid) return GDN_E_UNSUPPORTED;
  p.N = a->N;
  p.T = a->T;
  p.H = a->H;
  p.H_kv = a->H_kv;
  p.d = a->d;
  p.q = static_cast<const gdn::u16*>(a->q);
  p.q_stride = a->q_stride;
  p.k = static_cast<const gdn::u16*>(a->k);
  p.k_stride = a->k_stride;
  p.v = static_cast<const gdn::u16*>(a->v);
  p.v_stride = a->v_stride;
  p.out = static_cast<gdn::u16*>(a->out);
  p.out_stride = a->out_stride;
  p.cu = a->cu_seqlens;
  p.cache_len = a->cache_len;
  p.start = a->start;
  p.causal = a->causal != 0;
  p.visible = a->visible;
  p.doc = a->doc;
  p.slopes = a->slopes;
  p.window = a->window < kMaxWindow ? a->window : kMaxWindow;
  p.scale = a->scale;
  p.softcap = a->softcap;
  const int64_t group = a->H / a->H_kv;
  int64_t keys = (a->T + a->N - 1) / a->N;               // (a table has room for the new tokens as a rule)
  if (p.c.k) {
    int64_t held = (int64_t)a->table_width * a->cache.page;
    if (a->max_cached > 0 && a->max_cached + keys < held) held = a->max_cached + keys;
    if (held > keys) keys = held;
  }
  if (a->window > 0 && !(p.c.k && a->cache.pos) && keys > a->window + 128 / group + 64) keys = a->window + 128 / group + 64;
  gdn::plan_attn_extend(p, keys, gdn::current_device_cus());
  if (p.splits > 1) {
    const int64_t at = reinterpret_cast<uintptr_t>(a->workspace), heads = p.splits * a->T * a->H;
    p.part_o = reinterpret_cast<float*>(at);
    p.part_ml = reinterpret_cast<float*>(at + heads * a->d * 4);
    need = (heads * (a->d + 2) * 4 + 255) / 256 * 256;
  }
  return GDN_OK;
}

int plan_evict(const gdn_kv_evict_args* a, gdn::EvictLaunch& p, int64_t& need) {
  need = 0;
  if (!a) return GDN_E_NULL;
  if (a->N < 0 || a->N > 65535 || a->budget < 1 || a->recent < 0 || a->recent > a->budget) return GDN_E_SHAPE;
  const int st = check_cache(a->cache, a->N, a->block_table, a->table_stride, a->table_width, true, p.c);
  if (st != GDN_OK) return st;
  if (a->N > 0 && (!a->kv_len || !a->new_len)) return GDN_E_NULL;
  if (a->cache.num_pages > INT32_MAX / a->cache.page) return GDN_E_UNSUPPORTED;   // rows of the cache: 32-bit in the kernel
  p.N = a->N;
  // (a budget past the table's rows keeps them all)
  const int64_t rows = (int64_t)a->table_width * a->cache.page;
  p.budget = (int)(a->budget < rows ? a->budget : rows);
  p.recent = a->recent;
  p.kv_len = a->kv_len;
  p.new_len = a->new_len;
  if (a->N == 0) return GDN_OK;
  const int64_t lists = (int64_t)a->N * p.c.H_kv * p.budget;
  const int64_t pages = ((int64_t)p.budget + a->cache.page - 1) / a->cache.page;
  if (pages > kMaxGrid) return GDN_E_UNSUPPORTED;
  auto part = [&](int64_t bytes) {
    const int64_t at = need;
    need += (bytes + 255) / 256 * 256;
    return reinterpret_cast<void*>(reinterpret_cast<uintptr_t>(a->workspace) + at);
  };
  p.holes = static_cast<int32_t*>(part(lists * 4));
  p.movers = static_cast<int32_t*>(part(lists * 4));
  p.scales = static_cast<float*>(part(lists * 8));
  p.first = static_cast<int32_t*>(part((int64_t)a->N * p.c.H_kv * (pages + 1) * 4));
  return GDN_OK;
}

int check_workspace(const void* ws, int64_t bytes, int64_t need) {
  if (need == 0) return GDN_OK;
  if (!ws) return GDN_E_NULL;
  return bytes < need || !aligned(ws, 256) ? GDN_E_SHAPE : GDN_OK;
}

}  // namespace

extern "C" {

int gdn_kv_store(const gdn_kv_store_args* a, void* stream) {
  if (!a) return GDN_E_NULL;
  if (a->in_dtype != GDN_BF16) return GDN_E_DTYPE;
  if (a->N < 0 || a->T < 0 || a->T > INT32_MAX) return GDN_E_SHAPE;
  gdn::StoreLaunch p{};
  const int st = check_cache(a->cache, a->N, a->block_table, a->table_stride, a->table_width, false, p.c);
  if (st != GDN_OK) return st;
  if (!a->cu_seqlens && a->T != a->N) return GDN_E_SHAPE;
  if (a->T > 0 && (!a->k || !a->v)) return GDN_E_NULL;
  if (a->N > 0 && !a->cache_len) return GDN_E_NULL;
  if (!rows_ok(a->k, a->k_stride, p.c.H_kv, p.c.d) || !rows_ok(a->v, a->v_stride, p.c.H_kv, p.c.d)) return GDN_E_SHAPE;
  if (a->N == 0 || a->T == 0) return GDN_OK;
  const int64_t slots = a->cu_seqlens ? (a->T >> p.c.page_log2) + 2 * (int64_t)a->N : a->N;   // pages; for few tokens a workgroup takes two heads
  if (slots > kMaxGrid || (a->T <= gdn::kFewTokens * (int64_t)a->N && slots * p.c.H_kv > 2 * kMaxGrid)) return GDN_E_UNSUPPORTED;
  p.N = a->N;
  p.T = a->T;
  p.k = static_cast<const gdn::u16*>(a->k);
  p.k_stride = a->k_stride;
  p.v = static_cast<const gdn::u16*>(a->v);
  p.v_stride = a->v_stride;
  p.cu = a->cu_seqlens;
  p.cache_len = a->cache_len;
  p.start = a->start;
  return gdn::status_of_hip(gdn::launch_kv_store(p, (hipStream_t)stream));
}

int64_t gdn_attn_extend_workspace_size(const gdn_attn_extend_args* a) {
  gdn::AttnExtendLaunch p{};
  int64_t need = 0;
  const int st = plan_extend(a, p, need);
  return st == GDN_OK ? need : -(int64_t)st;
}

int gdn_attn_extend(const gdn_attn_extend_args* a, void* stream) {
  gdn::AttnExtendLaunch p{};
  int64_t need = 0;
  int st = plan_extend(a, p, need);
  if (st != GDN_OK || a->N == 0 || a->T == 0) return st;
  if (!a->workspace) {
    p.splits = 1;
  } else {
    st = check_workspace(a->workspace, a->workspace_bytes, need);
    if (st != GDN_OK) return st;
  }
  return gdn::status_of_hip(gdn::launch_attn_extend(p, (hipStream_t)stream));
}

int64_t gdn_attn_decode_workspace_size(const gdn_attn_decode_args* a) {
  gdn::AttnDecodeLaunch p{};
  int64_t need = 0;
  const int st = plan_decode(a, p, need);
  return st == GDN_OK ? need : -(int64_t)st;
}

int gdn_attn_decode(const gdn_attn_decode_args* a, void* stream) {
  gdn::AttnDecodeLaunch p{};
  int64_t need = 0;
  int st = plan_decode(a, p, need);
  if (st != GDN_OK || a->N == 0) return st;
  st = check_workspace(a->workspace, a->workspace_bytes, need);
  if (st != GDN_OK) return st;
  return gdn::status_of_hip(gdn::launch_attn_decode(p, (hipStream_t)stream));
}

int64_t gdn_kv_evict_workspace_size(const gdn_kv_evict_args* a) {
  gdn::EvictLaunch p{};
  int64_t need = 0;
  const int st = plan_evict(a, p, need);
  return st == GDN_OK ? need : -(int64_t)st;
}

int gdn_kv_evict(const gdn_kv_evict_args* a, void* stream) {
  gdn::EvictLaunch p{};
  int64_t need = 0;
  int st = plan_evict(a, p, need);
  if (st != GDN_OK || a->N == 0) return st;
  st = check_workspace(a->workspace, a->workspace_bytes, need);
  if (st != GDN_OK) return st;
  return gdn::status_of_hip(gdn::launch_kv_evict(p, (hipStream_t)stream));
}

}  // extern "C"
