// C-ABI entry points of a serving step's operators beside the attention layers (selective
// scan, RMS norm, pages): host-side validation, then the launches.  Declarations and the
// contract are in include/gdn.h.
#include "../../include/gdn.h"

#include <hip/hip_runtime.h>

#include <cmath>

#include "step_launch.h"

namespace {

constexpr int64_t kMaxGrid = (1 << 24) - 1;   // workgroups of 256 threads: a launch has fewer than 2^32 in a dimension

bool aligned(const void* p, uintptr_t bytes) { return reinterpret_cast<uintptr_t>(p) % bytes == 0; }
bool float_type(int32_t t) { return t == GDN_F32 || t == GDN_BF16; }
int64_t size_of(int32_t t) { return t == GDN_F32 ? 4 : t == GDN_BF16 ? 2 : 1; }

// An address range; empty ones meet nothing.
struct Range {
  uintptr_t at;
  int64_t bytes;
};
Range range(const void* p, int64_t bytes) { return {reinterpret_cast<uintptr_t>(p), p ? bytes : 0}; }
Range rows(const void* p, int64_t n, int64_t stride, int64_t width, int64_t size) {
  return range(p, n > 0 ? ((n - 1) * stride + width) * size : 0);
}
bool meet(const Range& a, const Range& b) {
  return a.bytes > 0 && b.bytes > 0 && a.at < b.at + (uintptr_t)b.bytes && b.at < a.at + (uintptr_t)a.bytes;
}

constexpr int64_t kMostBytes = (int64_t)1 << 61;   // of an operand: extents must not wrap

// A row operand: aligned to its element, rows of at least `width`.
bool rows_ok(const void* p, int64_t n, int64_t stride, int64_t width, int64_t size) {
  return aligned(p, size) && stride >= width && stride <= (int64_t)1 << 40 && n <= INT32_MAX &&
         stride <= kMostBytes / ((n > 0 ? n : 1) * size);
}

// Descriptor of a scan or update; need receives the workspace bytes with which a scan's sequences are cut.
int plan_selective(const gdn_selective_args* a, bool update, gdn::SelectiveLaunch& p, int64_t& need) {
  need = 0;
  if (!a) return GDN_E_NULL;
  if (!float_type(a->in_dtype) || !float_type(a->out_dtype)) return GDN_E_DTYPE;
  if (a->N < 0 || a->T < 0 || a->T > INT32_MAX || a->G <= 0 || a->D <= 0 || a->D > 1 << 24 || a->D % a->G != 0 ||
      a->num_slots < 0 || a->max_seqlen < 0 || (update && a->T != a->N))
    return GDN_E_SHAPE;
  if (a->states != 8 && a->states != 16 && a->states != 32 && a->states != 64 && a->states != 128) return GDN_E_UNSUPPORTED;
  if (!a->A || !a->pool) return GDN_E_NULL;
  if (a->N > 0 && (!a->slot || (!update && !a->cu_seqlens))) return GDN_E_NULL;
  if (a->T > 0 && (!a->x || !a->dt || !a->B || !a->C || !a->out)) return GDN_E_NULL;
  const int64_t in = size_of(a->in_dtype), out = size_of(a->out_dtype), bc = (int64_t)a->G * a->states;
  if (!rows_ok(a->x, a->T, a->x_stride, a->D, in) || !rows_ok(a->dt, a->T, a->dt_stride, a->D, in) ||
      !rows_ok(a->B, a->T, a->B_stride, bc, in) || !rows_ok(a->C, a->T, a->C_stride, bc, in) ||
      (a->z && !rows_ok(a->z, a->T, a->z_stride, a->D, in)) || !rows_ok(a->out, a->T, a->out_stride, a->D, out))
    return GDN_E_SHAPE;
  if (a->num_slots > kMostBytes / (a->D * a->states * 4)) return GDN_E_SHAPE;
  if (!aligned(a->A, 16) || !aligned(a->pool, 16) || !aligned(a->D_skip, 4) || !aligned(a->dt_bias, 4) || !aligned(a->slot, 4) ||
      (!update && (!aligned(a->cu_seqlens, 4) || !aligned(a->has_init, 4))))
    return GDN_E_SHAPE;
  const Range o = rows(a->out, a->T, a->out_stride, a->D, out);
  const Range pool = range(a->pool, a->num_slots * a->D * a->states * 4);
  if (meet(o, rows(a->x, a->T, a->x_stride, a->D, in)) || meet(o, rows(a->dt, a->T, a->dt_stride, a->D, in)) ||
      meet(o, rows(a->B, a->T, a->B_stride, bc, in)) || meet(o, rows(a->C, a->T, a->C_stride, bc, in)) ||
      meet(o, rows(a->z, a->T, a->z_stride, a->D, in)) || meet(o, pool))
    return GDN_E_SHAPE;
  const int64_t dg = a->D / a->G;
  // (the scan's workgroups have up to 512 threads, 64 channels each; the update's 1024 / states channels)
  const int64_t per = update ? 1024 / a->states : 64;
  if ((dg + per - 1) / per * a->G * a->N > kMaxGrid / 2) return GDN_E_UNSUPPORTED;
  p.N = a->N;
  p.G = a->G;
  p.T = a->T;
  p.D = a->D;
  p.states = a->states;
  p.softplus_on = a->dt_softplus != 0;
  p.in_bf16 = a->in_dtype == GDN_BF16;
  p.out_bf16 = a->out_dtype == GDN_BF16;
  p.x = a->x;
  p.x_stride = a->x_stride;
  p.dt = a->dt;
  p.dt_stride = a->dt_stride;
  p.B = a->B;
  p.B_stride = a->B_stride;
  p.C = a->C;
  p.C_stride = a->C_stride;
  p.z = a->z;
  p.z_stride = a->z_stride;
  p.A = a->A;
  p.D_skip = a->D_skip;
  p.dt_bias = a->dt_bias;
  p.cu = a->cu_seqlens;
  p.slot = a->slot;
  p.has_init = a->has_init;
  p.pool = a->pool;
  p.out = a->out;
  p.out_stride = a->out_stride;
  p.keep_pool = a->keep_pool != 0;
  p.segs = 1;
  if (update || a->N == 0) return GDN_OK;
  // (without a hint: four times the average, which ragged batches seldom exceed by much)
  int64_t longest = a->max_seqlen > 0 ? a->max_seqlen : (a->T + a->N - 1) / a->N * 4;
  gdn::plan_selective_scan(p, longest < a->T ? longest : a->T, gdn::current_device_cus());
  if (p.segs == 1) return GDN_OK;
  if ((dg + 63) / 64 * a->G * a->N * p.segs > kMaxGrid / 2) {
    p.segs = 1;
    return GDN_OK;
  }
  const int64_t rows = (2 * (a->T / p.seg_len) + 1) * a->D, states = rows * a->states * 4;   // (a multiple of 32 bytes)
  p.seg_state = static_cast<float*>(a->workspace);
  p.seg_delta = reinterpret_cast<float*>(reinterpret_cast<uintptr_t>(a->workspace) + states);
  need = states + rows * 4;
  return GDN_OK;
}

int plan_norm(const gdn_rms_norm_args* a, gdn::NormLaunch& p) {
  if (!a) return GDN_E_NULL;
  const bool e4m3 = a->out_dtype == GDN_E4M3;
  if (!float_type(a->in_dtype) || (!float_type(a->out_dtype) && !e4m3) || (a->weight && !float_type(a->weight_dtype)) ||
      (a->residual && !float_type(a->residual_dtype)))
    return GDN_E_DTYPE;
  if (a->T < 0 || a->T > INT32_MAX || a->H <= 0 || a->H > 8192 || a->d <= 0 || (int64_t)a->H * a->d > 1 << 20) return GDN_E_SHAPE;
  if (!(a->eps >= 0.0f) || !std::isfinite(a->eps) || !std::isfinite(a->offset)) return GDN_E_SHAPE;
  if (a->group != 0 && a->group != 64 && a->group != 128) return GDN_E_UNSUPPORTED;
  if (a->gate && a->residual) return GDN_E_UNSUPPORTED;
  if (a->T > 0 && (!a->x || !a->out || (e4m3 && !a->scale))) return GDN_E_NULL;
  const int64_t in = size_of(a->in_dtype), out = size_of(a->out_dtype), res = size_of(a->residual_dtype);
  const int64_t w = (int64_t)a->H * a->d;
  if (!rows_ok(a->x, a->T, a->x_stride, w, in) || (a->gate && !rows_ok(a->gate, a->T, a->gate_stride, w, in)) ||
      (a->residual && !rows_ok(a->residual, a->T, a->residual_stride, w, res)) ||
      !rows_ok(a->out, a->T, a->out_stride, w, out) || (a->weight && !aligned(a->weight, size_of(a->weight_dtype))) ||
      (e4m3 && !aligned(a->scale, 4)))
    return GDN_E_SHAPE;
  p.H = a->H;
  p.d = a->d;
  if (a->T > gdn::most_rms_norm_rows(p)) return GDN_E_UNSUPPORTED;
  p.group = a->group ? a->group : (int)w;
  p.groups = (int)((w + p.group - 1) / p.group);
  const Range written[3] = {rows(a->out, a->T, a->out_stride, w, out), rows(a->residual, a->T, a->residual_stride, w, res),
                            range(e4m3 ? a->scale : nullptr, a->T * p.groups * 4)};
  const Range read[3] = {rows(a->x, a->T, a->x_stride, w, in), rows(a->gate, a->T, a->gate_stride, w, in),
                         range(a->weight, a->weight ? a->d * size_of(a->weight_dtype) : 0)};
  for (int i = 0; i < 3; ++i) {
    for (int j = 0; j < 3; ++j)
      if (meet(written[i], read[j]) || (j < i && meet(written[i], written[j]))) return GDN_E_SHAPE;
  }
  p.T = a->T;
  p.in_bf16 = a->in_dtype == GDN_BF16;
  p.weight_bf16 = a->weight_dtype == GDN_BF16;
  p.residual_bf16 = a->residual_dtype == GDN_BF16;
  p.out_dtype = a->out_dtype;
  p.x = a->x;
  p.x_stride = a->x_stride;
  p.gate = a->gate;
  p.gate_stride = a->gate_stride;
  p.residual = a->residual;
  p.residual_stride = a->residual_stride;
  p.weight = a->weight;
  p.out = a->out;
  p.out_stride = a->out_stride;
  p.scale = a->scale;
  p.eps = a->eps;
  p.offset = a->offset;
  p.gate_first = a->gate_first != 0;
  return GDN_OK;
}

// The pool and block table of a pages call.
int check_pages(const int32_t* pool, int64_t capacity, int32_t N, int32_t page, const int32_t* table, int64_t stride,
                int32_t width) {
  if (capacity < 0 || capacity > INT32_MAX - 2 || N < 0 || N > 65535 || page <= 0 || page > 1 << 30 || width <= 0 ||
      stride < width || stride > (int64_t)1 << 40)
    return GDN_E_SHAPE;
  if (!pool || (N > 0 && !table)) return GDN_E_NULL;
  return aligned(pool, 4) && aligned(table, 4) ? GDN_OK : GDN_E_SHAPE;
}

}  // namespace

extern "C" {

int64_t gdn_selective_scan_workspace_size(const gdn_selective_args* a) {
  gdn::SelectiveLaunch p{};
  int64_t need = 0;
  const int st = plan_selective(a, false, p, need);
  return st == GDN_OK ? need : -(int64_t)st;
}

int gdn_selective_scan(const gdn_selective_args* a, void* stream) {
  gdn::SelectiveLaunch p{};
  int64_t need = 0;
  const int st = plan_selective(a, false, p, need);
  if (st != GDN_OK || a->N == 0) return st;
  if (!a->workspace) p.segs = 1;
  else if (need > 0 && (a->workspace_bytes < need || !aligned(a->workspace, 256))) return GDN_E_SHAPE;
  return gdn::status_of_hip(gdn::launch_selective_scan(p, (hipStream_t)stream));
}

int gdn_selective_update(const gdn_selective_args* a, void* stream) {
  gdn::SelectiveLaunch p{};
  int64_t need = 0;
  const int st = plan_selective(a, true, p, need);
  if (st != GDN_OK || a->N == 0) return st;
  return gdn::status_of_hip(gdn::launch_selective_update(p, (hipStream_t)stream));
}

int gdn_rms_norm(const gdn_rms_norm_args* a, void* stream) {
  gdn::NormLaunch p{};
  const int st = plan_norm(a, p);
  if (st != GDN_OK || a->T == 0) return st;
  return gdn::status_of_hip(gdn::launch_rms_norm(p, (hipStream_t)stream));
}

int gdn_plan_pages(const gdn_plan_pages_args* a, void* stream) {
  if (!a) return GDN_E_NULL;
  int st = check_pages(a->pool, a->capacity, a->N, a->page, a->block_table, a->table_stride, a->table_width);
  if (st != GDN_OK) return st;
  if (a->T < 0 || a->T > INT32_MAX) return GDN_E_SHAPE;
  if (!a->cu_seqlens || (a->N > 0 && (!a->held || !a->new_len || !a->cache_len || !a->kv_len))) return GDN_E_NULL;
  if (!aligned(a->held, 4) || !aligned(a->new_len, 4) || !aligned(a->start, 4) || !aligned(a->cu_seqlens, 4) ||
      !aligned(a->cache_len, 4) || !aligned(a->kv_len, 4) || !aligned(a->slots, 8) || !aligned(a->positions, 4) ||
      !aligned(a->seq, 4))
    return GDN_E_SHAPE;
  const int64_t n = a->N;
  const Range all[] = {range(a->pool, (a->capacity + 2) * 4), rows(a->block_table, n, a->table_stride, a->table_width, 4),
                       range(a->cu_seqlens, (n + 1) * 4), range(a->cache_len, n * 4), range(a->kv_len, n * 4),
                       range(a->slots, a->T * 8), range(a->positions, a->T * 4), range(a->seq, a->T * 4),
                       range(a->held, n * 4), range(a->new_len, n * 4), range(a->start, n * 4)};
  for (int i = 0; i < 8; ++i)      // what is written meets nothing else
    for (int j = i + 1; j < 11; ++j)
      if (meet(all[i], all[j])) return GDN_E_SHAPE;
  gdn::PlanPagesLaunch p{a->pool, a->capacity, a->N, a->page, a->T, a->held, a->new_len, a->start, a->block_table,
                         a->table_stride, a->table_width, a->cu_seqlens, a->cache_len, a->kv_len, a->slots, a->positions,
                         a->seq};
  return gdn::status_of_hip(gdn::launch_plan_pages(p, (hipStream_t)stream));
}

int gdn_release_pages(const gdn_release_pages_args* a, void* stream) {
  if (!a) return GDN_E_NULL;
  int st = check_pages(a->pool, a->capacity, a->N, a->page, a->block_table, a->table_stride, a->table_width);
  if (st != GDN_OK) return st;
  if (a->N == 0) return GDN_OK;
  if (!a->keep || !a->held) return GDN_E_NULL;
  if (!aligned(a->keep, 4) || !aligned(a->held, 4)) return GDN_E_SHAPE;
  const Range pool = range(a->pool, (a->capacity + 2) * 4);
  if (meet(pool, rows(a->block_table, a->N, a->table_stride, a->table_width, 4)) || meet(pool, range(a->keep, a->N * 4)) ||
      meet(pool, range(a->held, a->N * 4)))
    return GDN_E_SHAPE;
  gdn::ReleasePagesLaunch p{a->pool, a->capacity, a->N, a->page, a->keep, a->held, a->block_table, a->table_stride,
                            a->table_width};
  return gdn::status_of_hip(gdn::launch_release_pages(p, (hipStream_t)stream));
}

}  // extern "C"
