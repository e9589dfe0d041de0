// Writing and thinning of the paged 8-bit key/value cache: gdn_kv_store, gdn_kv_evict.
//
// Store: value = code * 2^e with one e per (page, kv head).  One workgroup per (page that a
// sequence touches, kv head, K or V) reads the new rows once into registers, takes their
// largest finite magnitude as an integer maximum over the bf16 bits, and writes codes and
// scale; where an older scale grows, the page's earlier codes are read and rounded again
// first.  No atomics and no second pass over the input: bound by HBM (2 bytes read and 1
// written per element; 8 x 4096 tokens, 8 heads of 128: 36 us, 5.6 TB/s; one token for each of
// 256 sequences onto held pages 7 us, 16 where 3 scales of 10 grow and nothing is in a cache).
//
// Evict: a kv head's rows are ranked by (newest, weight, row).  One workgroup per
// (sequence, kv head) finds the budget-th largest key by radix selection and lists, in row
// order, the dropped rows before `budget` and the kept rows behind it; the second launch
// moves row by row, one workgroup per page that receives any.  Sources lie at or past
// `budget`, destinations before it, so the moves need no order; the sources' scales are
// taken by the first launch, since a page across `budget` may change its own.  32 sequences
// of 8192 rows to 4096, 8 heads of 128: 21 us to choose, 94 to move 290 MB of rows in random
// order and to round again the rows of pages whose scale grows (200 MB); 66 where none grows.
#include "attn_common.h"

namespace gdn {
namespace {

constexpr int kStoreThreads = 256;

// The page of a store slot: rows [r0, r1) of it are new, its row 0 is (or would be) token
// tok0.  Sequence n has the slots floor(cu[n] / page) + 2 n + j for its j-th touched page: it
// touches at most floor(L / page) + 2, so slots of different sequences never meet and no
// prefix pass is needed.  False: nothing to do.
struct StoreSlot {
  int n, id, r0, r1, old;
  int64_t first, tok0;
};
__device__ __forceinline__ bool store_slot(const StoreLaunch& p, int w, int lane, StoreSlot& s) {
  const int lg = p.c.page_log2, page = 1 << lg;
  int j = 0, t0 = w, len = 1;
  s.n = w;
  if (p.cu) {
    s.n = find_last(p.N, lane, [&](int i) { return (p.cu[i] >> lg) + 2 * i <= w; });
    t0 = p.cu[s.n];
    len = p.cu[s.n + 1] - t0;
    j = w - ((t0 >> lg) + 2 * s.n);
  }
  s.old = p.cache_len[s.n];
  if (s.old < 0 || len <= 0 || j < 0) return false;
  s.first = ((int64_t)(s.old >> lg) + j) << lg;                    // the page's first row
  const int64_t end = (int64_t)s.old + len;
  if (s.first >= end || s.first > INT32_MAX - page) return false;
  s.r0 = s.old > s.first ? (int)(s.old - s.first) : 0;
  s.r1 = end - s.first < page ? (int)(end - s.first) : page;
  s.id = page_of(p.c, s.n, (int)s.first);
  s.tok0 = (int64_t)t0 + (s.first - s.old);
  return s.id >= 0;
}
// largest finite magnitude bits of eight bf16, NaN and infinities left out
__device__ __forceinline__ unsigned top_of(const u32x4& x, unsigned top) {
#pragma unroll
  for (int e = 0; e < 4; ++e) {
    const unsigned a = x[e] & 0x7fff, b = x[e] >> 16 & 0x7fff;
    top = max(top, max(a < 0x7f80 ? a : 0u, b < 0x7f80 ? b : 0u));
  }
  return top;
}
// eight bf16 as codes; NaN and infinities become NaN
__device__ __forceinline__ uint2 codes_of(const u32x4& x, float inv) {
  float f[8];
#pragma unroll
  for (int q = 0; q < 4; ++q) {
    f[2 * q] = bf_lo(x[q]);
    f[2 * q + 1] = bf_hi(x[q]);
  }
#pragma unroll
  for (int q = 0; q < 8; ++q)
    f[q] = (__float_as_uint(f[q]) & 0x7f800000u) == 0x7f800000u ? __uint_as_float(0x7fc00000u) : f[q] * inv;
  return make_uint2(to_f8x4(f[0], f[1], f[2], f[3]), to_f8x4(f[4], f[5], f[6], f[7]));
}
__device__ __forceinline__ void store_track(const StoreLaunch& p, const StoreSlot& s, int64_t row0, int r) {
  if (p.c.pos) p.c.pos[row0 + r] = (p.start ? p.start[s.n] : s.old) + (int)(s.first + r - s.old);
  if (p.c.weight) p.c.weight[row0 + r] = 0.f;
}

// NP: passes of 256 threads over a page's 16-byte (8 element) pieces, page * d / 8 / 256.
template <int D, int NP>
__global__ void __launch_bounds__(kStoreThreads) kv_store_kernel(const StoreLaunch p) {
  constexpr int kPer = D / 8;                       // pieces of a row
  __shared__ unsigned sTop[kStoreThreads / kWave];
  const int tid = threadIdx.x, h = blockIdx.y, isv = blockIdx.z;
  StoreSlot st;
  if (!store_slot(p, blockIdx.x, tid & 63, st)) return;
  const int r0 = st.r0, r1 = st.r1, id = st.id;
  const int64_t tok0 = st.tok0;
  const int64_t row0 = page_rows(p.c, id, h);
  const u16* src = isv ? p.v : p.k;
  const int64_t stride = isv ? p.v_stride : p.k_stride;
  uint8_t* codes = (isv ? p.c.v : p.c.k) + row0 * D;
  float* scale_at = (isv ? p.c.v_scale : p.c.k_scale) + (int64_t)id * p.c.H_kv + h;

  u32x4 x[NP];
  unsigned top = 0;
#pragma unroll
  for (int s = 0; s < NP; ++s) {
    const int i = tid + s * kStoreThreads, r = i / kPer, c = i % kPer;
    x[s] = u32x4{0, 0, 0, 0};
    if (r >= r0 && r < r1)
      x[s] = __builtin_nontemporal_load(reinterpret_cast<const u32x4*>(src + (tok0 + r) * stride + (int64_t)h * D + c * 8));
  }
#pragma unroll
  for (int s = 0; s < NP; ++s) top = top_of(x[s], top);
#pragma unroll
  for (int o = 32; o; o >>= 1) top = max(top, (unsigned)__shfl_xor((int)top, o, kWave));
  if ((tid & 63) == 0) sTop[tid >> 6] = top;
  const float was = r0 ? *scale_at : 0.f;
  __syncthreads();                                  // (also: every thread has read the old scale)
  top = max(max(sTop[0], sTop[1]), max(sTop[2], sTop[3]));
  int e = scale_exp_of(top);
  if (r0) {
    const int eo = min(exp_of(was), 120);
    if (e > eo) {                                   // the scale grows: round the earlier rows to it
      const float shrink = ldexpf(1.0f, eo - e);
#pragma unroll
      for (int s = 0; s < NP; ++s) {
        const int i = tid + s * kStoreThreads, r = i / kPer, c = i % kPer;
        if (r < r0) {
          uint2* at = reinterpret_cast<uint2*>(codes + (int64_t)r * D + c * 8);
          const uint2 w = *at;
          *at = make_uint2(f8x4_rescale(w.x, shrink), f8x4_rescale(w.y, shrink));
        }
      }
    }
    e = max(e, eo);
  }
  if (tid == 0) *scale_at = exp2_int(e);
  const float inv = exp2_int(-e);                   // e in [-64, 120]
#pragma unroll
  for (int s = 0; s < NP; ++s) {
    const int i = tid + s * kStoreThreads, r = i / kPer, c = i % kPer;
    if (r >= r0 && r < r1) *reinterpret_cast<uint2*>(codes + (int64_t)r * D + c * 8) = codes_of(x[s], inv);
  }
  if (!isv && tid >= r0 && tid < r1) store_track(p, st, row0, tid);
}

// The same for a few tokens per sequence (decode steps, verify batches): a wave per (page, kv
// head, K or V), four to a workgroup; the new rows' first 64 pieces stay in registers, more
// are read twice.
template <int D>
__global__ void __launch_bounds__(kStoreThreads) kv_store_few_kernel(const StoreLaunch p, int64_t items) {
  constexpr int kPer = D / 8;
  const int lane = threadIdx.x & 63;
  const int64_t item = (int64_t)blockIdx.x * (kStoreThreads / kWave) + __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
  if (item >= items) return;
  const int isv = item & 1, h = (int)((item >> 1) % p.c.H_kv);
  StoreSlot st;
  if (!store_slot(p, (int)((item >> 1) / p.c.H_kv), lane, st)) return;
  const int64_t row0 = page_rows(p.c, st.id, h);
  const int64_t stride = isv ? p.v_stride : p.k_stride;
  const u16* src = (isv ? p.v : p.k) + (st.tok0 + st.r0) * stride + (int64_t)h * D;
  uint8_t* codes = (isv ? p.c.v : p.c.k) + row0 * D;
  float* scale_at = (isv ? p.c.v_scale : p.c.k_scale) + (int64_t)st.id * p.c.H_kv + h;
  const float was = st.r0 ? *scale_at : 0.f;
  const int count = (st.r1 - st.r0) * kPer;
  auto piece = [&](int i) __attribute__((always_inline)) {
    return *reinterpret_cast<const u32x4*>(src + (i / kPer) * stride + (i % kPer) * 8);
  };
  u32x4 x{0, 0, 0, 0};
  if (lane < count) x = piece(lane);
  unsigned top = top_of(x, 0);
  for (int i = lane + kWave; i < count; i += kWave) top = top_of(piece(i), top);
#pragma unroll
  for (int o = 32; o; o >>= 1) top = max(top, (unsigned)__shfl_xor((int)top, o, kWave));
  int e = scale_exp_of(top);
  if (st.r0) {
    const int eo = min(exp_of(was), 120);
    if (e > eo) {                                   // the scale grows: round the earlier rows to it
      const float shrink = ldexpf(1.0f, eo - e);
      for (int i = lane; i < st.r0 * kPer; i += kWave) {
        uint2* at = reinterpret_cast<uint2*>(codes) + i;
        const uint2 w = *at;
        *at = make_uint2(f8x4_rescale(w.x, shrink), f8x4_rescale(w.y, shrink));
      }
    }
    e = max(e, eo);
  }
  if (lane == 0) *scale_at = exp2_int(e);           // (read by every lane above)
  const float inv = exp2_int(-e);
  uint2* to = reinterpret_cast<uint2*>(codes + (int64_t)st.r0 * D);
  if (lane < count) to[lane] = codes_of(x, inv);
  for (int i = lane + kWave; i < count; i += kWave) to[i] = codes_of(piece(i), inv);
  if (!isv)
    for (int r = st.r0 + lane; r < st.r1; r += kWave) store_track(p, st, row0, r);
}

template <int D>
hipError_t store_by_page(const StoreLaunch& p, dim3 grid, hipStream_t s) {
  switch ((D / 8 << p.c.page_log2) / kStoreThreads) {
    case 0:
    case 1: kv_store_kernel<D, 1><<<grid, kStoreThreads, 0, s>>>(p); break;
    case 2: kv_store_kernel<D, 2><<<grid, kStoreThreads, 0, s>>>(p); break;
    case 4: kv_store_kernel<D, 4><<<grid, kStoreThreads, 0, s>>>(p); break;
    case 8: kv_store_kernel<D, 8><<<grid, kStoreThreads, 0, s>>>(p); break;
    default: kv_store_kernel<D, 16><<<grid, kStoreThreads, 0, s>>>(p); break;
  }
  return hipGetLastError();
}

// ------------------------------------------------------------------ evict
constexpr int kBins = 2048;
constexpr int kCopies = 4;

// Weight -> unsigned key of the same order: NaN below every number, -0 equal to +0, and
// 0xffffffff left for the newest rows.
__device__ __forceinline__ unsigned weight_key(float w) {
  if (w != w) return 0;
  const unsigned u = __float_as_uint(w + 0.0f);
  return (u >> 31 ? ~u : u | 0x80000000u);          // -inf -> 0x007fffff, +inf -> 0xff800000
}

__device__ __forceinline__ int wave_scan(int v) {   // inclusive
#pragma unroll
  for (int o = 1; o < kWave; o <<= 1) {
    const int u = __shfl_up(v, o, kWave);
    if ((threadIdx.x & 63) >= o) v += u;
  }
  return v;
}

// Exclusive sums over a workgroup of W waves of up to three counts per thread, and their
// totals; buf: [3][W].  Two barriers.
template <int W, int K>
__device__ __forceinline__ void group_scan(int (&v)[K], int (&total)[K], int (*buf)[W]) {
  const int lane = threadIdx.x & 63, wave = threadIdx.x >> 6;
  int inc[K];
#pragma unroll
  for (int k = 0; k < K; ++k) {
    inc[k] = wave_scan(v[k]);
    if (lane == 63) buf[k][wave] = inc[k];
  }
  __syncthreads();
#pragma unroll
  for (int k = 0; k < K; ++k) {
    const int s = wave_scan(lane < W ? buf[k][lane] : 0);       // every wave scans the waves' sums
    total[k] = __builtin_amdgcn_readlane(s, W - 1);
    const int before = __shfl(s, wave, kWave) - buf[k][wave];
    v[k] = before + inc[k] - v[k];
  }
  __syncthreads();
}

// A workgroup of T threads.  KG: groups of four rows that a thread holds in registers (the
// whole sequence: 4 T KG rows); 0: any length, rows are read again for every pass.
template <int T, int KG>
__global__ void __launch_bounds__(T) evict_select_kernel(const EvictLaunch p) {
  constexpr int kSelThreads = T, kSelWaves = T / kWave;
  __shared__ int sHist[kCopies][kBins];
  __shared__ int sWave[2][kSelWaves];
  __shared__ int sPick[2];
  const int tid = threadIdx.x, wave = tid >> 6, h = blockIdx.x, n = blockIdx.y;
  const int lg = p.c.page_log2;
  const int64_t cap = (int64_t)p.c.table_width << lg;
  const int len = (int)min((int64_t)p.kv_len[n], cap);
  const int64_t slot = (int64_t)n * p.c.H_kv + h;
  const int pages = (p.budget + (1 << lg) - 1) >> lg;
  int* first = p.first + slot * (pages + 1);
  if (len <= p.budget) {
    if (tid == 0) first[pages] = 0;                 // nothing to move
    return;
  }
  // Four rows (r0 .. r0 + 3, one page) at a time; a row's place is its row over the whole
  // cache (page id and row in it; -1: a bad page).
  struct Rows {
    int4 pos;
    f32x4 w;
    int at;
  };
  auto load = [&](int r0) __attribute__((always_inline)) {
    Rows x;
    const int id = r0 < len ? page_of(p.c, n, r0) : -1, r = r0 & ((1 << lg) - 1);
    x.at = id < 0 ? -1 : (id << lg) + r;
    const int64_t row = page_rows(p.c, max(id, 0), h) + r;
    x.pos = *reinterpret_cast<const int4*>(p.c.pos + row);
    x.w = *reinterpret_cast<const f32x4*>(p.c.weight + row);
    return x;
  };
  Rows held[KG ? KG : 1];
  const int steps = KG ? KG : (len + 4 * kSelThreads - 1) / (4 * kSelThreads);
  auto row_of = [&](int s) __attribute__((always_inline)) { return 4 * (s * kSelThreads + tid); };
  int last = INT32_MIN;
  bool ok = true;                                   // a sequence with a bad page is left as it is
  auto look = [&](const Rows& x, int r0) __attribute__((always_inline)) {
    ok = ok && (x.at >= 0 || r0 >= len);
    if (r0 < len) last = max(last, x.pos.x);
    if (r0 + 1 < len) last = max(last, x.pos.y);
    if (r0 + 2 < len) last = max(last, x.pos.z);
    if (r0 + 3 < len) last = max(last, x.pos.w);
  };
  if constexpr (KG > 0) {
#pragma unroll
    for (int s = 0; s < KG; ++s) held[s] = load(row_of(s));
#pragma unroll
    for (int s = 0; s < KG; ++s) look(held[s], row_of(s));
  } else {
    for (int s = 0; s < steps; ++s) look(load(row_of(s)), row_of(s));
  }
#pragma unroll
  for (int o = 32; o; o >>= 1) last = max(last, __shfl_xor(last, o, kWave));
  if ((tid & 63) == 0) sWave[0][wave] = last;
  if (!__syncthreads_and(ok)) {
    if (tid == 0) first[pages] = -1;                // left alone
    return;
  }
  for (int i = 0; i < kSelWaves; ++i) last = max(last, sWave[0][i]);
  const int64_t newest = (int64_t)last - p.recent;
  auto keys_of = [&](const Rows& x, unsigned (&k)[4]) __attribute__((always_inline)) {
    k[0] = x.pos.x > newest ? 0xffffffffu : weight_key(x.w[0]);
    k[1] = x.pos.y > newest ? 0xffffffffu : weight_key(x.w[1]);
    k[2] = x.pos.z > newest ? 0xffffffffu : weight_key(x.w[2]);
    k[3] = x.pos.w > newest ? 0xffffffffu : weight_key(x.w[3]);
  };
  unsigned kept_keys[KG ? KG : 1][4];
  if constexpr (KG > 0) {
#pragma unroll
    for (int s = 0; s < KG; ++s) keys_of(held[s], kept_keys[s]);
  }

  // Radix selection of the budget-th largest key: digits of 11, 11 and 10 bits.  `want` of
  // the keys that share the digits found so far are still to be kept.  (Weights crowd into a
  // few bins, and lanes that count into one wait for each other: neighbours use copies.)
  unsigned found = 0, mask = 0;
  int want = p.budget;
#pragma unroll 1
  for (int d = 0; d < 3; ++d) {
    const int shift = d == 0 ? 21 : d == 1 ? 10 : 0, bins = d == 2 ? 1024 : kBins;
    __syncthreads();
#pragma unroll
    for (int i = 0; i < kCopies * kBins / kSelThreads; ++i) (&sHist[0][0])[tid + i * kSelThreads] = 0;
    __syncthreads();
    auto count = [&](const unsigned (&k)[4], int r0) __attribute__((always_inline)) {
#pragma unroll
      for (int e = 0; e < 4; ++e)
        if (r0 + e < len && (k[e] & mask) == found) atomicAdd(&sHist[tid & (kCopies - 1)][k[e] >> shift & (bins - 1)], 1);
    };
    if constexpr (KG > 0) {
#pragma unroll
      for (int s = 0; s < KG; ++s) count(kept_keys[s], row_of(s));
    } else {
      for (int s = 0; s < steps; ++s)
        if (row_of(s) < len) {
          unsigned k[4];
          keys_of(load(row_of(s)), k);
          count(k, row_of(s));
        }
    }
    __syncthreads();
    // suffix sums: thread t owns the bins from kBins - 1 - kOwn t down, so a prefix scan over
    // the threads counts from the largest key down
    constexpr int kOwn = kBins / T;
    const int b1 = kBins - 1 - kOwn * tid;
    int c[kOwn], sum[1] = {0}, all[1];
#pragma unroll
    for (int b = 0; b < kOwn; ++b) {
      c[b] = 0;
#pragma unroll
      for (int i = 0; i < kCopies; ++i) c[b] += sHist[i][b1 - b];
      sum[0] += c[b];
    }
    group_scan<kSelWaves, 1>(sum, all, sWave);
    int before = sum[0];
#pragma unroll
    for (int b = 0; b < kOwn; ++b) {
      if (before < want && want <= before + c[b]) {
        sPick[0] = b1 - b;
        sPick[1] = want - before;
      }
      before += c[b];
    }
    __syncthreads();
    found |= (unsigned)sPick[0] << shift;
    mask |= (unsigned)(bins - 1) << shift;
    want = sPick[1];
  }

  // In row order: keep keys above `found` and the first `want` equal ones; list the
  // dropped rows before budget and the kept rows behind it.
  int* holes = p.holes + slot * p.budget;
  int* movers = p.movers + slot * p.budget;
  f32x2* scales = reinterpret_cast<f32x2*>(p.scales) + slot * p.budget;
  int equal0 = 0, hole0 = 0, mover0 = 0;
  auto list = [&](const unsigned (&k)[4], int r0, int at) __attribute__((always_inline)) {
    int eq = 0;
#pragma unroll
    for (int e = 0; e < 4; ++e) eq += r0 + e < len && k[e] == found;
    int rk[1] = {eq}, eqs[1];
    group_scan<kSelWaves, 1>(rk, eqs, sWave);
    int rank = equal0 + rk[0];
    equal0 += eqs[0];
    bool hole[4], mover[4];
    int nh = 0, nm = 0;
#pragma unroll
    for (int e = 0; e < 4; ++e) {
      const int r = r0 + e;
      const bool in = r < len, same = in && k[e] == found;
      const bool keep = in && (k[e] > found || (same && rank < want));
      rank += same;
      hole[e] = in && r < p.budget && !keep;
      mover[e] = keep && r >= p.budget;
      nh += hole[e];
      nm += mover[e];
    }
    int at2[2] = {nh, nm}, sums[2];
    group_scan<kSelWaves, 2>(at2, sums, sWave);
    int hb = hole0 + at2[0], mb = mover0 + at2[1];
    hole0 += sums[0];
    mover0 += sums[1];
    if (r0 < p.budget && (r0 & ((1 << lg) - 1)) == 0) first[r0 >> lg] = hb;
    f32x2 sc{0.f, 0.f};
    if (nm) {
      const int64_t pg = (int64_t)(at >> lg) * p.c.H_kv + h;
      sc = f32x2{p.c.k_scale[pg], p.c.v_scale[pg]};
    }
#pragma unroll
    for (int e = 0; e < 4; ++e) {
      if (hole[e]) holes[hb++] = r0 + e;
      if (mover[e]) {
        movers[mb] = at + e;
        scales[mb++] = sc;
      }
    }
  };
  if constexpr (KG > 0) {
#pragma unroll
    for (int s = 0; s < KG; ++s)
      if (4 * s * kSelThreads < len) list(kept_keys[s], row_of(s), held[s].at);
  } else {
    for (int s = 0; s < steps; ++s) {
      unsigned k[4];
      const Rows x = load(row_of(s));
      keys_of(x, k);
      list(k, row_of(s), x.at);
    }
  }
  if (tid == 0) first[pages] = hole0;               // = mover0: budget rows are kept in all
}

template <int D>
__global__ void __launch_bounds__(256) evict_move_kernel(const EvictLaunch p) {
  __shared__ int sE[2][4];
  __shared__ unsigned sHole[4];                     // the page's rows that are filled
  const int tid = threadIdx.x, j = blockIdx.x, h = blockIdx.y, n = blockIdx.z;
  const int lg = p.c.page_log2, page = 1 << lg, pages = (p.budget + page - 1) >> lg;
  const int64_t slot = (int64_t)n * p.c.H_kv + h;
  const int* first = p.first + slot * (pages + 1);
  const int total = first[pages];
  if (j == 0 && h == 0 && tid == 0) {
    const int len = p.kv_len[n];
    p.new_len[n] = total >= 0 ? min(len, p.budget) : len;
  }
  if (total <= 0) return;
  const int a = first[j], b = j + 1 < pages ? first[j + 1] : total;
  if (a >= b) return;
  constexpr int kPer = D / 16;                      // 16-byte pieces of a row
  constexpr int kRows = 256 / kPer;                 // rows that the threads take at a time
  const int64_t to = page_of(p.c, n, j << lg) * (int64_t)p.c.H_kv + h;   // (the first launch checked the pages)
  const int* holes = p.holes + slot * p.budget;
  const int* movers = p.movers + slot * p.budget;
  const f32x2* scales = reinterpret_cast<const f32x2*>(p.scales) + slot * p.budget;
  const int c = tid % kPer;
  // This thread's piece of moved row m: all of a row's loads at once.
  struct Piece {
    uint4 k, v;
    int64_t from, dst;
    f32x2 s;
  };
  const int64_t row0 = to << lg;
  auto get = [&](int m) __attribute__((always_inline)) {
    Piece x;
    const int src = movers[m];
    x.s = scales[m];
    x.dst = row0 + (holes[m] & (page - 1));
    x.from = page_rows(p.c, src >> lg, h) + (src & (page - 1));
    x.k = *(reinterpret_cast<const uint4*>(p.c.k + x.from * D) + c);
    x.v = *(reinterpret_cast<const uint4*>(p.c.v + x.from * D) + c);
    return x;
  };
  Piece x;
  if (a + tid / kPer < b) x = get(a + tid / kPer);  // in flight while the scales are compared
  // the page's new scales
  const int ko = exp_of(p.c.k_scale[to]), vo = exp_of(p.c.v_scale[to]);
  int ke = ko, ve = vo;
  if (tid < 4) sHole[tid] = 0;
  __syncthreads();
  for (int i = a + tid; i < b; i += 256) {
    const f32x2 s = scales[i];
    ke = max(ke, exp_of(s.x));
    ve = max(ve, exp_of(s.y));
    const int r = holes[i] & (page - 1);
    atomicOr(&sHole[r >> 5], 1u << (r & 31));
  }
#pragma unroll
  for (int o = 32; o; o >>= 1) {
    ke = max(ke, __shfl_xor(ke, o, kWave));
    ve = max(ve, __shfl_xor(ve, o, kWave));
  }
  if ((tid & 63) == 0) {
    sE[0][tid >> 6] = ke;
    sE[1][tid >> 6] = ve;
  }
  __syncthreads();                                  // (and every thread has read the old scales)
  ke = max(max(sE[0][0], sE[0][1]), max(sE[0][2], sE[0][3]));
  ve = max(max(sE[1][0], sE[1][1]), max(sE[1][2], sE[1][3]));
  if (tid == 0) {
    p.c.k_scale[to] = exp2_int(ke);
    p.c.v_scale[to] = exp2_int(ve);
  }
  auto rescale = [](uint4 w, float f) __attribute__((always_inline)) {
    return make_uint4(f8x4_rescale(w.x, f), f8x4_rescale(w.y, f), f8x4_rescale(w.z, f), f8x4_rescale(w.w, f));
  };
  if (ke > ko || ve > vo) {                         // round the rows that stay to the new scales
    const int alive = min(page, p.budget - (j << lg));   // rows of the page before budget
    const float ks = ldexpf(1.0f, ko - ke), vs = ldexpf(1.0f, vo - ve);
    for (int r = tid / kPer; r < alive; r += kRows) {
      if (sHole[r >> 5] >> (r & 31) & 1) continue;
      uint4* kp = reinterpret_cast<uint4*>(p.c.k + (row0 + r) * D) + c;
      uint4* vp = reinterpret_cast<uint4*>(p.c.v + (row0 + r) * D) + c;
      if (ke > ko) *kp = rescale(*kp, ks);
      if (ve > vo) *vp = rescale(*vp, vs);
    }
  }
  for (int m = a + tid / kPer; m < b; m += kRows) {
    const int dk = exp_of(x.s.x) - ke, dv = exp_of(x.s.y) - ve;   // <= 0
    if (dk) x.k = rescale(x.k, ldexpf(1.0f, dk));
    if (dv) x.v = rescale(x.v, ldexpf(1.0f, dv));
    *(reinterpret_cast<uint4*>(p.c.k + x.dst * D) + c) = x.k;
    *(reinterpret_cast<uint4*>(p.c.v + x.dst * D) + c) = x.v;
    if (c == 0) {
      p.c.pos[x.dst] = p.c.pos[x.from];
      p.c.weight[x.dst] = p.c.weight[x.from];
    }
    if (m + kRows < b) x = get(m + kRows);
  }
}

}  // namespace

hipError_t launch_kv_store(const StoreLaunch& p, hipStream_t stream) {
  const int64_t slots = p.cu ? (p.T >> p.c.page_log2) + 2 * (int64_t)p.N : p.N;
  if (p.T <= kFewTokens * (int64_t)p.N) {
    const int64_t items = slots * p.c.H_kv * 2;
    const dim3 grid((unsigned)((items + kStoreThreads / kWave - 1) / (kStoreThreads / kWave)));
    switch (p.c.d) {
      case 64: kv_store_few_kernel<64><<<grid, kStoreThreads, 0, stream>>>(p, items); break;
      case 128: kv_store_few_kernel<128><<<grid, kStoreThreads, 0, stream>>>(p, items); break;
      default: kv_store_few_kernel<256><<<grid, kStoreThreads, 0, stream>>>(p, items); break;
    }
    return hipGetLastError();
  }
  const dim3 grid((unsigned)slots, (unsigned)p.c.H_kv, 2);
  switch (p.c.d) {
    case 64: return store_by_page<64>(p, grid, stream);
    case 128: return store_by_page<128>(p, grid, stream);
    default: return store_by_page<256>(p, grid, stream);
  }
}

hipError_t launch_kv_evict(const EvictLaunch& p, hipStream_t stream) {
  const dim3 heads((unsigned)p.c.H_kv, (unsigned)p.N);
  const int64_t rows = (int64_t)p.c.table_width << p.c.page_log2;   // the longest sequence
  // A small workgroup for few rows, since its barriers cost less (1000 rows: 256 threads 10.7
  // us, 1024 12.0), a large one for many (8192 rows, the whole call: 1024 threads 99 us, 512
  // 101, 256 112); as many keys per thread as keep a sequence in registers.
  if (rows <= 1024) evict_select_kernel<256, 1><<<heads, 256, 0, stream>>>(p);
  else if (rows <= 2048) evict_select_kernel<256, 2><<<heads, 256, 0, stream>>>(p);
  else if (rows <= 8192) evict_select_kernel<1024, 2><<<heads, 1024, 0, stream>>>(p);
  else if (rows <= 16384) evict_select_kernel<1024, 4><<<heads, 1024, 0, stream>>>(p);
  else evict_select_kernel<1024, 0><<<heads, 1024, 0, stream>>>(p);
  hipError_t e = hipGetLastError();
  if (e != hipSuccess) return e;
  const unsigned pages = (unsigned)(((int64_t)p.budget + (1 << p.c.page_log2) - 1) >> p.c.page_log2);
  const dim3 grid(pages, (unsigned)p.c.H_kv, (unsigned)p.N);
  switch (p.c.d) {
    case 64: evict_move_kernel<64><<<grid, 256, 0, stream>>>(p); break;
    case 128: evict_move_kernel<128><<<grid, 256, 0, stream>>>(p); break;
    default: evict_move_kernel<256><<<grid, 256, 0, stream>>>(p); break;
  }
  return hipGetLastError();
}

}  // namespace gdn
