// Writing and thinning of the paged 8-bit key/value cache: gdn_kv_store, gdn_kv_evict.
//
// Store: value = code * 2^e with one e per (page, kv head).  One workgroup per (page that a
// sequence touches, kv head, K or V) reads the new rows once into registers, takes their
// largest finite magnitude as an integer maximum over the bf16 bits, and writes codes and
// scale; where an older scale grows, the page's earlier codes are read and rounded again
// first.  No atomics and no second pass over the input: bound by HBM (2 bytes read and 1
// written per element).
//
// Evict: a kv head's rows are ranked by (newest, weight, row).  One workgroup per
// (sequence, kv head) finds the budget-th largest key by radix selection and lists, in row
// order, the dropped rows before `budget` and the kept rows behind it; the second launch
// moves row by row, one workgroup per page that receives any.  Sources lie at or past
// `budget`, destinations before it, so the moves need no order; the sources' scales are
// taken by the first launch, since a page across `budget` may change its own.
#include "attn_common.h"

namespace gdn {
namespace {

constexpr int kStoreThreads = 256;

// NP: passes of 256 threads over a page's 16-byte (8 element) pieces, page * d / 8 / 256.
template <int D, int NP>
__global__ void __launch_bounds__(kStoreThreads) kv_store_kernel(const StoreLaunch p) {
  constexpr int kPer = D / 8;                       // pieces of a row
  __shared__ unsigned sTop[kStoreThreads / kWave];
  const int tid = threadIdx.x, h = blockIdx.y, isv = blockIdx.z;
  const int lg = p.c.page_log2, page = 1 << lg;
  // block -> (sequence n, its j-th touched page).  Sequence n has the slots
  // floor(cu[n] / page) + 2 n + j: it touches at most floor(L / page) + 2 pages, so slots
  // of different sequences never meet and no prefix pass is needed.
  int n, j = 0, t0, len;
  if (p.cu == nullptr) {
    n = blockIdx.x;
    t0 = n;
    len = 1;
  } else {
    const int w = blockIdx.x;
    int lo = 0, hi = p.N;                           // largest n with slot0(n) <= w
    while (hi - lo > 1) {
      const int mid = (lo + hi) >> 1;
      if ((p.cu[mid] >> lg) + 2 * mid <= w) lo = mid; else hi = mid;
    }
    n = lo;
    t0 = p.cu[n];
    len = p.cu[n + 1] - t0;
    j = w - ((t0 >> lg) + 2 * n);
  }
  const int old = p.cache_len[n];
  if (old < 0 || len <= 0 || j < 0) return;
  const int64_t first = ((int64_t)(old >> lg) + j) << lg;          // the page's first row
  const int64_t end = (int64_t)old + len;
  if (first >= end || first > INT32_MAX - page) return;
  const int r0 = old > first ? (int)(old - first) : 0;             // new rows [r0, r1) of the page
  const int r1 = end - first < page ? (int)(end - first) : page;
  const int id = page_of(p.c, n, (int)first);
  if (id < 0) return;
  const int64_t row0 = page_rows(p.c, id, h);
  const int64_t tok0 = (int64_t)t0 + (first - old);                // token of the page's row 0
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
  for (int s = 0; s < NP; ++s)
#pragma unroll
    for (int e = 0; e < 4; ++e) {
      const unsigned a = x[s][e] & 0x7fff, b = x[s][e] >> 16 & 0x7fff;
      top = max(top, max(a < 0x7f80 ? a : 0u, b < 0x7f80 ? b : 0u));
    }
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
    if (r >= r0 && r < r1) {
      float f[8];
#pragma unroll
      for (int q = 0; q < 4; ++q) {
        f[2 * q] = bf_lo(x[s][q]);
        f[2 * q + 1] = bf_hi(x[s][q]);
      }
#pragma unroll
      for (int q = 0; q < 8; ++q)                   // NaN and infinities become NaN
        f[q] = (__float_as_uint(f[q]) & 0x7f800000u) == 0x7f800000u ? __uint_as_float(0x7fc00000u) : f[q] * inv;
      *reinterpret_cast<uint2*>(codes + (int64_t)r * D + c * 8) =
          make_uint2(to_f8x4(f[0], f[1], f[2], f[3]), to_f8x4(f[4], f[5], f[6], f[7]));
    }
  }
  if (!isv && tid < page && tid >= r0 && tid < r1) {
    if (p.c.pos) p.c.pos[row0 + tid] = (p.start ? p.start[n] : old) + (int)(first + tid - old);
    if (p.c.weight) p.c.weight[row0 + tid] = 0.f;
  }
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
constexpr int kSelThreads = 1024;
constexpr int kSelWaves = kSelThreads / kWave;
constexpr int kBins = 2048;

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

__global__ void __launch_bounds__(kSelThreads) evict_select_kernel(const EvictLaunch p) {
  __shared__ int sHist[kBins];
  __shared__ int sWave[3][kSelWaves];
  __shared__ int sPick[2];
  const int tid = threadIdx.x, wave = tid >> 6, h = blockIdx.x, n = blockIdx.y;
  const int lg = p.c.page_log2;
  const int64_t cap = (int64_t)p.c.table_width << lg;
  const int len = (int)min((int64_t)p.kv_len[n], cap);
  const int64_t slot = (int64_t)n * p.c.H_kv + h;
  const int pages = (p.budget + (1 << lg) - 1) >> lg;
  int* first = p.first + slot * (pages + 1);
  // pages all in range? (a sequence with a bad page is left as it is)
  bool ok = len > p.budget;
  if (ok)
    for (int j = tid; j << lg < len; j += kSelThreads) ok = ok && page_of(p.c, n, j << lg) >= 0;
  if (!__syncthreads_and(ok)) {
    if (tid == 0) first[pages] = len > p.budget ? -1 : 0;   // -1: left alone, 0: nothing to move
    return;
  }
  // Four rows (r0 .. r0 + 3, one page) at a time: their keys given the newest position.
  auto load = [&](int r0, int4& pos, f32x4& w, int64_t& row) __attribute__((always_inline)) {
    const int id = page_of(p.c, n, r0);
    row = page_rows(p.c, id, h) + (r0 & ((1 << lg) - 1));
    pos = *reinterpret_cast<const int4*>(p.c.pos + row);
    w = *reinterpret_cast<const f32x4*>(p.c.weight + row);
  };
  int last = INT32_MIN;
  for (int r0 = 4 * tid; r0 < len; r0 += 4 * kSelThreads) {
    int4 pos;
    f32x4 w;
    int64_t row;
    load(r0, pos, w, row);
    last = max(last, pos.x);
    if (r0 + 1 < len) last = max(last, pos.y);
    if (r0 + 2 < len) last = max(last, pos.z);
    if (r0 + 3 < len) last = max(last, pos.w);
  }
#pragma unroll
  for (int o = 32; o; o >>= 1) last = max(last, __shfl_xor(last, o, kWave));
  if ((tid & 63) == 0) sWave[0][wave] = last;
  __syncthreads();
  for (int i = 0; i < kSelWaves; ++i) last = max(last, sWave[0][i]);
  const int64_t newest = (int64_t)last - p.recent;
  auto keys = [&](int r0, unsigned (&k)[4]) __attribute__((always_inline)) {
    int4 pos;
    f32x4 w;
    int64_t row;
    load(r0, pos, w, row);
    k[0] = pos.x > newest ? 0xffffffffu : weight_key(w[0]);
    k[1] = pos.y > newest ? 0xffffffffu : weight_key(w[1]);
    k[2] = pos.z > newest ? 0xffffffffu : weight_key(w[2]);
    k[3] = pos.w > newest ? 0xffffffffu : weight_key(w[3]);
  };

  // Radix selection of the budget-th largest key: digits of 11, 11 and 10 bits.  `want` of
  // the keys that share the digits found so far are still to be kept.
  unsigned found = 0, mask = 0;
  int want = p.budget;
#pragma unroll 1
  for (int d = 0; d < 3; ++d) {
    const int shift = d == 0 ? 21 : d == 1 ? 10 : 0, bins = d == 2 ? 1024 : kBins;
    __syncthreads();
    for (int i = tid; i < kBins; i += kSelThreads) sHist[i] = 0;
    __syncthreads();
    for (int r0 = 4 * tid; r0 < len; r0 += 4 * kSelThreads) {
      unsigned k[4];
      keys(r0, k);
#pragma unroll
      for (int e = 0; e < 4; ++e)
        if (r0 + e < len && (k[e] & mask) == found) atomicAdd(&sHist[k[e] >> shift & (bins - 1)], 1);
    }
    __syncthreads();
    // suffix sums: thread t owns bins 2047 - 2 t and 2046 - 2 t, so a prefix scan over the
    // threads counts from the largest key down
    const int b1 = kBins - 1 - 2 * tid, c1 = sHist[b1], c0 = sHist[b1 - 1];
    const int inc = wave_scan(c1 + c0);
    if ((tid & 63) == 63) sWave[0][wave] = inc;
    __syncthreads();
    int before = inc - c1 - c0;
    for (int i = 0; i < wave; ++i) before += sWave[0][i];
    if (before < want && want <= before + c1) {
      sPick[0] = b1;
      sPick[1] = want - before;
    } else if (before + c1 < want && want <= before + c1 + c0) {
      sPick[0] = b1 - 1;
      sPick[1] = want - before - c1;
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
  for (int base = 0; base < len; base += 4 * kSelThreads) {
    const int r0 = base + 4 * tid;
    unsigned k[4] = {0, 0, 0, 0};
    int eq = 0;
    if (r0 < len) keys(r0, k);
#pragma unroll
    for (int e = 0; e < 4; ++e) eq += r0 + e < len && k[e] == found;
    const int eqi = wave_scan(eq);
    if ((tid & 63) == 63) sWave[0][wave] = eqi;
    __syncthreads();
    int rank = equal0 + eqi - eq;
    for (int i = 0; i < kSelWaves; ++i) {
      if (i < wave) rank += sWave[0][i];
      equal0 += sWave[0][i];
    }
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
    const int hi = wave_scan(nh), mi = wave_scan(nm);
    if ((tid & 63) == 63) {
      sWave[1][wave] = hi;
      sWave[2][wave] = mi;
    }
    __syncthreads();
    int hb = hole0 + hi - nh, mb = mover0 + mi - nm;
    for (int i = 0; i < kSelWaves; ++i) {
      if (i < wave) {
        hb += sWave[1][i];
        mb += sWave[2][i];
      }
      hole0 += sWave[1][i];
      mover0 += sWave[2][i];
    }
    if (r0 < p.budget && (r0 & ((1 << lg) - 1)) == 0) first[r0 >> lg] = hb;
    f32x2 sc{0.f, 0.f};
    if (nm) {
      const int64_t at = (int64_t)page_of(p.c, n, r0) * p.c.H_kv + h;
      sc = f32x2{p.c.k_scale[at], p.c.v_scale[at]};
    }
#pragma unroll
    for (int e = 0; e < 4; ++e) {
      if (hole[e]) holes[hb++] = r0 + e;
      if (mover[e]) {
        movers[mb] = r0 + e;
        scales[mb++] = sc;
      }
    }
    __syncthreads();                                // sWave is written again by the next rows
  }
  if (tid == 0) first[pages] = hole0;               // = mover0: budget rows are kept in all
}

template <int D>
__global__ void __launch_bounds__(256) evict_move_kernel(const EvictLaunch p) {
  __shared__ int sE[2][4];
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
  const int64_t to = page_of(p.c, n, j << lg) * (int64_t)p.c.H_kv + h;   // (the first launch checked the pages)
  const int* holes = p.holes + slot * p.budget;
  const int* movers = p.movers + slot * p.budget;
  const f32x2* scales = reinterpret_cast<const f32x2*>(p.scales) + slot * p.budget;
  // the page's new scales
  const int ko = exp_of(p.c.k_scale[to]), vo = exp_of(p.c.v_scale[to]);
  int ke = ko, ve = vo;
  for (int i = a + tid; i < b; i += 256) {
    const f32x2 s = scales[i];
    ke = max(ke, exp_of(s.x));
    ve = max(ve, exp_of(s.y));
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
  const int64_t row0 = to << lg;
  const int alive = min(page, p.budget - (j << lg));   // rows of the page before budget
  constexpr int kPer = D / 16;                      // 16-byte pieces of a row
  if (ke > ko || ve > vo) {
    const float ks = ldexpf(1.0f, ko - ke), vs = ldexpf(1.0f, vo - ve);
    for (int i = tid; i < alive * kPer; i += 256) {
      if (ke > ko) {
        uint4* at = reinterpret_cast<uint4*>(p.c.k + row0 * D) + i;
        const uint4 w = *at;
        *at = make_uint4(f8x4_rescale(w.x, ks), f8x4_rescale(w.y, ks), f8x4_rescale(w.z, ks), f8x4_rescale(w.w, ks));
      }
      if (ve > vo) {
        uint4* at = reinterpret_cast<uint4*>(p.c.v + row0 * D) + i;
        const uint4 w = *at;
        *at = make_uint4(f8x4_rescale(w.x, vs), f8x4_rescale(w.y, vs), f8x4_rescale(w.z, vs), f8x4_rescale(w.w, vs));
      }
    }
    __syncthreads();                                // the holes' old codes are written before the rows that fill them
  }
  for (int i = tid; i < (b - a) * kPer; i += 256) {
    const int m = a + i / kPer, c = i % kPer;
    const int src = movers[m];
    const int64_t from = page_rows(p.c, page_of(p.c, n, src), h) + (src & (page - 1));
    const int64_t dst = row0 + (holes[m] & (page - 1));
    const f32x2 s = scales[m];
    uint4 k = *(reinterpret_cast<const uint4*>(p.c.k + from * D) + c);
    uint4 v = *(reinterpret_cast<const uint4*>(p.c.v + from * D) + c);
    const int dk = exp_of(s.x) - ke, dv = exp_of(s.y) - ve;   // <= 0
    if (dk) {
      const float f = ldexpf(1.0f, dk);
      k = make_uint4(f8x4_rescale(k.x, f), f8x4_rescale(k.y, f), f8x4_rescale(k.z, f), f8x4_rescale(k.w, f));
    }
    if (dv) {
      const float f = ldexpf(1.0f, dv);
      v = make_uint4(f8x4_rescale(v.x, f), f8x4_rescale(v.y, f), f8x4_rescale(v.z, f), f8x4_rescale(v.w, f));
    }
    *(reinterpret_cast<uint4*>(p.c.k + dst * D) + c) = k;
    *(reinterpret_cast<uint4*>(p.c.v + dst * D) + c) = v;
    if (c == 0) {
      p.c.pos[dst] = p.c.pos[from];
      p.c.weight[dst] = p.c.weight[from];
    }
  }
}

}  // namespace

hipError_t launch_kv_store(const StoreLaunch& p, hipStream_t stream) {
  const int64_t slots = p.cu ? (p.T >> p.c.page_log2) + 2 * (int64_t)p.N : p.N;
  const dim3 grid((unsigned)slots, (unsigned)p.c.H_kv, 2);
  switch (p.c.d) {
    case 64: return store_by_page<64>(p, grid, stream);
    case 128: return store_by_page<128>(p, grid, stream);
    default: return store_by_page<256>(p, grid, stream);
  }
}

hipError_t launch_kv_evict(const EvictLaunch& p, hipStream_t stream) {
  evict_select_kernel<<<dim3((unsigned)p.c.H_kv, (unsigned)p.N), kSelThreads, 0, stream>>>(p);
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
