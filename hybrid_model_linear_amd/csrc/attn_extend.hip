// Attention of packed new tokens over their own keys and values and an optional cached
// 8-bit prefix (gdn_attn_extend).
//
//   o_i = sum_j p_ij v_j / sum_j p_ij,  p_ij = exp2(s_ij - m_i),  one pass with a running
//   maximum m and sum; s in units of log2, fp32.
//
// Bound by the matrix units (4 d flop per query head and visible pair; K and V are read
// from L2).  A workgroup takes 128 rows of one kv head: row f = token * G + g of the
// sequence's (token, query head of the group) pairs, G = H / H_kv, so the heads of a group
// share every K and V tile and short sequences still fill rows.  Each of its four waves
// owns 32 rows:
//   - S^T = K Q^T with 32x32x16 MFMA: a lane holds 32 of a 64-key tile's scores of one row
//     (lane % 32), so the softmax is lane-local but for one exchange of the two halves.
//   - O^T += V^T P^T: S^T's accumulator order is the B operand's once the 16 keys of a step
//     are taken as 8 (2 u + (e >> 2)) + 4 half + (e & 3), and V^T comes from the row-major V
//     tile by LDS transpose reads of 4 rows in that order.
// K and V tiles of 64 keys stand in LDS as bf16, double-buffered, their 16-byte pieces
// XOR-swizzled by row (operand and transpose reads without bank conflicts); the next
// tile's rows are loaded into registers while this one is computed.  Cached rows become
// bf16 times their page's power-of-two scale (exact) on the way into LDS.
// The weights are rounded to bf16 for the second product, their sum is not.
#include "attn_common.h"

namespace gdn {
namespace {

constexpr int kExtThreads = 256;
constexpr int kBM = 128;      // rows of a workgroup
constexpr int kBN = 64;       // keys of a tile
constexpr int kFlags = 4096;  // document mask: key tiles whose overlap is looked up ahead

// 16-byte piece c of row r of a [64][D] bf16 tile (element index).  Any 16 consecutive
// rows of one piece, and any 4-row group of 4 pieces, cover all banks.
template <int D>
__device__ __forceinline__ int tidx(int r, int c) {
  const int sw = D >= 128 ? ((r & 3) << 2 | (r >> 2 & 3)) : ((r >> 1 & 1) << 2 | (r >> 2 & 3));
  return r * D + ((c ^ sw) << 3);
}

struct ExtMask {                 // what decides whether row i sees key j (sequence-local tokens)
  int vis;                       // keys below are seen by every row (INT_MAX: not causal)
  int window;                    // 0: none
  const int32_t* doc;            // of the sequence's tokens, or null
};
__device__ __forceinline__ bool ext_seen(const ExtMask& k, int i, int j, int di, int dj) {
  bool ok = j <= i || j < k.vis;
  if (k.window > 0) ok = ok && abs(i - j) < k.window;
  if (k.doc) ok = ok && di == dj && di >= 0;
  return ok;
}

template <int D>
__global__ void __launch_bounds__(kExtThreads, D <= 128 ? 2 : 1) extend_kernel(const AttnExtendLaunch p) {
  constexpr int kU = D / 16;               // k steps of S^T
  constexpr int kDT = D / 32;              // 32-column tiles of O^T
  constexpr int kPc = D / 8;               // 16-byte pieces of a bf16 row
  constexpr int kSt = kBN * kPc / kExtThreads;   // pieces per thread of one tile (K or V)
  __shared__ __attribute__((aligned(16))) u16 sK[2][kBN * D], sV[2][kBN * D];
  __shared__ unsigned sFlag[kFlags / 16];  // 2 bits per key tile: overlaps, all one document
  __shared__ int sDoc[2];

  const int tid = threadIdx.x, wave = tid >> 6, lane = tid & 63, q32 = lane & 31, hh = lane >> 5;
  const int G = p.H / p.H_kv;
  // Heads fastest: consecutive workgroups go to the 8 XCDs in turn, so a head's tiles share
  // an L2.  Late tiles of a causal sequence see the most keys: they are launched first.
  const int h = blockIdx.x % p.H_kv;
  const int64_t w = (int64_t)(gridDim.x / p.H_kv) - 1 - blockIdx.x / p.H_kv;
  // slot w -> (sequence n, tile): sequence n's tiles begin at floor(cu[n] G / 128) + n
  int lo = 0, hi = p.N;
  while (hi - lo > 1) {
    const int mid = (lo + hi) >> 1;
    if ((int64_t)p.cu[mid] * G / kBM + mid <= w) lo = mid; else hi = mid;
  }
  const int n = lo, t0 = p.cu[n], L = p.cu[n + 1] - t0;
  const int64_t tile = w - ((int64_t)t0 * G / kBM + n);
  const int64_t f0 = tile * kBM;
  if (tile < 0 || f0 >= (int64_t)L * G) return;
  int P = p.cache_len ? p.cache_len[n] : 0;             // cached rows
  if (P < 0) return;
  const int start = p.start ? p.start[n] : P;           // position of token 0
  const int lg = p.c.page_log2;
  P = p.c.k ? (int)min((int64_t)P, (int64_t)p.c.table_width << lg) : 0;

  // this lane's row
  const int64_t f = f0 + wave * 32 + q32;
  const bool live = f < (int64_t)L * G;
  const int ti = live ? (int)(f / G) : L - 1, g = live ? (int)(f % G) : 0;
  const int hq = h * G + g;
  const int ta = (int)(f0 / G), tz = (int)(min(f0 + kBM - 1, (int64_t)L * G - 1) / G);   // the workgroup's tokens
  const int64_t fw = f0 + wave * 32;
  const int wa = (int)min(fw / G, (int64_t)L - 1), wz = (int)(min(fw + 31, (int64_t)L * G - 1) / G);   // the wave's

  ExtMask mk;
  mk.vis = p.causal ? (p.visible ? p.visible[n] : 0) : INT32_MAX;
  mk.window = p.window;
  mk.doc = p.doc ? p.doc + t0 : nullptr;
  const int di = mk.doc ? mk.doc[ti] : 0;

  bf16x8 q[kU];
#pragma unroll
  for (int u = 0; u < kU; ++u) {
    uint4 x = make_uint4(0, 0, 0, 0);
    if (live) x = *reinterpret_cast<const uint4*>(p.q + (int64_t)(t0 + ti) * p.q_stride + (int64_t)hq * D + 16 * u + 8 * hh);
    q[u] = as_bf16x8(x);
  }
  const float c1 = p.softcap > 0.f ? p.scale / p.softcap * 2.0f * kLog2e : p.scale * kLog2e;
  const float c2 = p.softcap * kLog2e;
  const float slope = p.slopes ? p.slopes[hq] * kLog2e : 0.f;

  // key tiles: cached ones, then the new tokens' [d0, d1)
  const int c1t = (P + kBN - 1) / kBN;
  int c0t = 0;
  if (p.window > 0 && !p.c.pos && P > 0) {              // cached rows a window leaves out of every row
    const int64_t first = (int64_t)start + ta - p.window + 1;
    c0t = (int)min((int64_t)c1t, max((int64_t)0, first) / kBN);
  }
  int last = min(L, max(tz + 1, min(mk.vis, L)));       // keys [first, last) are seen by some row
  int first = 0;
  if (p.window > 0) {
    first = (int)max((int64_t)0, (int64_t)ta - p.window + 1);
    last = (int)min((int64_t)last, (int64_t)tz + p.window);
  }
  const int d0 = first / kBN, d1 = (last + kBN - 1) / kBN;

  // Document mask: which key tiles hold a document of this workgroup's rows.
  if (mk.doc) {
    for (int i = tid; i < kFlags / 16; i += kExtThreads) sFlag[i] = 0;
    if (tid == 0) {
      sDoc[0] = INT32_MAX;
      sDoc[1] = -1;
    }
    __syncthreads();
    for (int t = ta + tid; t <= tz; t += kExtThreads) {
      const int d = mk.doc[t];
      atomicMin(&sDoc[0], d);
      atomicMax(&sDoc[1], d);
    }
    __syncthreads();
    const int dmin = sDoc[0], dmax = sDoc[1];
    for (int t = d0 + tid; t < min(d1, d0 + kFlags); t += kExtThreads) {
      bool any = false, all = dmin == dmax;
      for (int j = t * kBN; j < min(L, (t + 1) * kBN); ++j) {
        const int d = mk.doc[j];
        any = any || (d >= 0 && d >= dmin && d <= dmax);
        all = all && d == dmin && d >= 0;
      }
      atomicOr(&sFlag[(t - d0) >> 4], (any ? 1u : 0u) << 2 * ((t - d0) & 15) | (all ? 2u : 0u) << 2 * ((t - d0) & 15));
    }
    __syncthreads();
  }
  auto doc_flags = [&](int t) __attribute__((always_inline)) -> unsigned {
    return t - d0 < kFlags ? sFlag[(t - d0) >> 4] >> 2 * ((t - d0) & 15) & 3 : 1u;
  };
  // Tiles in order: x in [c0t, c1t) cached, then c1t + (t - d0).  The next tile at or after x.
  const int end = c1t + max(0, d1 - d0);
  auto skip = [&](int x) __attribute__((always_inline)) {
    if (mk.doc)
      while (x < end && !(doc_flags(x - c1t + d0) & 1)) ++x;
    return x;
  };

  float m = -INFINITY, l = 0.f;
  f32x16 o[kDT];
#pragma unroll
  for (int t = 0; t < kDT; ++t)
#pragma unroll
    for (int e = 0; e < 16; ++e) o[t][e] = 0.f;

  u32x4 rk[kSt], rv[kSt];                  // the next tile's pieces
  constexpr int kCp = D / 16;              // 16-code pieces of a cached row
  constexpr int kCt = kBN * kCp / kExtThreads;   // per thread: 1 (D = 64), 2, 4
  float rksc[kCt], rvsc[kCt];              // and their pages' scales
  auto load = [&](int x) __attribute__((always_inline)) {
    if (x < c1t) {
#pragma unroll
      for (int s = 0; s < kCt; ++s) {
        const int i = tid + s * kExtThreads, r = min(x * kBN + i / kCp, P - 1), c = i % kCp;
        const int id = page_of(p.c, n, r);
        const int64_t row = page_rows(p.c, max(id, 0), h) + (r & ((1 << lg) - 1));
        rk[s] = *reinterpret_cast<const u32x4*>(p.c.k + row * D + 16 * c);
        rv[s] = *reinterpret_cast<const u32x4*>(p.c.v + row * D + 16 * c);
        const int64_t sc = (int64_t)max(id, 0) * p.H_kv + h;
        rksc[s] = id < 0 ? 1.f : p.c.k_scale[sc];
        rvsc[s] = id < 0 ? 1.f : p.c.v_scale[sc];
        if (id < 0 || x * kBN + i / kCp >= P) {          // not held: finite, and masked below
          rk[s] = u32x4{0, 0, 0, 0};
          rv[s] = u32x4{0, 0, 0, 0};
        }
      }
    } else {
      const int j0 = (x - c1t + d0) * kBN, rows = min(kBN, L - j0);
      // rows past the sequence read as zeros (buffer range)
      const __amdgpu_buffer_rsrc_t bk = __builtin_amdgcn_make_buffer_rsrc(
          const_cast<u16*>(p.k + (int64_t)(t0 + j0) * p.k_stride + (int64_t)h * D), (short)0,
          (int)(((int64_t)(rows - 1) * p.k_stride + D) * 2), kBufWord3);
      const __amdgpu_buffer_rsrc_t bv = __builtin_amdgcn_make_buffer_rsrc(
          const_cast<u16*>(p.v + (int64_t)(t0 + j0) * p.v_stride + (int64_t)h * D), (short)0,
          (int)(((int64_t)(rows - 1) * p.v_stride + D) * 2), kBufWord3);
#pragma unroll
      for (int s = 0; s < kSt; ++s) {
        const int i = tid + s * kExtThreads, r = i / kPc, c = i % kPc;
        rk[s] = __builtin_amdgcn_raw_buffer_load_b128(bk, (int)((r * p.k_stride + c * 8) * 2), 0, 0);
        rv[s] = __builtin_amdgcn_raw_buffer_load_b128(bv, (int)((r * p.v_stride + c * 8) * 2), 0, 0);
      }
    }
  };
  auto land = [&](int x, int buf) __attribute__((always_inline)) {
    if (x < c1t) {
#pragma unroll
      for (int s = 0; s < kCt; ++s) {
        const int i = tid + s * kExtThreads, r = i / kCp, c = i % kCp;
#pragma unroll
        for (int e = 0; e < 2; ++e) {
          const uint2 a = f8x4_to_bf16(rk[s][2 * e], rksc[s]), b = f8x4_to_bf16(rk[s][2 * e + 1], rksc[s]);
          *reinterpret_cast<uint4*>(&sK[buf][tidx<D>(r, 2 * c + e)]) = make_uint4(a.x, a.y, b.x, b.y);
          const uint2 y = f8x4_to_bf16(rv[s][2 * e], rvsc[s]), z = f8x4_to_bf16(rv[s][2 * e + 1], rvsc[s]);
          *reinterpret_cast<uint4*>(&sV[buf][tidx<D>(r, 2 * c + e)]) = make_uint4(y.x, y.y, z.x, z.y);
        }
      }
    } else {
#pragma unroll
      for (int s = 0; s < kSt; ++s) {
        const int i = tid + s * kExtThreads, r = i / kPc, c = i % kPc;
        *reinterpret_cast<u32x4*>(&sK[buf][tidx<D>(r, c)]) = rk[s];
        *reinterpret_cast<u32x4*>(&sV[buf][tidx<D>(r, c)]) = rv[s];
      }
    }
  };

  int x = skip(c0t), buf = 0;
  if (x < end) {
    load(x);
    land(x, 0);
  }
  __syncthreads();
#pragma unroll 1
  while (x < end) {
    const int nx = skip(x + 1);
    if (nx < end) load(nx);
    const bool cached = x < c1t;
    const int j0 = (cached ? x : x - c1t + d0) * kBN;    // first key: cached row or token
    // does the wave see any of it, and all of it?
    bool none = false, full;
    if (cached) {
      full = j0 + kBN <= P && p.window == 0;
    } else {
      full = j0 + kBN <= L && (j0 + kBN - 1 <= wa || j0 + kBN <= mk.vis);
      none = j0 > wz && j0 >= mk.vis;
      if (p.window > 0) {
        full = full && wz - j0 < p.window && j0 + kBN - 1 - wa < p.window;
        none = none || wa - (j0 + kBN - 1) >= p.window;
      }
      if (mk.doc) full = full && (doc_flags(x - c1t + d0) & 2);
    }
    if (!none) {
      f32x16 s[2];
#pragma unroll
      for (int t = 0; t < 2; ++t) {
#pragma unroll
        for (int e = 0; e < 16; ++e) s[t][e] = 0.f;
#pragma unroll
        for (int u = 0; u < kU; ++u) {
          const bf16x8 a = as_bf16x8(*reinterpret_cast<const uint4*>(&sK[buf][tidx<D>(32 * t + q32, 2 * u + hh)]));
          s[t] = mfma32(a, q[u], s[t]);
        }
      }
      if (p.softcap > 0.f) {
#pragma unroll
        for (int i = 0; i < 32; ++i) s[i >> 4][i & 15] = capped(s[i >> 4][i & 15], c1, c2);
      } else {
#pragma unroll
        for (int i = 0; i < 32; ++i) s[i >> 4][i & 15] *= c1;
      }
      unsigned hidden = 0;                  // bit 16 t + e: key not seen by this lane's row
      if (cached) {
        if (p.window > 0 || p.slopes || !full) {
          const int qpos = start + ti;
#pragma unroll
          for (int t = 0; t < 2; ++t)
#pragma unroll
            for (int r4 = 0; r4 < 4; ++r4) {
              const int r = j0 + 32 * t + 8 * r4 + 4 * hh;        // four rows of one page
              int4 kp = make_int4(r, r + 1, r + 2, r + 3);
              const int id = r < P ? page_of(p.c, n, r) : -1;
              if (p.c.pos && id >= 0)
                kp = *reinterpret_cast<const int4*>(p.c.pos + page_rows(p.c, id, h) + (r & ((1 << lg) - 1)));
#pragma unroll
              for (int e = 0; e < 4; ++e) {
                const int dist = abs(qpos - (e == 0 ? kp.x : e == 1 ? kp.y : e == 2 ? kp.z : kp.w));
                s[t][4 * r4 + e] -= slope * (float)dist;
                if (id < 0 || r + e >= P || (p.window > 0 && dist >= p.window)) hidden |= 1u << (16 * t + 4 * r4 + e);
              }
            }
        } else {
          // a full tile can still have a page out of range
#pragma unroll
          for (int t = 0; t < 2; ++t)
#pragma unroll
            for (int r4 = 0; r4 < 4; r4 += 2)
              if (page_of(p.c, n, j0 + 32 * t + 8 * r4) < 0) hidden |= 0xffu << (16 * t + 4 * r4);
        }
      } else {
        if (p.slopes) {
          const float dq = (float)(ti - j0 - 4 * hh);
#pragma unroll
          for (int i = 0; i < 32; ++i)
            s[i >> 4][i & 15] -= slope * fabsf(dq - (float)(32 * (i >> 4) + 8 * (i >> 2 & 3) + (i & 3)));
        }
        if (!full) {
#pragma unroll
          for (int i = 0; i < 32; ++i) {
            const int j = j0 + 32 * (i >> 4) + 8 * (i >> 2 & 3) + 4 * hh + (i & 3);
            const int dj = mk.doc ? mk.doc[min(j, L - 1)] : 0;
            if (j >= L || !ext_seen(mk, ti, j, di, dj)) hidden |= 1u << i;
          }
        }
      }
      const bool masked = __any(hidden != 0);
      if (masked) {
#pragma unroll
        for (int i = 0; i < 32; ++i) s[i >> 4][i & 15] = hidden >> i & 1 ? -INFINITY : s[i >> 4][i & 15];
      }
      float mx = s[0][0];
#pragma unroll
      for (int i = 1; i < 32; ++i) mx = fmaxf(mx, s[i >> 4][i & 15]);
      mx = fmaxf(m, half_max(mx));
      if (__any(mx > m)) {
        const float fct = __builtin_amdgcn_exp2f(m == mx ? 0.f : m - mx);
        m = mx;
        l *= fct;
#pragma unroll
        for (int t = 0; t < kDT; ++t) o[t] *= fct;
      }
      const float base = m == -INFINITY ? 0.f : m;
      float ls = 0.f;
#pragma unroll
      for (int i = 0; i < 32; ++i) {
        s[i >> 4][i & 15] = __builtin_amdgcn_exp2f(s[i >> 4][i & 15] - base);
        ls += s[i >> 4][i & 15];
      }
      l += ls;
      // A masked weight is 0, and 0 times NaN or infinity would reach rows that do not see
      // the key: where a tile with hidden keys holds such a value, the product runs on
      // cleaned operands and the values are added to the rows that see them.
      unsigned long long dirty = 0;
      if (masked) {
        bool odd = false;
#pragma unroll
        for (int c = 0; c < kPc; ++c) {
          const u32x4 vv = *reinterpret_cast<const u32x4*>(&sV[buf][tidx<D>(lane, c)]);
#pragma unroll
          for (int e = 0; e < 4; ++e)
            odd = odd || (vv[e] & 0x7f80u) == 0x7f80u || (vv[e] & 0x7f800000u) == 0x7f800000u;
        }
        dirty = __ballot(odd);
      }
#pragma unroll
      for (int t = 0; t < 2; ++t)
#pragma unroll
        for (int u = 0; u < 2; ++u) {
          const bf16x8 pb = acc_to_op(s[t], u);
#pragma unroll
          for (int d = 0; d < kDT; ++d) {
            const int r = 32 * t + 16 * u + 4 * hh + ((lane & 15) >> 2), c = 4 * d + (lane >> 4 & 1) * 2 + ((lane & 3) >> 1);
            uint2 a0 = tr_read(&sV[buf][tidx<D>(r, c) + 4 * (lane & 1)]);
            uint2 a1 = tr_read(&sV[buf][tidx<D>(r + 8, c) + 4 * (lane & 1)]);
            if (dirty) {
              auto clean = [](unsigned v) {
                if ((v & 0x7f80u) == 0x7f80u) v &= 0xffff0000u;
                if ((v & 0x7f800000u) == 0x7f800000u) v &= 0xffffu;
                return v;
              };
              a0 = make_uint2(clean(a0.x), clean(a0.y));
              a1 = make_uint2(clean(a1.x), clean(a1.y));
            }
            o[d] = mfma32(join(a0, a1), pb, o[d]);
          }
        }
      for (unsigned long long left = dirty; left; left &= left - 1) {
        const int r = __builtin_ctzll(left);
        // key r of the tile sits in half (r >> 2) & 1, at bit 16 (r >> 5) + 4 (r >> 3 & 3) + (r & 3)
        const unsigned hid = (unsigned)__shfl((int)hidden, q32 + 32 * (r >> 2 & 1), kWave);
        if (hid >> (16 * (r >> 5) + 4 * (r >> 3 & 3) + (r & 3)) & 1) continue;
#pragma unroll
        for (int d = 0; d < kDT; ++d)
#pragma unroll
          for (int e = 0; e < 16; ++e) {
            const int col = 32 * d + acc_row(e, hh);
            const float v = bf16_to_f32(sV[buf][tidx<D>(r, col >> 3) + (col & 7)]);
            if ((__float_as_uint(v) & 0x7f800000u) == 0x7f800000u) o[d][e] += v;
          }
      }
    }
    if (nx < end) land(nx, buf ^ 1);
    __syncthreads();
    buf ^= 1;
    x = nx;
  }

  l += __shfl_xor(l, 32, kWave);
  if (!live) return;
  const float inv = l > 0.f ? 1.0f / l : (l == 0.f ? 0.f : l);   // nothing seen: zeros; a NaN sum stays NaN
  u16* at = p.out + (int64_t)(t0 + ti) * p.out_stride + (int64_t)hq * D;
#pragma unroll
  for (int d = 0; d < kDT; ++d)
#pragma unroll
    for (int r4 = 0; r4 < 4; ++r4)
      *reinterpret_cast<uint2*>(at + 32 * d + 8 * r4 + 4 * hh) =
          make_uint2(cvt2(o[d][4 * r4] * inv, o[d][4 * r4 + 1] * inv), cvt2(o[d][4 * r4 + 2] * inv, o[d][4 * r4 + 3] * inv));
}

}  // namespace

hipError_t launch_attn_extend(const AttnExtendLaunch& p, hipStream_t s) {
  const int64_t slots = p.T * (p.H / p.H_kv) / kBM + p.N;
  const dim3 grid((unsigned)(slots * p.H_kv));
  switch (p.d) {
    case 64: extend_kernel<64><<<grid, kExtThreads, 0, s>>>(p); break;
    case 128: extend_kernel<128><<<grid, kExtThreads, 0, s>>>(p); break;
    default: extend_kernel<256><<<grid, kExtThreads, 0, s>>>(p); break;
  }
  return hipGetLastError();
}

}  // namespace gdn
