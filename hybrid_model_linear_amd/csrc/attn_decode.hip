// Attention of one token per sequence over the paged 8-bit cache (gdn_attn_decode).
//
//   o_h = sum_r p_r v_r / sum_r p_r,  p_r = exp2(s_r - m),  s_r = log2(e) cap(scale q_h.k_r) + ...
//
// Bound by HBM: 2 d bytes of codes per row and kv head against 4 d H / H_kv flop.  The
// H / H_kv query heads of a kv head share the rows, so they are the 16 columns of one
// 16x16x32 MFMA tile and every code is read once.  A wave takes R = 64 rows at a time (32 at
// d = 256, whose codes would take the registers of its second wave per SIMD) with no LDS in
// the loop:
//   - S^T = K Q^T.  Row 4 g + r of tile t is row R / 4 g + 4 t + r of the R, so that lane
//     (query j, group g) ends up with the scores of R / 4 consecutive rows: one page (pages
//     hold 16 rows at least), and in the order in which the B operand of P wants them.  The d
//     axis of K is taken in 16-byte pieces straight from memory (Q is read in the same order).
//   - O^T = V^T P^T.  Lane (j, g) loads d / 16 bytes of each of its group's rows and
//     transposes 4 x 4 bytes at a time with byte permutes: it then holds the rows of each of
//     its d / 16 columns, the A operand's order.
// The next tile's K is loaded when this one's scores are formed, its V when the product is,
// page ids a tile before that.
// Codes become bf16 times their page's power-of-two scale, which is exact; the products
// are summed in fp32.  The weights p are rounded to bf16 for the second product (2^-8 of
// each weight at most, as the output's own rounding); their sum and the accumulated
// weights use the unrounded ones.
// The rows of a sequence are split over workgroups (and the waves of one); the partial
// (m, l, o) are joined in fp32 by a second launch, which also adds the weights: they
// need the final m and l, so the first launch leaves the scores.
// Measured, 8 kv heads: 64 sequences of 16384 rows 5.6 - 5.9 TB/s at d = 128 (pages of 16 rows
// 5.3), 5.3 at d = 64, 5.7 at d = 256; 256 sequences of 512 to 4096, d = 128: 182 us, 4.9 TB/s.
// 32 of 2000 to 8192, 32 query heads: 69 us and 5 for the join; a distance bias adds 5 to the
// first launch, accumulating 9 and 5 more to the join.
#include "attn_common.h"

namespace gdn {
namespace {

constexpr int kDecThreads = 256;
constexpr int kDecWaves = kDecThreads / kWave;
constexpr int kChunk = 64;                      // unit of the split over rows
constexpr int kRanked = 512;                    // sequences that are taken in order of length

// The 64-row chunks [t0, t1) that hold rows a sequence's query can see, and how many each
// split takes.
struct DecRange {
  int lo, hi;                                   // rows [lo, hi)
  int t0, t1, per;
};
__device__ __forceinline__ DecRange dec_range(const AttnDecodeLaunch& p, int n, int& qpos) {
  DecRange r;
  const int64_t cap = (int64_t)p.c.table_width << p.c.page_log2;
  const int len = p.kv_len[n];
  qpos = p.q_pos ? p.q_pos[n] : len - 1;
  r.lo = 0;
  r.hi = (int)min((int64_t)len, cap);           // (a padding row: negative)
  if (p.window > 0 && !p.c.pos) {               // a row's position is its index
    r.lo = max(0, (int)max((int64_t)qpos - p.window + 1, (int64_t)-1));
    r.hi = (int)min((int64_t)r.hi, (int64_t)qpos + p.window);
  }
  r.t0 = r.lo / kChunk;
  r.t1 = r.hi > r.lo ? (r.hi + kChunk - 1) / kChunk : r.t0;
  r.per = max((r.t1 - r.t0 + p.splits - 1) / p.splits, p.min_chunks);
  return r;
}

// The sequence of rank `pos` of N <= kRanked in order of length (0 the longest; in steps of
// an eighth bit and more: the lengths' top seven bits, equal ones by index), found by every
// wave for itself: the lanes hold all keys (which are distinct), and the answer's key is
// built bit by bit from the top, each bit kept if more than `pos` keys are at least as large.
// (Every workgroup does this, so it has to be short: a count over all pairs through LDS cost
// 256 x 2048 rows 25 us of 220, whole lengths in 64-bit keys 19.)
__device__ __forceinline__ int nth_longest(const int32_t* len, int N, int pos, int lane) {
  constexpr int kPer = kRanked / kWave;
  unsigned key[kPer], top = 1;
#pragma unroll
  for (int i = 0; i < kPer; ++i) {
    const int j = i * kWave + lane;
    key[i] = i * kWave < N && j < N ? (unsigned)max(len[j], 0) : 0;
    top = max(top, key[i]);
  }
#pragma unroll
  for (int o = 32; o; o >>= 1) top = max(top, (unsigned)__shfl_xor((int)top, o, kWave));
  const int shift = max(25 - __builtin_clz(__builtin_amdgcn_readfirstlane((int)top)), 0);
  const int ib = 32 - __builtin_clz(N);                  // an index takes ib bits (and none is 0)
#pragma unroll
  for (int i = 0; i < kPer; ++i) {
    const int j = i * kWave + lane;
    key[i] = j < N ? key[i] >> shift << ib | (unsigned)(N - j) : 0;
  }
  unsigned found = 0;
#pragma unroll 1
  for (unsigned bit = 1u << (ib + 6); bit; bit >>= 1) {
    const unsigned want = found | bit;
    int count = 0;
#pragma unroll
    for (int i = 0; i < kPer; ++i)
      if (i * kWave < N) count += __builtin_popcountll(__ballot(key[i] >= want));
    if (count > pos) found = want;
  }
  return N - (int)(found & ((1u << ib) - 1));
}

__device__ __forceinline__ float max_over_groups(float v) {     // lanes j, j + 16, j + 32, j + 48
  v = fmaxf(v, __shfl_xor(v, 16, kWave));
  return fmaxf(v, __shfl_xor(v, 32, kWave));
}
__device__ __forceinline__ float sum_over_groups(float v) {
  v += __shfl_xor(v, 16, kWave);
  return v + __shfl_xor(v, 32, kWave);
}

template <int W> struct VWord;                  // d / 16 bytes of a row
template <> struct VWord<1> { typedef uint32_t type; };
template <> struct VWord<2> { typedef u32x2 type; };
template <> struct VWord<4> { typedef u32x4 type; };
template <int W, typename T> __device__ __forceinline__ uint32_t word_of(const T& v, int i) {
  if constexpr (W == 1) return v; else return v[i];
}

template <int D>
__global__ void __launch_bounds__(kDecThreads, 2) decode_kernel(const AttnDecodeLaunch p) {
  constexpr int kR = D == 256 ? 32 : 64;        // rows of a wave's tile
  constexpr int kG = kR / 4;                    // rows of a lane group
  constexpr int kTS = kR / 16;                  // 16-row tiles of S^T
  constexpr int kT = D / 16;                    // 16-column tiles of O^T
  constexpr int kP = D / 64;                    // 16-byte pieces of a K row per lane
  constexpr int kW = D / 64;                    // 32-bit words of a V row per lane
  typedef typename VWord<kW>::type vword;
  __shared__ float sO[2][D][17];
  __shared__ float sML[2][2][16];
  const int tid = threadIdx.x, wave = tid >> 6, lane = tid & 63, j16 = lane & 15, g16 = lane >> 4;
  const int G = p.H / p.c.H_kv, groups = (G + 15) / 16;
  unsigned b = blockIdx.x;
  const int split = b % p.splits;
  b /= p.splits;
  const int gt = b % groups;
  b /= groups;
  const int h = b % p.c.H_kv;
  int n = b / p.c.H_kv;
  if (p.ranked) n = nth_longest(p.kv_len, p.N, n, lane);
  const int hq = h * G + gt * 16 + j16;         // this lane's query head
  const bool live = gt * 16 + j16 < G;
  const int lg = p.c.page_log2, pmask = (1 << lg) - 1;

  bf16x8 q[2 * kP];
#pragma unroll
  for (int s = 0; s < 2 * kP; ++s) {
    uint4 w = make_uint4(0, 0, 0, 0);
    if (live) w = *reinterpret_cast<const uint4*>(p.q + n * p.q_stride + (int64_t)hq * D + 64 * (s >> 1) + 16 * g16 + 8 * (s & 1));
    q[s] = as_bf16x8(w);
  }
  const float c1 = p.softcap > 0.f ? p.scale / p.softcap * 2.0f * kLog2e : p.scale * kLog2e;
  const float c2 = p.softcap * kLog2e;
  const float slope = p.slopes && live ? p.slopes[hq] * kLog2e : 0.f;
  const bool by_pos = p.c.pos && (p.slopes || p.window > 0);

  float m = -INFINITY, l = 0.f;
  f32x4 o[kT];
#pragma unroll
  for (int t = 0; t < kT; ++t) o[t] = f32x4{0.f, 0.f, 0.f, 0.f};

  // The page of the rows kG g .. of tile t (-1: out of range, or past the table).
  auto page_at = [&](int t, int g) __attribute__((always_inline)) { return page_of(p.c, n, t * kR + kG * g); };
  u32x4 kc[kTS][kP];
  vword vc[kG];
  int kid = -1, vid = -1;                       // pages of this lane's K rows and V rows: the next tile's to load
  int cur = -1;                                 // V page of the tile that is computed
  float ks = 1.f, vs = 1.f, ksn = 1.f, vsn = 1.f;
  auto load_k = [&](int t) __attribute__((always_inline)) {   // (and the scales of both)
    const int64_t row = page_rows(p.c, max(kid, 0), h);
    const uint8_t* base = p.c.k + row * D + 16 * g16;
#pragma unroll
    for (int s = 0; s < kTS; ++s) {
      const uint32_t r = (t * kR + kG * (j16 >> 2) + 4 * s + (j16 & 3)) & pmask;
#pragma unroll
      for (int c = 0; c < kP; ++c)
        kc[s][c] = __builtin_nontemporal_load(reinterpret_cast<const u32x4*>(base + r * D + 64 * c));
    }
    ksn = kid < 0 ? 1.f : p.c.k_scale[(int64_t)kid * p.c.H_kv + h];
    vsn = vid < 0 ? 1.f : p.c.v_scale[(int64_t)vid * p.c.H_kv + h];
  };
  int4 pc[kTS];                                 // positions of the rows
  auto load_v = [&](int t, int id) __attribute__((always_inline)) {
    if (by_pos) {
      const int32_t* at = p.c.pos + page_rows(p.c, max(id, 0), h) + ((t * kR + kG * g16) & pmask);
#pragma unroll
      for (int x = 0; x < kTS; ++x) pc[x] = *reinterpret_cast<const int4*>(at + 4 * x);
    }
    const uint8_t* base = p.c.v + page_rows(p.c, max(id, 0), h) * D + (D / 16) * j16;
    const uint32_t r0 = (t * kR + kG * g16) & pmask;
#pragma unroll
    for (int e = 0; e < kG; ++e)
      vc[e] = __builtin_nontemporal_load(reinterpret_cast<const vword*>(base + (r0 + e) * D));
  };
  auto ids = [&](int t) __attribute__((always_inline)) {
    kid = page_at(t, j16 >> 2);
    vid = page_at(t, g16);
  };

  auto start = [&](int t) __attribute__((always_inline)) {
    ids(t);
    load_k(t);
    load_v(t, vid);
    cur = vid;
    ids(t + kDecWaves);
  };
  // Where the first tile does not depend on the length, its loads do not wait for it.
  const bool early = p.splits == 1 && !(p.window > 0 && !p.c.pos);
  if (early) start(wave);
  int qpos;
  const DecRange rg = dec_range(p, n, qpos);
  if (p.kv_len[n] < 0) return;                  // a padding row
  // this split's tiles of kR rows
  const int c0 = rg.t0 + split * rg.per;
  const int tb = c0 * (kChunk / kR), te = min((int)min((int64_t)c0 + rg.per, (int64_t)rg.t1) * (kChunk / kR), (rg.hi + kR - 1) / kR);
  if (tb >= te && split > 0) return;            // (the join counts the splits that hold chunks)
  int t = tb + wave;
  if (!early && t < te) start(t);
#pragma unroll 1
  for (; t < te; t += kDecWaves) {
    const bool bad = cur < 0;
    ks = ksn;
    vs = vsn;
    // S^T = K Q^T, the K codes times their page's scale
    f32x4 s[kTS];
#pragma unroll
    for (int x = 0; x < kTS; ++x) {
      s[x] = f32x4{0.f, 0.f, 0.f, 0.f};
#pragma unroll
      for (int c = 0; c < kP; ++c) {
        s[x] = mfma1632(f8x8_to_op(kc[x][c][0], kc[x][c][1], ks), q[2 * c], s[x]);
        s[x] = mfma1632(f8x8_to_op(kc[x][c][2], kc[x][c][3], ks), q[2 * c + 1], s[x]);
      }
    }
    const bool more = t + kDecWaves < te;
    const int nid = vid;                        // V page of the next tile
    if (more) {                                 // in flight over the softmax and the second product
      load_k(t + kDecWaves);
      ids(t + 2 * kDecWaves);
    }
    const int r0 = t * kR + kG * g16;           // first of this lane's rows
#pragma unroll
    for (int x = 0; x < kTS; ++x)
#pragma unroll
      for (int e = 0; e < 4; ++e) s[x][e] = p.softcap > 0.f ? capped(s[x][e], c1, c2) : s[x][e] * c1;
    const bool partial = t * kR < rg.lo || t * kR + kR > rg.hi || __any(bad);
    unsigned hidden = 0;                        // bit 4 x + e: that row is not seen
    if (partial) {
#pragma unroll
      for (int i = 0; i < kG; ++i) hidden |= (bad || r0 + i < rg.lo || r0 + i >= rg.hi ? 1u : 0u) << i;
    }
    if (by_pos) {
#pragma unroll
      for (int x = 0; x < kTS; ++x) {
        const int4 kp = pc[x];
#pragma unroll
        for (int e = 0; e < 4; ++e) {
          const int dist = abs(qpos - (e == 0 ? kp.x : e == 1 ? kp.y : e == 2 ? kp.z : kp.w));
          s[x][e] -= slope * (float)dist;
          if (p.window > 0 && dist >= p.window) hidden |= 1u << (4 * x + e);
        }
      }
    } else if (p.slopes) {
#pragma unroll
      for (int i = 0; i < kG; ++i) s[i >> 2][i & 3] -= slope * (float)abs(qpos - (r0 + i));
    }
    if (__any(hidden != 0)) {
      // (the lane's rows lie on one page; behind the last row or outside of the window it may hold any scale)
      if (hidden == (1u << kG) - 1) vs = 1.f;
#pragma unroll
      for (int i = 0; i < kG; ++i) {
        const bool off = hidden >> i & 1;
        s[i >> 2][i & 3] = off ? -INFINITY : s[i >> 2][i & 3];
        if (off) {                              // what the row holds must not meet a weight of 0
          if constexpr (kW == 1) vc[i] = 0; else vc[i] = vword{};
        }
      }
    }
    if (p.accumulate && live) {
      float* at = p.scores + ((int64_t)n * p.H + hq) * p.score_cap + r0;
#pragma unroll
      for (int x = 0; x < kTS; ++x) *reinterpret_cast<f32x4*>(at + 4 * x) = s[x];
    }
    float mx = fmaxf(fmaxf(s[0][0], s[0][1]), fmaxf(s[0][2], s[0][3]));
#pragma unroll
    for (int x = 1; x < kTS; ++x) mx = fmaxf(mx, fmaxf(fmaxf(s[x][0], s[x][1]), fmaxf(s[x][2], s[x][3])));
    mx = max_over_groups(mx);
    if (__any(mx > m + 8.f)) {                  // (the maximum in use may lag the true one by 2^8)
      mx = fmaxf(m, mx);
      const float f = __builtin_amdgcn_exp2f(m == mx ? 0.f : m - mx);
      m = mx;
      l *= f;
#pragma unroll
      for (int x = 0; x < kT; ++x) o[x] *= f;
    }
    const float base = m == -INFINITY ? 0.f : m;   // a column that has seen nothing yet
#pragma unroll
    for (int x = 0; x < kTS; ++x)
#pragma unroll
      for (int e = 0; e < 4; ++e) {
        s[x][e] = __builtin_amdgcn_exp2f(s[x][e] - base);
        l += s[x][e];
      }
    bf16x8 pb[kTS / 2];
#pragma unroll
    for (int x = 0; x < kTS / 2; ++x) pb[x] = pair_to_op(s[2 * x], s[2 * x + 1]);
    // O^T += V^T P^T
#pragma unroll
    for (int w = 0; w < kW; ++w) {
      uint32_t tr[kTS][4];                      // [rows 4 i ..][column]: four rows of one column
#pragma unroll
      for (int i = 0; i < kTS; ++i) {
        const uint32_t a0 = word_of<kW>(vc[4 * i], w), a1 = word_of<kW>(vc[4 * i + 1], w);
        const uint32_t a2 = word_of<kW>(vc[4 * i + 2], w), a3 = word_of<kW>(vc[4 * i + 3], w);
        const uint32_t lo01 = __builtin_amdgcn_perm(a1, a0, 0x05010400), hi01 = __builtin_amdgcn_perm(a1, a0, 0x07030602);
        const uint32_t lo23 = __builtin_amdgcn_perm(a3, a2, 0x05010400), hi23 = __builtin_amdgcn_perm(a3, a2, 0x07030602);
        tr[i][0] = __builtin_amdgcn_perm(lo23, lo01, 0x05040100);
        tr[i][1] = __builtin_amdgcn_perm(lo23, lo01, 0x07060302);
        tr[i][2] = __builtin_amdgcn_perm(hi23, hi01, 0x05040100);
        tr[i][3] = __builtin_amdgcn_perm(hi23, hi01, 0x07060302);
      }
#pragma unroll
      for (int c = 0; c < 4; ++c)
#pragma unroll
        for (int x = 0; x < kTS / 2; ++x)
          o[4 * w + c] = mfma1632(f8x8_to_op(tr[2 * x][c], tr[2 * x + 1][c], vs), pb[x], o[4 * w + c]);
    }
    if (more) load_v(t + kDecWaves, nid);
    cur = nid;
  }

  // Join the waves: waves 2, 3 hand theirs to waves 0, 1, then wave 1 to wave 0.
  l = sum_over_groups(l);
#pragma unroll
  for (int step = 2; step; step >>= 1) {
    if (wave >= step && wave < 2 * step) {
      const int w = wave - step;
      if (g16 == 0) {
        sML[w][0][j16] = m;
        sML[w][1][j16] = l;
      }
#pragma unroll
      for (int x = 0; x < kT; ++x)
#pragma unroll
        for (int e = 0; e < 4; ++e) sO[w][kT * (4 * g16 + e) + x][j16] = o[x][e];
    }
    __syncthreads();
    if (wave < step) {
      const float m2 = sML[wave][0][j16], l2 = sML[wave][1][j16], mn = fmaxf(m, m2);
      const float f1 = mn == -INFINITY ? 0.f : __builtin_amdgcn_exp2f(m - mn);
      const float f2 = mn == -INFINITY ? 0.f : __builtin_amdgcn_exp2f(m2 - mn);
      m = mn;
      l = l * f1 + l2 * f2;
#pragma unroll
      for (int x = 0; x < kT; ++x)
#pragma unroll
        for (int e = 0; e < 4; ++e) o[x][e] = o[x][e] * f1 + sO[wave][kT * (4 * g16 + e) + x][j16] * f2;
    }
    __syncthreads();
  }
  if (wave != 0 || !live) return;
  const bool alone = rg.t1 - rg.t0 <= rg.per;   // no other split holds chunks
  if (alone) {
    const float inv = l > 0.f ? 1.0f / l : (l == 0.f ? 0.f : l);   // (a NaN sum stays NaN)
    u16* at = p.out + n * p.out_stride + (int64_t)hq * D;
#pragma unroll
    for (int e = 0; e < 4; ++e)                 // columns kT (4 g + e) .. + kT - 1
#pragma unroll
      for (int x = 0; x < kT; x += 4)
        *reinterpret_cast<uint2*>(at + kT * (4 * g16 + e) + x) =
            make_uint2(cvt2(o[x][e] * inv, o[x + 1][e] * inv), cvt2(o[x + 2][e] * inv, o[x + 3][e] * inv));
  } else {
    float* at = p.part_o + (((int64_t)n * p.H + hq) * p.splits + split) * D;
#pragma unroll
    for (int e = 0; e < 4; ++e)
#pragma unroll
      for (int x = 0; x < kT; x += 4)
        *reinterpret_cast<f32x4*>(at + kT * (4 * g16 + e) + x) = f32x4{o[x][e], o[x + 1][e], o[x + 2][e], o[x + 3][e]};
  }
  if ((!alone || p.accumulate) && g16 == 0) {
    float* at = p.part_ml + (((int64_t)n * p.H + hq) * p.splits + split) * 2;
    at[0] = m;
    at[1] = l;
  }
}

// Join: blockIdx.x = 0 .. H - 1: the partial outputs of one query head; the blocks behind
// (accumulate): 1024 rows of one kv head, four per thread.
constexpr int kAccRows = 4 * kDecThreads;
constexpr int kMaxSplits = kDecThreads;

template <int D>
__global__ void __launch_bounds__(kDecThreads) decode_join_kernel(const AttnDecodeLaunch p) {
  __shared__ float sM[64], sInv[64], sPart[8];
  const int tid = threadIdx.x, n = blockIdx.y;
  int qpos;
  const DecRange rg = dec_range(p, n, qpos);
  if (p.kv_len[n] < 0) return;
  const int used = (rg.t1 - rg.t0 + rg.per - 1) / rg.per;   // splits that hold chunks
  if ((int)blockIdx.x < p.H) {
    if (used <= 1) return;                      // written by the first launch
    __shared__ float sF[kMaxSplits];
    __shared__ f32x4 sAcc[kDecThreads];
    const int64_t row = ((int64_t)n * p.H + blockIdx.x) * p.splits;
    // factors of the partial sums: a thread per split (kMaxSplits = kDecThreads)
    const f32x2 ml = tid < used ? *reinterpret_cast<const f32x2*>(p.part_ml + (row + tid) * 2) : f32x2{-INFINITY, 0.f};
    float m = ml.x;
#pragma unroll
    for (int o = 32; o; o >>= 1) m = fmaxf(m, __shfl_xor(m, o, kWave));
    if ((tid & 63) == 0) sPart[tid >> 6] = m;
    __syncthreads();
    m = fmaxf(fmaxf(sPart[0], sPart[1]), fmaxf(sPart[2], sPart[3]));
    const float f = m == -INFINITY ? 0.f : __builtin_amdgcn_exp2f(ml.x - m);
    sF[tid] = f;
    float l = ml.y * f;
#pragma unroll
    for (int o = 32; o; o >>= 1) l += __shfl_xor(l, o, kWave);
    if ((tid & 63) == 0) sPart[4 + (tid >> 6)] = l;
    __syncthreads();
    l = sPart[4] + sPart[5] + sPart[6] + sPart[7];
    constexpr int kC = D / 4;                   // four columns per thread, kDecThreads / kC splits at a time
    const int c = tid % kC, part = tid / kC;
    const float* src = p.part_o + row * D + 4 * c;
    f32x4 o{0.f, 0.f, 0.f, 0.f};
#pragma unroll 4
    for (int s = part; s < used; s += kDecThreads / kC) o += *reinterpret_cast<const f32x4*>(src + (int64_t)s * D) * sF[s];
    sAcc[tid] = o;
    __syncthreads();
    if (part == 0) {
#pragma unroll
      for (int i = 1; i < kDecThreads / kC; ++i) o += sAcc[tid + i * kC];
      const float inv = l > 0.f ? 1.0f / l : (l == 0.f ? 0.f : l);
      *reinterpret_cast<uint2*>(p.out + n * p.out_stride + (int64_t)blockIdx.x * D + 4 * c) =
          make_uint2(cvt2(o[0] * inv, o[1] * inv), cvt2(o[2] * inv, o[3] * inv));
    }
    return;
  }
  // accumulated weights
  const int G = p.H / p.c.H_kv;
  const int blk = blockIdx.x - p.H, h = blk % p.c.H_kv;
  const int64_t first = (int64_t)(blk / p.c.H_kv) * kAccRows + (int64_t)rg.t0 * kChunk;
  if (first >= rg.hi || used == 0) return;
  const int r = (int)first + 4 * tid;
  f32x4 w{0.f, 0.f, 0.f, 0.f};
  // the row's weights and its first heads' scores, in flight while the statistics are joined
  constexpr int kPre = 4;
  const int id = r < rg.hi ? page_of(p.c, n, r) : -1;
  float* const at = p.c.weight + page_rows(p.c, max(id, 0), h) + (r & ((1 << p.c.page_log2) - 1));
  const float* const sc = p.scores + ((int64_t)n * p.H + h * G) * p.score_cap + r;
  f32x4 old{0.f, 0.f, 0.f, 0.f}, pre[kPre];
  if (id >= 0) {
    old = *reinterpret_cast<const f32x4*>(at);
#pragma unroll
    for (int g = 0; g < kPre; ++g)
      if (g < G) pre[g] = *reinterpret_cast<const f32x4*>(sc + g * p.score_cap);
  }
  for (int g0 = 0; g0 < G; g0 += 64) {
    const int gn = min(64, G - g0);
    __syncthreads();
    for (int g = tid >> 6; g < gn; g += kDecWaves) {   // a wave per head, a lane per split
      const f32x2* ml = reinterpret_cast<const f32x2*>(p.part_ml) + ((int64_t)n * p.H + h * G + g0 + g) * p.splits;
      f32x2 v[kMaxSplits / kWave];
      float m = -INFINITY, l = 0.f;
#pragma unroll
      for (int i = 0; i < kMaxSplits / kWave; ++i) {
        const int s = i * kWave + (tid & 63);
        v[i] = f32x2{-INFINITY, 0.f};
        if (s < used) v[i] = ml[s];
        m = fmaxf(m, v[i].x);
      }
#pragma unroll
      for (int o = 32; o; o >>= 1) m = fmaxf(m, __shfl_xor(m, o, kWave));
      const float base = m > -INFINITY ? m : 0.f;
#pragma unroll
      for (int i = 0; i < kMaxSplits / kWave; ++i) l += v[i].y * __builtin_amdgcn_exp2f(v[i].x - base);
#pragma unroll
      for (int o = 32; o; o >>= 1) l += __shfl_xor(l, o, kWave);
      if ((tid & 63) == 0) {
        sM[g] = base;
        sInv[g] = l > 0.f ? 1.0f / l : (l == 0.f ? 0.f : l);
      }
    }
    __syncthreads();
    auto add = [&](const f32x4& s, int g) __attribute__((always_inline)) {
#pragma unroll
      for (int e = 0; e < 4; ++e) w[e] += __builtin_amdgcn_exp2f(s[e] - sM[g]) * sInv[g];
    };
    if (id >= 0) {
      int g = 0;
      if (g0 == 0) {
#pragma unroll
        for (; g < kPre; ++g)
          if (g < gn) add(pre[g], g);
      }
#pragma unroll 4
      for (; g < gn; ++g) add(*reinterpret_cast<const f32x4*>(sc + (g0 + g) * p.score_cap), g);
    }
  }
  if (id < 0) return;
  if (p.window > 0 && p.c.pos) {                // hidden rows stay as they are, also where a head's sum is NaN
    const int4 kp = *reinterpret_cast<const int4*>(p.c.pos + (at - p.c.weight));
#pragma unroll
    for (int e = 0; e < 4; ++e)
      if (abs(qpos - (e == 0 ? kp.x : e == 1 ? kp.y : e == 2 ? kp.z : kp.w)) >= p.window) w[e] = 0.f;
  }
#pragma unroll
  for (int e = 0; e < 4; ++e)
    if (r + e >= rg.lo && r + e < rg.hi) at[e] = old[e] + w[e];
}

template <int D>
hipError_t launch_d(const AttnDecodeLaunch& p, int64_t max_rows, hipStream_t s) {
  const int G = p.H / p.c.H_kv;
  const int64_t blocks = (int64_t)p.splits * ((G + 15) / 16) * p.c.H_kv * p.N;
  decode_kernel<D><<<dim3((unsigned)blocks), kDecThreads, 0, s>>>(p);
  hipError_t e = hipGetLastError();
  if (e != hipSuccess || (p.splits == 1 && !p.accumulate)) return e;
  // (a range of max_rows rows can begin inside a chunk)
  const int64_t acc = p.accumulate ? (max_rows + kChunk + kAccRows - 1) / kAccRows * p.c.H_kv : 0;
  decode_join_kernel<D><<<dim3((unsigned)(p.H + acc), (unsigned)p.N), kDecThreads, 0, s>>>(p);
  return hipGetLastError();
}

}  // namespace

// How a call is cut: splits per (sequence, kv head, 16 query heads), the fewest chunks that
// one takes, and whether the longest sequences come first.  Two workgroups fit a CU.  Up to
// 16 sequences are cut into one round of workgroups (2 x 131000 rows, d = 256: 59 us, in two
// rounds 70; 16 x 5000, 8 heads of 128 39 and 48; 16 of 500 to 10000 47 and 48); more of them
// differ in length too much for one round, and two (32 of 100 to 8000 rows: 48 us, in one 66;
// 32 of 2000 to 8192 with weights 92, in four 106) with the longest first even that out (256 of
// 512 to 4096: 217 us in the order of the batch, 182; 256 of 2048 alike 196 and 208), at the
// cost of batches of like lengths (32 x 5000 77 us, in one round 69).  Shares of the batch's
// whole length, found on the device, were slower than the better of the two throughout.
void plan_attn_decode(AttnDecodeLaunch& p, int64_t max_rows, int cus) {
  const int64_t base = (int64_t)p.N * p.c.H_kv * ((p.H / p.c.H_kv + 15) / 16), chunks = (max_rows + kChunk - 1) / kChunk;
  p.min_chunks = 2 * (p.c.d == 256 ? 2 : 4);    // two tiles per wave
  const int64_t want = ((p.N > 16 ? 4 : 2) * (int64_t)cus + base - 1) / base;
  const int64_t most = (chunks + p.min_chunks - 1) / p.min_chunks;
  const int64_t s = want < most ? want : most;
  p.splits = (int)(s < 1 ? 1 : s > kMaxSplits ? kMaxSplits : s);
  p.ranked = p.N > 1 && p.N <= kRanked && base * p.splits > 2 * cus;
}

hipError_t launch_attn_decode(const AttnDecodeLaunch& p, hipStream_t s) {
  const int64_t rows = (int64_t)p.c.table_width << p.c.page_log2;
  switch (p.c.d) {
    case 64: return launch_d<64>(p, rows, s);
    case 128: return launch_d<128>(p, rows, s);
    default: return launch_d<256>(p, rows, s);
  }
}

}  // namespace gdn
