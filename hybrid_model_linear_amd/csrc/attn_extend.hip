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
//   - S^T = K Q^T with 32x32x16 MFMA: a lane holds half of a tile's scores of one row (lane
//     % 32), so the softmax is lane-local but for one exchange of the two halves.
//   - O^T += V^T P^T: S^T's accumulator order is the B operand's once the 16 keys of a step
//     are taken as 8 (2 u + (e >> 2)) + 4 half + (e & 3), and V^T comes from the row-major V
//     tile by LDS transpose reads of 4 rows in that order.
// K and V tiles of 64 keys stand in LDS as bf16, their 16-byte pieces XOR-swizzled by row
// (operand and transpose reads without bank conflicts).  New tokens' tiles are
// double-buffered and go from memory to LDS without passing through registers; the swizzle
// is on the global side.  Cached rows arrive as codes the same way; the lane that asked
// for a piece turns it into bf16 times its page's power-of-two scale (exact).
// The loop is a tile deep: while the matrix units form the scores of the next tile, the
// vector units turn this tile's into weights; then, under the second product, they cap and
// bias the next tile's scores and look for their maximum.  (One after the other, both kept
// the SIMDs busy 44% of the time each with hardly any overlap, even with two workgroups on
// a CU: 944 TFLOP/s at 8 x 4096 tokens, 32 / 8 heads, d = 128; now 1020 - 1060, where a
// library product of two matrices of 16384^2 normal values reaches 1390.)  Up to d = 128
// two workgroups fit a CU; at d = 256 one does (its output alone takes 128 registers).
// Keys are taken from the last to the first, the new tokens before the cached: with a
// distance bias the nearest keys set the maximum at once and the sums are not rescaled again.
// The weights are rounded to bf16 for the second product, their sum is not.
#include "attn_common.h"

namespace gdn {
namespace {

constexpr int kExtThreads = 256;
constexpr int kBM = 128;      // rows of a workgroup
constexpr int kMaxSplits = 16;
constexpr int kFlags = 4096;  // document mask: key tiles whose overlap is looked up ahead

typedef __attribute__((address_space(3))) const u32x4 lds_u32x4;
typedef __attribute__((address_space(3))) const u32x2 lds_u32x2;
typedef __attribute__((address_space(3))) u32x4 lds_u32x4w;

// LDS byte address (the 32-bit value of the pointer)
template <typename T> __device__ __forceinline__ uint32_t lds_at(const T* p) {
  return (uint32_t)(uintptr_t)(const __attribute__((address_space(3))) T*)p;
}
__device__ __forceinline__ bf16x8 lds_op(uint32_t at) { return __builtin_bit_cast(bf16x8, *(lds_u32x4*)(uintptr_t)at); }
__device__ __forceinline__ uint2 lds_tr(uint32_t at) {
  return __builtin_bit_cast(uint2, __builtin_amdgcn_ds_read_tr16_b64_v4i16((lds_v4i16*)(uintptr_t)at));
}

// Memory -> LDS, 16 bytes per lane: lane l's piece lands at `lds` + 16 l.  In inline
// assembly because the compiler, which cannot tell the two tile buffers apart, would wait
// for every load in flight before each LDS read; vm_wait() is the wait.
__device__ __forceinline__ void to_lds(u32x4 rsrc, uint32_t voff, uint32_t lds) {
  asm volatile("s_mov_b32 m0, %0\n\ts_nop 0\n\tbuffer_load_dwordx4 %1, %2, 0 offen lds"
               :: "s"(lds), "v"(voff), "s"(rsrc) : "memory", "m0");
}
__device__ __forceinline__ void vm_wait() { asm volatile("s_waitcnt vmcnt(0)" ::: "memory"); }
__device__ __forceinline__ uint32_t uni(uint32_t v) { return (uint32_t)__builtin_amdgcn_readfirstlane((int)v); }
// Buffer descriptor of `bytes` bytes at p (both the same in every lane); reads past the
// end give zeros.
__device__ __forceinline__ u32x4 buffer_of(const void* p, uint32_t bytes) {
  const uint64_t a = (uint64_t)(uintptr_t)p;
  return u32x4{uni((uint32_t)a), uni((uint32_t)(a >> 32)), uni(bytes), (unsigned)kBufWord3};
}

// XOR of a row's 16-byte pieces in a [rows][D] bf16 tile: any 16 consecutive rows of one
// piece, and any 4-row group of 4 pieces, cover all banks.
template <int D> __device__ __forceinline__ int row_swz(int r) {
  return D >= 128 ? ((r & 3) << 2 | (r >> 2 & 3)) : ((r >> 1 & 1) << 2 | (r >> 2 & 3));
}

// What happens to a score between the two products (a kernel per way: the vector work is laid
// out by hand under the matrix instructions).
enum Shape {
  kRaw = 0,       // nothing but a positive scale, which is left to the exponent
  kBias = 1,      // scale and distance bias (slopes may be null: a scale that is not positive)
  kCap = 2,       // tanh cap
  kCapBias = 3,
};

template <int D, bool CACHED, int SHAPE>
__global__ void __launch_bounds__(kExtThreads, D <= 128 ? 2 : 1) extend_kernel(const AttnExtendLaunch p) {
  constexpr int kBN = 64;                  // keys of a tile
  constexpr int kN2 = kBN / 32;
  constexpr int kS = 16 * kN2;             // scores per lane
  constexpr int kU = D / 16;               // k steps of S^T
  constexpr int kDT = D / 32;              // 32-column tiles of O^T
  constexpr int kPc = D / 8;               // 16-byte pieces of a bf16 row
  constexpr int kTile = kBN * D * 2;       // bytes of a K or V tile
  constexpr int kRpi = kWave / kPc;        // rows that one wave's load brings
  constexpr int kLd = kBN / kRpi / 4;      // loads per wave and tile
  constexpr int kKa = kU < 8 ? kU : 8, kVa = kDT < 4 ? kDT : 4;   // distinct operand addresses
  __shared__ __attribute__((aligned(1024))) unsigned char sT[4 * kTile];   // K, V, K, V
  __shared__ unsigned char sFlag[kFlags];  // per key tile: 1 overlaps the rows' documents, 2 is all of their one
  __shared__ int sDoc[2], sOdd;
  __shared__ __attribute__((aligned(16))) int sIds[4][64];
  __shared__ unsigned sBad[2];             // rows of a tile that hold NaN or infinity

  if (threadIdx.x == 0) sOdd = -1;         // (read after a barrier at least)
  const int tid = threadIdx.x, wave = (int)uni(threadIdx.x >> 6), lane = tid & 63, q32 = lane & 31, hh = lane >> 5;
  const int G = p.H / p.H_kv;
  // Heads fastest: consecutive workgroups go to the 8 XCDs in turn, so a head's tiles share
  // an L2.  Late tiles of a causal sequence see the most keys: they are launched first, and
  // from slot p.fold of the launch on the earliest.
  const int h = blockIdx.x % p.H_kv, pos = blockIdx.x / p.H_kv;
  const int w = pos < p.fold ? (int)(gridDim.x / p.H_kv) - 1 - pos : pos - p.fold;
  // slot w -> (sequence n, tile): sequence n's tiles begin at floor(cu[n] G / 128) + n
  const int n = find_last(p.N, threadIdx.x & 63, [&](int i) { return p.cu[i] * G / kBM + i <= w; });
  const int t0 = p.cu[n], L = p.cu[n + 1] - t0;
  const int rows = L * G, f0 = (w - (t0 * G / kBM + n)) * kBM;   // (T G stays below 2^31)
  if (f0 < 0 || f0 >= rows) return;
  int P = CACHED ? p.cache_len[n] : 0;                  // cached rows
  if (P < 0) return;
  const int start = p.start ? p.start[n] : P;           // position of token 0
  const int lg = p.c.page_log2, pmask = (1 << lg) - 1;
  if (CACHED) P = (int)min((int64_t)P, (int64_t)p.c.table_width << lg);

  // this lane's row, and the wave's and workgroup's tokens
  const int f = f0 + wave * 32 + q32;
  const bool live = f < rows;
  const int ti = live ? (int)((unsigned)f / (unsigned)G) : L - 1, g = live ? f - ti * G : 0;
  const int hq = h * G + g;
  const int ta = (int)uni((unsigned)f0 / (unsigned)G), tz = (int)uni((unsigned)(min(f0 + kBM, rows) - 1) / (unsigned)G);
  const int wa = __builtin_amdgcn_readlane(ti, 0), wz = __builtin_amdgcn_readlane(ti, 63);   // (a dead row counts as the last token)
  const int vis = p.causal ? (p.visible ? p.visible[n] : 0) : INT32_MAX;   // keys below: seen by every row
  const int32_t* doc = p.doc ? p.doc + t0 : nullptr;
  const int di = doc ? doc[ti] : 0;

  bf16x8 q[kU];
#pragma unroll
  for (int u = 0; u < kU; ++u) {
    uint4 x = make_uint4(0, 0, 0, 0);
    if (live) x = *reinterpret_cast<const uint4*>(p.q + (int64_t)(t0 + ti) * p.q_stride + (int64_t)hq * D + 16 * u + 8 * hh);
    q[u] = as_bf16x8(x);
  }
  // kRaw: scores stay q.k until the exponent; otherwise they are brought to units of log2 first.
  constexpr bool kHasBias = SHAPE & kBias, kHasCap = SHAPE & kCap;
  const float c1 = kHasCap ? p.scale / p.softcap * 2.0f * kLog2e : p.scale * kLog2e;
  const float c2 = p.softcap * kLog2e;
  float cs = SHAPE == kRaw ? c1 : 1.f;     // (kRaw: of this lane's row, raise() may change it)
  const float slope = kHasBias && p.slopes ? p.slopes[hq] * kLog2e : 0.f;
  const float slack = fminf(8.f / cs, 3e38f);   // the maximum in use may lag the true one by 2^8 (finite: the first raises it)

  // operand addresses in the first K and V tile (kTile bytes each: K, V, K, V)
  uint32_t ka[kKa], va[2][kVa];
  {
    const uint32_t base = lds_at(sT);
#pragma unroll
    for (int u = 0; u < kKa; ++u) ka[u] = base + q32 * (2 * D) + (((2 * u + hh) ^ row_swz<D>(q32)) << 4);
#pragma unroll
    for (int e = 0; e < 2; ++e)
#pragma unroll
      for (int d = 0; d < kVa; ++d) {
        const int r = 4 * hh + ((lane & 15) >> 2) + 8 * e, c = 4 * d + (lane >> 4 & 1) * 2 + ((lane & 3) >> 1);
        va[e][d] = base + kTile + r * (2 * D) + ((c ^ row_swz<D>(r)) << 4) + 8 * (lane & 1);
      }
  }

  float m = -INFINITY, base = 0.f, l = 0.f;   // base: m in units of log2, 0 while nothing is seen
  f32x16 o[kDT];
#pragma unroll
  for (int t = 0; t < kDT; ++t)
#pragma unroll
    for (int e = 0; e < 16; ++e) o[t][e] = 0.f;
  bf16x8 pb[2 * kN2];                      // the weights as operands, 16 keys each

  constexpr int kNS = kN2 * kU, kNP = 2 * kN2 * kDT;   // MFMAs of a tile's scores and of its product
  constexpr int kRing = 4;                 // operands in flight (3, 6 and 8 are no faster)
  auto k_op = [&](int i, uint32_t koff) __attribute__((always_inline)) {   // operand i of the K tile at koff
    const int t = i % kN2, u = i / kN2;
    return lds_op(ka[u & 7] + (koff + t * 32 * 2 * D + (u >> 3) * 256));
  };
  auto v_op = [&](int i, uint32_t voff) __attribute__((always_inline)) {
    const int k = i / kDT, d = i % kDT;
    const uint32_t imm = voff + 16 * k * 2 * D + (d >> 2) * 256;
    return join(lds_tr(va[0][d & 3] + imm), lds_tr(va[1][d & 3] + imm));
  };
  // One MFMA of the scores, and the read that its operand slot is free for.
  auto score = [&](int i, uint32_t koff, f32x16 (&s)[kN2], bf16x8 (&a)[kRing]) __attribute__((always_inline)) {
    f32x16 zero;
#pragma unroll
    for (int e = 0; e < 16; ++e) zero[e] = 0.f;
    s[i % kN2] = mfma32(a[i % kRing], q[i / kN2], i < kN2 ? zero : s[i % kN2]);
    if (i + kRing < kNS) a[i % kRing] = k_op(i + kRing, koff);
  };
  auto scores = [&](uint32_t koff, f32x16 (&s)[kN2]) __attribute__((always_inline)) {
    bf16x8 a[kRing];
#pragma unroll
    for (int i = 0; i < kRing; ++i) a[i] = k_op(i, koff);
    __builtin_amdgcn_sched_barrier(0);
#pragma unroll
    for (int i = 0; i < kNS; ++i) {
      score(i, koff, s, a);
      __builtin_amdgcn_sched_barrier(0);
    }
  };
  // Scores [a, b) of this lane -> weights; then (a step later, since an exponential's result
  // takes a few cycles) their part of the sum, and every eighth an operand.
  float ls[2];
  auto weigh = [&](int a, int b, f32x16 (&s)[kN2]) __attribute__((always_inline)) {
#pragma unroll
    for (int i = a; i < b; ++i) s[i >> 4][i & 15] = __builtin_amdgcn_exp2f(fmaf(s[i >> 4][i & 15], cs, -base));
  };
  auto gather = [&](int a, int b, const f32x16 (&s)[kN2]) __attribute__((always_inline)) {
#pragma unroll
    for (int i = a; i < b; ++i) {
      ls[i & 1] = i < 2 ? s[0][i] : ls[i & 1] + s[i >> 4][i & 15];
      if ((i & 7) == 7) pb[i >> 3] = acc_to_op(s[i >> 4], i >> 3 & 1);
    }
  };
  auto weights = [&](f32x16 (&s)[kN2]) __attribute__((always_inline)) {
    weigh(0, kS, s);
    gather(0, kS, s);
    l += ls[0] + ls[1];
  };
  // O^T += V^T P^T with the V tile `voff` bytes behind the first.
  auto product = [&](uint32_t voff) __attribute__((always_inline)) {
    bf16x8 a[kRing];
#pragma unroll
    for (int i = 0; i < kRing; ++i) a[i] = v_op(i, voff);
    __builtin_amdgcn_sched_barrier(0);
#pragma unroll
    for (int i = 0; i < kNP; ++i) {
      o[i % kDT] = mfma32(a[i % kRing], pb[i / kDT], o[i % kDT]);
      if (i + kRing < kNP) a[i % kRing] = v_op(i + kRing, voff);
      __builtin_amdgcn_sched_barrier(0);
    }
  };
  auto tile_max = [&](const f32x16 (&s)[kN2]) __attribute__((always_inline)) {
    float a = s[0][0];
#pragma unroll
    for (int i = 1; i < kS; ++i) a = fmaxf(a, s[i >> 4][i & 15]);
    return a;
  };
  // Makes m hold for a tile whose largest score in this lane is mx.
  auto raise = [&](float mx) __attribute__((always_inline)) {
    mx = half_max(mx);
    if (__any(mx > m + slack)) {
      mx = fmaxf(m, mx);
      const float fct = __builtin_amdgcn_exp2f(m == mx ? 0.f : (m - mx) * (SHAPE == kRaw ? c1 : 1.f));
      m = mx;
      // From 2^31 on m cs is off by 2^6 and more through its rounding, and weights would overflow
      // or vanish.  By a power of two it is exact, and as the next lower score is 2^6 away at
      // least, only the largest has a weight either way.
      if (SHAPE == kRaw) cs = fabsf(m * c1) >= 0x1p31f ? __uint_as_float(__float_as_uint(c1) & 0x7f800000u) : c1;
      base = m == -INFINITY ? 0.f : m * cs;
      l *= fct;
#pragma unroll
      for (int t = 0; t < kDT; ++t) o[t] *= fct;
    }
  };
  auto hide = [&](f32x16 (&s)[kN2], unsigned hidden, float& mx) __attribute__((always_inline)) {
    if (__any(hidden != 0)) {
#pragma unroll
      for (int i = 0; i < kS; ++i) s[i >> 4][i & 15] = hidden >> i & 1 ? -INFINITY : s[i >> 4][i & 15];
      mx = tile_max(s);
    }
  };
  // Score i to its final form but for the mask; dq: this row's position minus that of the tile's
  // first key of this lane, sl the slope.
  auto shape = [&](int i, f32x16 (&s)[kN2], float dq, float sl) __attribute__((always_inline)) {
    float x = s[i >> 4][i & 15];
    if (kHasCap) x = capped(x, c1, c2); else if (kHasBias) x *= c1;
    if (kHasBias) x -= sl * fabsf(dq - (float)(32 * (i >> 4) + 8 * (i >> 2 & 3) + (i & 3)));
    s[i >> 4][i & 15] = x;
  };
  // One step: weights of the tile in s under the scores of the next (s2), then this tile's
  // product, under which the new scores are shaped and their maximum is found; kRaw leaves
  // half of the weights to the first half of the product.  load(j) starts one of the loads
  // of later tiles; mask(s2, mx) hides scores of a tile that is seen in part.  The order is
  // fixed here, an MFMA and its share of vector work at a time with operands kRing MFMAs
  // ahead: left alone, the compiler waits for each read before its MFMA and puts the vector
  // work behind them all.
  auto step = [&](f32x16 (&s)[kN2], f32x16 (&s2)[kN2], uint32_t koff, uint32_t voff, float dq, float sl, auto loads,
                  auto load, auto mask) __attribute__((always_inline)) {
    // weights formed under the scores (half of them: 8 x 4096, d = 128 1.09 -> 1.06 ms; d = 256 no change)
    constexpr int kW = SHAPE == kRaw && D < 256 ? kS / 2 : kS;
    constexpr int kFirst = kW / 8;                      // of them, while the first operands are on their way
    constexpr int kH = kNP / 2, kQ = kH - 1, kLoads = decltype(loads)::value;
    auto part = [](int i, int n, int of, int from) { return from + i * of / n; };
    bf16x8 a[kRing];
#pragma unroll
    for (int i = 0; i < kRing; ++i) a[i] = k_op(i, koff);
    weigh(0, kFirst, s);
    __builtin_amdgcn_sched_barrier(0);
#pragma unroll
    for (int i = 0; i < kNS; ++i) {
      score(i, koff, s2, a);
      if (i + kRing >= kNS) a[i % kRing] = v_op(i + kRing - kNS, voff);
      weigh(part(i, kNS, kW - kFirst, kFirst), part(i + 1, kNS, kW - kFirst, kFirst), s);
      gather(i ? part(i - 1, kNS, kW - kFirst, kFirst) : 0, part(i, kNS, kW - kFirst, kFirst), s);
      if (i % (kNS / kLoads) == 0) load(i / (kNS / kLoads));
      __builtin_amdgcn_sched_barrier(0);
    }
    gather(part(kNS - 1, kNS, kW - kFirst, kFirst), kW, s);
    float mx = -INFINITY;
#pragma unroll
    for (int i = 0; i < kNP; ++i) {
      o[i % kDT] = mfma32(a[i % kRing], pb[i / kDT], o[i % kDT]);
      if (i + kRing < kNP) a[i % kRing] = v_op(i + kRing, voff);
      if (kW < kS) {                                    // (the second half's operands are whole a step before they are used)
        if (i < kQ) weigh(part(i, kQ, kS - kW, kW), part(i + 1, kQ, kS - kW, kW), s);
        if (i > 0 && i < kH) gather(part(i - 1, kQ, kS - kW, kW), part(i, kQ, kS - kW, kW), s);
      }
      const int n0 = kW < kS ? kH : 2, nn = kNP - n0;   // (the last scores are not there at once)
      if (i >= n0) {
        const int e0 = part(i - n0, nn, kS, 0), e1 = part(i + 1 - n0, nn, kS, 0);
#pragma unroll
        for (int e = e0; e < e1; ++e) shape(e, s2, dq, sl);
        const int m0 = SHAPE == kRaw ? e0 : i > n0 ? part(i - 1 - n0, nn, kS, 0) : 0, m1 = SHAPE == kRaw ? e1 : e0;
#pragma unroll
        for (int e = m0; e < m1; ++e) mx = fmaxf(mx, s2[e >> 4][e & 15]);
      }
      __builtin_amdgcn_sched_barrier(0);
    }
    if (SHAPE != kRaw) {
#pragma unroll
      for (int e = kS - (kS + kNP - 3) / (kNP - 2); e < kS; ++e) mx = fmaxf(mx, s2[e >> 4][e & 15]);
    }
    l += ls[0] + ls[1];
    // (formed here: the compiler would sink the vector work behind the branches of mask)
#pragma unroll
    for (int i = 0; i < kN2; ++i) asm volatile("" : "+v"(s2[i]));
    asm volatile("" : "+v"(l), "+v"(mx));
    mask(s2, mx);
    raise(mx);
  };
  // A copy of v that the compiler cannot see through: what the paths below compute from it
  // is computed there, and not kept in registers over the whole loop.
  auto opaque = [](int v) __attribute__((always_inline)) {
    asm volatile("" : "+v"(v));
    return v;
  };
  // Key of score i of a lane of half hh within its tile
  auto key = [](int i, int hh) __attribute__((always_inline)) { return 32 * (i >> 4) + 8 * (i >> 2 & 3) + 4 * hh + (i & 3); };
  // Bits of the scores whose keys lie in [lo, hi) of the tile.
  auto seen_bits = [&](int lo, int hi) __attribute__((always_inline)) {
    unsigned bits = 0;
    const int hh = opaque(lane) >> 5;
#pragma unroll
    for (int t = 0; t < kN2; ++t) {
      const int a = min(max(lo - 32 * t, 0), 32), b = min(max(hi - 32 * t, 0), 32);
      unsigned x = (unsigned)(((1ull << b) - 1) & ~((1ull << a) - 1)) >> 4 * hh & 0x0f0f0f0fu;   // keys of this half
      x = (x | x >> 4) & 0x00ff00ffu;
      bits |= ((x | x >> 8) & 0xffffu) << 16 * t;
    }
    return bits;
  };
  auto dist0 = [&](int qrel) __attribute__((always_inline)) {   // shape()'s dq; qrel: query minus the tile's first key
    return kHasBias ? (float)(qrel - 4 * (opaque(lane) >> 5)) : 0.f;
  };
  // The scores of the first tile, whole.
  auto first_scores = [&](f32x16 (&s)[kN2], float dq, float sl) __attribute__((always_inline)) {
    scores(0, s);
#pragma unroll
    for (int i = 0; i < kS; ++i) shape(i, s, dq, sl);
    return tile_max(s);
  };
  typedef u16 u16x2 __attribute__((ext_vector_type(2)));
  // A masked weight is 0, and 0 times NaN or infinity would reach rows that do not see the
  // key.  In a tile that some row sees only in part, scrub() looks at the V pieces that this
  // thread wrote (or asked for), sets such values to zero in LDS and returns the rows that held any
  // (the same in every thread); after the product, spill() adds them to the rows that see
  // them, read again from where they came.
  auto scrub = [&](int tile, auto piece_of, auto count) __attribute__((always_inline)) -> unsigned long long {
    constexpr int pieces = decltype(count)::value;
    const int ln = opaque(lane);
    auto piece = [&](int i) __attribute__((always_inline)) { return piece_of(i, ln); };
    u16x2 top = {0, 0};                                 // largest magnitude bits of each half word
#pragma unroll
    for (int i = 0; i < pieces; ++i) {
      const u32x4 v = *(lds_u32x4*)(uintptr_t)piece(i);
#pragma unroll
      for (int e = 0; e < 4; ++e) top = __builtin_elementwise_max(top, __builtin_bit_cast(u16x2, v[e] & 0x7fff7fffu));
    }
    if (__any(top.x >= 0x7f80 || top.y >= 0x7f80) && lane == 0) sOdd = tile;   // (each tile is looked at once)
    lds_sync();
    if ((int)uni((unsigned)sOdd) != tile) return 0;
    if (tid < 2) sBad[tid] = 0;
    __syncthreads();
#pragma unroll 1
    for (int i = 0; i < pieces; ++i) {
      const uint32_t at = piece(i);
      u32x4 v = *(lds_u32x4*)(uintptr_t)at;
      bool bad = false;
#pragma unroll
      for (int e = 0; e < 4; ++e) {
        unsigned x = v[e];
        if ((x & 0x7f80u) == 0x7f80u) x &= 0xffff0000u;
        if ((x & 0x7f800000u) == 0x7f800000u) x &= 0xffffu;
        bad = bad || x != v[e];
        v[e] = x;
      }
      if (bad) {
        *(lds_u32x4w*)(uintptr_t)at = v;
        const int r = (int)((at - lds_at(sT)) % kTile) / (2 * D);
        atomicOr(&sBad[r >> 5], 1u << (r & 31));
      }
    }
    __syncthreads();
    return (unsigned long long)uni(sBad[1]) << 32 | uni(sBad[0]);
  };
  auto spill = [&](unsigned long long bad, unsigned hidden, auto row) __attribute__((always_inline)) {
    const int ln = opaque(lane), q32 = ln & 31, hh = ln >> 5;
#pragma unroll 1
    for (; bad; bad &= bad - 1) {
      const int r = __builtin_ctzll(bad);
      // row r of the tile is key(i) of the lanes of half (r >> 2) & 1
      const unsigned hid = (unsigned)__shfl((int)hidden, q32 + 32 * (r >> 2 & 1), kWave);
      const bool see = !(hid >> (16 * (r >> 5) + 4 * (r >> 3 & 3) + (r & 3)) & 1);
      const auto value4 = row(r);
#pragma unroll
      for (int d = 0; d < kDT; ++d) {
        asm volatile("" ::: "memory");                  // (no loads ahead: this is the rare path)
#pragma unroll
        for (int r4 = 0; r4 < 4; ++r4) {
          const uint2 v = value4(32 * d + 8 * r4 + 4 * hh);   // four bf16
          const float x[4] = {bf_lo(v.x), bf_hi(v.x), bf_lo(v.y), bf_hi(v.y)};
#pragma unroll
          for (int e = 0; e < 4; ++e)
            if (see && (__float_as_uint(x[e]) & 0x7f800000u) == 0x7f800000u) o[d][4 * r4 + e] += x[e];
        }
      }
    }
  };

  // ---------------------------------------------------------------- new tokens
  int last = min(L, max(tz + 1, min(vis, L)));          // keys [first, last) are seen by some row
  int first = 0;
  if (p.window > 0) {
    first = (int)max((int64_t)0, (int64_t)ta - p.window + 1);
    last = (int)min((int64_t)last, (int64_t)tz + p.window);
  }
  int d0 = first / kBN, d1 = (last + kBN - 1) / kBN;    // tiles [d0, d1), from the last
  // Cached tiles x, x - 1, ... x0, without those that a window leaves out for every row
  int x0 = 0, x = CACHED ? (P + kBN - 1) / kBN - 1 : -1;
  if (CACHED && p.window > 0 && !p.c.pos) {             // (with `start` below P, rows ahead of the tokens too)
    x = (int)min((int64_t)x, max((int64_t)start + tz + p.window - 1, (int64_t)0) / kBN);
    x0 = (int)min((int64_t)(x + 1), max((int64_t)0, (int64_t)start + ta - p.window + 1) / kBN);
  }
  if (p.splits > 1) {                                   // this workgroup's part of both
    const int nd = max(d1 - d0, 0), nt = nd + x + 1 - x0;
    const int a = (int)((int64_t)nt * blockIdx.y / p.splits), b = (int)((int64_t)nt * (blockIdx.y + 1) / p.splits);
    d0 = d1 - min(b, nd);
    d1 -= min(a, nd);
    x0 = x + 1 - max(b - nd, 0);
    x -= max(a - nd, 0);
  }
  // Document mask: which key tiles hold a document of this workgroup's rows, a wave per
  // tile.  (Rows with a negative id see nothing: they take part as they come and give
  // zeros in the end.)
  if (doc) {
    if (tid == 0) {
      sDoc[0] = INT32_MAX;
      sDoc[1] = -1;
    }
    __syncthreads();
    for (int t = ta + tid; t <= tz; t += kExtThreads) {
      const int d = doc[t];
      if (d >= 0) {
        atomicMin(&sDoc[0], d);
        atomicMax(&sDoc[1], d);
      }
    }
    __syncthreads();
    const int dmin = sDoc[0], dmax = sDoc[1], lim = min(d1 - d0, kFlags);
    constexpr int kAhead = 8;
    for (int y = wave * kAhead; y < lim; y += 4 * kAhead) {
      int v[kAhead];
#pragma unroll
      for (int i = 0; i < kAhead; ++i) {
        const int j = (d1 - 1 - y - i) * kBN + lane;
        v[i] = j >= 0 && j < L ? doc[j] : -1;
      }
#pragma unroll
      for (int i = 0; i < kAhead; ++i) {
        const bool any = __any(v[i] >= 0 && v[i] >= dmin && v[i] <= dmax);
        const bool all = dmin == dmax && __all(v[i] == dmin);
        if (lane == 0 && y + i < lim) sFlag[y + i] = (any ? 1 : 0) | (all ? 2 : 0);
      }
    }
    __syncthreads();
  }
  // The next tile at or before t to look at, and whether it is all of the rows' one document:
  // flags of the 64 tiles from fb down are held as bits.  (Tiles past the table are looked at.)
  int fb = INT32_MAX;
  unsigned long long fany = 0, fall = 0;
  auto next = [&](int t, bool& all) __attribute__((always_inline)) {
    all = true;
    if (!doc) return t;
    while (t >= d0) {
      if (t <= fb - kWave) {
        fb = t;
        const int i = d1 - 1 - t + lane, flag = t - lane >= d0 ? (i < kFlags ? (int)sFlag[i] : 1) : 0;
        fany = __ballot(flag & 1);
        fall = __ballot(flag & 2);
      }
      const unsigned long long left = fany >> (fb - t);
      if (left) {
        t -= __builtin_ctzll(left);
        all = fall >> (fb - t) & 1;
        return t;
      }
      t = fb - kWave;
    }
    return t;
  };
  // Loads of tile t: this lane's piece of each of the wave's loads.  (Piece l % kPc of row
  // r in LDS is the row's piece (l % kPc) ^ swizzle(r); rows past the sequence read as zeros.)
  const uint32_t kst = (uint32_t)p.k_stride * 2, vst = (uint32_t)p.v_stride * 2;   // bytes
  const uint32_t ldsw = uni(lds_at(sT) + wave * 1024);
  const int fr = wave * kRpi + lane / kPc;              // row of the wave's first load; the next ones 4 kRpi further
  const uint32_t fc = (uint32_t)((lane % kPc) ^ row_swz<D>(fr)) << 4;
  auto fetch = [&](const char* src, uint32_t st, uint32_t row0, int t, uint32_t to, int s) __attribute__((always_inline)) {
    const int left = t >= d0 ? min(kBN, L - t * kBN) : 0;   // (behind the last tile nothing: zeros)
    const u32x4 rs = buffer_of(src + (int64_t)(t * kBN) * st, left > 0 ? (left - 1) * st + 2 * D : 0);
    // (8 rows on, the swizzle's bit 1 flips)
    to_lds(rs, row0 + s * (4 * kRpi * st) + (4 * kRpi * s & 8 ? fc ^ 32 : fc), ldsw + to + s * 4096);
  };
  const uint32_t rowk = fr * kst, rowv = fr * vst;
  const char* const ksrc = (const char*)(p.k + (int64_t)t0 * p.k_stride + (int64_t)h * D);
  const char* const vsrc = (const char*)(p.v + (int64_t)t0 * p.v_stride + (int64_t)h * D);
  auto fetch_k = [&](int t, uint32_t to, int s) __attribute__((always_inline)) { fetch(ksrc, kst, rowk, t, to, s); };
  auto fetch_v = [&](int t, uint32_t to, int s) __attribute__((always_inline)) { fetch(vsrc, vst, rowv, t, to + kTile, s); };
  // Tiles [wf, wl) are seen whole by all rows of the wave, [gf, gl) by the workgroup's
  // (documents aside): seen keys are a range, below the row's own or the prefix, inside the
  // window.
  auto whole = [&](int a, int z, int& from, int& to) __attribute__((always_inline)) {
    int hi = min(max(a + 1, min(vis, L)), L);
    from = 0;
    if (p.window > 0) {
      hi = (int)min((int64_t)hi, (int64_t)a + p.window);
      from = (max(z - p.window + 1, 0) + kBN - 1) / kBN;
    }
    to = hi / kBN;
  };
  int wf, wl, gf, gl;
  whole(wa, wz, wf, wl);
  whole(ta, tz, gf, gl);
  auto mask = [&](f32x16 (&s)[kN2], int t, bool all, float& mx) __attribute__((always_inline)) -> unsigned {
    const int j0 = t * kBN;
    unsigned hidden = 0;
    if (t < wf || t >= wl || !all) {
      int lo = 0, hi = min(max(ti + 1, vis), L) - j0;
      if (p.window > 0) {
        lo = ti - j0 - p.window + 1;
        hi = min(hi, ti - j0 + p.window);
      }
      hidden = ~seen_bits(lo, hi);
      if (!all) {                                       // the wave's own copy of the tile's ids
        const int ol = opaque(lane), oh = ol >> 5, j = j0 + ol;
        sIds[wave][ol] = j < L ? doc[j] : -1;
        lds_order();
#pragma unroll
        for (int i = 0; i < kS; i += 4) {
          const int4 dj = *reinterpret_cast<const int4*>(&sIds[wave][key(i, oh)]);
          if (dj.x != di) hidden |= 1u << i;
          if (dj.y != di) hidden |= 2u << i;
          if (dj.z != di) hidden |= 4u << i;
          if (dj.w != di) hidden |= 8u << i;
        }
        lds_order();
      }
      hide(s, hidden, mx);
    }
    return hidden;
  };
  bool all_t, all_x, all_2;                                      // (all of one document: tiles t, nx, n2)
  int t = next(d1 - 1, all_t);
  if (t >= d0) {
    int nx = next(t - 1, all_x), n2 = next(nx - 1, all_2);    // the tiles after t
#pragma unroll
    for (int i = 0; i < kLd; ++i) fetch_k(t, 0, i);
    vm_wait();
    lds_sync();
#pragma unroll
    for (int i = 0; i < kLd; ++i) fetch_v(t, 0, i);
#pragma unroll
    for (int i = 0; i < kLd; ++i) fetch_k(nx, 2 * kTile, i);
    f32x16 s0[kN2], s1[kN2];
    float mx = first_scores(s0, dist0(ti - t * kBN), slope);
    unsigned hidden = mask(s0, t, all_t, mx);
    raise(mx);
    // Tile t (scores in s, V `kV` bytes behind the first), the next one's K in the other pair.
    auto top = [&](uint32_t kV) __attribute__((always_inline)) -> unsigned long long {
      vm_wait();                                        // this wave's share has landed
      lds_sync();                                       // everyone's has, and nobody reads the last tiles
      if (t >= gf && t < gl && all_t) return 0;
      return scrub(t, [&](int i, int ln) { return ldsw + kV + kTile + i * 4096 + ln * 16; }, Par<kLd>{});
    };
    auto dirty = [&](unsigned long long bad) __attribute__((always_inline)) {
      spill(bad, hidden, [&](int r) {
        const u16* at = p.v + (int64_t)(t0 + min(t * kBN + r, L - 1)) * p.v_stride + (int64_t)h * D;
        return [=](int col) { return *reinterpret_cast<const uint2*>(at + col); };
      });
    };
    auto one = [&](f32x16 (&s)[kN2], f32x16 (&s2)[kN2], uint32_t kV) __attribute__((always_inline)) {
      const uint32_t kK = 2 * kTile - kV;
      const unsigned long long bad = top(kV);
      unsigned hid2 = 0;
      const auto load = [&](int i) __attribute__((always_inline)) {
        if (i < kLd) fetch_k(n2, kV, i); else fetch_v(nx, kK, i - kLd);
      };
      step(s, s2, kK, kV, dist0(ti - nx * kBN), slope, Par<2 * kLd>{}, load,
           [&](f32x16 (&f)[kN2], float& mx) __attribute__((always_inline)) { hid2 = mask(f, nx, all_x, mx); });
      if (bad) dirty(bad);
      hidden = hid2;
      t = nx;
      all_t = all_x;
      nx = n2;
      all_x = all_2;
      n2 = next(n2 - 1, all_2);
    };
    uint32_t off = 0;
    auto turn = [&]() __attribute__((always_inline)) {
      off ^= 2 * kTile;
#pragma unroll
      for (int i = 0; i < kN2; ++i) s0[i] = s1[i];
    };
    if constexpr (CACHED) {
      // (one copy of the step: with two, and the cached rows' loop behind them, registers spill)
#pragma unroll 1
      while (nx >= d0) {
        one(s0, s1, off);
        turn();
      }
    } else {
#pragma unroll 1
      while (nx >= d0) {
        one(s0, s1, 0);
        if (nx < d0) {
          turn();
          break;
        }
        one(s1, s0, 2 * kTile);
      }
    }
    const unsigned long long bad = top(off);
    weights(s0);
    product(off);
    if (bad) dirty(bad);
  }

  // ---------------------------------------------------------------- cached rows
  if constexpr (CACHED) {
    lds_sync();                                         // the new tokens' tiles are read
    constexpr int kCp = D / 16;                         // 16-code pieces of a row
    constexpr int kCr = kWave / kCp;                    // rows that one wave's load brings
    constexpr int kCt = kBN / kCr / 4;                  // loads per wave and tile
    // A load brings 4, 8 or 16 rows of one page, so page addresses and scales are the same in
    // every lane of a wave.  Lane l holds those of page pb + l of the sequence (its place in
    // units of 16 rows, -1: not there), 64 pages at a time; a load's are read out of the lanes.
    const bool big = lg >= 6;
    int pb = 0, punit = -1;
    float pks = 0.f, pvs = 0.f;
    auto pages = [&](int first) __attribute__((always_inline)) {
      pb = first;
      const int j = first + lane, id = j < ((P + pmask) >> lg) ? page_of(p.c, n, j << lg) : -1;
      const int64_t at = (int64_t)max(id, 0) * p.H_kv + h;
      punit = id < 0 ? -1 : (int)(at << (lg - 4));
      // (rows that are not there are zeros, which another page's scale could turn into NaN)
      pks = id < 0 ? 1.f : p.c.k_scale[at];
      pvs = id < 0 ? 1.f : p.c.v_scale[at];
    };
    auto lane_of = [&](int row) __attribute__((always_inline)) { return (row >> lg) - pb; };
    auto unit_of = [&](int pl) __attribute__((always_inline)) { return __builtin_amdgcn_readlane(punit, pl & 63); };   // (-1: not there)
    const uint32_t rlane = (uint32_t)(lane / kCp) * D + 16 * (lane % kCp);   // this lane's piece of a load
    const uint32_t raws = uni(lds_at(sT) + 2 * kTile + wave * 1024);   // codes: K and V, kTile / 2 bytes each, behind the first tiles
    auto fetch = [&](const uint8_t* src, uint32_t to, int unit, int s) __attribute__((always_inline)) {
      to_lds(buffer_of(src + (int64_t)unit * (16 * D) + (wave * kCr & 15) * D, kCr * D), rlane, to + s * 4096);
    };
    auto units = [&](int x, int* u) __attribute__((always_inline)) {   // places of a tile's loads (whole pages: of one)
      if (big) {
        const int first = max(unit_of(lane_of(x * kBN)), 0) + ((x * kBN & pmask) >> 4);
#pragma unroll
        for (int s = 0; s < kCt; ++s) u[s] = first + ((wave + 4 * s) * kCr >> 4);
      } else {
#pragma unroll
        for (int s = 0; s < kCt; ++s) {
          const int r = x * kBN + (wave + 4 * s) * kCr;
          u[s] = max(unit_of(lane_of(r)), 0) + ((r & pmask) >> 4);
        }
      }
    };
    auto fetch_all = [&](const uint8_t* src, uint32_t to, int x) __attribute__((always_inline)) {
      int u[kCt];
      units(x, u);
#pragma unroll
      for (int s = 0; s < kCt; ++s) fetch(src, to, u[s], s);
    };
    auto lane_f = [&](float v, int pl) __attribute__((always_inline)) {
      return __uint_as_float((unsigned)__builtin_amdgcn_readlane((int)__float_as_uint(v), pl & 63));
    };
    // Codes of tile x -> bf16 (rows that are not held -> zeros).
    auto put = [&](const u32x4& w, float sc, uint32_t at) __attribute__((always_inline)) {
#pragma unroll
      for (int e = 0; e < 2; ++e) {
        const uint2 a = f8x4_to_bf16(w[2 * e], sc), b = f8x4_to_bf16(w[2 * e + 1], sc);
        *(lds_u32x4w*)(uintptr_t)(at ^ 16 * e) = u32x4{a.x, a.y, b.x, b.y};
      }
    };
    auto convert = [&](uint32_t from, uint32_t to, float lane_scale, int x) __attribute__((always_inline)) {
      // (the rows of a lane's loads lie a multiple of 16 apart: one swizzle)
      const int ol = opaque(lane), pl = lane_of(x * kBN), r = wave * kCr + ol / kCp;
      const uint32_t at = lds_at(sT) + to + r * 2 * D + ((2 * (ol % kCp) ^ row_swz<D>(r)) << 4);
      u32x4 w[kCt];
#pragma unroll
      for (int s = 0; s < kCt; ++s) w[s] = *(lds_u32x4*)(uintptr_t)(from + s * 4096 + ol * 16);
      if (big && x * kBN + kBN <= P && unit_of(pl) >= 0) {
        const float sc = lane_f(lane_scale, pl);
#pragma unroll
        for (int s = 0; s < kCt; ++s) put(w[s], sc, at + s * (8 * kCr * D));
      } else {
#pragma unroll
        for (int s = 0; s < kCt; ++s) {
          const int r0 = 4 * s * kCr, l0 = lane_of(x * kBN + wave * kCr + r0);
          if (unit_of(l0) < 0 || x * kBN + r + r0 >= P) w[s] = u32x4{0, 0, 0, 0};
          put(w[s], lane_f(lane_scale, l0), at + s * (8 * kCr * D));
        }
      }
    };
    // Bit r: row x kBN + r is held.
    auto held = [&](int x) __attribute__((always_inline)) -> unsigned long long {
      if (big && x * kBN + kBN <= P && unit_of(lane_of(x * kBN)) >= 0) return ~0ull;
      unsigned long long bits = 0;
#pragma unroll
      for (int i = 0; i < 4; ++i) {                     // 16 rows lie on one page
        const int left = P - x * kBN - 16 * i;
        if (left > 0 && unit_of(lane_of(x * kBN + 16 * i)) >= 0)
          bits |= (left >= 16 ? 0xffffull : (1ull << left) - 1) << 16 * i;
      }
      return bits;
    };
    // Mask of tile x's scores (and the bias, where rows hold positions of their own); returns
    // the hidden keys.
    auto mask = [&](f32x16 (&s)[kN2], int x, unsigned long long now, float& mx) __attribute__((always_inline)) -> unsigned {
      unsigned hidden = 0;
      const int j0 = x * kBN, oh = opaque(lane) >> 5;
      if (now != ~0ull) {
#pragma unroll
        for (int i = 0; i < kS; i += 4) hidden |= ((unsigned)(~now >> key(i, oh)) & 15u) << i;
      }
      if (p.c.pos && (kHasBias || p.window > 0)) {
        const int qpos = start + ti;
#pragma unroll
        for (int i = 0; i < kS; i += 4) {
          asm volatile("" ::: "memory");                // (one at a time: registers)
          const int r = j0 + key(i, oh), pg = r < P ? page_of(p.c, n, r) : -1;
          int4 kp = make_int4(qpos, qpos, qpos, qpos);
          if (pg >= 0) kp = *reinterpret_cast<const int4*>(p.c.pos + page_rows(p.c, pg, h) + (r & pmask));
#pragma unroll
          for (int e = 0; e < 4; ++e) {
            const int dist = abs(qpos - (e == 0 ? kp.x : e == 1 ? kp.y : e == 2 ? kp.z : kp.w));
            if (kHasBias) s[i >> 4][(i & 15) + e] -= slope * (float)dist;
            if (p.window > 0 && dist >= p.window) hidden |= 1u << (i + e);
          }
        }
        mx = tile_max(s);
      } else if (p.window > 0 && (start + wz - j0 >= p.window || j0 + kBN - 1 - (start + wa) >= p.window)) {
        const int qrel = start + ti - j0;
        hidden |= ~seen_bits(qrel - p.window + 1, qrel + p.window);
      }
      hide(s, hidden, mx);
      return hidden;
    };
    if (x >= x0) {
      // K runs a tile ahead of V; x - 2 is the furthest tile whose pages are looked at
      auto block = [&](int x) __attribute__((always_inline)) { pages(max(((x * kBN + kBN - 1) >> lg) - (kWave - 1), 0)); };
      auto ahead = [&](int x) __attribute__((always_inline)) {
        if (lane_of(max(x - 2, x0) * kBN) < 0) block(x);
      };
      block(x);
      fetch_all(p.c.k, raws, x);
      vm_wait();
      convert(raws, 0, pks, x);
      lds_sync();
      fetch_all(p.c.v, raws + kTile / 2, x);
      fetch_all(p.c.k, raws, max(x - 1, x0));
      f32x16 s0[kN2], s1[kN2];
      const float sl = p.c.pos ? 0.f : slope;           // (positions of their own: mask() subtracts the bias)
      float mx = first_scores(s0, dist0(start + ti - x * kBN), sl);
      unsigned hidden = mask(s0, x, held(x), mx);
      raise(mx);
      auto top = [&](bool more) __attribute__((always_inline)) -> unsigned long long {
        vm_wait();                                      // this wave's codes have landed
        lds_sync();                                     // nobody reads the last tiles any more
        convert(raws + kTile / 2, kTile, pvs, x);
        if (more) convert(raws, 0, pks, x - 1);
        unsigned long long bad = 0;
        // (rows that are not held are zeros; only a window hides a held row from some rows)
        if (p.window > 0 && (p.c.pos || start + tz - x * kBN >= p.window || x * kBN + kBN - 1 - (start + ta) >= p.window))
          bad = scrub(-2 - x, [&](int i, int ln) { return lds_at(sT) + kTile + ((wave + 4 * (i >> 1)) * kCr + ln / kCp) * 2 * D +
                                                  (((2 * (ln % kCp) + (i & 1)) ^ row_swz<D>((wave + 4 * (i >> 1)) * kCr + ln / kCp)) << 4); },
                      Par<2 * kCt>{});
        lds_sync();
        return bad;
      };
      auto dirty = [&](unsigned long long bad) __attribute__((always_inline)) {
        spill(bad, hidden, [&](int r) {
          const int row = min(x * kBN + r, P - 1), pg = max(page_of(p.c, n, row), 0);
          const uint8_t* at = p.c.v + (page_rows(p.c, pg, h) + (row & pmask)) * D;
          const float sc = lane_f(pvs, lane_of(row));     // (code * scale may pass the largest float)
          return [=](int col) { return f8x4_to_bf16(*reinterpret_cast<const uint32_t*>(at + col), sc); };
        });
      };
      auto one = [&](f32x16 (&s)[kN2], f32x16 (&s2)[kN2]) __attribute__((always_inline)) {
        const unsigned long long bad = top(true);
        unsigned hid2 = 0;
        ahead(x);
        int uv[kCt], uk[kCt];
        units(x - 1, uv);
        units(max(x - 2, x0), uk);
        const auto load = [&](int i) __attribute__((always_inline)) {
          if (i < kCt) fetch(p.c.v, raws + kTile / 2, uv[i], i); else fetch(p.c.k, raws, uk[i - kCt], i - kCt);
        };
        step(s, s2, 0, 0, dist0(start + ti - (x - 1) * kBN), sl, Par<2 * kCt>{}, load,
             [&](f32x16 (&f)[kN2], float& mx) __attribute__((always_inline)) { hid2 = mask(f, x - 1, held(x - 1), mx); });
        if (bad) dirty(bad);
        hidden = hid2;
        --x;
      };
#pragma unroll 1
      while (x > x0) {
        one(s0, s1);
#pragma unroll
        for (int i = 0; i < kN2; ++i) s0[i] = s1[i];
      }
      const unsigned long long bad = top(false);
      weights(s0);
      product(0u);
      if (bad) dirty(bad);
      vm_wait();                                        // (the last tile's spare loads)
    }
  }

  l += __shfl_xor(l, 32, kWave);
  if (!live) return;
  if (p.splits > 1) {                                   // sums and outputs as they are, for extend_join_kernel
    const int64_t row = ((int64_t)blockIdx.y * p.T + t0 + ti) * p.H + hq;
    const bool none = doc && di < 0;
    if (hh == 0) *reinterpret_cast<float2*>(p.part_ml + 2 * row) = none ? make_float2(-INFINITY, 0.f) : make_float2(SHAPE == kRaw ? m * c1 : m, l);
    float* at = p.part_o + row * D;
#pragma unroll
    for (int d = 0; d < kDT; ++d)
#pragma unroll
      for (int r4 = 0; r4 < 4; ++r4)
        *reinterpret_cast<float4*>(at + 32 * d + 8 * r4 + 4 * hh) =
            none ? make_float4(0.f, 0.f, 0.f, 0.f)
                 : make_float4(o[d][4 * r4], o[d][4 * r4 + 1], o[d][4 * r4 + 2], o[d][4 * r4 + 3]);
    return;
  }
  float inv = l > 0.f ? 1.0f / l : (l == 0.f ? 0.f : l);   // nothing seen: zeros; a NaN sum stays NaN
  if (doc && di < 0) {                                  // a row outside of all documents
    inv = 0.f;
#pragma unroll
    for (int d = 0; d < kDT; ++d)
#pragma unroll
      for (int e = 0; e < 16; ++e) o[d][e] = 0.f;
  }
  u16* at = p.out + (int64_t)(t0 + ti) * p.out_stride + (int64_t)hq * D;
#pragma unroll
  for (int d = 0; d < kDT; ++d)
#pragma unroll
    for (int r4 = 0; r4 < 4; ++r4)
      *reinterpret_cast<uint2*>(at + 32 * d + 8 * r4 + 4 * hh) =
          make_uint2(cvt2(o[d][4 * r4] * inv, o[d][4 * r4 + 1] * inv), cvt2(o[d][4 * r4 + 2] * inv, o[d][4 * r4 + 3] * inv));
}

// Joins the parts of a row: o = sum_s o_s 2^(m_s - M) / sum_s l_s 2^(m_s - M), M the largest m_s.
// D / 4 lanes per (token, head), the heads of a token side by side.
template <int D> __global__ void __launch_bounds__(kExtThreads) extend_join_kernel(const AttnExtendLaunch p) {
  constexpr int kLanes = D / 4;
  const int t = blockIdx.x, hq = blockIdx.y * (kExtThreads / kLanes) + threadIdx.x / kLanes, c = threadIdx.x % kLanes * 4;
  if (t < p.cu[0] || t >= p.cu[p.N]) return;            // (in every lane; rows that no sequence holds)
  const int n = find_last(p.N, threadIdx.x & 63, [&](int i) { return p.cu[i] <= t; });
  if (hq >= p.H || (p.cache_len && p.cache_len[n] < 0)) return;
  const int64_t step = p.T * p.H, row = (int64_t)t * p.H + hq;
  float M = -INFINITY, l = 0.f;
#pragma unroll 4
  for (int s = 0; s < p.splits; ++s) M = fmaxf(M, p.part_ml[2 * (row + s * step)]);
  float4 o = make_float4(0.f, 0.f, 0.f, 0.f);
#pragma unroll 4
  for (int s = 0; s < p.splits; ++s) {
    const float2 ml = *reinterpret_cast<const float2*>(p.part_ml + 2 * (row + s * step));
    const float4 x = *reinterpret_cast<const float4*>(p.part_o + (row + s * step) * D + c);
    const float f = ml.x == -INFINITY ? 0.f : __builtin_amdgcn_exp2f(ml.x - M);   // (0 times a NaN sum stays NaN)
    l += ml.y * f;
    o.x += x.x * f;
    o.y += x.y * f;
    o.z += x.z * f;
    o.w += x.w * f;
  }
  const float inv = l > 0.f ? 1.0f / l : (l == 0.f ? 0.f : l);
  *reinterpret_cast<uint2*>(p.out + (int64_t)t * p.out_stride + (int64_t)hq * D + c) =
      make_uint2(cvt2(o.x * inv, o.y * inv), cvt2(o.z * inv, o.w * inv));
}

template <int D, int SHAPE>
hipError_t launch_shape(const AttnExtendLaunch& p, hipStream_t s) {
  const int64_t slots = p.T * (p.H / p.H_kv) / kBM + p.N;
  const dim3 grid((unsigned)(slots * p.H_kv), (unsigned)p.splits);
  if (p.c.k)
    extend_kernel<D, true, SHAPE><<<grid, kExtThreads, 0, s>>>(p);
  else
    extend_kernel<D, false, SHAPE><<<grid, kExtThreads, 0, s>>>(p);
  const hipError_t e = hipGetLastError();
  if (p.splits == 1 || e != hipSuccess) return e;
  constexpr int kRows = kExtThreads / (D / 4);
  extend_join_kernel<D><<<dim3((unsigned)p.T, (p.H + kRows - 1) / kRows), kExtThreads, 0, s>>>(p);
  return hipGetLastError();
}

template <int D>
hipError_t launch_d(const AttnExtendLaunch& p, hipStream_t s) {
  if (p.softcap > 0.f) return p.slopes ? launch_shape<D, kCapBias>(p, s) : launch_shape<D, kCap>(p, s);
  return p.slopes || !(p.scale > 0.f) ? launch_shape<D, kBias>(p, s) : launch_shape<D, kRaw>(p, s);
}

}  // namespace

// How a call is cut.  Parts of every row's keys: a workgroup walks its keys one tile after
// the other (about 1.25 us a tile, 2.5 at d = 256), so with few rows most of the chip waits
// for a few long walks: 16 tokens over 8000 cached rows, 32 / 8 heads, d = 128: 196 us
// whole, 25 in 16 parts; 512 over 8000 222 and 106; 64 over 16000, 16 / 2, d = 256: 667 and
// 62.  Parts cost a launch and their way through memory, about 5 us and 15 with all places
// taken by full tiles, and pay where the walk is shortened by more: 1024 new tokens 23 us
// whole, 36 in two parts; 8 over 600 22 and 18.  All parts have a place at once (two
// workgroups per CU, one at d = 256; twice as many for the sake of uneven sequences: 2 x 256
// over 7000, d = 256, 111 -> 128) and four tiles or more.  Tiles do not cross sequences: with
// many short ones the launch's workgroups are counted, one per sequence at least and up to one
// more that finds no rows, so that an eighth over is no second round (4 tokens each over 7000
// rows: 16 sequences, 32 / 8, d = 128: 4 parts 70 us, 16 80; 32 of 16 / 2, d = 256: 3 113, 16
// 133).  Where fewer than three have a place then, up to four even out the rounds (whole, in 4
// and in 16 parts: 48 sequences, 32 / 8, d = 128 243, 215 and 245 us; 64 of 16 / 2, d = 256 304,
// 249 and 246; but 64 of 32 / 8, d = 128 275, 285 and 327).
void plan_attn_extend(AttnExtendLaunch& p, int64_t keys, int cus) {
  const int64_t group = p.H / p.H_kv, places = (int64_t)cus * (p.d <= 128 ? 2 : 1);
  const int64_t wgs = (p.T * group + kBM - 1) / kBM * p.H_kv, grid = (p.T * group / kBM + p.N) * p.H_kv;
  const int64_t fit = 9 * places / (8 * grid), most = keys / (4 * 64);
  int64_t s = places / wgs;
  if (s > (fit >= 3 ? fit : 4)) s = fit >= 3 ? fit : 4;
  if (s > most) s = most;
  if (s > kMaxSplits) s = kMaxSplits;
  const double tiles = (double)keys / 64, step = p.d == 256 ? 2.5 : 1.25;
  p.splits = s > 1 && tiles * step * (double)(s - 1) / (double)s > 5 + 15.0 * (double)(s * wgs) / (double)places ? (int)s : 1;
  // Where every CU gets two workgroups (d <= 128) and there are few more, the second ones run
  // from the shortest walk up, so that a long and a short one share a CU: 2 x 1024 tokens, 32 / 8
  // heads, d = 128 34 -> 29 us, 4095, 16 / 4 83 -> 80.  With more of them it is better to go
  // on from the longest (5000 tokens, 16 / 4: 110 us, 118 so), and over a cache, where walks are
  // alike, in the order of the batch (4 x 512 over 7000 rows, 32 / 8: 276 us, 390 so).
  p.fold = p.causal && !p.c.k && p.d <= 128 && grid > cus && 4 * grid <= 9 * (int64_t)cus ? (cus + p.H_kv - 1) / p.H_kv : INT32_MAX;
}

hipError_t launch_attn_extend(const AttnExtendLaunch& p, hipStream_t s) {
  switch (p.d) {
    case 64: return launch_d<64>(p, s);
    case 128: return launch_d<128>(p, s);
    default: return launch_d<256>(p, s);
  }
}

}  // namespace gdn
