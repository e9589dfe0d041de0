// Device helpers of the softmax-attention kernels: e4m3 conversions, page lookups, the
// scores' cap.
#pragma once
#include "attn_launch.h"
#include "tile_ops.h"

namespace gdn {

constexpr float kLog2e = 1.4426950408889634f;

// Power-of-two scale 2^e of a row set whose largest finite |x| has the bf16 bits `top`
// (sign cleared): the smallest e >= -64 with |x| <= 448 2^e.  With |x| = 1.f 2^(E-127)
// and 448 = 1.75 2^8: e = E - 127 - 8, one more when 1.f > 1.75 (bf16: f > 0x60).
__device__ __forceinline__ int scale_exp_of(unsigned top) {
  const int e = (int)(top >> 7) - 135 + ((top & 0x7f) > 0x60 ? 1 : 0);
  return e < -64 ? -64 : e;
}
__device__ __forceinline__ float exp2_int(int e) { return __uint_as_float((unsigned)(e + 127) << 23); }
__device__ __forceinline__ int exp_of(float s) { return (int)(__float_as_uint(s) >> 23 & 0xff) - 127; }

// four e4m3 codes -> bf16 times the power-of-two scale (exact: three fraction bits)
__device__ __forceinline__ uint2 f8x4_to_bf16(uint32_t w, float scale) {
  return make_uint2(__builtin_bit_cast(uint32_t, __builtin_amdgcn_cvt_scalef32_pk_bf16_fp8(w, scale, false)),
                    __builtin_bit_cast(uint32_t, __builtin_amdgcn_cvt_scalef32_pk_bf16_fp8(w, scale, true)));
}
__device__ __forceinline__ bf16x8 f8x8_to_op(uint32_t lo, uint32_t hi, float scale) {
  return join(f8x4_to_bf16(lo, scale), f8x4_to_bf16(hi, scale));
}
// four floats -> e4m3, round to nearest even; |x| <= 448 or NaN (the caller's scale)
__device__ __forceinline__ uint32_t to_f8x4(float a, float b, float c, float d) {
  int w = __builtin_amdgcn_cvt_pk_fp8_f32(a, b, 0, false);
  return (uint32_t)__builtin_amdgcn_cvt_pk_fp8_f32(c, d, w, true);
}
// four codes rounded again to a scale 2^grow times as large
__device__ __forceinline__ uint32_t f8x4_rescale(uint32_t w, float shrink) {
  const f32x2 a = __builtin_amdgcn_cvt_pk_f32_fp8((int)w, false);
  const f32x2 b = __builtin_amdgcn_cvt_pk_f32_fp8((int)w, true);
  return to_f8x4(a.x * shrink, a.y * shrink, b.x * shrink, b.y * shrink);
}

// The page that holds row r of sequence n, or -1 when its id is out of range (or r lies
// past the table).
__device__ __forceinline__ int page_of(const CacheRef& c, int n, int r) {
  const int j = r >> c.page_log2;
  if (j >= c.table_width) return -1;
  const int id = c.table[(int64_t)n * c.table_stride + j];
  return id >= 0 && id < c.num_pages ? id : -1;
}
__device__ __forceinline__ int64_t page_rows(const CacheRef& c, int page, int h) {   // first row of (page, kv head)
  return ((int64_t)page * c.H_kv + h) << c.page_log2;
}

// Largest n in [0, N) with le(n), for le true at 0 and then false from some n on: 64 probes
// at a time, the same in every lane of a wave (which all take part).
template <typename F> __device__ __forceinline__ int find_last(int N, int lane, F le) {
  int lo = 0, hi = N;
  while (hi - lo > 1) {
    const int step = (hi - lo + kWave - 1) / kWave, i = lo + lane * step;
    const int n = __builtin_popcountll(__ballot(i < hi && (lane == 0 || le(i))));
    lo += (n - 1) * step;
    hi = min(hi, lo + step);
  }
  return lo;
}

// Raw score q.k -> score in units of log2, after scale and cap: with f1 = scale / cap and
// f2 = cap log2 e:  f2 tanh(f1 x), tanh(y) = 1 - 2 / (1 + e^2y).  Near 0 that form is
// off by a few 2^-24 absolutely, i.e. by cap 2^-22 in the score: below the error of the
// bf16 output for every cap that a call may have (8192 at most).
__device__ __forceinline__ float capped(float x, float f1x2log2e, float f2) {
  const float e = __builtin_amdgcn_exp2f(x * f1x2log2e);
  return fmaf(-2.0f * f2, __builtin_amdgcn_rcpf(1.0f + e), f2);
}

// Maximum over the two 32-lane halves, in every lane: the swap leaves one half's value of
// the pair in each result.  (Two registers: the instruction exchanges them in place.)
__device__ __forceinline__ float half_max(float v) {
  unsigned a = __float_as_uint(v), b = a;
  asm volatile("" : "+v"(b));
  const u32x2 r = __builtin_amdgcn_permlane32_swap(a, b, false, false);
  return fmaxf(__uint_as_float(r.x), __uint_as_float(r.y));
}

}  // namespace gdn
