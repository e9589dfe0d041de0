// Root-mean-square norm with the residual's addition, a gate and an output in 8 bits
// (gdn_rms_norm).  Each value is read once and written once, a few dozen operations apart:
// memory is the bound, so a row stays on chip between its two reductions (the parts' sums of
// squares, and in 8 bits the groups' maxima).
//   row_kernel : a row in the registers of 1, 4 or 16 waves, 8 values per thread and piece.
//   lds_kernel : rows or parts of fewer than 8 values: the row in LDS.  Rows too long for either
//                are read again for each pass (from the caches).
#include "step_launch.h"
#include "step_math.h"

namespace gdn {

namespace {

constexpr float kMinScale = 5.421010862427522e-20f;   // 2^-64

__device__ __forceinline__ bool not_finite(float v) { return (__float_as_uint(v) & 0x7f800000u) == 0x7f800000u; }
__device__ __forceinline__ float finite_abs(float v) { return not_finite(v) ? 0.0f : fabsf(v); }
__device__ __forceinline__ float nan_unless_finite(float v) { return not_finite(v) ? __uint_as_float(0x7fc00000u) : v; }
// v / scale, rounded once, with inv = 1 / scale: the product and what it leaves of v (exact in a
// fused one).  The product alone put about one code in a million on the other side of a border;
// two instructions a value, hidden behind memory but for the gated norm (134 -> 137 us at 32768 x 32 x 128).
__device__ __forceinline__ float quotient(float v, float scale, float inv) {
  const float q = v * inv;
  return fmaf(fmaf(-q, scale, v), inv, q);
}

// Maximum over aligned groups of `lanes` lanes (a power of two <= 64), in each of them.
__device__ __forceinline__ float lanes_max(float v, int lanes) {
  if (lanes >= 2) v = fmaxf(v, dpp_row<0xB1>(v));
  if (lanes >= 4) v = fmaxf(v, dpp_row<0x4E>(v));
  if (lanes >= 8) v = fmaxf(v, dpp_row<0x141>(v));
  if (lanes >= 16) v = fmaxf(v, dpp_row<0x140>(v));
  if (lanes >= 32) v = fmaxf(v, __shfl_xor(v, 16, kWave));
  if (lanes >= 64) v = fmaxf(v, __shfl_xor(v, 32, kWave));
  return v;
}
__device__ __forceinline__ float lanes_sum(float v, int lanes) {
  if (lanes >= 2) v += dpp_row<0xB1>(v);
  if (lanes >= 4) v += dpp_row<0x4E>(v);
  if (lanes >= 8) v += dpp_row<0x141>(v);
  if (lanes >= 16) v += dpp_row<0x140>(v);
  if (lanes >= 32) v += __shfl_xor(v, 16, kWave);
  if (lanes >= 64) v += __shfl_xor(v, 32, kWave);
  return v;
}

// ------------------------------------------------------------------ rows in registers
// Eight values from element i of a row operand on.  kWhole: in aligned pieces; else at any
// element (the card takes wide loads and stores at any address).
struct __attribute__((packed, aligned(1))) Loose4 { uint32_t u[4]; };
struct __attribute__((packed, aligned(1))) Loose2 { uint32_t u[2]; };

template <bool kWhole>
__device__ __forceinline__ Loose4 load_piece(const void* p) {
  if constexpr (kWhole) {
    const uint4 w = *static_cast<const uint4*>(p);
    return {{w.x, w.y, w.z, w.w}};
  } else {
    return *static_cast<const Loose4*>(p);
  }
}
template <bool kWhole>
__device__ __forceinline__ void load_values(const void* p, int bf16, int64_t i, float (&v)[8]) {
  if (bf16) {
    const Loose4 w = load_piece<kWhole>(static_cast<const u16*>(p) + i);
#pragma unroll
    for (int k = 0; k < 4; ++k) {
      v[2 * k] = __uint_as_float(w.u[k] << 16);
      v[2 * k + 1] = __uint_as_float(w.u[k] & 0xffff0000u);
    }
  } else {
    const Loose4 a = load_piece<kWhole>(static_cast<const float*>(p) + i), b = load_piece<kWhole>(static_cast<const float*>(p) + i + 4);
#pragma unroll
    for (int k = 0; k < 4; ++k) {
      v[k] = __uint_as_float(a.u[k]);
      v[4 + k] = __uint_as_float(b.u[k]);
    }
  }
}
// The values from `lo` on are written (0: all; 8: none).
template <bool kWhole>
__device__ __forceinline__ void store_piece(void* p, const Loose4& w) {
  if constexpr (kWhole) *static_cast<uint4*>(p) = make_uint4(w.u[0], w.u[1], w.u[2], w.u[3]);
  else *static_cast<Loose4*>(p) = w;
}
template <bool kWhole>
__device__ __forceinline__ void store_values(void* p, int bf16, int64_t i, int lo, const float (&v)[8]) {
  if (lo == 0) {
    if (bf16) {
      bf16x8 b;
#pragma unroll
      for (int k = 0; k < 8; ++k) b[k] = (__bf16)v[k];
      store_piece<kWhole>(static_cast<u16*>(p) + i, __builtin_bit_cast(Loose4, b));
    } else {
#pragma unroll
      for (int k = 0; k < 2; ++k)
        store_piece<kWhole>(static_cast<float*>(p) + i + 4 * k,
                            __builtin_bit_cast(Loose4, make_float4(v[4 * k], v[4 * k + 1], v[4 * k + 2], v[4 * k + 3])));
    }
  } else if (!kWhole && lo < 8) {
#pragma unroll
    for (int k = 1; k < 8; ++k)
      if (k >= lo) {
        if (bf16) static_cast<u16*>(p)[i + k] = f32_to_bf16(v[k]);
        else static_cast<float*>(p)[i + k] = v[k];
      }
  }
}
template <bool kWhole>
__device__ __forceinline__ void store_codes(uint8_t* p, int64_t i, int lo, const float (&v)[8]) {
  int a = __builtin_amdgcn_cvt_pk_fp8_f32(v[0], v[1], 0, false);
  a = __builtin_amdgcn_cvt_pk_fp8_f32(v[2], v[3], a, true);
  int b = __builtin_amdgcn_cvt_pk_fp8_f32(v[4], v[5], 0, false);
  b = __builtin_amdgcn_cvt_pk_fp8_f32(v[6], v[7], b, true);
  if (lo == 0) {
    if constexpr (kWhole) *reinterpret_cast<uint2*>(p + i) = make_uint2((uint32_t)a, (uint32_t)b);
    else *reinterpret_cast<Loose2*>(p + i) = {{(uint32_t)a, (uint32_t)b}};
  } else if (!kWhole && lo < 8) {
#pragma unroll
    for (int k = 1; k < 8; ++k)
      if (k >= lo) p[i + k] = (uint8_t)((k < 4 ? a : b) >> (k % 4 * 8));
  }
}

// A row of W = H d values, 8 <= W <= 512 K RW, over RW waves: piece j of thread r holds the values
// 8 (64 RW j + r) on.  A row's last piece, where it is short, begins earlier, at W - 8, and its
// first `lo` values, which are another piece's too, are 0 and not written; a piece past the row
// is all of that: every load is whole, in the row, and under no branch (one that is waits for its
// data before the next is sent).  part_lanes: lanes of a part for H > 1 (d / 8, a power of two up
// to 64); kAny: parts of any size from 8 on, of which a piece meets two at most: their sums are
// formed from the pieces' in LDS.
template <bool kWhole, int K, int RW, bool kAny>
__global__ void __launch_bounds__(RW > 4 ? RW * kWave : 256) row_kernel(NormLaunch p, int part_lanes) {
  constexpr int kRows = RW >= 4 ? 1 : 4 / RW, kRowThreads = RW * kWave;
  constexpr int kPieces = kAny ? K * kRowThreads : 1;
  __shared__ float sums[kRows][RW], tops[kRows][RW];
  __shared__ float front[kRows][kPieces], back[kRows][kPieces], part_rstd[kRows][kPieces];
  const int row = threadIdx.x / kRowThreads, r = threadIdx.x % kRowThreads, wave = r / kWave;
  const int64_t asked = (int64_t)blockIdx.x * kRows + row, t = min(asked, p.T - 1);
  const int W = p.H * p.d;
  float u[K][8], g[K][8];
  int at[K], lo[K];
#pragma unroll
  for (int j = 0; j < K; ++j) {
    const int from = (j * kRowThreads + r) * 8;
    at[j] = min(from, W - 8);
    lo[j] = asked < p.T ? min(from - at[j], 8) : 8;
  }
#pragma unroll
  for (int j = 0; j < K; ++j) load_values<kWhole>(p.x, p.in_bf16, t * p.x_stride + at[j], u[j]);
  if (p.residual) {
#pragma unroll
    for (int j = 0; j < K; ++j) load_values<kWhole>(p.residual, p.residual_bf16, t * p.residual_stride + at[j], g[j]);
#pragma unroll
    for (int j = 0; j < K; ++j) {
#pragma unroll
      for (int v = 0; v < 8; ++v) u[j][v] += g[j][v];
      store_values<kWhole>(p.residual, p.residual_bf16, t * p.residual_stride + at[j], lo[j], u[j]);
    }
  } else if (p.gate) {
#pragma unroll
    for (int j = 0; j < K; ++j) load_values<kWhole>(p.gate, p.in_bf16, t * p.gate_stride + at[j], g[j]);
#pragma unroll
    for (int j = 0; j < K; ++j)
#pragma unroll
      for (int v = 0; v < 8; ++v) {
        g[j][v] = step_silu(g[j][v]);
        if (p.gate_first) u[j][v] *= g[j][v];
      }
  }
#pragma unroll
  for (int j = 0; j < K; ++j)
#pragma unroll
    for (int v = 0; v < 8; ++v) u[j][v] = v < lo[j] ? 0.0f : u[j][v];
  // 1 / sqrt(mean + eps) of every piece's part (kAny: of its first `cut` values, and of the others)
  float rstd[K], rstd2[K];
  int cut[K], part[K];
  if constexpr (kAny) {
    const float per_d = 1.0f / (float)p.d;
#pragma unroll
    for (int j = 0; j < K; ++j) {
      // at / d: (at + 1/2) / d is at least 1/2d from a whole number, the product off by less
      part[j] = (int)(((float)at[j] + 0.5f) * per_d);
      cut[j] = (part[j] + 1) * p.d - at[j];
      float a = 0.0f, b = 0.0f;
#pragma unroll
      for (int v = 0; v < 8; ++v) {
        const float sq = u[j][v] * u[j][v];
        a += v < cut[j] ? sq : 0.0f;
        b += v < cut[j] ? 0.0f : sq;
      }
      front[row][j * kRowThreads + r] = a;
      back[row][j * kRowThreads + r] = b;
    }
    __syncthreads();
    for (int h = r; h < p.H; h += kRowThreads) {
      float sum = 0.0f;
      for (int i = h * p.d / 8; i <= ((h + 1) * p.d - 1) / 8; ++i) sum += min(8 * i, W - 8) >= h * p.d ? front[row][i] : back[row][i];
      part_rstd[row][h] = 1.0f / sqrtf(sum * per_d + p.eps);
    }
    __syncthreads();
#pragma unroll
    for (int j = 0; j < K; ++j) {
      rstd[j] = part_rstd[row][part[j]];
      rstd2[j] = part_rstd[row][min(part[j] + 1, p.H - 1)];
    }
  } else if (p.H == 1) {
    float sum = 0.0f;
#pragma unroll
    for (int j = 0; j < K; ++j)
#pragma unroll
      for (int v = 0; v < 8; ++v) sum = fmaf(u[j][v], u[j][v], sum);
    sum = group_sum<64>(sum);
    if constexpr (RW > 1) {
      if (r % kWave == 0) sums[row][wave] = sum;
      __syncthreads();
      sum = 0.0f;
#pragma unroll
      for (int w = 0; w < RW; ++w) sum += sums[row][w];
    }
    const float q = 1.0f / sqrtf(sum / (float)p.d + p.eps);
#pragma unroll
    for (int j = 0; j < K; ++j) rstd[j] = q;
  } else {
#pragma unroll
    for (int j = 0; j < K; ++j) {
      float sum = 0.0f;
#pragma unroll
      for (int v = 0; v < 8; ++v) sum = fmaf(u[j][v], u[j][v], sum);
      rstd[j] = 1.0f / sqrtf(lanes_sum(sum, part_lanes) / (float)p.d + p.eps);
    }
  }
#pragma unroll
  for (int j = 0; j < K; ++j) {
    if constexpr (kAny) {
#pragma unroll
      for (int v = 0; v < 8; ++v) {
        float w = 1.0f;
        if (p.weight) {
          const int i = v < cut[j] ? at[j] + v - part[j] * p.d : v - cut[j];
          w = (p.weight_bf16 ? bf16_to_f32(static_cast<const u16*>(p.weight)[i]) : static_cast<const float*>(p.weight)[i]) + p.offset;
        }
        u[j][v] *= (v < cut[j] ? rstd[j] : rstd2[j]) * w;
      }
    } else if (p.weight) {
      float w[8];
      load_values<kWhole>(p.weight, p.weight_bf16, p.H == 1 ? at[j] : at[j] & (p.d - 1), w);   // (parts are powers of two)
#pragma unroll
      for (int v = 0; v < 8; ++v) u[j][v] *= rstd[j] * (w[v] + p.offset);
    } else {
#pragma unroll
      for (int v = 0; v < 8; ++v) u[j][v] *= rstd[j];
    }
    if (p.gate && !p.gate_first) {
#pragma unroll
      for (int v = 0; v < 8; ++v) u[j][v] *= g[j][v];
    }
  }
  if (p.out_dtype != GDN_E4M3) {
#pragma unroll
    for (int j = 0; j < K; ++j)
      store_values<kWhole>(p.out, p.out_dtype == GDN_BF16, t * p.out_stride + at[j], lo[j], u[j]);
    return;
  }
  // the groups' largest magnitudes (fmaxf passes NaN over; infinities are looked for)
  float top[K];
  bool odd = false;
#pragma unroll
  for (int j = 0; j < K; ++j) {
    top[j] = 0.0f;
#pragma unroll
    for (int v = 0; v < 8; ++v) top[j] = fmaxf(top[j], fabsf(u[j][v]));
    odd |= top[j] == __uint_as_float(0x7f800000u);
  }
  if (odd) {
#pragma unroll
    for (int j = 0; j < K; ++j) {
      top[j] = 0.0f;
#pragma unroll
      for (int v = 0; v < 8; ++v) {
        top[j] = fmaxf(top[j], finite_abs(u[j][v]));
        u[j][v] = nan_unless_finite(u[j][v]);
      }
    }
  }
  if (p.group == W && p.groups == 1) {
    float m = top[0];
#pragma unroll
    for (int j = 1; j < K; ++j) m = fmaxf(m, top[j]);
    m = lanes_max(m, 64);
    if constexpr (RW > 1) {
      if (r % kWave == 0) tops[row][wave] = m;
      __syncthreads();
#pragma unroll
      for (int w = 0; w < RW; ++w) m = fmaxf(m, tops[row][w]);
    }
#pragma unroll
    for (int j = 0; j < K; ++j) top[j] = m;
  } else {
#pragma unroll
    for (int j = 0; j < K; ++j) top[j] = lanes_max(top[j], p.group / 8);
  }
  const int shift = p.group == 64 ? 6 : 7;
#pragma unroll
  for (int j = 0; j < K; ++j) {
    if (lo[j] == 8) continue;
    const float scale = fmaxf(top[j] / 448.0f, kMinScale), inv = 1.0f / scale;
    const int from = at[j] + lo[j];                         // (a multiple of 8)
    if (p.groups == 1 ? from == 0 : (from & (p.group - 1)) == 0) p.scale[t * p.groups + (p.groups == 1 ? 0 : from >> shift)] = scale;
    float c[8];
#pragma unroll
    for (int v = 0; v < 8; ++v) c[v] = quotient(u[j][v], scale, inv);
    store_codes<kWhole>(static_cast<uint8_t*>(p.out), t * p.out_stride + at[j], lo[j], c);
  }
}

// ------------------------------------------------------------------ rows of any shape
__device__ __forceinline__ float load_any(const void* p, int bf16, int64_t i) {
  return bf16 ? bf16_to_f32(static_cast<const u16*>(p)[i]) : static_cast<const float*>(p)[i];
}

__device__ __forceinline__ void store_any(void* p, int bf16, int64_t i, float v) {
  if (bf16) static_cast<u16*>(p)[i] = f32_to_bf16(v);
  else static_cast<float*>(p)[i] = v;
}

// A workgroup takes a row; its waves take the row's parts in turn for the sums of squares, then
// the groups that share a scale.  kStage: the row's values in LDS; else formed again.
template <bool kStage>
__global__ void __launch_bounds__(256) lds_kernel(NormLaunch p) {
  extern __shared__ float lds[];                      // rstd [H], then the row
  float* rstd = lds;
  float* kept = lds + p.H;
  const int64_t t = blockIdx.x;
  const int wave = threadIdx.x / kWave, lane = threadIdx.x % kWave;
  const int width = p.H * p.d;
  const int64_t xr = t * p.x_stride, gr = t * p.gate_stride, rr = t * p.residual_stride, orow = t * p.out_stride;
  auto value = [&](int e) {
    float u = load_any(p.x, p.in_bf16, xr + e);
    if (p.residual) u += load_any(p.residual, p.residual_bf16, rr + e);
    if (p.gate && p.gate_first) u *= step_silu(load_any(p.gate, p.in_bf16, gr + e));
    return u;
  };
  auto put_residual = [&](int e, float u) { store_any(p.residual, p.residual_bf16, rr + e, u); };
  if constexpr (kStage) {
    for (int e = threadIdx.x; e < width; e += 256) {
      const float u = value(e);
      kept[e] = u;
      if (p.residual) put_residual(e, u);
    }
    __syncthreads();
  }
  for (int h = wave; h < p.H; h += 4) {
    float sum = 0.0f;
    for (int i = lane; i < p.d; i += kWave) {
      const float u = kStage ? kept[h * p.d + i] : value(h * p.d + i);
      sum = fmaf(u, u, sum);
    }
    sum = group_sum<64>(sum);
    if (lane == 0) rstd[h] = 1.0f / sqrtf(sum / (float)p.d + p.eps);
  }
  __syncthreads();
  const float per_d = 1.0f / (float)p.d;
  auto result = [&](int e, float u) {
    // e / d: (e + 1/2) / d is at least 1/2d from a whole number, the product off by less (e < 2^21)
    const int h = (int)(((float)e + 0.5f) * per_d), i = e - h * p.d;
    float y = u * rstd[h];
    if (p.weight) y *= load_any(p.weight, p.weight_bf16, i) + p.offset;
    if (p.gate && !p.gate_first) y *= step_silu(load_any(p.gate, p.in_bf16, gr + e));
    return y;
  };
  if (p.out_dtype != GDN_E4M3) {
    for (int e = threadIdx.x; e < width; e += 256) {
      const float u = kStage ? kept[e] : value(e);
      store_any(p.out, p.out_dtype == GDN_BF16, orow + e, result(e, u));
      if (!kStage && p.residual) put_residual(e, u);
    }
    return;
  }
  if constexpr (kStage) {
    for (int e = threadIdx.x; e < width; e += 256) kept[e] = result(e, kept[e]);
    __syncthreads();
  }
  for (int k = wave; k < p.groups; k += 4) {
    const int lo = k * p.group, hi = min(width, lo + p.group);
    float top = 0.0f;
    for (int e = lo + lane; e < hi; e += kWave) top = fmaxf(top, finite_abs(kStage ? kept[e] : result(e, value(e))));
    const float scale = fmaxf(lanes_max(top, 64) / 448.0f, kMinScale), inv = 1.0f / scale;
    if (lane == 0) p.scale[t * p.groups + k] = scale;
    for (int e = lo + lane; e < hi; e += kWave) {
      const float u = kStage ? 0.0f : value(e);
      const float c = quotient(nan_unless_finite(kStage ? kept[e] : result(e, u)), scale, inv);
      static_cast<uint8_t*>(p.out)[orow + e] = (uint8_t)__builtin_amdgcn_cvt_pk_fp8_f32(c, 0.0f, 0, false);
      if (!kStage && p.residual) put_residual(e, u);
    }
  }
}

bool wide(const void* p, int64_t stride, int64_t size) {   // 8 values at a time, in pieces of 16 bytes (codes: 8)
  const int64_t piece = size == 1 ? 8 : 16;
  return reinterpret_cast<uintptr_t>(p) % piece == 0 && stride * size % piece == 0;
}

template <bool kWhole, int K, int RW, bool kAny>
void launch_rows(const NormLaunch& p, int part_lanes, hipStream_t stream) {
  constexpr int kRows = RW >= 4 ? 1 : 4 / RW;
  hipLaunchKernelGGL((row_kernel<kWhole, K, RW, kAny>), dim3((unsigned)((p.T + kRows - 1) / kRows)),
                     dim3(RW > 4 ? RW * kWave : 256), 0, stream, p, part_lanes);
}

template <bool kWhole, bool kAny>
void launch_row_sizes(const NormLaunch& p, int64_t W, int part_lanes, hipStream_t stream) {
  // A wave a row up to 1024 values where there are rows for every wave of the chip, else four
  // waves, which are done sooner.  (Three pieces a thread where two are too few: with four 777 x 5003
  // took 12.5 us for 10.9, 5000 x 20000 191 for 172.)
  const bool many = p.T >= 1024;
  if (many && W <= 512) launch_rows<kWhole, 1, 1, kAny>(p, part_lanes, stream);
  else if (many && W <= 1024) launch_rows<kWhole, 2, 1, kAny>(p, part_lanes, stream);
  else if (W <= 2048) launch_rows<kWhole, 1, 4, kAny>(p, part_lanes, stream);
  else if (W <= 4096) launch_rows<kWhole, 2, 4, kAny>(p, part_lanes, stream);
  else if (W <= 6144) launch_rows<kWhole, 3, 4, kAny>(p, part_lanes, stream);
  else if (W <= 8192) launch_rows<kWhole, 4, 4, kAny>(p, part_lanes, stream);
  else if (W <= 16384) launch_rows<kWhole, 2, 16, kAny>(p, part_lanes, stream);
  else if (W <= 24576) launch_rows<kWhole, 3, 16, kAny>(p, part_lanes, stream);
  else launch_rows<kWhole, 4, 16, kAny>(p, part_lanes, stream);
}

// Parts of d values that are no 8 times a power of two up to 64.
bool any_parts(const NormLaunch& p) {
  const int lanes = p.d / 8;
  return p.H > 1 && !(p.d % 8 == 0 && lanes <= 64 && (lanes & (lanes - 1)) == 0);
}
bool in_registers(const NormLaunch& p) {
  const int64_t W = (int64_t)p.H * p.d;
  return W >= 8 && W <= 32768 && (!any_parts(p) || p.d >= 8);
}

}  // namespace

int64_t most_rms_norm_rows(const NormLaunch& p) {
  const int64_t W = (int64_t)p.H * p.d, threads = in_registers(p) && W > 8192 ? 16 * kWave : 256;   // (of a workgroup)
  return (((int64_t)1 << 32) - 1) / threads;
}

hipError_t launch_rms_norm(const NormLaunch& p, hipStream_t stream) {
  const int64_t W = (int64_t)p.H * p.d, in = p.in_bf16 ? 2 : 4, res = p.residual_bf16 ? 2 : 4;
  const int64_t out = p.out_dtype == GDN_E4M3 ? 1 : p.out_dtype == GDN_BF16 ? 2 : 4;
  const bool whole = W % 8 == 0 && wide(p.x, p.x_stride, in) && (!p.gate || wide(p.gate, p.gate_stride, in)) &&
                     (!p.residual || wide(p.residual, p.residual_stride, res)) && wide(p.out, p.out_stride, out) &&
                     reinterpret_cast<uintptr_t>(p.weight) % 16 == 0;
  const int lanes = p.d / 8;
  if (in_registers(p)) {
    if (any_parts(p)) launch_row_sizes<false, true>(p, W, lanes, stream);
    else if (whole) launch_row_sizes<true, false>(p, W, lanes, stream);
    else launch_row_sizes<false, false>(p, W, lanes, stream);
  } else if ((W + p.H) * 4 <= 65536) {
    hipLaunchKernelGGL(lds_kernel<true>, dim3((unsigned)p.T), dim3(256), (W + p.H) * sizeof(float), stream, p);
  } else {
    hipLaunchKernelGGL(lds_kernel<false>, dim3((unsigned)p.T), dim3(256), p.H * sizeof(float), stream, p);
  }
  return hipGetLastError();
}

}  // namespace gdn
