// Root-mean-square norm with the residual's addition, a gate and an output in 8 bits
// (gdn_rms_norm).  Each value is read once and written once, a few dozen operations apart:
// memory is the bound, so a row stays on chip between its two reductions (the parts' sums of
// squares, and in 8 bits the groups' maxima).
//   row_kernel : a row in the registers of 1, 4 or 16 waves, 8 values (or, where rows are
//                unaligned or odd, one) per thread and piece.
//   lds_kernel : parts that no power of two of lanes covers: the row in LDS.  Rows too long
//                for either are read again for each pass (from the caches).
#include "step_launch.h"
#include "step_math.h"

namespace gdn {

namespace {

constexpr float kMinScale = 5.421010862427522e-20f;   // 2^-64

__device__ __forceinline__ bool not_finite(float v) { return (__float_as_uint(v) & 0x7f800000u) == 0x7f800000u; }
__device__ __forceinline__ float finite_abs(float v) { return not_finite(v) ? 0.0f : fabsf(v); }
__device__ __forceinline__ float nan_unless_finite(float v) { return not_finite(v) ? __uint_as_float(0x7fc00000u) : v; }

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
// V consecutive values at element i of a row operand.
template <int V>
__device__ __forceinline__ void load_values(const void* p, int bf16, int64_t i, float (&v)[V]) {
  if constexpr (V == 8) {
    if (bf16) {
      const uint4 w = *reinterpret_cast<const uint4*>(static_cast<const u16*>(p) + i);
      const uint32_t u[4] = {w.x, w.y, w.z, w.w};
#pragma unroll
      for (int k = 0; k < 4; ++k) {
        v[2 * k] = __uint_as_float(u[k] << 16);
        v[2 * k + 1] = __uint_as_float(u[k] & 0xffff0000u);
      }
    } else {
      const float4 a = *reinterpret_cast<const float4*>(static_cast<const float*>(p) + i);
      const float4 b = *reinterpret_cast<const float4*>(static_cast<const float*>(p) + i + 4);
      v[0] = a.x; v[1] = a.y; v[2] = a.z; v[3] = a.w;
      v[4] = b.x; v[5] = b.y; v[6] = b.z; v[7] = b.w;
    }
  } else {
    v[0] = bf16 ? bf16_to_f32(static_cast<const u16*>(p)[i]) : static_cast<const float*>(p)[i];
  }
}
template <int V>
__device__ __forceinline__ void store_values(void* p, int bf16, int64_t i, const float (&v)[V]) {
  if constexpr (V == 8) {
    if (bf16) {
      bf16x8 b;
#pragma unroll
      for (int k = 0; k < 8; ++k) b[k] = (__bf16)v[k];
      *reinterpret_cast<bf16x8*>(static_cast<u16*>(p) + i) = b;
    } else {
      *reinterpret_cast<float4*>(static_cast<float*>(p) + i) = make_float4(v[0], v[1], v[2], v[3]);
      *reinterpret_cast<float4*>(static_cast<float*>(p) + i + 4) = make_float4(v[4], v[5], v[6], v[7]);
    }
  } else {
    if (bf16) static_cast<u16*>(p)[i] = f32_to_bf16(v[0]);
    else static_cast<float*>(p)[i] = v[0];
  }
}
template <int V>
__device__ __forceinline__ void store_codes(uint8_t* p, int64_t i, const float (&v)[V]) {
  if constexpr (V == 8) {
    int a = __builtin_amdgcn_cvt_pk_fp8_f32(v[0], v[1], 0, false);
    a = __builtin_amdgcn_cvt_pk_fp8_f32(v[2], v[3], a, true);
    int b = __builtin_amdgcn_cvt_pk_fp8_f32(v[4], v[5], 0, false);
    b = __builtin_amdgcn_cvt_pk_fp8_f32(v[6], v[7], b, true);
    *reinterpret_cast<uint2*>(p + i) = make_uint2((uint32_t)a, (uint32_t)b);
  } else {
    p[i] = (uint8_t)__builtin_amdgcn_cvt_pk_fp8_f32(v[0], 0.0f, 0, false);
  }
}

// A row of W = H d <= 64 V K RW values over RW waves: piece j of thread r holds the values
// (64 RW j + r) V on.  part_lanes: lanes of a part for H > 1 (V = 8: d / 8, a power of two up
// to 64).  A value past W is 0 and takes part in nothing.
template <int V, int K, int RW>
__global__ void __launch_bounds__(RW > 4 ? RW * kWave : 256) row_kernel(NormLaunch p, int part_lanes) {
  constexpr int kRows = RW >= 4 ? 1 : 4 / RW, kRowThreads = RW * kWave;
  __shared__ float sums[kRows][RW];
  __shared__ float tops[kRows][V == 1 ? K * RW : RW];
  const int row = threadIdx.x / kRowThreads, r = threadIdx.x % kRowThreads, wave = r / kWave;
  const int64_t t = (int64_t)blockIdx.x * kRows + row;
  const bool here = t < p.T;
  const int W = p.H * p.d;
  float u[K][V], g[K][V];
  int at[K];
#pragma unroll
  for (int j = 0; j < K; ++j) {
    at[j] = (j * kRowThreads + r) * V;
    if (!here || at[j] >= W) at[j] = -1;
  }
#pragma unroll
  for (int j = 0; j < K; ++j) {
#pragma unroll
    for (int v = 0; v < V; ++v) u[j][v] = 0.0f;
    if (at[j] >= 0) load_values<V>(p.x, p.in_bf16, t * p.x_stride + at[j], u[j]);
  }
  if (p.residual) {
#pragma unroll
    for (int j = 0; j < K; ++j)
      if (at[j] >= 0) load_values<V>(p.residual, p.residual_bf16, t * p.residual_stride + at[j], g[j]);
#pragma unroll
    for (int j = 0; j < K; ++j) {
      if (at[j] < 0) continue;
#pragma unroll
      for (int v = 0; v < V; ++v) u[j][v] += g[j][v];
      store_values<V>(p.residual, p.residual_bf16, t * p.residual_stride + at[j], u[j]);
    }
  } else if (p.gate) {
#pragma unroll
    for (int j = 0; j < K; ++j) {
#pragma unroll
      for (int v = 0; v < V; ++v) g[j][v] = 0.0f;
      if (at[j] >= 0) load_values<V>(p.gate, p.in_bf16, t * p.gate_stride + at[j], g[j]);
    }
#pragma unroll
    for (int j = 0; j < K; ++j)
#pragma unroll
      for (int v = 0; v < V; ++v) {
        g[j][v] = step_silu(g[j][v]);
        if (p.gate_first) u[j][v] *= g[j][v];
      }
  }
  // 1 / sqrt(mean + eps) of every piece's part
  float rstd[K];
  if (p.H == 1) {
    float sum = 0.0f;
#pragma unroll
    for (int j = 0; j < K; ++j)
#pragma unroll
      for (int v = 0; v < V; ++v) sum = fmaf(u[j][v], u[j][v], sum);
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
      for (int v = 0; v < V; ++v) sum = fmaf(u[j][v], u[j][v], sum);
      rstd[j] = 1.0f / sqrtf(lanes_sum(sum, part_lanes) / (float)p.d + p.eps);
    }
  }
#pragma unroll
  for (int j = 0; j < K; ++j) {
    float w[V];
#pragma unroll
    for (int v = 0; v < V; ++v) w[v] = 1.0f;
    if (p.weight && at[j] >= 0) {
      load_values<V>(p.weight, p.weight_bf16, p.H == 1 ? at[j] : at[j] & (p.d - 1), w);   // (parts are powers of two)
#pragma unroll
      for (int v = 0; v < V; ++v) w[v] += p.offset;
    }
#pragma unroll
    for (int v = 0; v < V; ++v) {
      u[j][v] *= rstd[j] * w[v];
      if (p.gate && !p.gate_first) u[j][v] *= g[j][v];
    }
  }
  if (p.out_dtype != GDN_E4M3) {
#pragma unroll
    for (int j = 0; j < K; ++j)
      if (at[j] >= 0) store_values<V>(p.out, p.out_dtype == GDN_BF16, t * p.out_stride + at[j], u[j]);
    return;
  }
  // the groups' largest magnitudes (fmaxf passes NaN over; infinities are looked for)
  float top[K];
  bool odd = false;
#pragma unroll
  for (int j = 0; j < K; ++j) {
    top[j] = 0.0f;
#pragma unroll
    for (int v = 0; v < V; ++v) top[j] = fmaxf(top[j], fabsf(u[j][v]));
    odd |= top[j] == __uint_as_float(0x7f800000u);
  }
  if (odd) {
#pragma unroll
    for (int j = 0; j < K; ++j) {
      top[j] = 0.0f;
#pragma unroll
      for (int v = 0; v < V; ++v) {
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
  } else if constexpr (V == 8) {
#pragma unroll
    for (int j = 0; j < K; ++j) top[j] = lanes_max(top[j], p.group / 8);
  } else {                      // a wave's piece is 64 values: one group, or half of one
#pragma unroll
    for (int j = 0; j < K; ++j) top[j] = lanes_max(top[j], 64);
    if (p.group == 128) {
#pragma unroll
      for (int j = 0; j < K; ++j)
        if (r % kWave == 0) tops[row][j * RW + wave] = top[j];
      __syncthreads();
#pragma unroll
      for (int j = 0; j < K; ++j) top[j] = fmaxf(top[j], tops[row][(j * RW + wave) ^ 1]);
    }
  }
#pragma unroll
  for (int j = 0; j < K; ++j) {
    if (at[j] < 0) continue;
    const float scale = fmaxf(top[j] / 448.0f, kMinScale), inv = 1.0f / scale;
    const int shift = p.groups == 1 ? 20 : p.group == 64 ? 6 : 7;
    if ((at[j] & ((1 << shift) - 1)) == 0) p.scale[t * p.groups + (at[j] >> shift)] = scale;
    float c[V];
#pragma unroll
    for (int v = 0; v < V; ++v) c[v] = u[j][v] * inv;
    store_codes<V>(static_cast<uint8_t*>(p.out), t * p.out_stride + at[j], c);
  }
}

// ------------------------------------------------------------------ rows of any shape
__device__ __forceinline__ float load_any(const void* p, int bf16, int64_t i) {
  return bf16 ? bf16_to_f32(static_cast<const u16*>(p)[i]) : static_cast<const float*>(p)[i];
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
  auto put_residual = [&](int e, float u) {
    const float v[1] = {u};
    store_values<1>(p.residual, p.residual_bf16, rr + e, v);
  };
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
  auto result = [&](int e, float u) {
    const int h = e / p.d, i = e - h * p.d;
    float y = u * rstd[h];
    if (p.weight) y *= load_any(p.weight, p.weight_bf16, i) + p.offset;
    if (p.gate && !p.gate_first) y *= step_silu(load_any(p.gate, p.in_bf16, gr + e));
    return y;
  };
  if (p.out_dtype != GDN_E4M3) {
    for (int e = threadIdx.x; e < width; e += 256) {
      const float u = kStage ? kept[e] : value(e);
      const float y[1] = {result(e, u)};
      store_values<1>(p.out, p.out_dtype == GDN_BF16, orow + e, y);
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
      const float c[1] = {nan_unless_finite(kStage ? kept[e] : result(e, u)) * inv};
      store_codes<1>(static_cast<uint8_t*>(p.out), orow + e, c);
      if (!kStage && p.residual) put_residual(e, u);
    }
  }
}

bool wide(const void* p, int64_t stride, int64_t size) {   // 8 values at a time, in pieces of 16 bytes (codes: 8)
  const int64_t piece = size == 1 ? 8 : 16;
  return reinterpret_cast<uintptr_t>(p) % piece == 0 && stride * size % piece == 0;
}

template <int V, int K, int RW>
void launch_rows(const NormLaunch& p, int part_lanes, hipStream_t stream) {
  constexpr int kRows = RW >= 4 ? 1 : 4 / RW;
  hipLaunchKernelGGL((row_kernel<V, K, RW>), dim3((unsigned)((p.T + kRows - 1) / kRows)), dim3(RW > 4 ? RW * kWave : 256), 0,
                     stream, p, part_lanes);
}

}  // namespace

hipError_t launch_rms_norm(const NormLaunch& p, hipStream_t stream) {
  const int64_t W = (int64_t)p.H * p.d, in = p.in_bf16 ? 2 : 4, res = p.residual_bf16 ? 2 : 4;
  const int64_t out = p.out_dtype == GDN_E4M3 ? 1 : p.out_dtype == GDN_BF16 ? 2 : 4;
  const bool eight = W % 8 == 0 && wide(p.x, p.x_stride, in) && (!p.gate || wide(p.gate, p.gate_stride, in)) &&
                     (!p.residual || wide(p.residual, p.residual_stride, res)) && wide(p.out, p.out_stride, out) &&
                     reinterpret_cast<uintptr_t>(p.weight) % 16 == 0;
  const int lanes = p.d / 8;
  const bool parts = p.H == 1 || (eight && p.d % 8 == 0 && lanes <= 64 && (lanes & (lanes - 1)) == 0);
  if (parts && eight && W <= 32768) {
    // A wave a row up to 2048 values where there are rows for every wave of the chip, else four
    // waves, which are done sooner.
    const bool many = p.T >= 1024;
    if (many && W <= 512) launch_rows<8, 1, 1>(p, lanes, stream);
    else if (many && W <= 1024) launch_rows<8, 2, 1>(p, lanes, stream);
    else if (W <= 2048) launch_rows<8, 1, 4>(p, lanes, stream);
    else if (W <= 4096) launch_rows<8, 2, 4>(p, lanes, stream);
    else if (W <= 8192) launch_rows<8, 4, 4>(p, lanes, stream);
    else if (W <= 16384) launch_rows<8, 2, 16>(p, lanes, stream);
    else launch_rows<8, 4, 16>(p, lanes, stream);
  } else if (p.H == 1 && W <= 8192) {
    if (W <= 256) launch_rows<1, 4, 1>(p, lanes, stream);
    else if (W <= 1024) launch_rows<1, 4, 4>(p, lanes, stream);
    else if (W <= 4096) launch_rows<1, 4, 16>(p, lanes, stream);
    else launch_rows<1, 8, 16>(p, lanes, stream);
  } else if ((W + p.H) * 4 <= 65536) {
    hipLaunchKernelGGL(lds_kernel<true>, dim3((unsigned)p.T), dim3(256), (W + p.H) * sizeof(float), stream, p);
  } else {
    hipLaunchKernelGGL(lds_kernel<false>, dim3((unsigned)p.T), dim3(256), p.H * sizeof(float), stream, p);
  }
  return hipGetLastError();
}

}  // namespace gdn
