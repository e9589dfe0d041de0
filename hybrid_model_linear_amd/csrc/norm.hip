// Root-mean-square norm with the residual's addition, a gate and an output in 8 bits
// (gdn_rms_norm).  A workgroup takes a token's row: its waves take the row's H parts in
// turn for the sums of squares, then the groups of values that share a scale.
#include "step_launch.h"
#include "step_math.h"

namespace gdn {

namespace {

constexpr float kMinScale = 5.421010862427522e-20f;   // 2^-64

__device__ __forceinline__ float load_any(const void* p, int bf16, int64_t i) {
  return bf16 ? bf16_to_f32(static_cast<const u16*>(p)[i]) : static_cast<const float*>(p)[i];
}

// e4m3 code of v / scale (a value that is not finite: NaN)
__device__ __forceinline__ uint8_t e4m3_code(float v, float scale) {
  if ((__float_as_uint(v) & 0x7f800000u) == 0x7f800000u) return 0x7f;
  return (uint8_t)__builtin_amdgcn_cvt_pk_fp8_f32(v / scale, 0.0f, 0, false);
}

__device__ __forceinline__ float finite_abs(float v) {
  return (__float_as_uint(v) & 0x7f800000u) == 0x7f800000u ? 0.0f : fabsf(v);
}

__device__ __forceinline__ float wave_max(float v) {
#pragma unroll
  for (int s = 32; s; s >>= 1) v = fmaxf(v, __shfl_xor(v, s, kWave));
  return v;
}

__global__ void __launch_bounds__(256) norm_kernel(NormLaunch p) {
  extern __shared__ float rstd[];                     // [H]
  const int64_t t = blockIdx.x;
  const int wave = threadIdx.x / kWave, lane = threadIdx.x % kWave;
  const int width = p.H * p.d;
  const int64_t xr = t * p.x_stride, gr = t * p.gate_stride, rr = t * p.residual_stride, orow = t * p.out_stride;
  // the value that is normalised
  auto value = [&](int e) {
    float u = load_any(p.x, p.in_bf16, xr + e);
    if (p.gate && p.gate_first) u *= step_silu(load_any(p.gate, p.in_bf16, gr + e));
    return u;
  };
  for (int h = wave; h < p.H; h += 4) {
    float sum = 0.0f;
    for (int i = lane; i < p.d; i += kWave) {
      float u = value(h * p.d + i);
      if (p.residual) u += load_any(p.residual, p.residual_bf16, rr + h * p.d + i);
      sum = fmaf(u, u, sum);
    }
    sum = group_sum<64>(sum);
    if (lane == 0) rstd[h] = 1.0f / sqrtf(sum / (float)p.d + p.eps);
  }
  __syncthreads();
  auto result = [&](int e) {
    const int h = e / p.d, i = e - h * p.d;
    float u = value(e);
    if (p.residual) u += load_any(p.residual, p.residual_bf16, rr + e);
    float y = u * rstd[h];
    if (p.weight) y *= load_any(p.weight, p.weight_bf16, i) + p.offset;
    if (p.gate && !p.gate_first) y *= step_silu(load_any(p.gate, p.in_bf16, gr + e));
    return y;
  };
  for (int k = wave; k < p.groups; k += 4) {
    const int lo = k * p.group, hi = min(width, lo + p.group);
    float scale = 1.0f;
    if (p.out_dtype == GDN_E4M3) {
      float top = 0.0f;
      for (int e = lo + lane; e < hi; e += kWave) top = fmaxf(top, finite_abs(result(e)));
      scale = fmaxf(wave_max(top) / 448.0f, kMinScale);
      if (lane == 0) p.scale[t * p.groups + k] = scale;
    }
    for (int e = lo + lane; e < hi; e += kWave) {
      const float y = result(e);
      if (p.out_dtype == GDN_E4M3) static_cast<uint8_t*>(p.out)[orow + e] = e4m3_code(y, scale);
      else if (p.out_dtype == GDN_BF16) static_cast<u16*>(p.out)[orow + e] = f32_to_bf16(y);
      else static_cast<float*>(p.out)[orow + e] = y;
      if (p.residual) {
        const float u = value(e) + load_any(p.residual, p.residual_bf16, rr + e);
        if (p.residual_bf16) static_cast<u16*>(p.residual)[rr + e] = f32_to_bf16(u);
        else static_cast<float*>(p.residual)[rr + e] = u;
      }
    }
  }
}

}  // namespace

hipError_t launch_rms_norm(const NormLaunch& p, hipStream_t stream) {
  hipLaunchKernelGGL(norm_kernel, dim3((unsigned)p.T), dim3(256), p.H * sizeof(float), stream, p);
  return hipGetLastError();
}

}  // namespace gdn
