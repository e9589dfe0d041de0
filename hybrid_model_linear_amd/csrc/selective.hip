// Selective state space scan: packed prompts (gdn_selective_scan) and one token per row
// (gdn_selective_update).  Per channel c with states h[i]:
//   h[i] = exp(delta A[c, i]) h[i] + delta x B[i],   y = sum_i C[i] h[i] + D_skip[c] x
// A thread walks one channel with its states in registers.
#include "step_launch.h"
#include "step_math.h"

namespace gdn {

namespace {

constexpr int kBlock = 64;          // channels of a workgroup, all of one group
constexpr float kLog2e = 1.4426950408889634f;

template <typename In>
struct TokenIn {
  const In *x, *dt, *B, *C, *z;
  int64_t x_stride, dt_stride, B_stride, C_stride, z_stride;
};

template <typename In>
TokenIn<In> token_in(const SelectiveLaunch& p) {
  return {static_cast<const In*>(p.x), static_cast<const In*>(p.dt), static_cast<const In*>(p.B),
          static_cast<const In*>(p.C), static_cast<const In*>(p.z), p.x_stride, p.dt_stride, p.B_stride, p.C_stride,
          p.z_stride};
}

// Channel of this thread: workgroups do not cross groups.
__device__ __forceinline__ bool channel_of(const SelectiveLaunch& p, int blk, int64_t& c, int& g) {
  const int64_t dg = p.D / p.G;
  const int per = (int)((dg + kBlock - 1) / kBlock);
  g = blk / per;
  const int64_t in = (int64_t)(blk % per) * kBlock + threadIdx.x;
  c = g * dg + in;
  return in < dg;
}

// One token of one channel: h is updated, y returned.
template <typename In, int NS>
__device__ __forceinline__ float token_step(const SelectiveLaunch& p, const TokenIn<In>& in, int64_t t, int64_t c, int g,
                                            const float* A, float bias, float skip, float (&h)[NS]) {
  const float x = Elem<In>::load(in.x, t * in.x_stride + c);
  float delta = Elem<In>::load(in.dt, t * in.dt_stride + c) + bias;
  if (p.softplus_on) delta = step_softplus(delta);
  const float dx = delta * x;
  float y = skip * x;
#pragma unroll
  for (int i = 0; i < NS; ++i) {
    const float b = Elem<In>::load(in.B, t * in.B_stride + (int64_t)g * NS + i);
    const float cc = Elem<In>::load(in.C, t * in.C_stride + (int64_t)g * NS + i);
    h[i] = fmaf(h[i], __builtin_amdgcn_exp2f(delta * (A[i] * kLog2e)), dx * b);
    y = fmaf(cc, h[i], y);
  }
  if (in.z) y *= step_silu(Elem<In>::load(in.z, t * in.z_stride + c));
  return y;
}

template <typename In, typename Out, int NS, bool kUpdate>
__global__ void __launch_bounds__(kBlock) selective_kernel(SelectiveLaunch p, TokenIn<In> in, int blocks) {
  const int n = blockIdx.x / blocks;
  int64_t c;
  int g;
  if (!channel_of(p, blockIdx.x % blocks, c, g)) return;
  const int32_t slot = p.slot[n];
  if (slot < 0) return;
  const int64_t first = kUpdate ? n : p.cu[n], end = kUpdate ? n + 1 : p.cu[n + 1];
  const float* A = p.A + c * NS;
  float* state = p.pool + ((int64_t)slot * p.D + c) * NS;
  const bool init = kUpdate || !p.has_init || p.has_init[n] != 0;
  float h[NS];
#pragma unroll
  for (int i = 0; i < NS; ++i) h[i] = init ? state[i] : 0.0f;
  const float bias = p.dt_bias ? p.dt_bias[c] : 0.0f, skip = p.D_skip ? p.D_skip[c] : 0.0f;
  for (int64_t t = first; t < end; ++t)
    Elem<Out>::store(static_cast<Out*>(p.out), t * p.out_stride + c, token_step<In, NS>(p, in, t, c, g, A, bias, skip, h));
  if (!kUpdate && p.keep_pool) return;
#pragma unroll
  for (int i = 0; i < NS; ++i) state[i] = h[i];
}

template <typename In, typename Out, bool kUpdate>
void launch(const SelectiveLaunch& p, hipStream_t stream) {
  const int64_t dg = p.D / p.G;
  const int blocks = (int)((dg + kBlock - 1) / kBlock * p.G);
  const dim3 grid((unsigned)(blocks * (int64_t)p.N)), block(kBlock);
  const TokenIn<In> in = token_in<In>(p);
#define SELECTIVE(NS) \
  case NS: hipLaunchKernelGGL((selective_kernel<In, Out, NS, kUpdate>), grid, block, 0, stream, p, in, blocks); break
  switch (p.states) {
    SELECTIVE(8);
    SELECTIVE(16);
    SELECTIVE(32);
    SELECTIVE(64);
    SELECTIVE(128);
  }
#undef SELECTIVE
}

template <bool kUpdate>
hipError_t launch_types(const SelectiveLaunch& p, hipStream_t stream) {
  if (p.in_bf16) {
    if (p.out_bf16) launch<u16, u16, kUpdate>(p, stream); else launch<u16, float, kUpdate>(p, stream);
  } else {
    if (p.out_bf16) launch<float, u16, kUpdate>(p, stream); else launch<float, float, kUpdate>(p, stream);
  }
  return hipGetLastError();
}

}  // namespace

hipError_t launch_selective_scan(const SelectiveLaunch& p, hipStream_t stream) { return launch_types<false>(p, stream); }
hipError_t launch_selective_update(const SelectiveLaunch& p, hipStream_t stream) { return launch_types<true>(p, stream); }

}  // namespace gdn
