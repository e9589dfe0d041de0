// Selective state space scan: packed prompts (gdn_selective_scan) and one token per row
// (gdn_selective_update).  Per channel c with states h[i]:
//   h[i] = exp(delta A[c, i]) h[i] + delta x B[i],   y = sum_i C[i] h[i] + D_skip[c] x
//
// The scan's bound is vector arithmetic: per token, channel and state a product, an
// exponential (the time of two other instructions), a product and two fused ones, ~26 cycles
// of a SIMD for 64 of them, where the bytes of a token and channel are 8 (at 32768 tokens x 4096
// channels, 16 states: 0.44 ms of instructions, softplus and gate among them, to 0.19 ms of
// memory; measured 0.56 ms).
// A lane is a channel, the states are dealt out over the 4 or 8 waves of a workgroup: so
// each wave reads B and C of its states as broadcasts, whole rows of x, dt, z are read and
// written, and what there is once per token and channel (softplus, gate, conversions) is
// dealt out over the waves by tokens.  Through LDS go delta and delta x to all waves and each
// wave's part of y back; two buffers of each, so that a tile of tokens costs one barrier.
#include "step_launch.h"
#include "step_math.h"
#include "tile_ops.h"

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

int64_t channel_blocks(const SelectiveLaunch& p) { return (p.D / p.G + kBlock - 1) / kBlock * p.G; }

// Channel of this lane: workgroups do not cross groups.
__device__ __forceinline__ bool channel_of(const SelectiveLaunch& p, int blk, int64_t& c, int& g) {
  const int64_t dg = p.D / p.G;
  const int per = (int)((dg + kBlock - 1) / kBlock);
  g = blk / per;
  const int64_t in = (int64_t)(blk % per) * kBlock + threadIdx.x % kBlock;
  c = g * dg + (in < dg ? in : dg - 1);
  return in < dg;
}

// ------------------------------------------------------------------ scan
// Waves that the states are dealt out over, and tokens of a tile.
template <int NS> constexpr int kWaves = NS <= 32 ? 4 : 8;
template <int NS> constexpr int kTile = NS <= 32 ? 16 : 8;

enum Pass {
  kWhole,      // a workgroup walks a sequence
  kStates,     // ... a segment, for its last state (from zeros; the first one from the sequence's start) and its sum of delta
  kSegment     // ... a segment, from the state that the segments before it leave
};

template <typename In, typename Out, int NS, int kPass>
__global__ void __launch_bounds__(kWaves<NS>* kWave, 2) scan_kernel(SelectiveLaunch p, TokenIn<In> in, int blocks) {
  constexpr int NW = kWaves<NS>, SPL = NS / NW, TT = kTile<NS>, TW = TT / NW;
  constexpr int kOut = kPass != kStates;                    // y is formed
  constexpr int kBC = kOut ? 2 : 1;                         // B, or B and C
  constexpr int kValues = TT * kBC * NS, kFill = (kValues + NW * kWave - 1) / (NW * kWave);   // of a tile; of a thread
  static_assert(TT % NW == 0 && NS % NW == 0, "tiles divide evenly");
  __shared__ __attribute__((aligned(16))) float2 steps[2][TT][kBlock];           // delta, delta x
  __shared__ __attribute__((aligned(16))) float bc[2][TT][NW][kBC][SPL];
  __shared__ float part[kOut ? 2 : 1][kOut ? TT : 1][kOut ? NW : 1][kBlock];     // each wave's part of y
  const int wave = __builtin_amdgcn_readfirstlane(threadIdx.x / kWave), lane = threadIdx.x % kWave;
  const int blk = blockIdx.x % blocks, rest = blockIdx.x / blocks;
  const int cuts = kPass == kWhole ? 1 : kPass == kStates ? p.segs - 1 : p.segs;
  const int n = rest / cuts, seg = rest % cuts;
  int64_t c;
  int g;
  const bool mine = channel_of(p, blk, c, g);
  const int32_t slot = p.slot[n];
  if (slot < 0) return;
  int64_t first = __builtin_amdgcn_readfirstlane(p.cu[n]), end = __builtin_amdgcn_readfirstlane(p.cu[n + 1]);
  // A sequence of `pieces` segments keeps its states in that many rows of the workspace from
  // 2 (its first token / seg_len) on: one for each segment but the last, and its start state
  // (whose slot of the pool the last segment writes).  One segment needs none.
  bool last = true;
  int pieces = 1;
  int64_t seg_row = 0;
  if constexpr (kPass != kWhole) {
    const int len = (int)p.seg_len;
    pieces = max(1, min((int)(((uint32_t)(end - first) + len - 1) / (uint32_t)len), p.segs));
    if (seg >= (kPass == kStates ? pieces - 1 : pieces)) return;
    seg_row = 2 * ((int)first / len) * p.D;
    last = seg == pieces - 1;
    first += (int64_t)seg * len;
    if (!last) end = first + len;
  }
  const int64_t at = c * NS + wave * SPL;                   // this lane's states in an [D, states] matrix
  float* state = p.pool + (int64_t)slot * p.D * NS + at;
  const bool init = !p.has_init || p.has_init[n] != 0;
  float A[SPL], h[SPL];
#pragma unroll
  for (int i = 0; i < SPL; ++i) A[i] = p.A[at + i] * kLog2e;
  const int64_t row = p.D * NS;
  float* kept = p.seg_state + seg_row * NS + at;            // of the sequence's first segment
  if (kPass == kSegment && pieces > 1) {
    const float* from = seg == 0 ? kept + (pieces - 1) * row : kept;
#pragma unroll
    for (int i = 0; i < SPL; ++i) h[i] = from[i];
    for (int s = 1; s < seg; ++s) {
      const float sum = p.seg_delta[seg_row + s * p.D + c];
#pragma unroll
      for (int i = 0; i < SPL; ++i) {
        const float e = from[s * row + i];     // (a state of 0 stays 0 where a growing factor overflows)
        h[i] = h[i] != 0.0f ? fmaf(h[i], __builtin_amdgcn_exp2f(sum * A[i]), e) : e;
      }
    }
  } else {
#pragma unroll
    for (int i = 0; i < SPL; ++i) h[i] = init && seg == 0 ? state[i] : 0.0f;
    if (kPass == kStates && seg == 0 && mine) {
#pragma unroll
      for (int i = 0; i < SPL; ++i) kept[(pieces - 1) * row + i] = h[i];
    }
  }
  const float bias = p.dt_bias ? p.dt_bias[c] : 0.0f, skip = p.D_skip ? p.D_skip[c] : 0.0f;

  // A tile's operands in registers: of TW tokens (this wave's share), and of B and C.  Tiles are
  // fetched two ahead, in turn into two sets of registers from which they are staged and finished
  // without being moved (a copy, a branch around the loads, or a conversion behind them, would wait
  // for them); without z its loads read x.
  struct Operands { In x[TW], dt[TW], z[TW], bc[kFill]; } set[2];
  const uint32_t at_c = (uint32_t)c * sizeof(In), at_out = (uint32_t)c * sizeof(Out);
  const int64_t row0 = first + wave * TW;
  const In *x_at = in.x + row0 * in.x_stride, *dt_at = in.dt + row0 * in.dt_stride;
  const int64_t z_stride = in.z ? in.z_stride : in.x_stride;
  const In* z_at = in.z ? in.z + row0 * z_stride : x_at;
  Out* out_at = static_cast<Out*>(p.out) + row0 * p.out_stride;
  // (the empty statement keeps the sum of a row's scalar address and the channel's 32-bit offset for the load itself)
  auto of = [&](const In* row, uint32_t off) {
    auto* from = (const __attribute__((address_space(1))) char*)row;
    asm("" : "+s"(from));
    return *(const __attribute__((address_space(1))) In*)(from + off);
  };
  const In* bc_at[kFill];                                   // this thread's values of B and C
  int64_t bc_step[kFill];
  int bc_token[kFill], bc_to[kFill];                        // their token of the tile; their place in LDS
#pragma unroll
  for (int k = 0; k < kFill; ++k) {
    const int e = k * NW * kWave + threadIdx.x, i = e % (kBC * NS), s = i % NS;
    bc_token[k] = e / (kBC * NS);                           // (past the tile: read as its first, not written)
    const int64_t stride = i < NS ? in.B_stride : in.C_stride;
    bc_at[k] = (i < NS ? in.B : in.C) + (first + (bc_token[k] < TT ? bc_token[k] : 0)) * stride + (int64_t)g * NS + s;
    bc_to[k] = ((bc_token[k] * NW + s / SPL) * kBC + i / NS) * SPL + s % SPL;
    bc_step[k] = TT * stride;
  }
  auto fetch = [&](Operands& r) __attribute__((always_inline)) {
    uint32_t off = at_c;
    asm("" : "+v"(off));
#pragma unroll
    for (int q = 0; q < TW; ++q) {
      r.x[q] = of(x_at + q * in.x_stride, off);
      r.dt[q] = of(dt_at + q * in.dt_stride, off);
      if (kOut) r.z[q] = of(z_at + q * z_stride, off);
    }
#pragma unroll
    for (int k = 0; k < kFill; ++k) r.bc[k] = *bc_at[k];
  };
  auto advance = [&](bool on) __attribute__((always_inline)) {
    x_at += on ? TT * in.x_stride : 0;
    dt_at += on ? TT * in.dt_stride : 0;
    z_at += on ? TT * z_stride : 0;
#pragma unroll
    for (int k = 0; k < kFill; ++k) bc_at[k] += on ? bc_step[k] : 0;
  };
  // Their part that is the same for all states, into LDS; tokens from `left` on count as zeros
  // (`whole`: there are none).
  auto stage = [&](int buf, const Operands& r, auto whole, int left) __attribute__((always_inline)) {
    constexpr bool kAll = decltype(whole)::value;
    float delta[TW];
#pragma unroll
    for (int q = 0; q < TW; ++q) delta[q] = Elem<In>::load(&r.dt[q], 0) + bias;
    if (p.softplus_on) {
#pragma unroll
      for (int q = 0; q < TW; ++q) delta[q] = step_softplus(delta[q]);
    }
#pragma unroll
    for (int q = 0; q < TW; ++q) {
      const int k = wave * TW + q;
      const bool live = kAll || k < left;
      steps[buf][k][lane] = make_float2(live ? delta[q] : 0.0f, live ? delta[q] * Elem<In>::load(&r.x[q], 0) : 0.0f);
    }
    float* to = &bc[buf][0][0][0][0];
#pragma unroll
    for (int k = 0; k < kFill; ++k)
      if (kValues % (NW * kWave) == 0 || bc_token[k] < TT)
        to[bc_to[k]] = kAll || bc_token[k] < left ? Elem<In>::load(&r.bc[k], 0) : 0.0f;
  };
  float sum = 0.0f;                                          // of delta (kStates)
  // The tile's tokens in turn, LDS reads a step of kStep tokens ahead of their use.  Those that are
  // not there are not walked: their delta of 0 would leave a state as it is, but not under an A of -inf.
  constexpr int kStep = SPL <= 4 ? 2 : 1;
  auto walk = [&](int buf, auto whole, int left) __attribute__((always_inline)) {
    float2 d[2][kStep];
    float b[2][kStep][SPL], cc[2][kStep][SPL];
    auto read = [&](int s) __attribute__((always_inline)) {
#pragma unroll
      for (int j = 0; j < kStep; ++j) {
        const int k = s * kStep + j;
        d[s & 1][j] = steps[buf][k][lane];
#pragma unroll
        for (int i = 0; i < SPL; ++i) {
          b[s & 1][j][i] = bc[buf][k][wave][0][i];
          if constexpr (kOut) cc[s & 1][j][i] = bc[buf][k][wave][kBC - 1][i];
        }
      }
    };
    read(0);
#pragma unroll
    for (int s = 0; s < TT / kStep; ++s) {
      if (s + 1 < TT / kStep) read(s + 1);
      __builtin_amdgcn_sched_barrier(0);
#pragma unroll
      for (int j = 0; j < kStep; ++j) {
        if (!decltype(whole)::value && s * kStep + j >= left) continue;
        const float2 dd = d[s & 1][j];
        float y = 0.0f;
#pragma unroll
        for (int i = 0; i < SPL; ++i) {
          h[i] = fmaf(h[i], __builtin_amdgcn_exp2f(dd.x * A[i]), dd.y * b[s & 1][j][i]);
          if constexpr (kOut) y = fmaf(cc[s & 1][j][i], h[i], y);
        }
        if constexpr (kOut) part[buf][s * kStep + j][wave][lane] = y;
        else sum += dd.x;
      }
      if constexpr (!kOut) {       // (no write keeps the steps apart: what they form is not to be formed all at once)
#pragma unroll
        for (int i = 0; i < SPL; ++i) asm volatile("" : "+v"(h[i]));
        lds_order();
      }
      __builtin_amdgcn_sched_barrier(0);
    }
  };
  auto finish = [&](int buf, const Operands& r, auto whole, int left) __attribute__((always_inline)) {
    if constexpr (kOut) {
      uint32_t off = at_out;
      asm("" : "+v"(off));
      float y[TW];
#pragma unroll
      for (int q = 0; q < TW; ++q) {
        y[q] = skip * Elem<In>::load(&r.x[q], 0);
#pragma unroll
        for (int w = 0; w < NW; ++w) y[q] += part[buf][wave * TW + q][w][lane];
      }
      if (in.z) {
#pragma unroll
        for (int q = 0; q < TW; ++q) y[q] *= step_silu(Elem<In>::load(&r.z[q], 0));
      }
#pragma unroll
      for (int q = 0; q < TW; ++q)
        if ((decltype(whole)::value || wave * TW + q < left) && mine) {
          auto* to = (__attribute__((address_space(1))) char*)(out_at + q * p.out_stride);
          asm("" : "+s"(to));
          Out v;
          Elem<Out>::store(&v, 0, y[q]);
          *(__attribute__((address_space(1))) Out*)(to + off) = v;
        }
      out_at += TT * p.out_stride;
    }
  };
  const int tokens = first < end ? (int)(end - first) : 0, tiles = tokens / TT, tail = tokens % TT;
  if (tiles > 0) {
    fetch(set[0]);
    stage(0, set[0], Par<1>{}, TT);
    advance(tiles > 1);
    fetch(set[1]);
    lds_sync();
    // Tile k: walked; the next one staged behind it; finished; the one after the next fetched (the
    // last one again where there is none).
    auto turn = [&](auto parity, int k) __attribute__((always_inline)) {
      constexpr int kBuf = decltype(parity)::value;
      walk(kBuf, Par<1>{}, TT);
      stage(1 - kBuf, set[1 - kBuf], Par<1>{}, TT);
      lds_sync();
      finish(kBuf, set[kBuf], Par<1>{}, TT);
      advance(k + 2 < tiles);
      fetch(set[kBuf]);
    };
    int k = 0;
    for (; k + 1 < tiles; k += 2) {
      turn(Par<0>{}, k);
      turn(Par<1>{}, k + 1);
    }
    if (k < tiles) turn(Par<0>{}, k);
    advance(true);
  }
  if (tail > 0) {
    Operands r;
#pragma unroll
    for (int q = 0; q < TW; ++q) {
      const bool there = wave * TW + q < tail;
      r.x[q] = there ? of(x_at + q * in.x_stride, at_c) : In(0);
      r.dt[q] = there ? of(dt_at + q * in.dt_stride, at_c) : In(0);
      if (kOut) r.z[q] = there ? of(z_at + q * z_stride, at_c) : In(0);
    }
#pragma unroll
    for (int k = 0; k < kFill; ++k) r.bc[k] = bc_token[k] < tail ? *bc_at[k] : In(0);
    lds_sync();                     // (the last turns' buffers have been read)
    stage(0, r, Par<0>{}, tail);
    lds_sync();
    walk(0, Par<0>{}, tail);
    lds_sync();
    finish(0, r, Par<0>{}, tail);
  }
  if (!mine) return;
  if constexpr (kPass == kStates) {
#pragma unroll
    for (int i = 0; i < SPL; ++i) kept[seg * row + i] = h[i];
    if (wave == 0) p.seg_delta[seg_row + seg * p.D + c] = sum;
  } else if (last && !p.keep_pool) {
#pragma unroll
    for (int i = 0; i < SPL; ++i) state[i] = h[i];
  }
}

template <typename In, typename Out, int NS>
void launch_scan(const SelectiveLaunch& p, hipStream_t stream) {
  const int64_t blocks = channel_blocks(p);
  const dim3 block(kWaves<NS> * kWave);
  const TokenIn<In> in = token_in<In>(p);
  auto grid = [&](int cuts) { return dim3((unsigned)(blocks * p.N * cuts)); };
  if (p.segs == 1) {
    hipLaunchKernelGGL((scan_kernel<In, Out, NS, kWhole>), grid(1), block, 0, stream, p, in, (int)blocks);
    return;
  }
  hipLaunchKernelGGL((scan_kernel<In, Out, NS, kStates>), grid(p.segs - 1), block, 0, stream, p, in, (int)blocks);
  hipLaunchKernelGGL((scan_kernel<In, Out, NS, kSegment>), grid(p.segs), block, 0, stream, p, in, (int)blocks);
}

// ------------------------------------------------------------------ update
// One token per row: the states are read and written once and little else is (memory-bound).
// A lane takes four states of a channel, NS / 4 lanes a channel, whose sum over the states is
// formed across them; a workgroup takes 1024 / NS channels of kRows rows, for which A is loaded
// once and whose states are all in flight together.
template <typename In, bool kVec>
__device__ __forceinline__ void load_four(const In* p, float (&v)[4]) {
  if constexpr (!kVec) {
#pragma unroll
    for (int i = 0; i < 4; ++i) v[i] = Elem<In>::load(p, i);
  } else if constexpr (sizeof(In) == 4) {
    const float4 w = *reinterpret_cast<const float4*>(p);
    v[0] = w.x; v[1] = w.y; v[2] = w.z; v[3] = w.w;
  } else {
    const uint2 w = *reinterpret_cast<const uint2*>(p);
    v[0] = __uint_as_float(w.x << 16); v[1] = __uint_as_float(w.x & 0xffff0000u);
    v[2] = __uint_as_float(w.y << 16); v[3] = __uint_as_float(w.y & 0xffff0000u);
  }
}

template <typename In, typename Out, int NS, int kRows, bool kVec>
__global__ void __launch_bounds__(256) update_kernel(SelectiveLaunch p, TokenIn<In> in, int blocks) {
  constexpr int kLanes = NS / 4, kChannels = 256 / kLanes;
  const int blk = blockIdx.x % blocks, n0 = blockIdx.x / blocks * kRows;
  const int dg = (int)(p.D / p.G), per = (dg + kChannels - 1) / kChannels, g = blk / per;
  const int within = blk % per * kChannels + threadIdx.x / kLanes, i0 = threadIdx.x % kLanes * 4;
  const bool mine = within < dg;
  const int64_t c = (int64_t)g * dg + (mine ? within : dg - 1), at = c * NS + i0;
  int32_t slot[kRows];
  float4 state[kRows];
  float x[kRows], dt[kRows], z[kRows], b[kRows][4], cc[kRows][4];
#pragma unroll
  for (int r = 0; r < kRows; ++r) slot[r] = n0 + r < p.N ? p.slot[n0 + r] : -1;
#pragma unroll
  for (int r = 0; r < kRows; ++r) {
    if (slot[r] < 0) continue;
    const int64_t n = n0 + r, bc = (int64_t)g * NS + i0;
    state[r] = *reinterpret_cast<const float4*>(p.pool + (int64_t)slot[r] * p.D * NS + at);
    x[r] = Elem<In>::load(in.x + n * in.x_stride, c);
    dt[r] = Elem<In>::load(in.dt + n * in.dt_stride, c);
    if (in.z) z[r] = Elem<In>::load(in.z + n * in.z_stride, c);
    load_four<In, kVec>(in.B + n * in.B_stride + bc, b[r]);
    load_four<In, kVec>(in.C + n * in.C_stride + bc, cc[r]);
  }
  const float4 a4 = *reinterpret_cast<const float4*>(p.A + at);
  const float A[4] = {a4.x * kLog2e, a4.y * kLog2e, a4.z * kLog2e, a4.w * kLog2e};
  const float bias = p.dt_bias ? p.dt_bias[c] : 0.0f, skip = p.D_skip ? p.D_skip[c] : 0.0f;
#pragma unroll
  for (int r = 0; r < kRows; ++r) {
    if (slot[r] < 0) continue;
    float delta = dt[r] + bias;
    if (p.softplus_on) delta = step_softplus(delta);
    const float dx = delta * x[r];
    float h[4] = {state[r].x, state[r].y, state[r].z, state[r].w}, y = 0.0f;
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      h[i] = fmaf(h[i], __builtin_amdgcn_exp2f(delta * A[i]), dx * b[r][i]);
      y = fmaf(cc[r][i], h[i], y);
    }
    y = group_sum<kLanes>(y);
    if (!mine) continue;
    *reinterpret_cast<float4*>(p.pool + (int64_t)slot[r] * p.D * NS + at) = make_float4(h[0], h[1], h[2], h[3]);
    if (i0 == 0) {
      y = fmaf(skip, x[r], y);
      if (in.z) y *= step_silu(z[r]);
      Elem<Out>::store(static_cast<Out*>(p.out) + (n0 + r) * p.out_stride, c, y);
    }
  }
}

template <typename In, typename Out, int NS>
void launch_update(const SelectiveLaunch& p, hipStream_t stream) {
  constexpr int kChannels = 1024 / NS;
  const int64_t blocks = (p.D / p.G + kChannels - 1) / kChannels * p.G;
  const TokenIn<In> in = token_in<In>(p);
  const auto four = [](const In* q, int64_t stride) { return reinterpret_cast<uintptr_t>(q) % (4 * sizeof(In)) == 0 && stride % 4 == 0; };
  const bool vec = four(in.B, in.B_stride) && four(in.C, in.C_stride);
#define UPDATE(ROWS, VEC)                                                                                             \
  hipLaunchKernelGGL((update_kernel<In, Out, NS, ROWS, VEC>), dim3((unsigned)(blocks * ((p.N + ROWS - 1) / ROWS))), \
                     dim3(256), 0, stream, p, in, (int)blocks)
  // One row a workgroup while that leaves places free (latency), else two: 256 rows x 4096 channels
  // 31.2 us with one, 29.9 with two, 31.2 with four, 38 with eight.
  if (blocks * p.N < 4096) {
    if (vec) UPDATE(1, true); else UPDATE(1, false);
  } else {
    if (vec) UPDATE(2, true); else UPDATE(2, false);
  }
#undef UPDATE
}

template <typename In, typename Out>
void launch_states(const SelectiveLaunch& p, bool update, hipStream_t stream) {
#define SELECTIVE(NS) \
  case NS: if (update) launch_update<In, Out, NS>(p, stream); else launch_scan<In, Out, NS>(p, stream); break
  switch (p.states) {
    SELECTIVE(8);
    SELECTIVE(16);
    SELECTIVE(32);
    SELECTIVE(64);
    SELECTIVE(128);
  }
#undef SELECTIVE
}

hipError_t launch_types(const SelectiveLaunch& p, bool update, hipStream_t stream) {
  if (p.in_bf16) {
    if (p.out_bf16) launch_states<u16, u16>(p, update, stream); else launch_states<u16, float>(p, update, stream);
  } else {
    if (p.out_bf16) launch_states<float, u16>(p, update, stream); else launch_states<float, float>(p, update, stream);
  }
  return hipGetLastError();
}

}  // namespace

void plan_selective_scan(SelectiveLaunch& p, int64_t longest, int cus) {
  // In tokens of one workgroup: uncut, the longest sequence walks alone while the others share
  // the chip, which is full at 1.4 workgroups of four waves per CU (0.7 of eight); cut, all
  // tokens are counted 1.5 times, plus one segment and a launch.  (The states are formed twice, the
  // first time without y, which is 1.83 times the recurrence's cycles; 1.5 is what fits the
  // measurements, since a walk at 1.4 workgroups a CU does not fill its SIMDs.)
  // Measured, us, 16 states, uncut / cut: one of 4096 x 4096 channels 400 / 124, two 400 / 232, four
  // 409 / 411, eight 569 / 758; one of 256 x 1024 31 / 20; 8192 and 31 of 500 x 4096 824 / 520; the
  // rule is within 10% of the best number of segments over 18 such shapes.
  // Segments: four workgroups (two of eight waves) a CU, no shorter than two tiles.  (The LDS of
  // the pass that forms y holds three a CU at 8, 16 and 64 states, 53 KB each, two at 32 and 128.)
  constexpr int kShortest = 32, kLaunch = 80;      // tokens of a segment, and the launch's worth
  static_assert(kShortest + kLaunch == GDN_SELECTIVE_UNCUT, "the header's promise");
  p.segs = 1;
  p.seg_len = longest;
  const int eight = p.states > 32;
  const int64_t work = channel_blocks(p) * p.T;
  int64_t len = work / (eight ? 2 * cus : 4 * cus) / 16 * 16;
  if (len < longest / 128) len = longest / 128;
  len = (len < kShortest ? kShortest : len + 15) / 16 * 16;
  if (15 * work / (eight ? 7 * cus : 14 * cus) + len + kLaunch >= longest) return;
  p.seg_len = len;
  p.segs = (int)((longest + len - 1) / len);
}

hipError_t launch_selective_scan(const SelectiveLaunch& p, hipStream_t stream) { return launch_types(p, false, stream); }
hipError_t launch_selective_update(const SelectiveLaunch& p, hipStream_t stream) { return launch_types(p, true, stream); }

}  // namespace gdn
