// Launch descriptors between step_abi.cpp and the kernels of a serving step's operators
// beside the attention layers: the selective scan, the RMS norm and the pages of a step.
// Validation happens before these are filled; the kernels trust them.
#pragma once
#include <hip/hip_runtime.h>
#include <stdint.h>

#include "gdn.h"
#include "gdn_common.h"

namespace gdn {

struct SelectiveLaunch {
  int N, G;
  int64_t T, D;
  int states;
  int softplus_on;
  int in_bf16, out_bf16;
  const void* x;
  int64_t x_stride;
  const void* dt;
  int64_t dt_stride;
  const void* B;
  int64_t B_stride;
  const void* C;
  int64_t C_stride;
  const void* z;              // or null
  int64_t z_stride;
  const float* A;             // [D, states]
  const float* D_skip;        // [D] or null
  const float* dt_bias;       // [D] or null
  const int32_t* cu;          // [N + 1]
  const int32_t* slot;        // [N]
  const int32_t* has_init;    // [N] or null
  float* pool;                // [num_slots, D, states]
  void* out;
  int64_t out_stride;
  int keep_pool;
  // Sequences cut into segments of seg_len tokens, the last of `segs` taking the rest; segs 1: not cut.
  int segs;
  int64_t seg_len;
  float* seg_state;           // [2 (T / seg_len) + 1, D, states]
  float* seg_delta;           // [2 (T / seg_len) + 1, D]
};

// Segments of a scan on a card of this many CUs: segs and seg_len.
void plan_selective_scan(SelectiveLaunch& p, int64_t longest, int cus);

struct NormLaunch {
  int64_t T;
  int H, d;
  int in_bf16, weight_bf16, residual_bf16;
  int out_dtype;              // gdn_dtype
  const void* x;
  int64_t x_stride;
  const void* gate;           // or null
  int64_t gate_stride;
  void* residual;             // or null
  int64_t residual_stride;
  const void* weight;         // or null
  void* out;
  int64_t out_stride;
  float* scale;               // [T, groups]
  float eps, offset;
  int gate_first;
  int group;                  // values of a scale (the whole row's H d for group 0)
  int groups;                 // scales of a row
};

struct PlanPagesLaunch {
  int32_t* pool;
  int64_t capacity;
  int N, page;
  int64_t T;
  const int32_t* held;
  const int32_t* new_len;
  const int32_t* start;       // or null
  int32_t* table;
  int64_t table_stride;
  int table_width;
  int32_t* cu;
  int32_t* cache_len;
  int32_t* kv_len;
  int64_t* slots;             // or null
  int32_t* positions;         // or null
  int32_t* seq;               // or null
};

struct ReleasePagesLaunch {
  int32_t* pool;
  int64_t capacity;
  int N, page;
  const int32_t* keep;
  const int32_t* held;
  const int32_t* table;
  int64_t table_stride;
  int table_width;
};

// Most rows of a norm of this width (H, d): a launch has fewer than 2^32 threads.
int64_t most_rms_norm_rows(const NormLaunch& p);

hipError_t launch_selective_scan(const SelectiveLaunch& p, hipStream_t stream);
hipError_t launch_selective_update(const SelectiveLaunch& p, hipStream_t stream);
hipError_t launch_rms_norm(const NormLaunch& p, hipStream_t stream);
hipError_t launch_plan_pages(const PlanPagesLaunch& p, hipStream_t stream);
hipError_t launch_release_pages(const ReleasePagesLaunch& p, hipStream_t stream);

int status_of_hip(hipError_t e);
int current_device_cus();

}  // namespace gdn
