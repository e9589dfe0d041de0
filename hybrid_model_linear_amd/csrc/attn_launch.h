// Launch descriptors of the softmax-attention kernels, between attn_abi.cpp and the
// kernels.  Validation happens before these are filled; the kernels trust the pointers,
// sizes and strides, and bound everything that is device data (lengths, page ids).
#pragma once
#include <hip/hip_runtime.h>
#include <stdint.h>

#include "gdn.h"
#include "gdn_common.h"

namespace gdn {

// The paged 8-bit cache and the block table of a call.
struct CacheRef {
  uint8_t* k;               // e4m3 [num_pages, H_kv, page, d]; null: no cache
  uint8_t* v;
  float* k_scale;           // [num_pages, H_kv], powers of two
  float* v_scale;
  int32_t* pos;             // [num_pages, H_kv, page] or null
  float* weight;            // likewise
  int64_t num_pages;
  int page_log2;
  int H_kv;
  int d;
  const int32_t* table;     // [N, table_width]
  int64_t table_stride;
  int table_width;
};

// Tokens per sequence, on average, up to which a wave takes a page and head, not a workgroup.
// wave / workgroup, us, 8 heads of 128: 256 sequences of 1 token 6.0 / 13.0, of 8 7.7 / 14.8;
// 32 of 8 4.4 / 4.7, of 16 5.4 / 5.1, of 64 11.1 / 6.3; one of 8 3.8 / 3.4, of 64 9.3 / 4.1.
constexpr int kFewTokens = 8;

struct StoreLaunch {
  CacheRef c;
  int N;
  int64_t T;
  const u16* k;
  int64_t k_stride;
  const u16* v;
  int64_t v_stride;
  const int32_t* cu;        // [N + 1] or null (one token per sequence)
  const int32_t* cache_len;
  const int32_t* start;     // or null
};

struct AttnExtendLaunch {
  CacheRef c;
  int N;
  int64_t T;
  int H;
  int H_kv, d;
  const u16* q;
  int64_t q_stride;
  const u16* k;
  int64_t k_stride;
  const u16* v;
  int64_t v_stride;
  u16* out;
  int64_t out_stride;
  const int32_t* cu;
  const int32_t* cache_len; // or null (no cache)
  const int32_t* start;     // or null
  int causal;
  const int32_t* visible;   // or null
  const int32_t* doc;       // or null
  const float* slopes;      // or null
  int window;               // 0 = none
  float scale;
  float softcap;            // 0 = none
  int splits;               // parts of every row's keys
  int fold;                 // slot of the launch from which the shortest walks come first
  float* part_o;            // [splits, T, H, d] unscaled outputs (splits > 1)
  float* part_ml;           // [splits, T, H, 2] running maximum and sum (splits > 1)
};

struct AttnDecodeLaunch {
  CacheRef c;
  int N;
  int H;
  const u16* q;
  int64_t q_stride;
  u16* out;
  int64_t out_stride;
  const int32_t* kv_len;
  const int32_t* q_pos;     // or null
  const float* slopes;      // or null
  int window;
  float scale;
  float softcap;
  int accumulate;
  int min_chunks;           // fewest 64-row chunks of a split
  int ranked;               // workgroups in order of the sequences' lengths
  int splits;               // workgroups per (sequence, kv head, group of 16 query heads)
  float* part_o;            // [N, H, splits, d] partial sums (splits > 1)
  float* part_ml;           // [N, H, splits, 2] running maximum and sum (splits > 1 or accumulate)
  float* scores;            // [N, H, score_cap] (accumulate): scores in units of log2
  int64_t score_cap;
};

struct EvictLaunch {
  CacheRef c;
  int N;
  int budget;
  int recent;
  const int32_t* kv_len;
  int32_t* new_len;
  int32_t* holes;           // [N, H_kv, budget] rows to fill, ascending
  int32_t* movers;          // [N, H_kv, budget] rows that fill them (rows of the whole cache, one head's)
  float* scales;            // [N, H_kv, budget, 2] k and v scale of the movers' pages
  int32_t* first;           // [N, H_kv, pages + 1] first entry of `holes` in each page before budget
};

hipError_t launch_kv_store(const StoreLaunch& p, hipStream_t stream);
void plan_attn_extend(AttnExtendLaunch& p, int64_t keys, int cus);   // splits, fold
hipError_t launch_attn_extend(const AttnExtendLaunch& p, hipStream_t stream);
void plan_attn_decode(AttnDecodeLaunch& p, int64_t max_rows, int cus);   // splits, min_chunks, ranked
hipError_t launch_attn_decode(const AttnDecodeLaunch& p, hipStream_t stream);
hipError_t launch_kv_evict(const EvictLaunch& p, hipStream_t stream);

// The C ABI's per-thread record of the last HIP error (gdn_abi.cpp): the status of a launch.
int status_of_hip(hipError_t e);
int current_device_cus();

}  // namespace gdn
