// The pages of a step (gdn_plan_pages, gdn_release_pages): sums over the requests before
// each one, then lists that they index.
//
// A workgroup of 256 threads looks after a slice of 256 requests, blockIdx.y splits the
// slice's tokens and pages further.  Every workgroup adds up the requests in front of its
// slice for itself (they are few, and in the caches), scans its own, and finds the request
// of a token or page by bisection of the scan in LDS: one launch, and no workgroup waits
// for another.  The number of free pages, which all of them read first, is written by the
// last one to finish.  (A release whose table has entries without a page is walked once more by
// that one alone.)
#include "step_launch.h"

namespace gdn {

namespace {

constexpr int kThreads = 256;

// ceil(rows / page), rows < 2^31, page <= 2^30
__device__ __forceinline__ int32_t pages_of(int32_t rows, int32_t page) {
  return (int32_t)(((uint32_t)rows + (uint32_t)page - 1) / (uint32_t)page);
}

// Inclusive sums over the workgroup's threads of a pair; `a`, `b` become them.
__device__ __forceinline__ void scan_pair(int64_t& a, int64_t& b, int64_t (&wave_sums)[2][kThreads / kWave]) {
  const int lane = threadIdx.x % kWave, wave = threadIdx.x / kWave;
#pragma unroll
  for (int s = 1; s < kWave; s <<= 1) {
    const int64_t x = __shfl_up(a, s, kWave), y = __shfl_up(b, s, kWave);
    if (lane >= s) { a += x; b += y; }
  }
  if (lane == kWave - 1) { wave_sums[0][wave] = a; wave_sums[1][wave] = b; }
  __syncthreads();
  for (int w = 0; w < wave; ++w) { a += wave_sums[0][w]; b += wave_sums[1][w]; }
  __syncthreads();
}

// Sum of a pair over the workgroup, in every thread.
__device__ __forceinline__ void sum_pair(int64_t& a, int64_t& b, int64_t (&wave_sums)[2][kThreads / kWave]) {
#pragma unroll
  for (int s = kWave / 2; s; s >>= 1) { a += __shfl_xor(a, s, kWave); b += __shfl_xor(b, s, kWave); }
  if (threadIdx.x % kWave == 0) { wave_sums[0][threadIdx.x / kWave] = a; wave_sums[1][threadIdx.x / kWave] = b; }
  __syncthreads();
  a = b = 0;
  for (int w = 0; w < kThreads / kWave; ++w) { a += wave_sums[0][w]; b += wave_sums[1][w]; }
  __syncthreads();
}

// First k in [0, 256) with ends[k] > v (ends non-decreasing, ends[255] > v).
__device__ __forceinline__ int find(const int32_t* ends, int32_t v) {
  int lo = 0;
#pragma unroll
  for (int s = 128; s; s >>= 1)
    if (ends[lo + s - 1] <= v) lo += s;
  return lo;
}

// True in every thread of the last workgroup of the launch to come here; `arrivals` is 0
// before and after the launch.  `mark` (0 or 1, uniform) becomes the number of workgroups that
// came with 1: they are counted in the upper half, there being 511 workgroups at most.
__device__ __forceinline__ bool last_to_arrive(int32_t* arrivals, int* flag, int& mark) {
  const int total = gridDim.x * gridDim.y;
  if (total == 1) return true;
  __threadfence();
  __syncthreads();
  if (threadIdx.x == 0) {
    const int before = __hip_atomic_fetch_add(arrivals, 1 + (mark << 16), __ATOMIC_ACQ_REL, __HIP_MEMORY_SCOPE_AGENT);
    *flag = (before & 0xffff) == total - 1 ? 1 + (before >> 16) + mark : 0;
    if (*flag) __hip_atomic_store(arrivals, 0, __ATOMIC_RELAXED, __HIP_MEMORY_SCOPE_AGENT);
  }
  __syncthreads();
  const bool last = *flag != 0;
  mark = *flag - 1;
  if (last) __threadfence();
  return last;
}

__device__ __forceinline__ int32_t load_agent(const int32_t* p) {
  return __hip_atomic_load(p, __ATOMIC_RELAXED, __HIP_MEMORY_SCOPE_AGENT);
}

// A sum as LDS holds it: what counts lies below 2^31 (the tokens below T, the pages below the capacity).
__device__ __forceinline__ int32_t narrow(int64_t v) { return (int32_t)min(v, (int64_t)INT32_MAX); }

struct Request {
  int64_t held, tokens, lo, need;
  bool live;
};

__device__ __forceinline__ Request request_of(const PlanPagesLaunch& p, int32_t held, int32_t add) {
  Request r{};
  r.held = held;
  const bool real = held >= 0 && add >= 0;
  r.tokens = real ? add : 0;
  const int64_t rows = (int64_t)held + add;
  const bool fits = real && rows <= INT32_MAX;
  r.lo = pages_of(real ? held : 0, p.page);
  const int32_t hi = pages_of(fits ? (int32_t)rows : 0, p.page);
  r.live = fits && hi <= p.table_width;
  r.need = r.live ? hi - r.lo : 0;
  return r;
}

// f(a[m], b[m]) for this thread's m below n, four loads of each at once.
template <typename Load, typename F>
__device__ __forceinline__ void for_each_pair(int n, Load load, F f) {
  for (int m0 = threadIdx.x; m0 < n; m0 += 4 * kThreads) {
    int32_t a[4], b[4];
#pragma unroll
    for (int k = 0; k < 4; ++k) load(min(m0 + k * kThreads, n - 1), a[k], b[k]);
#pragma unroll
    for (int k = 0; k < 4; ++k)
      if (m0 + k * kThreads < n) f(a[k], b[k]);
  }
}

__global__ void __launch_bounds__(kThreads) plan_kernel(PlanPagesLaunch p) {
  __shared__ int64_t wave_sums[2][kThreads / kWave];
  __shared__ int32_t token_end[kThreads], page_end[kThreads];   // inclusive sums within the slice
  __shared__ int32_t held_of[kThreads], lo_of[kThreads];        // held -1: not served
  __shared__ int flag;
  const int tid = threadIdx.x, base = blockIdx.x * kThreads, part = blockIdx.y, parts = gridDim.y;
  const int64_t count = min(max((int64_t)p.pool[0], (int64_t)0), p.capacity);
  const int32_t* stack = p.pool + 2;
  int64_t tokens0 = 0, pages0 = 0;
  for_each_pair(min(base, p.N), [&](int m, int32_t& a, int32_t& b) { a = p.held[m]; b = p.new_len[m]; },
                [&](int32_t a, int32_t b) {
                  const Request r = request_of(p, a, b);
                  tokens0 += r.tokens;
                  pages0 += r.need;
                });
  sum_pair(tokens0, pages0, wave_sums);
  const int n = base + tid;
  const Request r = n < p.N ? request_of(p, p.held[n], p.new_len[n]) : Request{};
  int64_t te = r.tokens, pe = r.need;
  scan_pair(te, pe, wave_sums);
  const bool served = r.live && pages0 + pe <= count && tokens0 + te <= p.T;
  token_end[tid] = narrow(te);
  page_end[tid] = narrow(pe);
  held_of[tid] = served ? (int32_t)r.held : -1;
  lo_of[tid] = (int32_t)r.lo;
  if (part == 0 && n < p.N) {
    p.cu[n + 1] = (int32_t)min(tokens0 + te, p.T);
    p.cache_len[n] = served ? (int32_t)r.held : -1;
    p.kv_len[n] = served ? (int32_t)(r.held + r.tokens) : -1;
  }
  if (part == 0 && base == 0 && tid == 0) p.cu[0] = 0;
  __syncthreads();
  // new pages, in order (a served request's are all on the stack, below `left`)
  const int stride = parts * kThreads, place = part * kThreads + tid;
  const int32_t left = (int32_t)max(count - pages0, (int64_t)0);
  const int32_t pages = min(page_end[kThreads - 1], left);
  for (int64_t i = place; i < pages; i += stride) {
    const int k = find(page_end, (int32_t)i);
    if (held_of[k] < 0) continue;
    p.table[(int64_t)(base + k) * p.table_stride + lo_of[k] + (i - (k ? page_end[k - 1] : 0))] = stack[left - 1 - i];
  }
  // tokens; the last slice also those behind the last request
  const int32_t mine = token_end[kThreads - 1];
  const int32_t room = (int32_t)max(p.T - tokens0, (int64_t)0);
  const int32_t stop = blockIdx.x == gridDim.x - 1 ? room : min(mine, room);
  const uint32_t page = p.page;
  for (int64_t i64 = place; i64 < stop; i64 += stride) {
    const int32_t i = (int32_t)i64;
    int64_t slot = -1;
    int32_t position = -1, owner = -1;
    if (i < mine) {
      const int k = find(token_end, i);
      if (held_of[k] >= 0) {
        const uint32_t in = i - (k ? token_end[k - 1] : 0), row = held_of[k] + in;
        const uint32_t entry = row / page, rest = row - entry * page;
        owner = base + k;
        const int32_t id = entry >= (uint32_t)lo_of[k] ? stack[left - 1 - ((k ? page_end[k - 1] : 0) + (int32_t)entry - lo_of[k])]
                                                       : p.table[(int64_t)owner * p.table_stride + entry];
        if (id >= 0) slot = (int64_t)id * page + rest;
        position = (int32_t)((p.start ? (uint32_t)p.start[owner] : (uint32_t)held_of[k]) + in);
      }
    }
    const int64_t t = tokens0 + i;
    if (p.slots) p.slots[t] = slot;
    if (p.positions) p.positions[t] = position;
    if (p.seq) p.seq[t] = owner;
  }
  int mark = 0;
  if (!last_to_arrive(p.pool + 1, &flag, mark)) return;
  int64_t taken = 0, none = 0;
  if (gridDim.x * gridDim.y > 1) {
    for_each_pair(p.N, [&](int m, int32_t& a, int32_t& b) { a = load_agent(p.cache_len + m); b = load_agent(p.kv_len + m); },
                  [&](int32_t a, int32_t b) { taken += a >= 0 ? pages_of(b, p.page) - pages_of(a, p.page) : 0; });
  } else {
    taken = served ? r.need : 0;
  }
  sum_pair(taken, none, wave_sums);
  if (tid == 0) p.pool[0] = (int32_t)(count - taken);
}

__device__ __forceinline__ int32_t given_back(const ReleasePagesLaunch& p, int32_t keep, int32_t held, int32_t& lo) {
  const bool some = keep >= 0 && held > keep;
  lo = pages_of(some ? keep : 0, p.page);
  const int32_t hi = some ? min(pages_of(held, p.page), p.table_width) : 0;
  return hi > lo ? hi - lo : 0;
}

__global__ void __launch_bounds__(kThreads) release_kernel(ReleasePagesLaunch p) {
  __shared__ int64_t wave_sums[2][kThreads / kWave];
  __shared__ int32_t page_end[kThreads], lo_of[kThreads];
  __shared__ int flag;
  const int tid = threadIdx.x, base = blockIdx.x * kThreads, part = blockIdx.y, parts = gridDim.y;
  const int64_t count = min(max((int64_t)p.pool[0], (int64_t)0), p.capacity);
  int32_t* stack = p.pool + 2;
  int64_t before = 0, none = 0;
  int32_t lo = 0;
  const auto load = [&](int m, int32_t& a, int32_t& b) { a = p.keep[m]; b = p.held[m]; };
  for_each_pair(min(base, p.N), load, [&](int32_t a, int32_t b) { int32_t at; before += given_back(p, a, b, at); });
  sum_pair(before, none, wave_sums);
  int64_t pe = base + tid < p.N ? given_back(p, p.keep[base + tid], p.held[base + tid], lo) : 0;
  scan_pair(pe, none, wave_sums);
  page_end[tid] = narrow(pe);
  lo_of[tid] = lo;
  __syncthreads();
  // (as far as the stack's capacity goes)
  const int64_t pages = min((int64_t)page_end[kThreads - 1], p.capacity - count - before);
  auto entry = [&](int first, int32_t i) {            // the i-th of the slice whose requests begin at `first`
    const int k = find(page_end, i);
    return p.table[(int64_t)(first + k) * p.table_stride + lo_of[k] + i - (k ? page_end[k - 1] : 0)];
  };
  bool hole = false;
  for (int64_t i = (int64_t)part * kThreads + tid; i < pages; i += (int64_t)parts * kThreads) {
    const int32_t id = entry(base, (int32_t)i);
    stack[count + before + i] = id;
    hole |= id < 0;
  }
  int holes = __syncthreads_or(hole) != 0;
  if (!last_to_arrive(p.pool + 1, &flag, holes)) return;
  int64_t total = 0;
  none = 0;
  if (holes == 0) {
    for_each_pair(p.N, load, [&](int32_t a, int32_t b) { int32_t at; total += given_back(p, a, b, at); });
    sum_pair(total, none, wave_sums);
  } else {
    // Entries without a page do not come to the stack: all of them in order once more, a thread
    // eight at a time, each at the number of pages before it.  (Rare, and not worth a count of
    // every other release's pages ahead of its writes.)
    constexpr int kEach = 8;
    for (int first = 0; first < p.N; first += kThreads) {
      const int n = first + tid;
      pe = n < p.N ? given_back(p, p.keep[n], p.held[n], lo) : 0;
      scan_pair(pe, none, wave_sums);                  // (its barriers end the last slice's look-ups)
      page_end[tid] = narrow(pe);
      lo_of[tid] = lo;
      __syncthreads();
      const int64_t all = page_end[kThreads - 1];
      for (int64_t i0 = 0; i0 < all && count + total < p.capacity; i0 += kThreads * kEach) {
        int32_t id[kEach];
        int64_t mine = 0;
#pragma unroll
        for (int q = 0; q < kEach; ++q) {
          const int64_t i = i0 + tid * kEach + q;
          id[q] = i < all ? entry(first, (int32_t)i) : -1;
          mine += id[q] >= 0;
        }
        int64_t at = mine, chunk = mine;
        scan_pair(at, none, wave_sums);
        sum_pair(chunk, none, wave_sums);
        at += count + total - mine;
#pragma unroll
        for (int q = 0; q < kEach; ++q) {
          if (id[q] < 0) continue;
          if (at < p.capacity) stack[at] = id[q];
          ++at;
        }
        total += chunk;
      }
    }
  }
  if (tid == 0) p.pool[0] = (int32_t)min(count + total, p.capacity);
}

int parts_of(int64_t items, int64_t slices) {
  // 1024 tokens or pages a workgroup, on average over the slices; no more than 256 workgroups or so,
  // each of which adds up the requests in front of it
  const int64_t want = (items / slices + 1023) / 1024, most = (255 + slices) / slices;
  return (int)(want > most ? most : want < 1 ? 1 : want);
}

}  // namespace

hipError_t launch_plan_pages(const PlanPagesLaunch& p, hipStream_t stream) {
  const int64_t slices = p.N > 0 ? (p.N + kThreads - 1) / kThreads : 1;
  hipLaunchKernelGGL(plan_kernel, dim3((unsigned)slices, parts_of(p.T, slices)), dim3(kThreads), 0, stream, p);
  return hipGetLastError();
}

hipError_t launch_release_pages(const ReleasePagesLaunch& p, hipStream_t stream) {
  const int64_t slices = (p.N + kThreads - 1) / kThreads;
  hipLaunchKernelGGL(release_kernel, dim3((unsigned)slices, parts_of((int64_t)p.N * p.table_width, slices)), dim3(kThreads), 0,
                     stream, p);
  return hipGetLastError();
}

}  // namespace gdn
