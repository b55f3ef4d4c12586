// ss_pack.hip -- rows, sequences and slots of a serving batch, from its requests' lengths (gfx950).
//
// The batch's rows: one of every request that decodes a token, in the requests'
// order, then the rows of every prompt, in that order, as many as there is room
// for.  All of it is prefix sums over the requests: of the steps, of the prompts
// and of the prompts' rows.
#include "ss_device.h"
#include "ss_internal.h"

namespace ss {
namespace {

constexpr int kScanThreads = 1024;

struct Counts {
  int32_t steps, prompts;
  int64_t rows;  // of prompts
};
__device__ __forceinline__ Counts operator+(Counts a, Counts b) {
  return {a.steps + b.steps, a.prompts + b.prompts, a.rows + b.rows};
}
struct Request {
  int32_t rows, seen, slot;
  bool step, prompt;
};
__device__ __forceinline__ Request request(const PackParams& p, int i) {
  Request q{0, 0, -1, false, false};
  if (i < p.requests) {
    q.slot = p.slots[i];
    q.seen = p.seen[i];
    const int32_t n = p.new_tokens[i];
    q.rows = q.slot >= 0 && n > 0 ? n : 0;
    q.step = q.rows == 1 && q.seen > 0;
    q.prompt = q.rows > 0 && !q.step;
  }
  return q;
}
__device__ __forceinline__ Counts counts(const Request& q) { return {q.step, q.prompt, q.prompt ? q.rows : 0}; }

// sums over the threads before this one (before) and over all
__device__ __forceinline__ void block_sums(Counts own, Counts* waves, Counts& before, Counts& all) {
  const int lane = threadIdx.x % 64, wave = threadIdx.x / 64;
  Counts run = own;
#pragma unroll
  for (int off = 1; off < 64; off <<= 1) {
    const Counts o = {__shfl_up(run.steps, off, 64), __shfl_up(run.prompts, off, 64), __shfl_up(run.rows, off, 64)};
    if (lane >= off) run = run + o;
  }
  __syncthreads();  // the last round's sums are read
  if (lane == 63) waves[wave] = run;
  __syncthreads();
  before = {run.steps - own.steps, run.prompts - own.prompts, run.rows - own.rows};
  all = {0, 0, 0};
#pragma unroll 2
  for (int k = 0; k < kScanThreads / 64; ++k) {
    if (k < wave) before = before + waves[k];
    all = all + waves[k];
  }
}

// ---- up to 4096 requests: one launch --------------------------------------------------------
// Every workgroup takes the sums over all requests, ITEMS a thread, and lists in LDS the
// requests that have rows, in the rows' order.  It writes what goes by request for its
// share of the waves and by row for its rows, whose requests it finds in the list by
// bisection.  Reading all requests in each workgroup (48 KiB at most, from L2) costs less
// than a second launch that waits for the first: 64 requests and 2048 rows 3.9 us against
// 14.4 + 2.8, 4001 and 65536 rows 6.8 against 30 + 5.3.  Bound by latency: a load, two
// barriers, the bisection's reads of LDS.  4096 requests fill 4 a thread and 48 KiB of
// LDS, which two workgroups have room for on a CU.
struct Sums {
  uint32_t number;  // of steps, and of prompts * 2^16
  uint32_t rows;    // of prompts, up to 2^31 - 1
};
__device__ __forceinline__ Sums operator+(Sums a, Sums b) {
  const uint32_t r = a.rows + b.rows;
  return {a.number + b.number, r < 0x7fffffffu ? r : 0x7fffffffu};
}
template <int THREADS, int ITEMS>
__global__ void __launch_bounds__(THREADS) pack_kernel(PackParams p) {
  constexpr int kMost = THREADS * ITEMS;
  __shared__ Sums waves[THREADS / 64];
  __shared__ int32_t start[kMost], who[kMost];
  __shared__ uint32_t base[kMost];
  __shared__ int32_t last;
  const int tid = threadIdx.x, lane = tid % 64, wave = tid / 64;
  int32_t n[ITEMS], slot[ITEMS], seen[ITEMS];
  if (ITEMS == 4 && 4 * tid + 3 < p.requests) {
    typedef int32_t int4_t __attribute__((ext_vector_type(4)));
    const int4_t a = reinterpret_cast<const int4_t*>(p.new_tokens)[tid], b = reinterpret_cast<const int4_t*>(p.slots)[tid],
                 c = reinterpret_cast<const int4_t*>(p.seen)[tid];
#pragma unroll
    for (int e = 0; e < ITEMS; ++e) {
      n[e] = a[e % 4];
      slot[e] = b[e % 4];
      seen[e] = c[e % 4];
    }
  } else {
#pragma unroll
    for (int e = 0; e < ITEMS; ++e) {
      const int i = ITEMS * tid + e;
      const bool in = i < p.requests;
      n[e] = in ? p.new_tokens[i] : 0;
      slot[e] = in ? p.slots[i] : -1;
      seen[e] = in ? p.seen[i] : 0;
    }
  }
  Sums own{0, 0};
#pragma unroll
  for (int e = 0; e < ITEMS; ++e) {
    if (slot[e] < 0 || n[e] < 0) n[e] = 0;
    const bool step = n[e] == 1 && seen[e] > 0;
    own = own + Sums{step ? 1u : n[e] > 0 ? 0x10000u : 0u, step ? 0u : (uint32_t)n[e]};
  }
  // sums over the lanes before this one; saturating sums are not taken apart again, so the
  // scan leaves this lane's own out
  Sums run = own;
#pragma unroll
  for (int off = 1; off < 64; off <<= 1) {
    const Sums o = {(uint32_t)__shfl_up((int)run.number, off, 64), (uint32_t)__shfl_up((int)run.rows, off, 64)};
    if (lane >= off) run = run + o;
  }
  if (lane == 63) waves[wave] = run;
  if (tid == 0) last = 0;
  Sums before = {(uint32_t)__shfl_up((int)run.number, 1, 64), (uint32_t)__shfl_up((int)run.rows, 1, 64)};
  if (lane == 0) before = {0, 0};
  __syncthreads();
  Sums all{0, 0};
  {
    Sums front{0, 0};
#pragma unroll
    for (int k = 0; k < THREADS / 64; ++k) {
      if (k == wave) front = all;
      all = all + waves[k];
    }
    before = front + before;
  }
  const uint32_t most = (uint32_t)p.tokens, steps = all.number & 0xffffu;
  const uint32_t listed_steps = steps < most ? steps : most;
  const int32_t end = (int32_t)(steps + all.rows < most ? steps + all.rows : most);
  const bool write = (uint32_t)wave % gridDim.x == blockIdx.x;
  int32_t listed = 0;
#pragma unroll
  for (int e = 0; e < ITEMS; ++e) {
    const int i = ITEMS * tid + e;
    const bool step = n[e] == 1 && seen[e] > 0;
    const uint32_t nstep = before.number & 0xffffu, nprompt = before.number >> 16;
    const uint32_t at = step ? nstep : steps + before.rows;
    const uint32_t left = at < most ? most - at : 0u, taken = (uint32_t)n[e] < left ? (uint32_t)n[e] : left;
    if (taken) {
      const uint32_t k = step ? nstep : steps + nprompt;
      start[k] = (int32_t)at;
      who[k] = i;
      base[k] = (uint32_t)(seen[e] > 0 ? seen[e] : 0) - at;
      if (!step) listed = (int32_t)nprompt + 1;
    }
    if (write && i < p.requests) {
      p.rows[i] = taken ? (int32_t)at : -1;
      p.taken[i] = (int32_t)taken;
      if (taken && step) p.step_slots[nstep] = slot[e];
      if (taken && !step) {
        p.cu[nprompt] = (int32_t)at;
        p.prompt_slots[nprompt] = slot[e];
        p.has_state[nprompt] = seen[e] > 0;
      }
    }
    before = before + Sums{step ? 1u : n[e] > 0 ? 0x10000u : 0u, step ? 0u : (uint32_t)n[e]};
  }
  if (listed) atomicMax(&last, listed);
  __syncthreads();
  listed = last;
  const int first = (int)blockIdx.x * THREADS + tid, stride = (int)gridDim.x * THREADS;
  for (int i = first; i <= p.requests; i += stride) {
    if (i >= listed) p.cu[i] = end;
    if (i >= p.requests) continue;
    if (i >= (int)listed_steps) p.step_slots[i] = -1;
    if (i >= listed) {
      p.prompt_slots[i] = -1;
      p.has_state[i] = 0;
    }
  }
  int top = 1;
  while (2 * top < listed) top *= 2;
  for (int64_t k = first; k < p.tokens; k += stride) {
    int32_t request = -1, position = -1;
    if (k < end) {
      int at = (int)k;
      if (k >= listed_steps) {
        at = (int)steps;  // the last prompt that starts at this row or before it
        for (int b = top; b; b /= 2)
          if (at + b < (int)steps + listed && start[at + b] <= k) at += b;
      }
      request = who[at];
      position = (int32_t)(base[at] + (uint32_t)k);
    }
    p.row_request[k] = request;
    p.row_position[k] = position;
  }
}

// ---- more requests: what goes by request and by sequence in one workgroup, then what goes by row ----
__global__ void __launch_bounds__(kScanThreads) pack_requests_kernel(PackParams p) {
  __shared__ Counts waves[kScanThreads / 64];
  const int tid = threadIdx.x;
  Counts own{0, 0, 0}, before, total;
  for (int i = tid; i < p.requests; i += kScanThreads) own = own + counts(request(p, i));
  block_sums(own, waves, before, total);
  const int64_t most = p.tokens, steps = total.steps;
  Counts base{0, 0, 0};
  for (int i0 = 0; i0 < p.requests; i0 += kScanThreads) {
    const int i = i0 + tid;
    const Request q = request(p, i);
    Counts all;
    block_sums(counts(q), waves, before, all);
    before = before + base;
    base = base + all;
    if (i >= p.requests) continue;
    const int64_t at = q.step ? before.steps : steps + before.rows, left = most - at;
    const int32_t taken = left <= 0 ? 0 : q.rows < left ? q.rows : (int32_t)left;
    p.rows[i] = taken ? (int32_t)at : -1;
    p.taken[i] = taken;
    if (taken && q.step) p.step_slots[before.steps] = q.slot;
    if (taken && q.prompt) {
      p.cu[before.prompts] = (int32_t)at;
      p.prompt_slots[before.prompts] = q.slot;
      p.has_state[before.prompts] = q.seen > 0;
    }
  }
  // behind the last step and the last prompt: prompts that had no row are not listed, which
  // are the last ones; the first of them is the one that no row was left for
  const int32_t end = (int32_t)(steps + total.rows < most ? steps + total.rows : most);
  const int32_t listed_steps = (int32_t)(steps < most ? steps : most);
  __syncthreads();
  int32_t listed = 0;  // prompts with a row
  if (steps + total.rows <= most) {
    listed = total.prompts;
  } else {
    Counts run{0, 0, 0};
    for (int i0 = 0; i0 < p.requests; i0 += kScanThreads) {
      const Request q = request(p, i0 + tid);
      Counts all;
      block_sums(counts(q), waves, before, all);
      before = before + run;
      run = run + all;
      listed += __syncthreads_count(q.prompt && steps + before.rows < most);
    }
  }
  for (int i = tid; i <= p.requests; i += kScanThreads) {
    if (i >= listed) p.cu[i] = end;
    if (i < p.requests) {
      if (i >= listed_steps) p.step_slots[i] = -1;
      if (i >= listed) {
        p.prompt_slots[i] = -1;
        p.has_state[i] = 0;
      }
    }
  }
}

// What goes by row.  A wave writes every gridDim.y-th run of kRun rows of a request, and
// the waves behind the last request the rows of none.
constexpr int kRun = 4096;
__global__ void __launch_bounds__(256) pack_rows_kernel(PackParams p) {
  const int i = (int)blockIdx.x * 4 + (int)threadIdx.x / 64, lane = threadIdx.x % 64;
  if (i < p.requests) {
    const int n = p.taken[i], at = p.rows[i];
    const int32_t seen = p.seen[i] > 0 ? p.seen[i] : 0;
    for (int64_t first = (int64_t)blockIdx.y * kRun; first < n; first += (int64_t)gridDim.y * kRun) {
      const int end = n < first + kRun ? n : (int)(first + kRun);
      for (int k = (int)first + lane; k < end; k += 64) {
        p.row_request[at + k] = i;
        p.row_position[at + k] = (int32_t)((uint32_t)seen + (uint32_t)k);
      }
    }
  } else {
    const int64_t begin = p.cu[p.requests];
    const int64_t step = (int64_t)gridDim.y * 64 * ((int)gridDim.x * 4 - p.requests);
    for (int64_t k = begin + ((int64_t)(i - p.requests) * gridDim.y + blockIdx.y) * 64 + lane; k < p.tokens; k += step) {
      p.row_request[k] = -1;
      p.row_position[k] = -1;
    }
  }
}

}  // namespace

hipError_t launch_pack(const PackParams& p, hipStream_t st) {
  if (p.requests <= 4096) {
    const int threads = p.requests <= 256 ? 256 : 1024;
    const int64_t rows = ((int64_t)p.tokens + threads - 1) / threads;
    const dim3 grid((uint32_t)(rows < 256 ? rows : 256));
    if (threads == 256) hipLaunchKernelGGL((pack_kernel<256, 1>), grid, dim3(256), 0, st, p);
    else hipLaunchKernelGGL((pack_kernel<1024, 4>), grid, dim3(1024), 0, st, p);
    return hipGetLastError();
  }
  hipLaunchKernelGGL(pack_requests_kernel, dim3(1), dim3(kScanThreads), 0, st, p);
  const hipError_t e = hipGetLastError();
  if (e != hipSuccess) return e;
  const int64_t x = p.requests / 4 + 8, runs = ((int64_t)p.tokens + kRun - 1) / kRun, most = ((int64_t)1 << 22) / x;
  const dim3 grid((uint32_t)x, (uint32_t)(runs < 64 ? (runs < most ? runs : most) : most < 64 ? most : 64));
  hipLaunchKernelGGL(pack_rows_kernel, grid, dim3(256), 0, st, p);
  return hipGetLastError();
}

}  // namespace ss
