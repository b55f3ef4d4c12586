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
  for (int k = 0; k < kScanThreads / 64; ++k) {
    if (k < wave) before = before + waves[k];
    all = all + waves[k];
  }
}

// One workgroup: what goes by request and by sequence
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
  hipLaunchKernelGGL(pack_requests_kernel, dim3(1), dim3(kScanThreads), 0, st, p);
  const hipError_t e = hipGetLastError();
  if (e != hipSuccess) return e;
  const int64_t x = p.requests / 4 + 8, runs = ((int64_t)p.tokens + kRun - 1) / kRun, most = ((int64_t)1 << 22) / x;
  const dim3 grid((uint32_t)x, (uint32_t)(runs < 64 ? (runs < most ? runs : most) : most < 64 ? most : 64));
  hipLaunchKernelGGL(pack_rows_kernel, grid, dim3(256), 0, st, p);
  return hipGetLastError();
}

}  // namespace ss
