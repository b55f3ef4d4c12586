// ss_prompt.hip -- the Mamba-2 SSD scan of packed prompts on MFMA (gfx950).
//
// Page "Mamba" (walkthrough), "Deep dive: Mamba-2 and state-space duality":
// per head, with the state H[p][n] (headdim 64 x dstate N),
//   H_t = exp(Delta_t A) H_{t-1} + Delta_t x_t B_t^T,  y_t = H_t C_t + D x_t,
// computed in chunks of Q = 256 steps; with cs the running sum of Delta A from
// a chunk's first step,
//   S   = sum_j exp(cs_last - cs_j) Delta_j x_j B_j^T          (the chunk's own state)
//   E'  = exp(cs_last) E + S                                   (E enters the chunk)
//   Y_i = exp(cs_i) E C_i + sum_{j<=i} exp(cs_i - cs_j) Delta_j (C_i . B_j) x_j.
// The prompts of a batch lie one behind the other (cu: their row offsets);
// chunks are counted from each prompt's first row (ss_packed.h), so that no
// chunk holds two prompts, and every prompt's state comes from and goes to
// its slot of a pool.  Three kernels:
//   prompt_state_kernel  per (chunk, a few heads): S, and the decay over the chunk;
//                        further workgroups compute C B^T per (chunk, group);
//   prompt_pass_kernel   per (prompt of several chunks, head, 1024 elements): E of
//                        every chunk, in the place of its S, and the final state;
//   prompt_scan_kernel   per (chunk, head): Y, skip, gate.
// All chunks of a prompt run at once, whatever its length; only the
// element-wise pass walks them in order.  24 ragged prompts of 16384 tokens (24
// heads, state 128, bf16, gate): 50, 25 and 88 us; one prompt of 32769 tokens
// (state 64, fp16): 68-72, 21 and 118-126 us.  Of the bytes, 4 times the fp32 states
// (276 MB of the first) are the price of the chunks' independence: a walk over the
// chunks inside a workgroup, as in ss_ssd.hip, has no such traffic and as many
// workgroups as prompts have heads.
//
// Precision: products of 16-bit inputs run on the matrix cores as they are.
// Computed operands are multiplied as sums of bf16 parts (ss_mfma.h): the
// weighted x that makes the states in three, E and the decayed C B^T, which
// make y, in two.  States stay in fp32.
#include "ss_device.h"
#include "ss_internal.h"
#include "ss_mfma.h"
#include "ss_packed.h"
#include "ss_state.h"

namespace ss {
namespace {

constexpr int kLogQ = 8;
constexpr int kQ = 1 << kLogQ;  // chunk length
constexpr int kP = 64;          // headdim
constexpr int kJB = 64;         // time piece of a chunk

template <int IO>
__device__ __forceinline__ float step_size(const SsdPromptParams& p, float raw, int h) {
  const float xd = raw + (p.dt_bias ? p.dt_bias[h] : 0.0f);
  return p.softplus ? softplus_f(xd) : xd;
}

// ---- pass 1: the chunks' own states, and C B^T --------------------------------
// State workgroup = (chunk, HB heads of a group): S of ss_state.h with u = x, V = B
// and w_j = exp(sum of Delta A behind j) Delta_j, from a sum that runs backwards,
// so that no difference of long sums enters the state.  A prompt of one chunk (or
// none) is done with its state here: E is its slot's and goes to the workspace,
// E' = decay E + S to the slot, and the pass between the chunks leaves it out.
template <int IO, int N, int HB>
__device__ __forceinline__ void state_role(const SsdPromptParams& p, int place, int g, int h0, int heads,
                                           StateLds<N, HB, 1, 1, IO == SS_F16>& lds) {
  const int tid = threadIdx.x, lane = tid % 64, wave = tid / 64, team = tid / 256, t = tid % 256;
  const SeqChunk q = find_chunk<kLogQ>(p.cu, p.nseqs, p.tokens, place);
  if (q.chunk < 0 || (q.chunk > 0 && q.chunk * kQ >= q.len)) return;
  const bool single = q.len <= kQ;
  const int slot = single ? uniform(slot_of(p.slots, q.seq, p.nslots)) : -1;
  const bool carried = slot >= 0 && p.has_state && p.has_state[q.seq] != 0;
  float* state = p.state + ((int64_t)(slot < 0 ? 0 : slot) * p.nheads + h0) * (kP * N);
  if (q.len == 0) {  // a state that is not carried starts, and ends, as zeros
    if (slot >= 0 && !carried)
      for (int k = tid; k < heads * (kP * N / 4); k += kStateThreads)
        reinterpret_cast<f32x4*>(state)[k] = f32x4{0.0f, 0.0f, 0.0f, 0.0f};
    return;
  }
  const int left = q.len - q.chunk * kQ, rows = left < kQ ? left : kQ;
  const int64_t row0 = q.begin + (int64_t)q.chunk * kQ;
#pragma unroll
  for (int hb = 0; hb < HB; hb += 2) {  // two heads at a time, 256 threads each
    const int h = h0 + hb + team;
    const bool in = t < rows && hb + team < heads;
    const float delta = in ? step_size<IO>(p, load_io<IO>(p.dt, (row0 + t) * p.dt_stride + h), h) : 0.0f;
    float v = in ? delta * p.A[h] : 0.0f;  // sum from this step to the end of the wave's 64
#pragma unroll
    for (int off = 1; off < 64; off <<= 1) {
      const float o = __shfl_down(v, off, 64);
      if (lane + off < 64) v += o;
    }
    if (lane == 0) lds.wave[team][wave % 4] = v;
    __syncthreads();
    float behind = __shfl_down(v, 1, 64);
    if (lane == 63) behind = 0.0f;
    const float* sum = lds.wave[team];
    for (int w = 3; w > wave % 4; --w) behind += sum[w];
    if (hb + team < HB) lds.w[hb + team][t] = in ? exp2_hw(behind * kLog2e) * delta : 0.0f;  // in: its head is there
    if (t == 0 && hb + team < heads)
      p.ws_decay[(int64_t)place * p.nheads + h] = lds.decay[hb + team] =
          exp2_hw((sum[0] + sum[1] + sum[2] + sum[3]) * kLog2e);
    if (hb + 2 < HB) __syncthreads();
  }
  const int64_t xrow = p.x_stride, brow = p.b_stride;
  const __amdgpu_buffer_rsrc_t xv[1] = {
      rows_view(static_cast<const char*>(p.x) + (row0 * xrow + h0 * kP) * 2, xrow * 2, rows, heads * (kP * 2))};
  const __amdgpu_buffer_rsrc_t bv[1] = {
      rows_view(static_cast<const char*>(p.Bm) + (row0 * brow + g * N) * 2, brow * 2, rows, N * 2)};
  float* ws = p.ws_state + ((int64_t)place * p.nheads + h0) * (kP * N);
  chunk_states<IO, N, HB, 1, 1, IO == SS_F16>(
      lds, xv, xrow, bv, brow, rows, heads, [&](int hb, int at, const f32x4 (&S)[N / 32]) {
        f32x4 E[N / 32];
#pragma unroll
        for (int t = 0; t < N / 32; ++t) {
          E[t] = f32x4{0.0f, 0.0f, 0.0f, 0.0f};
          if (carried) E[t] = *reinterpret_cast<const f32x4*>(state + hb * (kP * N) + at + 16 * t);
        }
        const float decay = lds.decay[hb];
#pragma unroll
        for (int t = 0; t < N / 32; ++t) {
          *reinterpret_cast<f32x4*>(ws + hb * (kP * N) + at + 16 * t) = single ? E[t] : S[t];
          if (slot >= 0) {
#pragma unroll
            for (int e = 0; e < 4; ++e) E[t][e] = fmaf(decay, E[t][e], S[t][e]);
            *reinterpret_cast<f32x4*>(state + hb * (kP * N) + at + 16 * t) = E[t];
          }
        }
      });
}

// C B^T workgroup = (chunk, group, half of the rows): for the half's rows i and
// the columns j up to the end of i's piece of 64, in fp32, in the order in which the output pass
// reads its operands: element (i, j) of row tile it = i / 16 and k-step
// kt = j / 32 is float j % 8 of lane i % 16 + 16 ((j % 32) / 8), 8 floats a
// lane, so that pass reads whole contiguous kilobytes.  Wave w has row tile
// 8 half + w; the product is built transposed (B C^T), so that a lane holds 4
// consecutive columns of one row.
template <int IO, int N>
__device__ __forceinline__ void cb_role(const SsdPromptParams& p, int place, int g, int half) {
  const int lane = threadIdx.x % 64, wave = threadIdx.x / 64;
  const SeqChunk q = find_chunk<kLogQ>(p.cu, p.nseqs, p.tokens, place);
  if (q.chunk < 0 || q.chunk * kQ >= q.len) return;
  const int left = q.len - q.chunk * kQ, rows = left < kQ ? left : kQ;
  const int it = 8 * half + wave;
  if (16 * it >= rows) return;
  const int64_t row0 = q.begin + (int64_t)q.chunk * kQ;
  const int64_t brow = p.b_stride * 2, crow = p.c_stride * 2;
  const auto bv = rows_view(static_cast<const char*>(p.Bm) + row0 * brow + g * N * 2, brow, rows, N * 2);
  const auto cv = rows_view(static_cast<const char*>(p.Cm) + row0 * crow + g * N * 2, crow, rows, N * 2);
  u32x4v c[N / 32];
#pragma unroll
  for (int ks = 0; ks < N / 32; ++ks)
    c[ks] = vload16(cv, (uint32_t)((16 * it + lane % 16) * crow + (32 * ks + 8 * (lane / 16)) * 2));
  float* CB = p.ws_cb + ((int64_t)place * p.ngroups + g) * (kQ * kQ);
  u32x4v b[N / 32];
  auto load_b = [&](int jt) {
#pragma unroll
    for (int ks = 0; ks < N / 32; ++ks)
      b[ks] = vload16(bv, (uint32_t)((16 * jt + lane % 16) * brow + (32 * ks + 8 * (lane / 16)) * 2));
  };
  load_b(0);
  const int j1 = 4 * (it / 4) + 4;
  for (int jt = 0; jt < j1; ++jt) {
    f32x4 acc = f32x4{0.0f, 0.0f, 0.0f, 0.0f};
#pragma unroll
    for (int ks = 0; ks < N / 32; ++ks) acc = mfma_t<IO>::run(as_vec<IO>(b[ks]), as_vec<IO>(c[ks]), acc);
    if (jt + 1 < j1) load_b(jt + 1);
    const int to = lane % 16 + 16 * (2 * (jt & 1) + lane / 32);
    *reinterpret_cast<f32x4*>(CB + cb_at(it, jt / 2) + to * 8 + 4 * ((lane / 16) & 1)) = acc;
  }
}

template <int IO, int N, int HB>
__global__ void __launch_bounds__(kStateThreads, IO == SS_F16 ? 2 : 4) prompt_state_kernel(SsdPromptParams p) {
  __shared__ StateLds<N, HB, 1, 1, IO == SS_F16> lds;
  // a (chunk, group) has 2 workgroups for C B^T, which take longest, then `parts`
  // for the states, all on one XCD
  const int hpg = p.nheads / p.ngroups, parts = (hpg + HB - 1) / HB;
  const int lb = (int)xcd_logical_block(), r = lb % (parts + 2), g = (lb / (parts + 2)) % p.ngroups;
  const int place = lb / (parts + 2) / p.ngroups;
  if (r < 2) {
    cb_role<IO, N>(p, place, g, 1 - r);
  } else {
    const int h = (r - 2) * HB, left = hpg - h;
    state_role<IO, N, HB>(p, place, g, g * hpg + h, left < HB ? left : HB, lds);
  }
}

// ---- pass 2: the states between the chunks -----------------------------------------
// Workgroup = (prompt, head, 1024 elements), a thread 4 elements: E <- the
// slot's state (or 0); per chunk, S <- E in memory and E <- decay E + S.  AHEAD
// chunks' S are loaded ahead; a chunk's view is empty behind the last one.
template <int N, int AHEAD>
__global__ void __launch_bounds__(256) prompt_pass_kernel(SsdPromptParams p) {
  constexpr int kParts = kP * N / 1024;
  const int part = (int)(blockIdx.x % kParts);
  const int h = (int)((blockIdx.x / kParts) % (uint32_t)p.nheads);
  const int s = (int)(blockIdx.x / kParts / (uint32_t)p.nheads);
  const int e = part * 1024 + 4 * (int)threadIdx.x;
  const int begin = uniform(seq_row(p.cu, s, p.tokens)), end = uniform(seq_row(p.cu, s + 1, p.tokens));
  const int n = end > begin ? (end - begin + kQ - 1) >> kLogQ : 0;
  if (n <= 1) return;  // done with its chunk
  const int first = (begin >> kLogQ) + s;
  const int slot = uniform(slot_of(p.slots, s, p.nslots));
  f32x4* state = reinterpret_cast<f32x4*>(p.state + ((int64_t)(slot < 0 ? 0 : slot) * p.nheads + h) * (kP * N) + e);
  f32x4 E = f32x4{0.0f, 0.0f, 0.0f, 0.0f};
  if (slot >= 0 && p.has_state && p.has_state[s] != 0) E = *state;
  float* ws = p.ws_state + ((int64_t)first * p.nheads + h) * (kP * N);
  const float* dec = p.ws_decay + (int64_t)first * p.nheads + h;
  const int64_t step = (int64_t)p.nheads * (kP * N);
  // chunk c's state, empty behind the last: what is out of range reads 0 and is not written
  auto at = [&](int c) { return make_rsrc(ws + c * step, c < n ? (uint32_t)(kP * N * 4) : 0u); };
  f32x4 S[AHEAD];
  float d[AHEAD];
  auto load = [&](int k, int c) {
    if (AHEAD == 4 && c >= n) return;  // short prompts: most of the loads ahead are behind the end
    S[k] = __builtin_bit_cast(f32x4, vload16(at(c), (uint32_t)(e * 4)));
    d[k] = __builtin_bit_cast(float, __builtin_amdgcn_raw_buffer_load_b32(
        make_rsrc(dec + (int64_t)c * p.nheads, c < n ? 4u : 0u), 0, 0, 0));
  };
#pragma unroll
  for (int k = 0; k < AHEAD; ++k) load(k, k);
  for (int c = 0; c < n; c += AHEAD) {
#pragma unroll
    for (int k = 0; k < AHEAD; ++k) {
      if (k && k % 4 == 0 && c + k >= n) break;
      const f32x4 own = S[k];
      const float decay = d[k];
      load(k, c + k + AHEAD);
      __builtin_amdgcn_raw_buffer_store_b128(__builtin_bit_cast(u32x4v, E), at(c + k), (uint32_t)(e * 4), 0, 0);
      if (c + k < n) {
#pragma unroll
        for (int i = 0; i < 4; ++i) E[i] = fmaf(decay, E[i], own[i]);
      }
    }
  }
  if (slot >= 0) *state = E;
}

// ---- pass 3: outputs of a chunk ------------------------------------------------------
// Workgroup = (chunk, head), 512 threads.  Y is built transposed, Y^T[p][i], so
// that a lane ends with 4 consecutive channels of one step i.  The chunk's 256
// rows are 8 blocks of 32; waves w and w + 4 take the two 16-row halves of
// blocks w and 7 - w, so that every wave does the same causal work:
//   Y^T = E C^T scaled by exp(cs_i)  +  x^T M^T,
// M[i][j] = CB[i][j] exp(cs_i - cs_j) Delta_j for j <= i, built in registers.
// cs is kept as its sum inside a piece of 64 steps (sCs; what the float leaves goes
// into sRow and the columns' factors) and the sums over whole pieces (sTot), in
// powers of two: pairs inside a piece take a difference of the former, a
// pair across pieces two factors, exp(cs_i - end of j's piece) and
// exp(end of j's piece - cs_j), one exp per row and one per column.  fp16's lo
// part of x takes E's place once E C^T is done, so that two workgroups share a
// CU (one prompt of 32769 tokens: 122 us, 137 us with one).  C B^T and y go
// through range-checked views, whose addresses take one register, and the gate
// is loaded in the place of a next piece behind the last: at two workgroups to a
// CU nothing is spilled, but 4 registers of bf16 at states below 128 (87 and 118-126 us;
// 94 and 122 us with 8 and 12 registers spilled, whose stores went to HBM).  Of
// the 88 us, the loads, E's staging and the stores alone take about 52, near what
// their 230 MB need, and the products do not hide behind them.  Several heads one
// after the other in a workgroup, the next one's loads ahead, leave one workgroup
// to a CU and take longer (24 ragged prompts: 160 us against 95).
constexpr int kScanThreads = 512;
template <int IO, int N>
__global__ void __launch_bounds__(kScanThreads, 4) prompt_scan_kernel(SsdPromptParams p) {
  constexpr bool kTwo = IO == SS_F16;  // x and C need a lo part
  constexpr int kHS = N + 8;           // row stride of E in LDS: 16 rows' fragments in different banks
  __shared__ __attribute__((aligned(16))) float sCs[kQ];   // log2 of the decay from the piece's first step,
  __shared__ float sRow[kQ];                               // 2^lo, lo what that float leaves of it (step_log2),
  __shared__ __attribute__((aligned(16))) float sOwn[kQ];  // and 2^-lo_j Delta_j
  __shared__ __attribute__((aligned(16))) float sWp[kQ];   // exp(piece's end - cs_j) Delta_j
  __shared__ float sTot[4];
  __shared__ __attribute__((aligned(16))) uint16_t sX0[kQ * kP];
  __shared__ __attribute__((aligned(16))) uint16_t sU[kTwo && 2 * kP * kHS < kQ * kP ? kQ * kP : 2 * kP * kHS];
  uint16_t* const sX[2] = {sX0, sU};
  uint16_t* const sE[2] = {sU, sU + kP * kHS};
  const int tid = threadIdx.x, lane = tid % 64, wave = tid / 64;
  const int lb = (int)xcd_logical_block();  // the heads of one chunk share its C and CB in an XCD's L2
  const int h = lb % p.nheads, place = lb / p.nheads;
  const SeqChunk q = find_chunk<kLogQ>(p.cu, p.nseqs, p.tokens, place);
  if (q.chunk < 0 || q.chunk * kQ >= q.len) return;
  const int left = q.len - q.chunk * kQ, rows = left < kQ ? left : kQ;
  const int64_t row0 = q.begin + (int64_t)q.chunk * kQ;
  const int g = h / (p.nheads / p.ngroups);
  const int64_t xrow = p.x_stride * 2, crow = p.c_stride * 2;
  const int half = wave / 4;
  const int blk[2] = {wave % 4, 7 - wave % 4};
  const int ir[2] = {32 * blk[0] + 16 * half, 32 * blk[1] + 16 * half};  // first row of each block

  // ---- prologue: every operand's load, then the sums, then LDS
  const auto dv = rows_view(static_cast<const char*>(p.dt) + (row0 * p.dt_stride + h) * 2, p.dt_stride * 2, rows, 2);
  const raw_t<IO> dr = bload<IO>(dv, tid < kQ ? (uint32_t)(tid * p.dt_stride * 2) : kOffNone);
  const auto xv = rows_view(static_cast<const char*>(p.x) + row0 * xrow + h * kP * 2, xrow, rows, kP * 2);
  u32x4v xr[4];
#pragma unroll
  for (int k = 0; k < 4; ++k) xr[k] = vload16(xv, (uint32_t)((tid / 8 + 64 * k) * xrow + (tid % 8) * 16));
  const f32x4* E = reinterpret_cast<const f32x4*>(p.ws_state + ((int64_t)place * p.nheads + h) * (kP * N));
  f32x4 er[N / 32];
#pragma unroll
  for (int k = 0; k < N / 32; ++k) er[k] = E[tid + kScanThreads * k];
  const auto cv = rows_view(static_cast<const char*>(p.Cm) + row0 * crow + g * N * 2, crow, rows, N * 2);
  u32x4v cf[2][N / 32];
#pragma unroll
  for (int b = 0; b < 2; ++b)
#pragma unroll
    for (int ks = 0; ks < N / 32; ++ks)
      cf[b][ks] = vload16(cv, (uint32_t)((ir[b] + lane % 16) * crow + (32 * ks + 8 * (lane / 16)) * 2));
  if (tid < kQ) {
    const float delta = tid < rows ? step_size<IO>(p, bits_f32<IO>(dr), h) : 0.0f;
    const double sum = scan_up(step_log2(delta, p.A[h]));
    const float hi = (float)sum, lo = (float)(sum - (double)hi);
    sCs[tid] = hi;
    sRow[tid] = exp2_hw(lo);
    sOwn[tid] = exp2_hw(-lo) * delta;
    sWp[tid] = exp2_hw((float)(__shfl(sum, 63, 64) - sum)) * delta;
    if (lane == 63) sTot[wave] = hi;
  }
#pragma unroll
  for (int k = 0; k < 4; ++k) {
    const int at = tm_off<kP>(tid / 8 + 64 * k, 8 * (tid % 8));
    if constexpr (kTwo) {
      u32x4v hi, lo;
      split8<IO>(xr[k], hi, lo);
      *reinterpret_cast<u32x4v*>(&sX[0][at]) = hi;
      xr[k] = lo;
    } else {
      *reinterpret_cast<u32x4v*>(&sX[0][at]) = xr[k];
    }
  }
#pragma unroll
  for (int k = 0; k < N / 32; ++k) {
    const int item = 4 * (tid + kScanThreads * k);  // E[item / N][item % N ..]
    const int at = (item / N) * kHS + item % N;
    uint32_t a0, a1, b0, b1;
    split2(er[k][0], er[k][1], a0, b0);
    split2(er[k][2], er[k][3], a1, b1);
    *reinterpret_cast<uint2*>(&sE[0][at]) = make_uint2(a0, a1);
    *reinterpret_cast<uint2*>(&sE[1][at]) = make_uint2(b0, b1);
  }
  __syncthreads();
  // sums over the whole pieces before each piece
  float before[4];
  before[0] = 0.0f;
#pragma unroll
  for (int k = 1; k < 4; ++k) before[k] = before[k - 1] + sTot[k - 1];

  // ---- Y_off = E C^T, scaled by exp(cs_i)
  f32x4 acc[2][4];  // [block][p tile]: p = 16 pt + 4 (lane / 16) + r, i = ir + lane % 16
#pragma unroll
  for (int b = 0; b < 2; ++b)
#pragma unroll
    for (int pt = 0; pt < 4; ++pt) acc[b][pt] = f32x4{0.0f, 0.0f, 0.0f, 0.0f};
#pragma unroll
  for (int ks = 0; ks < N / 32; ++ks) {
    u32x4v ch[2], cl[2];
#pragma unroll
    for (int b = 0; b < 2; ++b) {
      if constexpr (kTwo) split8<IO>(cf[b][ks], ch[b], cl[b]);
      else ch[b] = cf[b][ks];
    }
#pragma unroll
    for (int pt = 0; pt < 4; ++pt) {
      const int at = (16 * pt + lane % 16) * kHS + 32 * ks + 8 * (lane / 16);
      const bf16x8 eh = bfv(*reinterpret_cast<const u32x4v*>(&sE[0][at]));
      const bf16x8 el = bfv(*reinterpret_cast<const u32x4v*>(&sE[1][at]));
#pragma unroll
      for (int b = 0; b < 2; ++b) acc[b][pt] = BF::run(el, bfv(ch[b]), acc[b][pt]);
      if constexpr (kTwo) {
#pragma unroll
        for (int b = 0; b < 2; ++b) acc[b][pt] = BF::run(eh, bfv(cl[b]), acc[b][pt]);
      }
#pragma unroll
      for (int b = 0; b < 2; ++b) acc[b][pt] = BF::run(eh, bfv(ch[b]), acc[b][pt]);
    }
  }
#pragma unroll
  for (int b = 0; b < 2; ++b) {
    const float bf = blk[b] / 2 == 0 ? before[0] : blk[b] / 2 == 1 ? before[1] : blk[b] / 2 == 2 ? before[2] : before[3];
    const float sc = exp2_hw(sCs[ir[b] + lane % 16] + bf);
#pragma unroll
    for (int pt = 0; pt < 4; ++pt) acc[b][pt] *= sc;
  }

  if constexpr (kTwo) {
    __syncthreads();  // E is used up
#pragma unroll
    for (int k = 0; k < 4; ++k)
      *reinterpret_cast<u32x4v*>(&sX[1][tm_off<kP>(tid / 8 + 64 * k, 8 * (tid % 8))]) = xr[k];
    __syncthreads();
  }

  // ---- Y_diag += x^T M^T, piece by piece
  const auto cbv = make_rsrc(p.ws_cb + ((int64_t)place * p.ngroups + g) * (kQ * kQ), kQ * kQ * 4);
  const auto yv = rows_view(static_cast<char*>(p.y) + (row0 * p.nheads + h) * (kP * 2), (int64_t)p.nheads * (kP * 2), rows,
                            kP * 2);
  const auto zv = rows_view(p.z ? static_cast<const char*>(p.z) + row0 * p.z_stride * 2 + h * kP * 2 : nullptr,
                            p.z_stride * 2, rows, kP * 2);
  const float Dh = p.D ? p.D[h] : 0.0f;
#pragma unroll
  for (int b = 0; b < 2; ++b) {
    if (ir[b] >= rows) continue;
    const int i = ir[b] + lane % 16;  // this lane's row
    const int dpiece = blk[b] / 2;    // the piece that holds it
    const float csi = sCs[i];
    const uint32_t cb = (uint32_t)(cb_at(ir[b] / 16, 0) + lane * 8) * 4u;
    uint2 zr[4];
    f32x4 cur[2][2], nxt[2][2];
#pragma unroll
    for (int ks = 0; ks < 2; ++ks)
#pragma unroll
      for (int e = 0; e < 2; ++e) cur[ks][e] = __builtin_bit_cast(f32x4, vload16(cbv, cb + ks * 2048 + 16 * e));
    for (int piece = 0; piece <= dpiece; ++piece) {
      const int jb = kJB * piece;
      if (piece < dpiece) {
#pragma unroll
        for (int ks = 0; ks < 2; ++ks)
#pragma unroll
          for (int e = 0; e < 2; ++e)
            nxt[ks][e] = __builtin_bit_cast(f32x4, vload16(cbv, cb + (2 * piece + 2 + ks) * 2048 + 16 * e));
      } else {  // the last piece: the gate instead
#pragma unroll
        for (int pt = 0; pt < 4; ++pt)
          zr[pt] = vload8(zv, (uint32_t)(i * p.z_stride * 2 + (16 * pt + 4 * (lane / 16)) * 2));
      }
      const bool diag = piece == dpiece;
      float between = csi;  // log2 of the decay from the end of this piece to row i
      for (int k = piece + 1; k < dpiece; ++k) between += sTot[k];
      const float ei = exp2_hw(between);
#pragma unroll
      for (int ks = 0; ks < 2; ++ks) {
        if (ks == 1 && diag && blk[b] % 2 == 0) continue;  // columns behind all of the block's rows
        const int j0 = jb + 32 * ks + 8 * (lane / 16);
        float m[8];
        if (diag) {
          const f32x4 c0 = *reinterpret_cast<const f32x4*>(&sCs[j0]), c1 = *reinterpret_cast<const f32x4*>(&sCs[j0 + 4]);
          const f32x4 d0 = *reinterpret_cast<const f32x4*>(&sOwn[j0]), d1 = *reinterpret_cast<const f32x4*>(&sOwn[j0 + 4]);
#pragma unroll
          for (int e = 0; e < 8; ++e) {
            const float csj = e < 4 ? c0[e & 3] : c1[e & 3], dj = e < 4 ? d0[e & 3] : d1[e & 3];
            const float v = cur[ks][e / 4][e & 3] * exp2_hw(csi - csj) * dj;
            m[e] = j0 + e <= i ? v : 0.0f;
          }
        } else {
          const f32x4 w0 = *reinterpret_cast<const f32x4*>(&sWp[j0]), w1 = *reinterpret_cast<const f32x4*>(&sWp[j0 + 4]);
#pragma unroll
          for (int e = 0; e < 8; ++e) m[e] = cur[ks][e / 4][e & 3] * ((e < 4 ? w0[e & 3] : w1[e & 3]) * ei);
        }
        u32x4v mh, ml;
#pragma unroll
        for (int e = 0; e < 4; ++e) {
          uint32_t a, c;
          split2(m[2 * e], m[2 * e + 1], a, c);
          mh[e] = a;
          ml[e] = c;
        }
        bf16x8 xa[kTwo ? 2 : 1][4];  // A[m = p][k = step] = x^T, from the time-major tile
#pragma unroll
        for (int i = 0; i < (kTwo ? 2 : 1); ++i)
#pragma unroll
          for (int pt = 0; pt < 4; ++pt)
            xa[i][pt] = bfv(tm_frag(&sX[i][(jb + 32 * ks) * kP], tm_lane_off<kP>(16 * pt, 0, lane),
                                    tm_lane_off<kP>(16 * pt, 1, lane)));
#pragma unroll
        for (int pt = 0; pt < 4; ++pt) acc[b][pt] = BF::run(xa[0][pt], bfv(ml), acc[b][pt]);
        if constexpr (kTwo) {
#pragma unroll
          for (int pt = 0; pt < 4; ++pt) acc[b][pt] = BF::run(xa[kTwo ? 1 : 0][pt], bfv(mh), acc[b][pt]);
        }
#pragma unroll
        for (int pt = 0; pt < 4; ++pt) acc[b][pt] = BF::run(xa[0][pt], bfv(mh), acc[b][pt]);
      }
#pragma unroll
      for (int ks = 0; ks < 2; ++ks)
#pragma unroll
        for (int e = 0; e < 2; ++e) cur[ks][e] = nxt[ks][e];
    }
    // ---- D skip, gate, store (rows past the chunk are dropped by the range check)
    {
      const float row = sRow[i];
#pragma unroll
      for (int pt = 0; pt < 4; ++pt) {
        const int p0 = 16 * pt + 4 * (lane / 16);
        const uint2 xw = *reinterpret_cast<const uint2*>(&sX[0][tm_off<kP>(i, p0)]);
        float x[4] = {__uint_as_float(xw.x << 16), __uint_as_float(xw.x & 0xffff0000u), __uint_as_float(xw.y << 16),
                      __uint_as_float(xw.y & 0xffff0000u)};
        if constexpr (kTwo) {
          const uint2 lw = *reinterpret_cast<const uint2*>(&sX[kTwo ? 1 : 0][tm_off<kP>(i, p0)]);
          x[0] += __uint_as_float(lw.x << 16);
          x[1] += __uint_as_float(lw.x & 0xffff0000u);
          x[2] += __uint_as_float(lw.y << 16);
          x[3] += __uint_as_float(lw.y & 0xffff0000u);
        }
        float o[4];
#pragma unroll
        for (int r = 0; r < 4; ++r) o[r] = fmaf(Dh, x[r], row * acc[b][pt][r]);
        if (p.z) {
          o[0] *= silu_f(low16<IO>(zr[pt].x));
          o[1] *= silu_f(high16<IO>(zr[pt].x));
          o[2] *= silu_f(low16<IO>(zr[pt].y));
          o[3] *= silu_f(high16<IO>(zr[pt].y));
        }
        vstore8(yv, (uint32_t)(i * p.nheads * (kP * 2) + p0 * 2), pack2<IO>(o[0], o[1]), pack2<IO>(o[2], o[3]));
      }
    }
  }
}

template <int IO, int N, int HB>
void launch_state(const SsdPromptParams& p, hipStream_t st) {
  const uint32_t parts = (uint32_t)((p.nheads / p.ngroups + HB - 1) / HB);
  hipLaunchKernelGGL((prompt_state_kernel<IO, N, HB>), dim3((uint32_t)p.chunks * (uint32_t)p.ngroups * (parts + 2)),
                     dim3(kStateThreads), 0, st, p);
}
template <int IO, int N>
hipError_t launch_prompt_n(const SsdPromptParams& p, hipStream_t st) {
  const uint32_t chunks = (uint32_t)p.chunks, heads = (uint32_t)p.nheads;
  switch (state_heads((int64_t)p.chunks * p.ngroups, p.nheads / p.ngroups, device_cus())) {
    case 1: launch_state<IO, N, 1>(p, st); break;
    case 2: launch_state<IO, N, 2>(p, st); break;
    default: launch_state<IO, N, 3>(p, st); break;
  }
  hipError_t e = hipGetLastError();
  if (e != hipSuccess) return e;
  // no prompt has two chunks where all rows fit one: five prompts of 131 tokens take
  // 15.6 us without the launch, 17.9 us with it
  const uint32_t pass = p.tokens <= kQ ? 0 : (uint32_t)p.nseqs * heads * (kP * N / 1024);
  if (pass == 0) {
  } else if (pass_ahead(pass, p.chunks, p.nseqs, device_cus()) == 16)
    hipLaunchKernelGGL((prompt_pass_kernel<N, 16>), dim3(pass), dim3(256), 0, st, p);
  else
    hipLaunchKernelGGL((prompt_pass_kernel<N, 4>), dim3(pass), dim3(256), 0, st, p);
  e = hipGetLastError();
  if (e != hipSuccess) return e;
  hipLaunchKernelGGL((prompt_scan_kernel<IO, N>), dim3(chunks * heads), dim3(kScanThreads), 0, st, p);
  return hipGetLastError();
}
template <int IO>
hipError_t launch_prompt_io(const SsdPromptParams& p, hipStream_t st) {
  switch (p.dstate) {
    case 32: return launch_prompt_n<IO, 32>(p, st);
    case 64: return launch_prompt_n<IO, 64>(p, st);
    case 96: return launch_prompt_n<IO, 96>(p, st);
    default: return launch_prompt_n<IO, 128>(p, st);
  }
}

}  // namespace

hipError_t launch_ssd_prompt(const SsdPromptParams& p, hipStream_t st) {
  return p.io == SS_F16 ? launch_prompt_io<SS_F16>(p, st) : launch_prompt_io<SS_BF16>(p, st);
}

}  // namespace ss
