// ss_ssd_bwd.hip -- gradients of the Mamba-2 SSD scan on MFMA (gfx950).
//
// Of the scan of ss_ssd.hip (page "Mamba" (walkthrough), "Deep dive: Mamba-2
// and state-space duality"), per head, a_t = exp(Delta_t A), state H[p][n]:
//   H_t = a_t H_{t-1} + Delta_t x_t B_t^T,  y_t = (H_t C_t + D x_t) silu(z_t).
// With g = dy silu(z) and G_t the gradient of H_t,
//   G_t = g_t C_t^T + a_{t+1} G_{t+1} (the final state's gradient behind the end),
//   dC_t = H_t^T g_t,  dB_t = Delta_t G_t^T x_t,  dx_t = Delta_t G_t B_t + D g_t,
//   da_t = a_t <G_t, H_{t-1}>  (the gradient of Delta_t A),
//   dDelta_t = x_t . G_t B_t + A da_t,  dh0 = a_0 G_0.
// Computed in chunks of Q = 256 steps, cs the running sum of Delta A in a
// chunk, E the state that enters it and R the gradient of the state that
// leaves it:
//   E' = exp(cs_last) E + sum_j exp(cs_last - cs_j) Delta_j x_j B_j^T
//   R' = exp(cs_last) R + sum_i exp(cs_i) g_i C_i^T   (R' leaves the chunk before)
//   G_j B_j = sum_{i>=j} exp(cs_i - cs_j) (C_i . B_j) g_i + exp(cs_last - cs_j) R B_j
//   S_ij = exp(cs_i - cs_j) Delta_j (g_i . x_j),  j <= i, summed over a group's heads:
//   dC_i = sum_j S_ij B_j + sum_h exp(cs_i) E^T g_i
//   dB_j = sum_i S_ij C_i + sum_h Delta_j exp(cs_last - cs_j) R^T x_j
// and for the decays, with W_ij = (C_i . B_j) S_ij, e_i = exp(cs_i) C_i . E^T g_i and
// r_j = Delta_j exp(cs_last - cs_j) B_j . R^T x_j,
//   da_t = sum_{j < t <= i} W_ij + sum_{i>=t} e_i + sum_{j<t} r_j + exp(cs_last) <R, E>.
// The pairs around a step t of a piece k of 64 steps are summed as
//   i and j in k:         sum_{i>=t} sum_{j<t} W_ij, rows' sums first,
//   i in k, j before k:   sum_{i>=t} sum_j W_ij;  j in k, i behind: sum_{j<t} sum_i W_ij,
//   i behind k, j before: one number for the piece,
// so that no terms cancel (sum_{i>=t} (row_i - col_i), shorter, loses what its
// errors add up to over the steps: 1e-5 of dA over 600 steps, 1e-7 this way).
// Kernels:
//   bwd_planes   (fp16 or gated) the operands' planes of bf16 parts, g among them
//   bwd_state    per (chunk, one to three heads of a group, E or R): what a chunk adds
//                to E and to R; further workgroups: B C^T (and C B^T if gated) per (chunk, group)
//   bwd_pass_pair, two kinds of workgroups:
//     pass       per (row, head, 1024 elements): E of every chunk, then R and
//                <R, E> backwards, dh0
//     pair       per (chunk, group, pair of pieces of 64): all heads of the group, S
//                and the sums of W
//   bwd_scan     per (chunk, head): G_j B_j, dx; if gated, others rebuild y for dz
//   bwd_out      per (chunk, group, dC or dB, half the rows, half the states): dC or
//                dB, e or r
//   bwd_delta    per (chunk, head): da, ddt, and the chunk's part of dA, ddt_bias, dD
//   bwd_sum      per head: dA, ddt_bias, dD
// At the bench layer (B = 8, L = 2048, 24 heads, state 128, bf16) state, pass_pair,
// scan, out, delta and sum take 68, 75, 56, 67, 11 and 5 us, of which the bytes they
// move need 48, 80, 35, 53, 6 and 0 at 4.9 TB/s (E, R and S are read back partly
// from the last level cache); at two workgroups or less to a CU, their loads,
// products and LDS phases hide each other only in part.
// No atomics: every sum has a fixed order.  Computed operands are multiplied
// as sums of bf16 parts (ss_mfma.h), three where the result stays in fp32 (E,
// R, t and S's products, which dA, ddt_bias, dD and dh0 sum up), two where it
// is rounded to 16 bits (dx, dz, dB, dC); states and sums are fp32.
#include "ss_device.h"
#include "ss_internal.h"
#include "ss_mfma.h"
#include "ss_state.h"

namespace ss {
namespace {

constexpr int kQ = 256;  // chunk length
constexpr int kP = 64;   // headdim
constexpr int kJB = 64;  // time piece of a chunk

// MODE: 0 bf16, 1 bf16 with a gate, 2 fp16, 3 fp16 with a gate
template <int MODE> constexpr int io_of() { return MODE >= 2 ? SS_F16 : SS_BF16; }
template <int MODE> constexpr int data_parts() { return MODE >= 2 ? 2 : 1; }               // of x, B, C
template <int MODE> constexpr int g_parts() { return MODE % 2 ? 3 : data_parts<MODE>(); }  // of g

struct Chunk {
  int place, rows;
  int64_t row0;  // first row, counted over the batch
};
__device__ __forceinline__ Chunk chunk_of(const SsdBwdParams& p, int place) {
  Chunk q;
  q.place = place;
  const int b = place / p.nchunks, c = place - b * p.nchunks;
  const int64_t left = p.seqlen - (int64_t)c * kQ;
  q.rows = left < kQ ? (int)left : kQ;
  q.row0 = b * p.seqlen + (int64_t)c * kQ;
  return q;
}
// a view of `cols` columns of a plane, from a chunk's first row on
__device__ __forceinline__ __amdgpu_buffer_rsrc_t plane_view(const uint16_t* at, int64_t row0, int64_t row, int col,
                                                             int cols, int rows) {
  return rows_view(at ? at + row0 * row + col : nullptr, row * 2, rows, cols * 2);
}
__device__ __forceinline__ float lo_f(uint32_t w) { return __uint_as_float(w << 16); }
__device__ __forceinline__ float hi_f(uint32_t w) { return __uint_as_float(w & 0xffff0000u); }
// four values from their parts' words
template <int NP>
__device__ __forceinline__ void join4(const uint2 (&w)[NP], float (&v)[4]) {
#pragma unroll
  for (int i = NP - 1; i >= 0; --i) {
    const float a[4] = {lo_f(w[i].x), hi_f(w[i].x), lo_f(w[i].y), hi_f(w[i].y)};
#pragma unroll
    for (int e = 0; e < 4; ++e) v[e] = i == NP - 1 ? a[e] : v[e] + a[e];
  }
}

// ---- the operands' planes ---------------------------------------------------------
struct PlaneJob {
  const void* src;
  const void* gate;  // null, or multiply by silu(gate)
  uint16_t* part[3];
  int parts;
  int64_t n;         // multiple of 8
  int64_t blocks;
};
struct PlaneJobs { PlaneJob j[4]; int n; };
constexpr int64_t kPlaneBlocks = 16384;  // workgroups of one plane
template <int IO>
__global__ void __launch_bounds__(256) bwd_planes_kernel(PlaneJobs a) {
  int64_t blk = blockIdx.x;
  int k = 0;
  while (k + 1 < a.n && blk >= a.j[k].blocks) blk -= a.j[k++].blocks;
  const PlaneJob q = a.j[k];
  for (int64_t i = (blk * 256 + threadIdx.x) * 8; i < q.n; i += q.blocks * 2048) {
    const u32x4v w = *reinterpret_cast<const u32x4v*>(static_cast<const uint16_t*>(q.src) + i);
    u32x4v z = u32x4v{0u, 0u, 0u, 0u};
    if (q.gate) z = *reinterpret_cast<const u32x4v*>(static_cast<const uint16_t*>(q.gate) + i);
    u32x4v part[3];
#pragma unroll
    for (int e = 0; e < 4; ++e) {
      float v0 = low16<IO>(w[e]), v1 = high16<IO>(w[e]);
      if (q.gate) {
        v0 *= silu_f(low16<IO>(z[e]));
        v1 *= silu_f(high16<IO>(z[e]));
      }
      uint32_t v[3];
      split3(v0, v1, v);
#pragma unroll
      for (int m = 0; m < 3; ++m) part[m][e] = v[m];
    }
#pragma unroll
    for (int m = 0; m < 3; ++m)
      if (m < q.parts) *reinterpret_cast<u32x4v*>(q.part[m] + i) = part[m];
  }
}

// ---- what a chunk adds to E and to R ------------------------------------------------
// Workgroup = (chunk, HB heads of a group, E or R), the sums of ss_state.h:
// E: u = x, V = B, w_j = exp(sum of Delta A behind j) Delta_j, from the last
// document start on; R: u = g, V = C, w_i = exp(cs_i), before the first start.
template <int MODE, int N, int HB, bool R>
using StateOf = StateLds<N, HB, R ? g_parts<MODE>() : data_parts<MODE>(), data_parts<MODE>(), false>;

template <int MODE, int N, int HB, bool R>
__device__ __forceinline__ void state_role(const SsdBwdParams& p, int place, int g, int h0, int heads,
                                           StateOf<MODE, N, HB, R>& lds) {
  constexpr int UP = R ? g_parts<MODE>() : data_parts<MODE>(), VP = data_parts<MODE>();
  constexpr int IO = io_of<MODE>();
  const int tid = threadIdx.x, lane = tid % 64, team = tid / 256, t = tid % 256, wave = t / 64;
  const Chunk q = chunk_of(p, place);
  // documents: starts at or before each step of the chunk
  int seg = 0, starts = 0, first = kQ;
  if (p.seq_idx) {
    const int64_t at = q.row0 + t;
    const bool st = t < q.rows && at % p.seqlen != 0 && p.seq_idx[at] != p.seq_idx[at - 1];
    const uint64_t m = __builtin_amdgcn_ballot_w64(st);
    if (lane == 0 && team == 0) {
      lds.count[wave] = (int)__builtin_popcountll(m);
      lds.first[wave] = m ? 64 * wave + (int)__builtin_ctzll(m) : kQ;
    }
    seg = (int)__builtin_popcountll(m & (lane == 63 ? ~0ull : (2ull << lane) - 1));
    __syncthreads();
    for (int w = 0; w < wave; ++w) seg += lds.count[w];
    starts = lds.count[0] + lds.count[1] + lds.count[2] + lds.count[3];
    first = min(min(lds.first[0], lds.first[1]), min(lds.first[2], lds.first[3]));
    if (!R && h0 == 0 && team == 0) p.ws_seg[(int64_t)place * kQ + t] = seg;
  }
#pragma unroll
  for (int hb = 0; hb < HB; hb += 2) {  // two heads at a time, 256 threads each
    const int h = h0 + hb + team;
    const bool mine = hb + team < heads, in = mine && t < q.rows;
    float delta = 0.0f;
    if (in) {
      const float xd = load_io<IO>(p.dt, (q.row0 + t) * p.nheads + h) + (p.dt_bias ? p.dt_bias[h] : 0.0f);
      delta = p.softplus ? softplus_f(xd) : xd;
    }
    const float A = mine ? p.A[h] : 0.0f;
    // R: the sum up to this step in the wave's 64, a power of two in two floats
    // (step_log2); E: of Delta A from this step on.
    float v = delta * A, low = 0.0f;
    if constexpr (R) {
      const double c = scan_up(step_log2(delta, A));
      v = (float)c;
      low = (float)(c - (double)v);
    } else {
#pragma unroll
      for (int off = 1; off < 64; off <<= 1) {
        const float o = __shfl_down(v, off, 64);
        if (lane + off < 64) v += o;
      }
    }
    float* sum = lds.wave[team];
    if (lane == (R ? 63 : 0)) sum[wave] = v;
    __syncthreads();
    const int64_t at = ((int64_t)place * p.nheads + h) * kQ + t;
    float w = 0.0f;
    if (mine) {
      if constexpr (R) {
        const float behind = (__shfl(v, 63, 64) - v) + (__shfl(low, 63, 64) - low);
        p.ws_cs[at] = v;
        p.ws_cl[at] = low;
        p.ws_from[at] = exp2_hw(v);
        p.ws_to[at] = exp2_hw(behind);
        for (int k = 0; k < wave; ++k) v += sum[k];
        w = t < first ? exp2_hw(v) : 0.0f;
        p.ws_wc[at] = w;
      } else {
        p.ws_delta[at] = delta;
        float behind = __shfl_down(v, 1, 64);
        if (lane == 63) behind = 0.0f;
        for (int k = 3; k > wave; --k) behind += sum[k];
        w = seg == starts ? exp2_hw(behind * kLog2e) : 0.0f;
        p.ws_wb[at] = w;
        w *= delta;
        if (t == 0)
          p.ws_decay[(int64_t)place * p.nheads + h] =
              starts ? 0.0f : exp2_hw((sum[0] + sum[1] + sum[2] + sum[3]) * kLog2e);
      }
    }
    if (hb + team < HB) lds.w[hb + team][t] = in ? w : 0.0f;
    if (hb + 2 < HB) __syncthreads();
  }
  const int64_t urow = (int64_t)p.nheads * kP, vrow = (int64_t)p.ngroups * N;
  __amdgpu_buffer_rsrc_t uv[UP], vv[VP];
#pragma unroll
  for (int i = 0; i < UP; ++i) uv[i] = plane_view(R ? p.gp[i] : p.xp[i % 2], q.row0, urow, h0 * kP, heads * kP, q.rows);
#pragma unroll
  for (int i = 0; i < VP; ++i) vv[i] = plane_view(R ? p.cp[i] : p.bp[i], q.row0, vrow, g * N, N, q.rows);
  float* const base = R ? p.ws_R : p.ws_E;
  const int nheads = p.nheads;
  chunk_states<IO, N, HB, UP, VP, false>(
      lds, uv, urow, vv, vrow, q.rows, heads, [=](int hb, int at, const f32x4 (&v)[N / 32]) {
        float* out = base + ((int64_t)place * nheads + h0 + hb) * (kP * N) + at;
#pragma unroll
        for (int t = 0; t < N / 32; ++t) *reinterpret_cast<f32x4*>(out + 16 * t) = v[t];
      });
}

// C B^T (REV false: rows i of C, columns j of B up to the row's piece) or B C^T
// (REV true: rows j of B, columns i of C from the row's piece to the last) of a
// chunk in operand order, fp32; rows past the chunk come out as zeros.
template <int MODE, int N, bool REV>
__device__ __forceinline__ void cb_role(const SsdBwdParams& p, int place, int g, int half) {
  constexpr int IO = io_of<MODE>();
  const int lane = threadIdx.x % 64, wave = threadIdx.x / 64;
  const Chunk q = chunk_of(p, place);
  const int it = 8 * half + wave, piece = it / 4;
  if (16 * it >= q.rows) return;
  const int64_t row = (int64_t)p.ngroups * N;
  const auto bv = plane_view(static_cast<const uint16_t*>(REV ? p.Cm : p.Bm), q.row0, row, g * N, N, q.rows);
  const auto cv = plane_view(static_cast<const uint16_t*>(REV ? p.Bm : p.Cm), q.row0, row, g * N, N, q.rows);
  u32x4v c[N / 32];
#pragma unroll
  for (int ks = 0; ks < N / 32; ++ks)
    c[ks] = vload16(cv, (uint32_t)((16 * it + lane % 16) * row * 2 + (32 * ks + 8 * (lane / 16)) * 2));
  float* CB = (REV ? p.ws_bc : p.ws_cb) + ((int64_t)place * p.ngroups + g) * (kQ * kQ);
  const int j1 = REV ? 4 * ((q.rows + kJB - 1) / kJB) : 4 * piece + 4;
  u32x4v b[N / 32];
  auto load_b = [&](int jt) {
#pragma unroll
    for (int ks = 0; ks < N / 32; ++ks)
      b[ks] = vload16(bv, (uint32_t)((16 * jt + lane % 16) * row * 2 + (32 * ks + 8 * (lane / 16)) * 2));
  };
  load_b(REV ? 4 * piece : 0);
  for (int jt = REV ? 4 * piece : 0; jt < j1; ++jt) {
    f32x4 acc = f32x4{0.0f, 0.0f, 0.0f, 0.0f};
#pragma unroll
    for (int ks = 0; ks < N / 32; ++ks) acc = mfma_t<IO>::run(as_vec<IO>(b[ks]), as_vec<IO>(c[ks]), acc);
    if (jt + 1 < j1) load_b(jt + 1);
    const int to = lane % 16 + 16 * (2 * (jt & 1) + lane / 32);
    *reinterpret_cast<f32x4*>(CB + cb_at(it, jt / 2) + to * 8 + 4 * ((lane / 16) & 1)) = acc;
  }
}

template <int MODE, int N, int HB>
__global__ void __launch_bounds__(kStateThreads, MODE == 0 ? 4 : 2) bwd_state_kernel(SsdBwdParams p) {
  __shared__ union {
    StateOf<MODE, N, HB, false> e;
    StateOf<MODE, N, HB, true> r;
  } lds;
  // a (chunk, group) has 2 workgroups for B C^T and, if gated, 2 for C B^T, which
  // take longest, then 2 * parts for the states, all on one XCD
  constexpr int kCb = MODE % 2 ? 4 : 2;
  const int hpg = p.nheads / p.ngroups, parts = (hpg + HB - 1) / HB, per = kCb + 2 * parts;
  const int lb = (int)xcd_logical_block(), r = lb % per, g = (lb / per) % p.ngroups, place = lb / per / p.ngroups;
  if (r < 2) {
    cb_role<MODE, N, true>(p, place, g, r);
  } else if (r < kCb) {
    cb_role<MODE, N, false>(p, place, g, 1 - r % 2);
  } else {
    const int h = (r - kCb) / 2 * HB, left = hpg - h, heads = left < HB ? left : HB;
    if (r & 1) state_role<MODE, N, HB, true>(p, place, g, g * hpg + h, heads, lds.r);
    else state_role<MODE, N, HB, false>(p, place, g, g * hpg + h, heads, lds.e);
  }
}

// ---- E forwards, R backwards ----------------------------------------------------------
// Workgroup = (batch row, head, 1024 elements), a thread 4 elements.  <R, E> of a
// chunk: each wave leaves the sum of its 256 elements.
template <int N>
__device__ __forceinline__ void pass_role(const SsdBwdParams& p, uint32_t block) {
  constexpr int kParts = kP * N / 1024, kAhead = 4;
  const int part = (int)(block % kParts);
  const int h = (int)((block / kParts) % (uint32_t)p.nheads);
  const int64_t b = block / kParts / (uint32_t)p.nheads;
  const int e = part * 1024 + 4 * (int)threadIdx.x, n = p.nchunks;
  const int64_t first = b * n * p.nheads + h, step = (int64_t)p.nheads * (kP * N);
  const float* dec = p.ws_decay + first;
  const int64_t row = (b * p.nheads + h) * (kP * N) + e;
  float* wE = p.ws_E + first * (kP * N) + e;
  float* wR = p.ws_R + first * (kP * N) + e;
  f32x4 S[kAhead], F[kAhead];
  float d[kAhead];
  {
    f32x4 E = f32x4{0.0f, 0.0f, 0.0f, 0.0f};
    if (p.h0) E = *reinterpret_cast<const f32x4*>(p.h0 + row);
#pragma unroll
    for (int k = 0; k < kAhead; ++k)
      if (k < n) {
        S[k] = *reinterpret_cast<const f32x4*>(wE + k * step);
        d[k] = dec[(int64_t)k * p.nheads];
      }
    for (int c = 0; c < n; c += kAhead) {
#pragma unroll
      for (int k = 0; k < kAhead; ++k)
        if (c + k < n) {
          const f32x4 own = S[k];
          const float decay = d[k];
          if (c + k + kAhead < n) {
            S[k] = *reinterpret_cast<const f32x4*>(wE + (c + k + kAhead) * step);
            d[k] = dec[(int64_t)(c + k + kAhead) * p.nheads];
          }
          *reinterpret_cast<f32x4*>(wE + (c + k) * step) = E;
#pragma unroll
          for (int i = 0; i < 4; ++i) E[i] = fmaf(decay, E[i], own[i]);
        }
    }
  }
  f32x4 Rg = f32x4{0.0f, 0.0f, 0.0f, 0.0f};
  if (p.dfinal) Rg = *reinterpret_cast<const f32x4*>(p.dfinal + row);
#pragma unroll
  for (int k = 0; k < kAhead; ++k)
    if (k < n) {
      S[k] = *reinterpret_cast<const f32x4*>(wR + (n - 1 - k) * step);
      F[k] = *reinterpret_cast<const f32x4*>(wE + (n - 1 - k) * step);  // this thread's own store
      d[k] = dec[(int64_t)(n - 1 - k) * p.nheads];
    }
  for (int c = 0; c < n; c += kAhead) {
#pragma unroll
    for (int k = 0; k < kAhead; ++k)
      if (c + k < n) {
        const int at = n - 1 - c - k, nx = at - kAhead;
        const f32x4 own = S[k], E = F[k];
        const float decay = d[k];
        if (nx >= 0) {
          S[k] = *reinterpret_cast<const f32x4*>(wR + nx * step);
          F[k] = *reinterpret_cast<const f32x4*>(wE + nx * step);
          d[k] = dec[(int64_t)nx * p.nheads];
        }
        *reinterpret_cast<f32x4*>(wR + at * step) = Rg;
        float v = Rg[0] * E[0] + Rg[1] * E[1] + (Rg[2] * E[2] + Rg[3] * E[3]);
        v = row_sum(v);
        v += __shfl_xor(v, 16, 64);
        v += __shfl_xor(v, 32, 64);
        if (threadIdx.x % 64 == 0)
          p.ws_dot[(first + (int64_t)at * p.nheads) * (4 * kParts) + 4 * part + threadIdx.x / 64] = decay * v;
#pragma unroll
        for (int i = 0; i < 4; ++i) Rg[i] = fmaf(decay, Rg[i], own[i]);
      }
  }
  if (p.dh0) *reinterpret_cast<f32x4*>(p.dh0 + row) = Rg;
}

// ---- dx (rev), or y for dz --------------------------------------------------------------
// Workgroup = (chunk, head), 512 threads, laid out as prompt_scan_kernel: out
// rows o, source rows s, out^T[p][o] = sum_s u_s[p] M[o][s] + f_o sum_n K[p][n] v_o[n].
//   rev:  s >= o, u = g, M = exp(cs_s - cs_o) (C_s . B_o),         K = R, v = B, f = exp(cs_last - cs_o)
//   else: s <= o, u = x, M = exp(cs_o - cs_s) Delta_s (C_o . B_s), K = E, v = C, f = exp(cs_o)
// A pair in different pieces of 64 takes a factor per row and one per column,
// both through the piece's end, a pair inside a piece the exp of a difference (of
// sums in two floats: step_log2).
constexpr int kScanThreads = 512;
// Where z is given, workgroups of both take turns in one launch; u's second part
// takes K's place once K is used up, so that two workgroups share a CU (gated
// fp16, B = 2, L = 1001, 8 heads, state 64: the gradients take 77 us, 86 us with
// two launches; B = 4, L = 2048, 24 heads: 296 against 298 us).
template <int MODE, int N>
__global__ void __launch_bounds__(kScanThreads, 4) bwd_scan_kernel(SsdBwdParams p) {
  constexpr int IO = io_of<MODE>();
  // two parts at the most: dx and dz are rounded to 16 bits
  constexpr int UP = g_parts<MODE>() > 1 ? 2 : 1, VP = data_parts<MODE>();
  constexpr int kHS = N + 8;
  __shared__ __attribute__((aligned(16))) float sCs[kQ];   // log2 of the decay from the piece's first step
  __shared__ __attribute__((aligned(16))) float sCol[kQ];  // a source row's factor in other pieces
  // of lo, what that float leaves of the sum (step_log2):
  __shared__ __attribute__((aligned(16))) float sOwn[kQ];  // a source row's factor in its own piece: 2^lo, or 2^-lo Delta
  __shared__ float sRow[kQ];                               // an out row's at the end: 2^-lo Delta, or 2^lo
  __shared__ __attribute__((aligned(16))) int sSeg[kQ];
  __shared__ float sTot[4], sTotLo[4];
  __shared__ __attribute__((aligned(16))) uint16_t u0[kQ * kP];
  __shared__ __attribute__((aligned(16))) uint16_t ku[UP > 1 && 2 * kP * kHS < kQ * kP ? kQ * kP : 2 * kP * kHS];
  uint16_t* const sU[2] = {u0, ku};
  uint16_t* const sK[2] = {ku, ku + kP * kHS};
  const int tid = threadIdx.x, lane = tid % 64, wave = tid / 64;
  const int all = (int)xcd_logical_block();  // the heads of one chunk share its B, C and C B^T in an XCD's L2
  const int lb = MODE % 2 ? all >> 1 : all;
  const bool rev = MODE % 2 ? all & 1 : true;
  const int h = lb % p.nheads;
  const Chunk q = chunk_of(p, lb / p.nheads);
  const int rows = q.rows, g = h / (p.nheads / p.ngroups);
  const int64_t xrow = (int64_t)p.nheads * kP, vrow = (int64_t)p.ngroups * N;
  const int64_t ph = (int64_t)q.place * p.nheads + h;
  const int half = wave / 4;
  const int blk[2] = {wave % 4, 7 - wave % 4};
  const int orow[2] = {32 * blk[0] + 16 * half, 32 * blk[1] + 16 * half};
  const int lastp = (rows - 1) / kJB;

  u32x4v ur[UP][4];
#pragma unroll
  for (int i = 0; i < UP; ++i) {
    const auto uv = plane_view(rev ? p.gp[i] : i < data_parts<MODE>() ? p.xp[i] : nullptr, q.row0, xrow, h * kP, kP, rows);
#pragma unroll
    for (int k = 0; k < 4; ++k)
      ur[i][k] = vload16(uv, (uint32_t)((tid / 8 + 64 * k) * xrow * 2 + (tid % 8) * 16));
  }
  const f32x4* K = reinterpret_cast<const f32x4*>((rev ? p.ws_R : p.ws_E) + ph * (kP * N));
  f32x4 kr[N / 32];
#pragma unroll
  for (int k = 0; k < N / 32; ++k) kr[k] = K[tid + kScanThreads * k];
  u32x4v vf[VP][2][N / 32];
#pragma unroll
  for (int i = 0; i < VP; ++i) {
    const auto vv = plane_view(rev ? p.bp[i] : p.cp[i], q.row0, vrow, g * N, N, rows);
#pragma unroll
    for (int b = 0; b < 2; ++b)
#pragma unroll
      for (int ks = 0; ks < N / 32; ++ks)
        vf[i][b][ks] = vload16(vv, (uint32_t)((orow[b] + lane % 16) * vrow * 2 + (32 * ks + 8 * (lane / 16)) * 2));
  }
  if (tid < kQ) {
    const float delta = p.ws_delta[ph * kQ + tid], cs = p.ws_cs[ph * kQ + tid], lo = p.ws_cl[ph * kQ + tid];
    const float col = (rev ? p.ws_from : p.ws_to)[ph * kQ + tid];
    const float up = exp2_hw(lo), down = exp2_hw(-lo) * delta;
    sCs[tid] = cs;
    sCol[tid] = rev ? col : col * delta;
    sOwn[tid] = rev ? up : down;
    sRow[tid] = rev ? down : up;
    if (lane == 63) {
      sTot[wave] = cs;
      sTotLo[wave] = lo;
    }
    if (p.seq_idx) sSeg[tid] = p.ws_seg[(int64_t)q.place * kQ + tid];
  }
#pragma unroll
  for (int k = 0; k < 4; ++k) {
    *reinterpret_cast<u32x4v*>(&sU[0][tm_off<kP>(tid / 8 + 64 * k, 8 * (tid % 8))]) = ur[0][k];
  }
#pragma unroll
  for (int k = 0; k < N / 32; ++k) {
    const int item = 4 * (tid + kScanThreads * k);
    const int at = (item / N) * kHS + item % N;
    uint32_t a0, a1, b0, b1;
    split2(kr[k][0], kr[k][1], a0, b0);
    split2(kr[k][2], kr[k][3], a1, b1);
    *reinterpret_cast<uint2*>(&sK[0][at]) = make_uint2(a0, a1);
    *reinterpret_cast<uint2*>(&sK[1][at]) = make_uint2(b0, b1);
  }
  __syncthreads();

  f32x4 acc[2][4];  // [block][p tile]: p = 16 pt + 4 (lane / 16) + r, o = orow + lane % 16
#pragma unroll
  for (int b = 0; b < 2; ++b)
#pragma unroll
    for (int pt = 0; pt < 4; ++pt) acc[b][pt] = f32x4{0.0f, 0.0f, 0.0f, 0.0f};
#pragma unroll
  for (int ks = 0; ks < N / 32; ++ks)
#pragma unroll
    for (int pt = 0; pt < 4; ++pt) {
      const int at = (16 * pt + lane % 16) * kHS + 32 * ks + 8 * (lane / 16);
      const bf16x8 kh = bfv(*reinterpret_cast<const u32x4v*>(&sK[0][at]));
      const bf16x8 kl = bfv(*reinterpret_cast<const u32x4v*>(&sK[1][at]));
#pragma unroll
      for (int b = 0; b < 2; ++b) acc[b][pt] = BF::run(kl, bfv(vf[0][b][ks]), acc[b][pt]);
      if constexpr (VP > 1) {
#pragma unroll
        for (int b = 0; b < 2; ++b) acc[b][pt] = BF::run(kh, bfv(vf[VP - 1][b][ks]), acc[b][pt]);
      }
#pragma unroll
      for (int b = 0; b < 2; ++b) acc[b][pt] = BF::run(kh, bfv(vf[0][b][ks]), acc[b][pt]);
    }
#pragma unroll
  for (int b = 0; b < 2; ++b) {
    const int o = orow[b] + lane % 16, piece = blk[b] / 2;
    float arg = rev ? (sTot[piece] - sCs[o]) + sTotLo[piece] : sCs[o];
    if (rev) {
      for (int k = piece + 1; k < 4; ++k) arg += sTot[k];
    } else {
      for (int k = 0; k < piece; ++k) arg += sTot[k];
    }
    float f = exp2_hw(arg);
    if (p.seq_idx && sSeg[o] != (rev ? sSeg[rows - 1] : 0)) f = 0.0f;
#pragma unroll
    for (int pt = 0; pt < 4; ++pt) acc[b][pt] *= f;
  }

  if constexpr (UP > 1) {
    __syncthreads();  // K is used up
#pragma unroll
    for (int k = 0; k < 4; ++k)
      *reinterpret_cast<u32x4v*>(&sU[1][tm_off<kP>(tid / 8 + 64 * k, 8 * (tid % 8))]) = ur[UP - 1][k];
    __syncthreads();
  }

  const float* CB = (rev ? p.ws_bc : p.ws_cb) + ((int64_t)q.place * p.ngroups + g) * (kQ * kQ);
  const float Dh = p.D ? p.D[h] : 0.0f;
#pragma unroll
  for (int b = 0; b < 2; ++b) {
    if (orow[b] >= rows) continue;
    const int o = orow[b] + lane % 16, piece = blk[b] / 2;
    const float cso = sCs[o];
    const float base = rev ? (sTot[piece] - cso) + sTotLo[piece] : cso;  // log2 of the decay from or to the piece's end
    const int sego = p.seq_idx ? sSeg[o] : 0;
    const float* cb = CB + cb_at(orow[b] / 16, 0) + lane * 8;
    const int s0 = rev ? piece : 0, s1 = rev ? lastp : piece;
    f32x4 cur[2][2], nxt[2][2];
#pragma unroll
    for (int ks = 0; ks < 2; ++ks)
#pragma unroll
      for (int e = 0; e < 2; ++e) cur[ks][e] = *reinterpret_cast<const f32x4*>(cb + (2 * s0 + ks) * 512 + 4 * e);
    for (int sp = s0; sp <= s1; ++sp) {
      if (sp < s1) {
#pragma unroll
        for (int ks = 0; ks < 2; ++ks)
#pragma unroll
          for (int e = 0; e < 2; ++e) nxt[ks][e] = *reinterpret_cast<const f32x4*>(cb + (2 * sp + 2 + ks) * 512 + 4 * e);
      }
      const bool diag = sp == piece;
      float arg = base;  // log2 of the decay between this row and the source piece's end towards it
      for (int k = rev ? piece + 1 : sp + 1; k < (rev ? sp : piece); ++k) arg += sTot[k];
      const float fo = exp2_hw(arg);
#pragma unroll
      for (int ks = 0; ks < 2; ++ks) {
        // steps all behind (rev: before) the block's rows
        if (diag && ks == (rev ? 0 : 1) && blk[b] % 2 == (rev ? 1 : 0)) continue;
        const int s = kJB * sp + 32 * ks + 8 * (lane / 16);
        float m[8];
        if (diag) {
          const f32x4 c0 = *reinterpret_cast<const f32x4*>(&sCs[s]), c1 = *reinterpret_cast<const f32x4*>(&sCs[s + 4]);
          const f32x4 d0 = *reinterpret_cast<const f32x4*>(&sOwn[s]), d1 = *reinterpret_cast<const f32x4*>(&sOwn[s + 4]);
#pragma unroll
          for (int e = 0; e < 8; ++e) {
            const float css = e < 4 ? c0[e & 3] : c1[e & 3];
            const float v = cur[ks][e / 4][e & 3] * exp2_hw(rev ? css - cso : cso - css) *
                            (e < 4 ? d0[e & 3] : d1[e & 3]);
            m[e] = (rev ? s + e >= o : s + e <= o) ? v : 0.0f;
          }
        } else {
          const f32x4 w0 = *reinterpret_cast<const f32x4*>(&sCol[s]), w1 = *reinterpret_cast<const f32x4*>(&sCol[s + 4]);
#pragma unroll
          for (int e = 0; e < 8; ++e) m[e] = cur[ks][e / 4][e & 3] * ((e < 4 ? w0[e & 3] : w1[e & 3]) * fo);
        }
        if (p.seq_idx) {
#pragma unroll
          for (int e = 0; e < 8; ++e) m[e] = sSeg[s + e] == sego ? m[e] : 0.0f;
        }
        u32x4v mh, ml;
#pragma unroll
        for (int e = 0; e < 4; ++e) {
          uint32_t a, c;
          split2(m[2 * e], m[2 * e + 1], a, c);
          mh[e] = a;
          ml[e] = c;
        }
        bf16x8 ua[UP][4];
#pragma unroll
        for (int i = 0; i < UP; ++i)
#pragma unroll
          for (int pt = 0; pt < 4; ++pt)
            ua[i][pt] = bfv(tm_frag(&sU[i][(kJB * sp + 32 * ks) * kP], tm_lane_off<kP>(16 * pt, 0, lane),
                                    tm_lane_off<kP>(16 * pt, 1, lane)));
#pragma unroll
        for (int pt = 0; pt < 4; ++pt) acc[b][pt] = BF::run(ua[0][pt], bfv(ml), acc[b][pt]);
        if constexpr (UP > 1) {
#pragma unroll
          for (int pt = 0; pt < 4; ++pt) acc[b][pt] = BF::run(ua[UP - 1][pt], bfv(mh), acc[b][pt]);
        }
#pragma unroll
        for (int pt = 0; pt < 4; ++pt) acc[b][pt] = BF::run(ua[0][pt], bfv(mh), acc[b][pt]);
      }
#pragma unroll
      for (int ks = 0; ks < 2; ++ks)
#pragma unroll
        for (int e = 0; e < 2; ++e) cur[ks][e] = nxt[ks][e];
    }
    const int64_t out = (q.row0 + o) * xrow + h * kP;
    if (o >= rows) continue;
    const float row = sRow[o];
#pragma unroll
    for (int pt = 0; pt < 4; ++pt) {
      const int p0 = 16 * pt + 4 * (lane / 16);
      uint2 uw[UP];
#pragma unroll
      for (int i = 0; i < UP; ++i) uw[i] = *reinterpret_cast<const uint2*>(&sU[i][tm_off<kP>(o, p0)]);
      float u[4], r[4];  // of row o: g, or x
      join4<UP>(uw, u);
      if (rev) {
#pragma unroll
        for (int e = 0; e < 4; ++e) r[e] = fmaf(Dh, u[e], row * acc[b][pt][e]);
      } else {
        const uint2 zw = *reinterpret_cast<const uint2*>(static_cast<const uint16_t*>(p.z) + out + p0);
        const uint2 dw = *reinterpret_cast<const uint2*>(static_cast<const uint16_t*>(p.dy) + out + p0);
        const float z[4] = {low16<IO>(zw.x), high16<IO>(zw.x), low16<IO>(zw.y), high16<IO>(zw.y)};
        const float dy[4] = {low16<IO>(dw.x), high16<IO>(dw.x), low16<IO>(dw.y), high16<IO>(dw.y)};
#pragma unroll
        for (int e = 0; e < 4; ++e) {
          const float sg = sigmoid_f(z[e]);
          r[e] = dy[e] * fmaf(Dh, u[e], row * acc[b][pt][e]) * (sg * fmaf(z[e], 1.0f - sg, 1.0f));
        }
      }
      *reinterpret_cast<uint2*>(static_cast<uint16_t*>(rev ? p.dx : p.dz) + out + p0) =
          make_uint2(pack2<IO>(r[0], r[1]), pack2<IO>(r[2], r[3]));
    }
  }
}

// ---- S and the sums of W -----------------------------------------------------------------
// Workgroup = (chunk, group, pair of 64-step pieces ib >= jb), all heads of the
// group in turn; wave w has the rows i of tile w of ib and all columns j of jb,
// lane l the row i = l % 16 and the columns 16 t + 4 (l / 16) + r: S^T is built
// as x_j . g_i (A = x from LDS, B = g from memory) and summed over the heads in
// registers.  The columns' x and vectors of the next head are on their way
// while this head is worked on, two buffers in turn, one barrier per head.
// Of W = (C_i . B_j) S_ij it leaves, per head,
//   ib > jb: its sums over j of every row, and over i of every column, the
//            latter without Delta_j (x . G B takes those);
//   ib = jb: the columns' sums too (i >= j), and for every j the sum over i > j
//            of the row's sums up to j, sum_{i>j} sum_{m<=j} W_im: the pairs
//            around step j + 1, formed without terms that cancel.
// A column's sum over the 16 lanes of a row tile is a halving exchange (45
// instructions for 16 columns); the waves' parts meet in LDS once per batch of
// heads.  The decay between two pieces is a factor per row, one per column and
// one for the pieces between; inside a piece it is the exp of a difference, of
// sums kept as two floats.
constexpr int kBatch = 16;
constexpr int kPairs = 10;
__device__ __forceinline__ int pair_of(int ib, int jb) { return ib * (ib + 1) / 2 + jb; }
// rows of 64 channels in LDS, their 16-byte pieces swapped by the row, so that
// 8 rows' pieces of one column lie in different banks
__device__ __forceinline__ int row64_off(int row, int col) {
  return row * kP + 8 * ((col >> 3) ^ (row & 7)) + (col & 7);
}

// 16 values per lane summed over the 16 lanes of a DPP row: lane l of the row
// receives the sum of value l.  In each of four steps a lane keeps the half of
// its values that one bit of l names and adds its partner's; the partners (8
// away, mirrored in 8, 2 away, 1 away) differ in that bit and in no earlier one.
template <int CTRL>
__device__ __forceinline__ float half_sum(float a, float b, bool upper) {
  const float keep = upper ? b : a, send = upper ? a : b;
  return keep + __int_as_float(__builtin_amdgcn_update_dpp(0, __float_as_int(send), CTRL, 0xf, 0xf, true));
}
__device__ __forceinline__ float transpose_sum(const f32x4 (&v)[4]) {
  const int l = threadIdx.x % 16;
  float a[8], b[4], c[2];
#pragma unroll
  for (int k = 0; k < 8; ++k) a[k] = half_sum<0x128>(v[k / 4][k % 4], v[2 + k / 4][k % 4], l & 8);  // row_ror:8
#pragma unroll
  for (int k = 0; k < 4; ++k) b[k] = half_sum<0x141>(a[k], a[4 + k], l & 4);                        // row_half_mirror
#pragma unroll
  for (int k = 0; k < 2; ++k) c[k] = half_sum<0x4E>(b[k], b[2 + k], l & 2);                         // quad_perm ^2
  return half_sum<0xB1>(c[0], c[1], l & 1);                                                         // quad_perm ^1
}

template <int MODE>
struct PairLds {
  union {
    float part[kBatch][2][4][64];  // [head][columns' sums, pairs around][wave][column]
    float S[64 * 65];              // after the heads
  };
  __attribute__((aligned(16))) uint16_t x[2][data_parts<MODE>()][kJB * kP];
  __attribute__((aligned(16))) float vec[2][3][kJB];  // Delta_j; the columns' factors, or their sums (step_log2)
};

template <int MODE, int N, bool DIAG>
__device__ __forceinline__ void pair_role(const SsdBwdParams& p, const Chunk& q, int g, int ib, int jb,
                                          PairLds<MODE>& lds) {
  constexpr int IO = io_of<MODE>();
  constexpr int GP = g_parts<MODE>(), XP = data_parts<MODE>();
  const int tid = threadIdx.x, lane = tid % 64, wave = tid / 64, quad = lane / 16, l16 = lane % 16;
  const int rows = q.rows, pr = pair_of(ib, jb);
  const int hpg = p.nheads / p.ngroups;
  const int64_t xrow = (int64_t)p.nheads * kP, vrow = (int64_t)p.ngroups * N;
  const int il = kJB * ib + 16 * wave + l16, jl = 4 * quad, j0 = kJB * jb + jl;  // columns j0 + 16 t + r

  // C_i . B_j, the same for every head
  f32x4 cb[4];
  {
    const auto bv = plane_view(static_cast<const uint16_t*>(p.Bm), q.row0, vrow, g * N, N, rows);
    const auto cv = plane_view(static_cast<const uint16_t*>(p.Cm), q.row0, vrow, g * N, N, rows);
#pragma unroll
    for (int t = 0; t < 4; ++t) cb[t] = f32x4{0.0f, 0.0f, 0.0f, 0.0f};
#pragma unroll
    for (int ks = 0; ks < N / 32; ++ks) {
      const auto c = as_vec<IO>(vload16(cv, (uint32_t)(il * vrow * 2 + (32 * ks + 8 * quad) * 2)));
#pragma unroll
      for (int t = 0; t < 4; ++t)
        cb[t] = mfma_t<IO>::run(
            as_vec<IO>(vload16(bv, (uint32_t)((kJB * jb + 16 * t + l16) * vrow * 2 + (32 * ks + 8 * quad) * 2))), c, cb[t]);
    }
  }
  uint32_t same = 0xffffu;  // bit 4 t + r: column j of tile t counts for row i
  if (p.seq_idx) {
    const int32_t* seg = p.ws_seg + (int64_t)q.place * kQ;
    const int si = seg[il];
    same = 0u;
#pragma unroll
    for (int t = 0; t < 4; ++t)
#pragma unroll
      for (int r = 0; r < 4; ++r) same |= (uint32_t)(seg[j0 + 16 * t + r] == si) << (4 * t + r);
  }
  if constexpr (DIAG) {
#pragma unroll
    for (int t = 0; t < 4; ++t)
#pragma unroll
      for (int r = 0; r < 4; ++r)
        if (j0 + 16 * t + r > il) same &= ~(1u << (4 * t + r));
  }
  f32x4 S[4];
#pragma unroll
  for (int t = 0; t < 4; ++t) S[t] = f32x4{0.0f, 0.0f, 0.0f, 0.0f};

  // a head's operands on their way: x of the columns (row tid / 8 + 32 k,
  // channels 8 (tid % 8) ..), one vector element, the factors of this lane's row, and
  // its g, of which two heads' take turns
  u32x4v xr[XP][2], gf[2][GP][2];
  float vr = 0.0f, fn, ln = 0.0f, mid[2] = {0.0f, 0.0f};
  const int uwave = uniform(wave);
  const float* const vec = uwave == 0 ? p.ws_delta : uwave == 1 ? (DIAG ? p.ws_cs : p.ws_to) : p.ws_cl;
  auto load_x = [&](int h) {
    const int64_t at = ((int64_t)q.place * p.nheads + h) * kQ;
#pragma unroll
    for (int i = 0; i < XP; ++i) {
      const auto xv = plane_view(p.xp[i], q.row0, xrow, h * kP, kP, rows);
#pragma unroll
      for (int k = 0; k < 2; ++k)
        xr[i][k] = vload16(xv, (uint32_t)((kJB * jb + tid / 8 + 32 * k) * xrow * 2 + (tid % 8) * 16));
    }
    if (uwave < (DIAG ? 3 : 2)) vr = vec[at + kJB * jb + lane];
    fn = (DIAG ? p.ws_cs : p.ws_from)[at + il];
    if constexpr (DIAG) {
      ln = p.ws_cl[at + il];
    } else {  // the sums over the pieces between
#pragma unroll
      for (int k = 0; k < 2; ++k)
        if (jb + 1 + k < ib) mid[k] = p.ws_cs[at + kJB * (jb + 1 + k) + kJB - 1];
    }
  };
  auto load_g = [&](int u, int h) {
#pragma unroll
    for (int i = 0; i < GP; ++i) {
      const auto gv = plane_view(p.gp[i], q.row0, xrow, h * kP, kP, rows);
#pragma unroll
      for (int ks = 0; ks < 2; ++ks) gf[u][i][ks] = vload16(gv, (uint32_t)(il * xrow * 2 + (32 * ks + 8 * quad) * 2));
    }
  };
  const int hend = (g + 1) * hpg;
  load_x(g * hpg);
  load_g(0, g * hpg);
  for (int h0 = 0; h0 < hpg; h0 += kBatch) {
    const int nb = hpg - h0 < kBatch ? hpg - h0 : kBatch;
    for (int hb0 = 0; hb0 < nb; hb0 += 2)
#pragma unroll
    for (int turn = 0; turn < 2; ++turn) {
      const int hb = hb0 + turn, h = g * hpg + h0 + hb;
      if (hb >= nb) break;
      const int64_t ph = (int64_t)q.place * p.nheads + h;
#pragma unroll
      for (int i = 0; i < XP; ++i)
#pragma unroll
        for (int k = 0; k < 2; ++k)
          *reinterpret_cast<u32x4v*>(&lds.x[turn][i][row64_off(tid / 8 + 32 * k, 8 * (tid % 8))]) = xr[i][k];
      if (uwave < (DIAG ? 3 : 2)) lds.vec[turn][wave][lane] = vr;
      const float f = DIAG ? fn : fn * exp2_hw(mid[0] + mid[1]), l = ln;
      if (h + 1 < hend) {
        load_x(h + 1);
        load_g(1 - turn, h + 1);
      }
      __syncthreads();
      f32x4 a[4];
#pragma unroll
      for (int t = 0; t < 4; ++t) a[t] = f32x4{0.0f, 0.0f, 0.0f, 0.0f};
#pragma unroll
      for (int ks = 0; ks < 2; ++ks)
#pragma unroll
        for (int j = XP - 1; j >= 0; --j) {
          bf16x8 xf[4];
#pragma unroll
          for (int t = 0; t < 4; ++t)
            xf[t] = bfv(*reinterpret_cast<const u32x4v*>(&lds.x[turn][j][row64_off(16 * t + l16, 32 * ks + 8 * quad)]));
#pragma unroll
          for (int i = GP - 1; i >= 0; --i)
            if (i + j <= 2)
#pragma unroll
              for (int t = 0; t < 4; ++t) a[t] = BF::run(xf[t], bfv(gf[turn][i][ks]), a[t]);
        }
      float xd = 0.0f;
#pragma unroll
      for (int t = 0; t < 4; ++t) {
        const f32x4 ej = *reinterpret_cast<const f32x4*>(&lds.vec[turn][1][jl + 16 * t]);
        if constexpr (DIAG) {
          const f32x4 lj = *reinterpret_cast<const f32x4*>(&lds.vec[turn][2][jl + 16 * t]);
#pragma unroll
          for (int r = 0; r < 4; ++r) {
            if (t == wave) xd = j0 + 16 * t + r == il ? a[t][r] : xd;
            const float e = exp2_hw((f - ej[r]) + (l - lj[r]));
            a[t][r] = (same >> (4 * t + r)) & 1u ? a[t][r] * e : 0.0f;
          }
        } else {
#pragma unroll
          for (int r = 0; r < 4; ++r) a[t][r] *= ej[r] * f;
          if (p.seq_idx) {
#pragma unroll
            for (int r = 0; r < 4; ++r) a[t][r] = (same >> (4 * t + r)) & 1u ? a[t][r] : 0.0f;
          }
        }
      }
      // a: S_ij without Delta_j
      f32x4 W[4];
      float row = 0.0f, base = 0.0f;
#pragma unroll
      for (int t = 0; t < 4; ++t) {
        const f32x4 dj = *reinterpret_cast<const f32x4*>(&lds.vec[turn][0][jl + 16 * t]);
        f32x4 v;
#pragma unroll
        for (int r = 0; r < 4; ++r) {
          S[t][r] = fmaf(a[t][r], dj[r], S[t][r]);
          W[t][r] = cb[t][r] * a[t][r];
          if constexpr (DIAG) {
            v[r] = r ? fmaf(W[t][r], dj[r], v[r - 1]) : W[t][0] * dj[0];
          } else {
            row = fmaf(W[t][r], dj[r], row);
          }
        }
        if constexpr (DIAG) {
          // the row's sums up to each j: inside a lane's 4 columns, over the quads
          // of a tile (lanes 16 apart), over the tiles
          const QuadSums s = quad_sums(v[3]);
          const float before = base + s.before;
#pragma unroll
          for (int r = 0; r < 4; ++r) a[t][r] = il > j0 + 16 * t + r ? v[r] + before : 0.0f;
          base += s.all;
        }
      }
      lds.part[hb][0][wave][16 * (l16 / 4) + jl + l16 % 4] = transpose_sum(W);
      if constexpr (DIAG) {
        lds.part[hb][1][wave][16 * (l16 / 4) + jl + l16 % 4] = transpose_sum(a);
        if (quad == (l16 >> 2)) p.ws_xd[ph * kQ + il] = xd;
      } else {
        row = quad_sum(row);
        if (quad == 0) p.ws_prow[(ph * kPairs + pr) * kJB + 16 * wave + l16] = row;
      }
    }
    __syncthreads();
    for (int k = tid; k < nb * 64; k += 256) {
      const int hb = k / 64, j = k % 64;
      const auto& v = lds.part[hb];
      const int64_t to = (((int64_t)q.place * p.nheads + g * hpg + h0 + hb) * kPairs + pr) * kJB + j;
      p.ws_pcol[to] = (v[0][0][j] + v[0][1][j]) + (v[0][2][j] + v[0][3][j]);
      if constexpr (DIAG) p.ws_prow[to] = (v[1][0][j] + v[1][1][j]) + (v[1][2][j] + v[1][3][j]);
    }
    __syncthreads();
  }

  // S as operand fragments, two parts, for dC (a lane a row i, 8 columns) and for
  // dB (a lane a column j, 8 rows): [dC, dB][part][tile][k-step][lane][8], where
  // element e of a k-step's quad is step 4 quad + e of its first tile, or of its
  // second for e >= 4
  uint32_t* out = p.ws_S + (((int64_t)q.place * p.ngroups + g) * kPairs + pr) * (2 * kJB * kJB);
#pragma unroll
  for (int t = 0; t < 4; ++t)
#pragma unroll
    for (int r = 0; r < 4; ++r) lds.S[(16 * wave + l16) * 65 + 16 * t + jl + r] = S[t][r];
  __syncthreads();
#pragma unroll
  for (int side = 0; side < 2; ++side) {
    if (side) {
#pragma unroll
      for (int t = 0; t < 4; ++t)
#pragma unroll
        for (int r = 0; r < 4; ++r) S[t][r] = lds.S[(16 * t + jl + r) * 65 + 16 * wave + l16];
    }
#pragma unroll
    for (int ks = 0; ks < 2; ++ks) {
      u32x4v part[2];
#pragma unroll
      for (int e = 0; e < 4; ++e) {
        uint32_t hi, lo;
        split2(S[2 * ks + e / 2][2 * (e % 2)], S[2 * ks + e / 2][2 * (e % 2) + 1], hi, lo);
        part[0][e] = hi;
        part[1][e] = lo;
      }
#pragma unroll
      for (int k = 0; k < 2; ++k)
        *reinterpret_cast<u32x4v*>(out + ((((side * 2 + k) * 4 + wave) * 2 + ks) * 64 + lane) * 4) = part[k];
    }
  }
}

// The pass between the chunks' states and the pairs need nothing of each other;
// the former waits for memory, the latter computes, so they share a launch, the
// pairs' workgroups first, which live longer (bench layer: 75 us; 94 us as two
// launches, 98 us with one's eight workgroups, one on each XCD, after the
// other's eight, 103 us with the pass first).
inline uint32_t pass_octets(const SsdBwdParams& p) {
  return (uint32_t)((p.batch * p.nheads * (kP * p.dstate / 1024) + 7) / 8);
}
inline uint32_t pair_octets(const SsdBwdParams& p) {
  return (uint32_t)((p.batch * p.nchunks * p.ngroups + 7) / 8 * kPairs);
}
template <int MODE, int N>
__global__ void __launch_bounds__(256, MODE == 0 ? 3 : 2)
    bwd_pass_pair_kernel(SsdBwdParams p, uint32_t passes, uint32_t pairs) {
  __shared__ PairLds<MODE> lds;
  uint32_t octet = blockIdx.x / 8u;
  const bool pass = octet >= pairs;
  octet = pass ? octet - pairs : octet;
  if (pass) {
    const uint32_t block = octet * 8u + blockIdx.x % 8u;
    if (block < (uint32_t)(p.batch * p.nheads * (kP * N / 1024))) pass_role<N>(p, block);
    return;
  }
  // the pairs of one chunk's group share an XCD's L2, and of an XCD's pairs the
  // ib = jb ones, which take longest, come first
  const int units = (int)p.batch * p.nchunks * p.ngroups, xcd = (int)(blockIdx.x % 8u);
  const int u0 = (int)((int64_t)units * xcd / 8), n = (int)((int64_t)units * (xcd + 1) / 8) - u0;
  int l = (int)octet, ib, jb, unit;
  if (l < 4 * n) {
    unit = u0 + l / 4;
    ib = jb = l % 4;
  } else {
    l -= 4 * n;
    if (l >= 6 * n) return;
    unit = u0 + l / 6;
    l %= 6;
    ib = l < 1 ? 1 : l < 3 ? 2 : 3;
    jb = l - ib * (ib - 1) / 2;
  }
  const int g = unit % p.ngroups;
  const Chunk q = chunk_of(p, unit / p.ngroups);
  if (kJB * ib >= q.rows) return;
  if (ib == jb) pair_role<MODE, N, true>(p, q, g, ib, jb, lds);
  else pair_role<MODE, N, false>(p, q, g, ib, jb, lds);
}

// ---- dC and dB -----------------------------------------------------------------------------
// Workgroup = (chunk, group, dC or dB, half of the rows, half of the states), 256
// threads, wave w the rows f = 32 w .. 32 w + 31 of the half:
//   dC: f = i: F = g, K = E, v = C, u = B, w_f = exp(cs_f), d = 1
//   dB: f = j: F = x, K = R, v = B, u = C, w_f = exp(cs_last - cs_f), d = Delta
//   out_f[n] = sum_h d_f w_f sum_p K[p][n] F_f[p] + sum_s S_fs u_s[n]
// and per head v_f . (w_f K^T F_f) (e; r and x . G B's share of it, without
// Delta).  The heads' K are staged in LDS by turns of two buffers (three parts,
// [p][16 n] tiles read back transposed): the K of the head after the next is on
// its way while this head is multiplied, the next one's F while its K is staged,
// one barrier per head.  S comes as operand fragments from bwd_pair, with u's
// pieces staged in LDS.
// Bound by HBM and the phases' waits: at the bench layer 68 us for 259 MB (E, R, x
// and g; the halves' second reads are the L2's), the matrix units busy for a
// quarter of it.  Two register sets for F, so that it is loaded a multiplication
// earlier, take 72 us (gated bf16 at state 128, where they spill: 641 against 599
// us of the whole); 32 states a workgroup, which read x and g twice as often, 78
// us; all rows in one workgroup of 512 threads 67 us, and 23.5 against 14.1 us
// where a few chunks (B = 2, L = 1001, 8 heads) leave CUs idle.
constexpr int kOutThreads = 256;
// element (row, c) of a [rows][16] tile: blocks of 4 rows swapped so that the
// transposing reads of rows 8 apart hit different banks
__device__ __forceinline__ int t16_off(int row, int c) { return (row ^ (((row >> 3) & 1) << 2)) * 16 + c; }

template <int MODE, int N, bool DB>
__device__ __forceinline__ void out_role(const SsdBwdParams& p, int lb, uint16_t* lds) {
  constexpr int IO = io_of<MODE>();
  constexpr int FP = DB ? data_parts<MODE>() : g_parts<MODE>(), UP = data_parts<MODE>();
  constexpr int NH = N / 2, NT = NH / 16;                    // states and state tiles of the half
  constexpr int kItems = kP * NH / 4, kPer = (kItems + kOutThreads - 1) / kOutThreads;
  constexpr int kBuf = 3 * kP * NH;
  const int tid = threadIdx.x, lane = tid % 64, wave = tid / 64, quad = lane / 16, l16 = lane % 16;
  const int half = lb & 1, upper = (lb >> 1) & 1, g = (lb >> 2) % p.ngroups;
  const Chunk q = chunk_of(p, (lb >> 2) / p.ngroups);
  const int rows = q.rows, n0 = NH * half, f0 = kQ / 2 * upper;
  if (f0 >= rows) return;
  const int hpg = p.nheads / p.ngroups;
  const int64_t xrow = (int64_t)p.nheads * kP, vrow = (int64_t)p.ngroups * N;
  const int fr[2] = {f0 + 32 * wave + l16, f0 + 32 * wave + 16 + l16};  // this lane's rows
  const auto vv = plane_view(static_cast<const uint16_t*>(DB ? p.Bm : p.Cm), q.row0, vrow, g * N, N, rows);
  uint2 vn[2][NT];
#pragma unroll
  for (int b = 0; b < 2; ++b)
#pragma unroll
    for (int t = 0; t < NT; ++t) vn[b][t] = vload8(vv, (uint32_t)(fr[b] * vrow * 2 + (n0 + 16 * t + 4 * quad) * 2));
  f32x4 tot[2][NT];
#pragma unroll
  for (int b = 0; b < 2; ++b)
#pragma unroll
    for (int t = 0; t < NT; ++t) tot[b][t] = f32x4{0.0f, 0.0f, 0.0f, 0.0f};

  f32x4 kr[kPer];
  u32x4v F[FP][2][2];
  float wf[2], df[2];
  auto load_k = [&](int h) {
    const float* K = (DB ? p.ws_R : p.ws_E) + ((int64_t)q.place * p.nheads + h) * (kP * N) + n0;
#pragma unroll
    for (int k = 0; k < kPer; ++k) {
      const int item = tid + kOutThreads * k;
      if (kItems % kOutThreads == 0 || item < kItems)
        kr[k] = *reinterpret_cast<const f32x4*>(K + (item / (NH / 4)) * N + 4 * (item % (NH / 4)));
    }
  };
  auto load_f = [&](int h) {
#pragma unroll
    for (int i = 0; i < FP; ++i) {
      const auto fv = plane_view(DB ? p.xp[i % 2] : p.gp[i], q.row0, xrow, h * kP, kP, rows);
#pragma unroll
      for (int b = 0; b < 2; ++b)
#pragma unroll
        for (int ks = 0; ks < 2; ++ks)
          F[i][b][ks] = vload16(fv, (uint32_t)(fr[b] * xrow * 2 + (32 * ks + 8 * quad) * 2));
    }
    const int64_t at = ((int64_t)q.place * p.nheads + h) * kQ;
#pragma unroll
    for (int b = 0; b < 2; ++b) {
      wf[b] = (DB ? p.ws_wb : p.ws_wc)[at + fr[b]];
      df[b] = DB ? p.ws_delta[at + fr[b]] : 1.0f;
    }
  };
  auto stage_k = [&](uint16_t* buf) {
#pragma unroll
    for (int k = 0; k < kPer; ++k) {
      const int item = tid + kOutThreads * k;
      if (kItems % kOutThreads == 0 || item < kItems) {
        const int pr = item / (NH / 4), n = 4 * (item % (NH / 4));
        uint32_t a[3], b[3];
        split3(kr[k][0], kr[k][1], a);
        split3(kr[k][2], kr[k][3], b);
        const int at = (n / 16) * (kP * 16) + t16_off(pr, n % 16);
#pragma unroll
        for (int i = 0; i < 3; ++i) *reinterpret_cast<uint2*>(&buf[i * kP * NH + at]) = make_uint2(a[i], b[i]);
      }
    }
  };
  load_k(g * hpg);
  load_f(g * hpg);
  stage_k(lds);
  if (hpg > 1) load_k(g * hpg + 1);
  for (int hg0 = 0; hg0 < hpg; hg0 += 2)
#pragma unroll
  for (int u = 0; u < 2; ++u) {
    const int hg = hg0 + u, h = g * hpg + hg;
    if (hg >= hpg) break;
    const uint16_t* buf = lds + u * kBuf;
    __syncthreads();
    f32x4 a[2][NT];
#pragma unroll
    for (int t = 0; t < NT; ++t)
#pragma unroll
      for (int b = 0; b < 2; ++b) a[b][t] = f32x4{0.0f, 0.0f, 0.0f, 0.0f};
#pragma unroll
    for (int ks = 0; ks < 2; ++ks) {
      const int r0 = 32 * ks + 8 * quad + l16 / 4, c = 4 * (l16 % 4);
      const int o0 = t16_off(r0, c), o1 = t16_off(r0 + 4, c);
#pragma unroll
      for (int j = 2; j >= 0; --j) {
        bf16x8 kp[NT];
#pragma unroll
        for (int t = 0; t < NT; ++t) kp[t] = bfv(tm_frag(buf + j * kP * NH + t * (kP * 16), o0, o1));
#pragma unroll
        for (int i = FP - 1; i >= 0; --i)
          if (i + j <= 2)
#pragma unroll
            for (int t = 0; t < NT; ++t)
#pragma unroll
              for (int b = 0; b < 2; ++b) a[b][t] = BF::run(kp[t], bfv(F[i][b][ks]), a[b][t]);
      }
    }
    const float w[2] = {wf[0], wf[1]}, d[2] = {df[0], df[1]};
    if (hg + 1 < hpg) {  // the next head's K into the other buffer, the one after on its way
      load_f(h + 1);
      stage_k(lds + (1 - u) * kBuf);
      if (hg + 2 < hpg) load_k(h + 2);
    }
    const int64_t to = ((int64_t)half * p.batch * p.nchunks * p.nheads + (int64_t)q.place * p.nheads + h) * kQ;
#pragma unroll
    for (int b = 0; b < 2; ++b) {
      float vt = 0.0f;
#pragma unroll
      for (int t = 0; t < NT; ++t) {
        const float v[4] = {low16<IO>(vn[b][t].x), high16<IO>(vn[b][t].x), low16<IO>(vn[b][t].y), high16<IO>(vn[b][t].y)};
#pragma unroll
        for (int r = 0; r < 4; ++r) {
          vt = fmaf(v[r], a[b][t][r], vt);
          tot[b][t][r] = fmaf(DB ? w[b] * d[b] : w[b], a[b][t][r], tot[b][t][r]);
        }
      }
      vt = quad_sum(vt * w[b]);
      if (quad == 0) (DB ? p.ws_r : p.ws_e)[to + fr[b]] = vt;
    }
  }

  // ---- sum_s S_fs u_s
  __amdgpu_buffer_rsrc_t up[UP];
#pragma unroll
  for (int i = 0; i < UP; ++i) up[i] = plane_view(DB ? p.cp[i] : p.bp[i], q.row0, vrow, g * N + n0, NH, rows);
  const uint32_t* Sw = p.ws_S + ((int64_t)q.place * p.ngroups + g) * kPairs * (2 * kJB * kJB);
  const int fb = 2 * upper + wave / 2;  // the piece that holds this wave's rows
  const int lastp = (rows - 1) / kJB, fend = 2 * upper + 1 < lastp ? 2 * upper + 1 : lastp;
  const int s0 = DB ? 2 * upper : 0, s1 = DB ? lastp : fend;  // the pieces that any of the rows meets
  constexpr int kUItems = kJB * NH / 8, kU = (kUItems + kOutThreads - 1) / kOutThreads;
  u32x4v ur[UP][kU];  // the next piece of u on its way
  auto load_u = [&](int sb) {
#pragma unroll
    for (int k = 0; k < kU; ++k) {
      const int item = tid + kOutThreads * k;
      const uint32_t at = (uint32_t)((kJB * sb + item / (NH / 8)) * vrow * 2 + 16 * (item % (NH / 8)));
#pragma unroll
      for (int i = 0; i < UP; ++i) ur[i][k] = vload16(up[i], item < kUItems ? at : kOffNone);
    }
  };
  load_u(s0);
  for (int sb = s0; sb <= s1; ++sb) {
    const bool mine = fb <= lastp && (DB ? sb >= fb : sb <= fb);
    const uint32_t* Sp = Sw + (mine ? pair_of(DB ? sb : fb, DB ? fb : sb) : 0) * (2 * kJB * kJB) + (DB ? kJB * kJB : 0);
    u32x4v sp[2][2][2];  // [k-step][part][row tile]
    if (mine) {
#pragma unroll
      for (int ks = 0; ks < 2; ++ks)
#pragma unroll
        for (int k = 0; k < 2; ++k)
#pragma unroll
          for (int b = 0; b < 2; ++b)
            sp[ks][k][b] =
                *reinterpret_cast<const u32x4v*>(Sp + (((k * 4 + 2 * (wave % 2) + b) * 2 + ks) * 64 + lane) * 4);
    }
    __syncthreads();
#pragma unroll
    for (int k = 0; k < kU; ++k) {
      const int item = tid + kOutThreads * k, s = item / (NH / 8), n = 8 * (item % (NH / 8));
      const int at = (n / 16) * (kJB * 16) + t16_off(s, n % 16);
      if (kUItems % kOutThreads == 0 || item < kUItems)
#pragma unroll
        for (int i = 0; i < UP; ++i) *reinterpret_cast<u32x4v*>(&lds[i * kJB * NH + at]) = ur[i][k];
    }
    __syncthreads();
    if (sb < s1) load_u(sb + 1);
    if (!mine) continue;
#pragma unroll
    for (int ks = 0; ks < 2; ++ks) {
      const int r0 = 32 * ks + 4 * quad + l16 / 4, c = 4 * (l16 % 4);
      const int o0 = t16_off(r0, c), o1 = t16_off(r0 + 16, c);
#pragma unroll
      for (int t = 0; t < NT; ++t) {
        const bf16x8 uh = bfv(tm_frag(lds + t * (kJB * 16), o0, o1));
#pragma unroll
        for (int b = 0; b < 2; ++b) {
          tot[b][t] = BF::run(uh, bfv(sp[ks][1][b]), tot[b][t]);
          if constexpr (UP > 1)
            tot[b][t] = BF::run(bfv(tm_frag(lds + kJB * NH + t * (kJB * 16), o0, o1)), bfv(sp[ks][0][b]), tot[b][t]);
          tot[b][t] = BF::run(uh, bfv(sp[ks][0][b]), tot[b][t]);
        }
      }
    }
  }
  uint16_t* out = static_cast<uint16_t*>(DB ? p.dB : p.dC) + q.row0 * vrow + g * N + n0;
#pragma unroll
  for (int b = 0; b < 2; ++b)
    if (fr[b] < rows)
#pragma unroll
      for (int t = 0; t < NT; ++t)
        *reinterpret_cast<uint2*>(out + fr[b] * vrow + 16 * t + 4 * quad) =
            make_uint2(pack2<IO>(tot[b][t][0], tot[b][t][1]), pack2<IO>(tot[b][t][2], tot[b][t][3]));
}

template <int MODE, int N>
__global__ void __launch_bounds__(kOutThreads, 2) bwd_out_kernel(SsdBwdParams p) {
  constexpr int kHeads = 2 * 3 * kP * (N / 2), kSteps = data_parts<MODE>() * kJB * (N / 2);
  __shared__ __attribute__((aligned(16))) uint16_t lds[kHeads > kSteps ? kHeads : kSteps];
  const int lb = (int)xcd_logical_block(), n = (int)p.batch * p.nchunks * p.ngroups * 4;
  if (lb < n) out_role<MODE, N, false>(p, lb, lds);
  else out_role<MODE, N, true>(p, lb - n, lds);
}

// ---- da, ddt ----------------------------------------------------------------------------
// sum of v over the workgroup's 256 threads, in every thread
__device__ __forceinline__ float block_sum(float v, float* sWave) {
  v = row_sum(v);
  v += __shfl_xor(v, 16, 64);
  v += __shfl_xor(v, 32, 64);
  __syncthreads();
  if (threadIdx.x % 64 == 0) sWave[threadIdx.x / 64] = v;
  __syncthreads();
  return (sWave[0] + sWave[1]) + (sWave[2] + sWave[3]);
}

template <int IO>
__global__ void __launch_bounds__(256) bwd_delta_kernel(SsdBwdParams p) {
  __shared__ float sA[4], sB[4];
  const int tid = threadIdx.x, lane = tid % 64, wave = tid / 64;  // a wave is a piece
  const int h = (int)(blockIdx.x % (uint32_t)p.nheads);
  const Chunk q = chunk_of(p, (int)(blockIdx.x / (uint32_t)p.nheads));
  const int64_t ph = (int64_t)q.place * p.nheads + h, at = ph * kQ + tid;
  const int64_t other = p.batch * p.nchunks * p.nheads * kQ;  // the second half of the states
  const float* prow = p.ws_prow + ph * kPairs * kJB + lane;
  const float* pcol = p.ws_pcol + ph * kPairs * kJB + lane;
  const int lastp = (q.rows - 1) / kJB;
  const bool in = tid < q.rows;
  float around = 0.0f, row = 0.0f, col = 0.0f, e = 0.0f, out = 0.0f, xg = 0.0f, xd = 0.0f, delta = 0.0f, raw = 0.0f;
  if (in) {
    delta = p.ws_delta[at];
    if (lane > 0) around = prow[pair_of(wave, wave) * kJB - 1];  // the pairs around this step
    for (int k = 0; k < wave; ++k) row += prow[pair_of(wave, k) * kJB];
    for (int k = wave + 1; k <= lastp; ++k) col += pcol[pair_of(k, wave) * kJB];
    e = p.ws_e[at] + p.ws_e[other + at];
    out = p.ws_r[at] + p.ws_r[other + at];
    xg = (pcol[pair_of(wave, wave) * kJB] + col) + out;
    col *= delta;
    out *= delta;
    xd = p.ws_xd[at];
    raw = load_io<IO>(p.dt, (q.row0 + tid) * p.nheads + h) + (p.dt_bias ? p.dt_bias[h] : 0.0f);
  }
  const int nd = p.dstate / 4;
  float dot = 0.0f;
  for (int k = lane; k < nd; k += 64) dot += p.ws_dot[ph * nd + k];
  // the pairs around the whole piece: rows of later pieces, columns of earlier ones
  for (int i = wave + 1; i <= lastp; ++i)
    if (kJB * i + lane < q.rows)
      for (int j = 0; j < wave; ++j) dot += prow[pair_of(i, j) * kJB];
  dot = row_sum(dot);
  dot += __shfl_xor(dot, 16, 64);
  dot += __shfl_xor(dot, 32, 64);
  // from this step on (row, e), and before this step (col, out)
  float b = out;
#pragma unroll
  for (int off = 1; off < 64; off <<= 1) {
    const float u1 = __shfl_down(row, off, 64), u2 = __shfl_down(e, off, 64);
    const float v1 = __shfl_up(col, off, 64), v2 = __shfl_up(b, off, 64);
    if (lane + off < 64) {
      row += u1;
      e += u2;
    }
    if (lane >= off) {
      col += v1;
      b += v2;
    }
  }
  if (lane == 0) sA[wave] = e;
  if (lane == 63) sB[wave] = b;
  __syncthreads();
  float a = around + row;
  const float before = __shfl_up(col, 1, 64);
  b = __shfl_up(b, 1, 64);
  if (lane == 0) b = 0.0f;
  if (lane > 0) a += before;
  for (int k = wave + 1; k < 4; ++k) e += sA[k];
  for (int k = 0; k < wave; ++k) b += sB[k];
  a += e;
  const float da = in ? a + b + dot : 0.0f;
  float dr = fmaf(p.A[h], da, xg);
  if (p.softplus) dr *= sigmoid_f(raw);
  if (in) store_io<IO>(p.ddt, (q.row0 + tid) * p.nheads + h, dr);
  __syncthreads();
  const float s0 = block_sum(delta * da, sA), s1 = block_sum(in ? dr : 0.0f, sB), s2 = block_sum(xd, sA);
  if (tid == 0) {
    float* part = p.ws_part + ph * 3;
    part[0] = s0;
    part[1] = s1;
    part[2] = s2;
  }
}

__global__ void __launch_bounds__(256) bwd_sum_kernel(SsdBwdParams p) {
  __shared__ float sW[4];
  const int h = blockIdx.x;
  const int places = (int)p.batch * p.nchunks;
  float v[3] = {0.0f, 0.0f, 0.0f};
  for (int k = threadIdx.x; k < places; k += 256)
#pragma unroll
    for (int e = 0; e < 3; ++e) v[e] += p.ws_part[((int64_t)k * p.nheads + h) * 3 + e];
#pragma unroll
  for (int e = 0; e < 3; ++e) v[e] = block_sum(v[e], sW);
  if (threadIdx.x == 0) {
    p.dA[h] = v[0];
    if (p.ddt_bias) p.ddt_bias[h] = v[1];
    if (p.dD) p.dD[h] = v[2];
  }
}

#define SS_LAUNCH(k, grid, block)                                       \
  do {                                                                  \
    hipLaunchKernelGGL(k, dim3((uint32_t)(grid)), dim3(block), 0, st, p); \
    const hipError_t e_ = hipGetLastError();                            \
    if (e_ != hipSuccess) return e_;                                    \
  } while (0)

template <int MODE, int N, int HB>
hipError_t launch_state(const SsdBwdParams& p, hipStream_t st) {
  const int64_t groups = p.batch * p.nchunks * p.ngroups, parts = (p.nheads / p.ngroups + HB - 1) / HB;
  SS_LAUNCH((bwd_state_kernel<MODE, N, HB>), groups * ((MODE % 2 ? 4 : 2) + 2 * parts), kStateThreads);
  return hipSuccess;
}
template <int MODE, int N>
hipError_t launch_n(const SsdBwdParams& p, hipStream_t st) {
  const int64_t places = p.batch * p.nchunks, heads = places * p.nheads;
  constexpr bool gate = MODE % 2 != 0;
  hipError_t e;
  switch (state_heads(2 * places * p.ngroups, p.nheads / p.ngroups, device_cus())) {
    case 1: e = launch_state<MODE, N, 1>(p, st); break;
    case 2: e = launch_state<MODE, N, 2>(p, st); break;
    default: e = launch_state<MODE, N, 3>(p, st); break;
  }
  if (e != hipSuccess) return e;
  const uint32_t passes = pass_octets(p), pairs = pair_octets(p);
  hipLaunchKernelGGL((bwd_pass_pair_kernel<MODE, N>), dim3(8u * (passes + pairs)), dim3(256), 0, st, p, passes, pairs);
  e = hipGetLastError();
  if (e != hipSuccess) return e;
  SS_LAUNCH((bwd_scan_kernel<MODE, N>), gate ? 2 * heads : heads, kScanThreads);
  SS_LAUNCH((bwd_out_kernel<MODE, N>), places * p.ngroups * 8, kOutThreads);
  SS_LAUNCH((bwd_delta_kernel<io_of<MODE>()>), heads, 256);
  SS_LAUNCH(bwd_sum_kernel, p.nheads, 256);
  return hipSuccess;
}
template <int MODE>
hipError_t launch_mode(const SsdBwdParams& p, hipStream_t st) {
  switch (p.dstate) {
    case 32: return launch_n<MODE, 32>(p, st);
    case 64: return launch_n<MODE, 64>(p, st);
    case 96: return launch_n<MODE, 96>(p, st);
    default: return launch_n<MODE, 128>(p, st);
  }
}

}  // namespace

hipError_t launch_ssd_bwd(int32_t io, const SsdBwdParams& p, hipStream_t st) {
  PlaneJobs a{};
  const int64_t rows = p.batch * p.seqlen;
  const int parts = io == SS_F16 ? 2 : 1;
  auto add = [&](const void* src, const void* gate, const uint16_t* const* to, int n_parts, int64_t n) {
    if (n_parts == 1) return;
    PlaneJob& j = a.j[a.n++];
    j = PlaneJob{src, gate, {}, n_parts, n, n / 2048 < kPlaneBlocks ? (n + 2047) / 2048 : kPlaneBlocks};
    for (int i = 0; i < n_parts; ++i) j.part[i] = const_cast<uint16_t*>(to[i]);
  };
  add(p.dy, p.z, p.gp, p.z ? 3 : parts, rows * p.nheads * kP);
  add(p.x, nullptr, p.xp, parts, rows * p.nheads * kP);
  add(p.Bm, nullptr, p.bp, parts, rows * p.ngroups * p.dstate);
  add(p.Cm, nullptr, p.cp, parts, rows * p.ngroups * p.dstate);
  if (a.n) {
    int64_t blocks = 0;
    for (int k = 0; k < a.n; ++k) blocks += a.j[k].blocks;
    if (io == SS_F16) hipLaunchKernelGGL((bwd_planes_kernel<SS_F16>), dim3((uint32_t)blocks), dim3(256), 0, st, a);
    else hipLaunchKernelGGL((bwd_planes_kernel<SS_BF16>), dim3((uint32_t)blocks), dim3(256), 0, st, a);
    const hipError_t e = hipGetLastError();
    if (e != hipSuccess) return e;
  }
  if (io == SS_F16) return p.z ? launch_mode<3>(p, st) : launch_mode<2>(p, st);
  return p.z ? launch_mode<1>(p, st) : launch_mode<0>(p, st);
}

}  // namespace ss
