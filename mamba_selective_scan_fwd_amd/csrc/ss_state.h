// ss_state.h -- the states that chunks add (gfx950).  Internal to libss.so.
//
// For HB heads that share V (a group's B or C): out_h[p][n] = sum_t w_h[t] u_h[t][p]
// V[t][n] over the rows of a chunk, u (rows, heads, 64) and V (rows, groups, N)
// time-major, on the matrix cores with the time as the inner axis.
//
// Workgroup: 512 threads, HB heads of one chunk, so that V's pieces of 64 steps
// are staged once for all of them.  The steps are (piece, head): w u in three
// bf16 parts lies in one of two LDS buffers in turn and is read back transposed
// together with V, while the next step's w u is made for the other; one barrier
// a step.  Wave w has the channels 16 (w % 4) .. and the half w / 4 of the
// states, of every head (the accumulators stay in registers over all pieces).
// A head's u of the next piece is loaded as soon as this piece's is in LDS, so
// its way is HB steps long.
#pragma once

#include "ss_mfma.h"
#include "ss_plan.h"

namespace ss {

// ---- decays inside a chunk ----------------------------------------------------------
// exp(Delta_t A) as a power of two, in 64 bits.  The weight of step j in step i is
// 2 to the difference of two running sums of these over up to 64 steps: after
// steps that forget everything the sums are large where the difference between
// neighbours is small, and its error is the sums' own.  One float leaves 2^-24 of
// the sum (32 steps of Delta A = -320 and 32 small ones: weights near 1 off by
// 2e-3); the sums are formed in 64 bits and kept as two floats hi + lo.  The scans
// take a pair's exponent from hi alone and lo as factors 2^lo, of the column with
// what else scales it and of the row at the end, so that a pair costs no more.
// Beyond +-2^20 a decay is 0 or infinite in every product that fp32 holds; the
// bound keeps lo within 2, and its power finite.
__device__ __forceinline__ double step_log2(float delta, float A) {
  constexpr double kMost = 1048576.0;
  const double v = (double)delta * (double)A * 1.4426950408889634074;
  return v < -kMost ? -kMost : v > kMost ? kMost : v;
}
// sum of v over this lane and those before it
__device__ __forceinline__ double scan_up(double v) {
  const int lane = threadIdx.x % 64;
#pragma unroll
  for (int off = 1; off < 64; off <<= 1) {
    const double o = __shfl_up(v, off, 64);
    if (lane >= off) v += o;
  }
  return v;
}

constexpr int kStateThreads = 512;
constexpr int kStatePiece = 64;

// SPLIT: the operands are fp16 data as they are (one plane each), V's two bf16
// parts are made here; else they are planes of bf16 parts.
template <int N, int HB, int UP, int VP, bool SPLIT>
struct StateLds {
  float w[HB][256];
  float wave[2][4];
  float decay[HB];
  int first[4], count[4];
  __attribute__((aligned(16))) uint16_t u[2][3][kStatePiece * 64];
  __attribute__((aligned(16))) uint16_t v[SPLIT ? 2 : VP][N / 32][kStatePiece * 32];
};

// uv, vv: views of the planes from the chunk's first row on (rows past it read as
// zeros); the heads' columns start 64 channels apart.  uv ends with the columns of
// the last of `heads` in the last row.  Heads past `heads` are worked on and not
// stored: w (LDS) is 0 for them, as for rows past the chunk, and their u is what
// follows in the same plane, the next row's columns, or zeros behind the view's
// end.  store(hb, at, v) takes NT
// pieces of 4 elements of head hb's (64, N) at at, at + 16 ..
template <int IO, int N, int HB, int UP, int VP, bool SPLIT, class Store>
__device__ __forceinline__ void chunk_states(StateLds<N, HB, UP, VP, SPLIT>& lds, const __amdgpu_buffer_rsrc_t (&uv)[UP],
                                             int64_t urow, const __amdgpu_buffer_rsrc_t (&vv)[VP], int64_t vrow,
                                             int rows, int heads, Store store) {
  constexpr int NT = N / 32;  // state tiles of a wave
  constexpr int kV = SPLIT ? 2 : VP, kVItems = kStatePiece * N / 8, kVPer = (kVItems + kStateThreads - 1) / kStateThreads;
  const int tid = threadIdx.x, lane = tid % 64, wave = tid / 64, pt = wave % 4, nh = wave / 4;
  u32x4v ur[HB][UP], vr[VP][kVPer];
  auto load_u = [&](int hb, int j0) {
#pragma unroll
    for (int i = 0; i < UP; ++i)
      ur[hb][i] = vload16(uv[i], (uint32_t)((j0 + tid / 8) * urow * 2 + hb * 128 + (tid % 8) * 16));
  };
  auto load_v = [&](int j0) {
#pragma unroll
    for (int i = 0; i < VP; ++i)
#pragma unroll
      for (int k = 0; k < kVPer; ++k) {
        const int item = tid + kStateThreads * k;
        vr[i][k] = vload16(vv[i], kVItems % kStateThreads == 0 || item < kVItems
                                      ? (uint32_t)((j0 + item / (N / 8)) * vrow * 2 + (item % (N / 8)) * 16)
                                      : kOffNone);
      }
  };
  // w u of head hb, for the piece its registers hold
  auto stage = [&](int hb, int j0, int turn) {
    const int row = tid / 8;
    const float w = lds.w[hb][j0 + row];
    u32x4v part[3];
#pragma unroll
    for (int e = 0; e < 4; ++e) {
      float a, b;
      if constexpr (SPLIT) {
        a = low16<IO>(ur[hb][0][e]);
        b = high16<IO>(ur[hb][0][e]);
      } else {
        a = __uint_as_float(ur[hb][UP - 1][e] << 16);
        b = __uint_as_float(ur[hb][UP - 1][e] & 0xffff0000u);
#pragma unroll
        for (int i = UP - 2; i >= 0; --i) {
          a += __uint_as_float(ur[hb][i][e] << 16);
          b += __uint_as_float(ur[hb][i][e] & 0xffff0000u);
        }
      }
      uint32_t v[3];
      split3(a * w, b * w, v);
#pragma unroll
      for (int i = 0; i < 3; ++i) part[i][e] = v[i];
    }
#pragma unroll
    for (int i = 0; i < 3; ++i)
      *reinterpret_cast<u32x4v*>(&lds.u[turn][i][tm_off<64>(row, 8 * (tid % 8))]) = part[i];
  };
  load_v(0);
#pragma unroll
  for (int hb = 0; hb < HB; ++hb) load_u(hb, 0);

  const int uo[2] = {tm_lane_off<64>(16 * pt, 0, lane), tm_lane_off<64>(16 * pt, 1, lane)};
  const int vo[2][2] = {{tm_lane_off<32>(0, 0, lane), tm_lane_off<32>(0, 1, lane)},
                        {tm_lane_off<32>(16, 0, lane), tm_lane_off<32>(16, 1, lane)}};
  f32x4 acc[HB][NT];
#pragma unroll
  for (int hb = 0; hb < HB; ++hb)
#pragma unroll
    for (int t = 0; t < NT; ++t) acc[hb][t] = f32x4{0.0f, 0.0f, 0.0f, 0.0f};
  __syncthreads();  // the weights are there
  stage(0, 0, 0);
  load_u(0, kStatePiece);
  int turn = 0;
  for (int j0 = 0; j0 < rows; j0 += kStatePiece) {
    const bool more = j0 + kStatePiece < rows;
    __syncthreads();  // the last piece's V is used up
#pragma unroll
    for (int k = 0; k < kVPer; ++k) {
      const int item = tid + kStateThreads * k;
      if (kVItems % kStateThreads == 0 || item < kVItems) {
        const int s = item / (N / 8), n = 8 * (item % (N / 8)), at = tm_off<32>(s, n % 32);
        if constexpr (SPLIT) {
          u32x4v hi, lo;
          split8<IO>(vr[0][k], hi, lo);
          *reinterpret_cast<u32x4v*>(&lds.v[0][n / 32][at]) = hi;
          *reinterpret_cast<u32x4v*>(&lds.v[kV - 1][n / 32][at]) = lo;
        } else {
#pragma unroll
          for (int i = 0; i < VP; ++i) *reinterpret_cast<u32x4v*>(&lds.v[i][n / 32][at]) = vr[i][k];
        }
      }
    }
    load_v(j0 + kStatePiece);  // past the rows: zeros, no memory is read
    __syncthreads();
#pragma unroll
    for (int hb = 0; hb < HB; ++hb) {
      // the next step's operand is made while this one's is multiplied
#pragma unroll
      for (int ks = 0; ks < kStatePiece; ks += 32) {
        bf16x8 up[3];  // [k = step][n = channel]
#pragma unroll
        for (int i = 0; i < 3; ++i) up[i] = bfv(tm_frag(&lds.u[turn][i][ks * 64], uo[0], uo[1]));
#pragma unroll
        for (int j = 0; j < kV; ++j) {
          bf16x8 vp[NT];  // [m = state][k = step]
#pragma unroll
          for (int t = 0; t < NT; ++t) {
            const int nt = NT * nh + t;
            vp[t] = bfv(tm_frag(&lds.v[j][nt / 2][ks * 32], nt & 1 ? vo[1][0] : vo[0][0], nt & 1 ? vo[1][1] : vo[0][1]));
          }
#pragma unroll
          for (int i = 2 - j; i >= 0; --i)
#pragma unroll
            for (int t = 0; t < NT; ++t) acc[hb][t] = BF::run(vp[t], up[i], acc[hb][t]);
        }
      }
      if (hb + 1 < HB) {
        stage(hb + 1, j0, turn ^ 1);
        load_u(hb + 1, j0 + kStatePiece);
        __syncthreads();
      } else if (more) {
        stage(0, j0 + kStatePiece, turn ^ 1);
        load_u(0, j0 + 2 * kStatePiece);
      }
      turn ^= 1;
    }
  }
#pragma unroll
  for (int hb = 0; hb < HB; ++hb)
    if (hb < heads) store(hb, (16 * pt + lane % 16) * N + 16 * NT * nh + 4 * (lane / 16), acc[hb]);
}

}  // namespace ss
