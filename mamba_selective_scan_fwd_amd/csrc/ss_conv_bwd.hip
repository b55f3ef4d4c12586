// ss_conv_bwd.hip -- gradients of the depthwise causal conv1d + SiLU (gfx950).
//
// Of the convolution of ss_conv.hip (page "Mamba" (walkthrough), Part IV
// Stage 2), pre[t] = bias + sum_k w[k] x[t-W+1+k], out = silu(pre):
//   dpre[t]  = dout[t] s (1 + pre (1 - s)),  s = sigmoid(pre[t])
//   dx[t]    = sum_{m<W} w[W-1-m] dpre[t+m]
//   dw[k]    = sum_{b,t} dpre[t] x[t-W+1+k],  dbias = sum_{b,t} dpre[t]
// with the same document resets and window before the row as the forward
// ("niverel-mamba" README, "seq_idx strict reset"); the window's gradient is
// dx continued to t < 0, and a gradient of conv_final is added to the inputs
// it holds.  pre is rebuilt from x.
//
// A streaming stencil (x, dout and dx once each), bound by HBM and by the vector
// units about alike (8 x 1536 rows of 2048 bf16 steps: 37 us, 4.1 TB/s, the
// latter busy for three quarters of it; 16 steps a thread, which rebuild less,
// take 39): a thread
// covers 8 consecutive steps of one row, takes 4 inputs before and 4 inputs
// and gradients behind them from the neighbours' lines (L1 hits), and rebuilds
// pre for its 8 steps and the W - 1 behind.  Rows begin at any element, so the
// 16-byte accesses are unaligned ones where a row's length is odd; only a
// chunk that a row's end cuts goes element by element.  The 256 chunks of 8
// steps of a unit run over the batch rows of one channel, short rows too.
// dw and dbias: each workgroup sums its units in registers, then over its
// threads, and leaves one partial sum per (channel, part); a second kernel
// adds the parts in order, so results do not depend on timing.
#include <string.h>

#include "ss_device.h"
#include "ss_internal.h"

namespace ss {
namespace {

constexpr int kBwdThreads = 256;
constexpr int kPer = 8;

template <int IO, int M>
__device__ __forceinline__ void load_run(const void* base, int64_t at, float* v) {  // M consecutive elements
  if constexpr (IO == SS_F32) {
    memcpy(v, static_cast<const float*>(base) + at, 4 * M);
  } else {
    uint32_t w[M / 2];
    memcpy(w, static_cast<const uint16_t*>(base) + at, 2 * M);
#pragma unroll
    for (int i = 0; i < M / 2; ++i) {
      v[2 * i] = bits_f32<IO>((raw_t<IO>)(w[i] & 0xffffu));
      v[2 * i + 1] = bits_f32<IO>((raw_t<IO>)(w[i] >> 16));
    }
  }
}

template <int IO, int W, bool SEQ>
__global__ void __launch_bounds__(kBwdThreads) conv1d_bwd_kernel(ConvBwdParams p) {
  const int tid = threadIdx.x, lane = tid % 64, wave = tid / 64;
  const int part = (int)(blockIdx.x % (uint32_t)p.parts);
  const int d = (int)(blockIdx.x / (uint32_t)p.parts);
  const int L = (int)p.seqlen, nc = (L + kPer - 1) / kPer;
  float w[W];
#pragma unroll
  for (int k = 0; k < W; ++k) w[k] = p.w[(int64_t)d * W + k];
  const float bias = p.bias ? p.bias[d] : 0.0f;
  float dw[W], db = 0.0f;
#pragma unroll
  for (int k = 0; k < W; ++k) dw[k] = 0.0f;

  for (int64_t unit = part; unit < p.units; unit += p.parts) {
    const int64_t c = unit * kBwdThreads + tid;  // chunk of the channel: batch row c / nc
    if (c >= p.batch * nc) break;
    const int64_t b = p.batch * (int64_t)nc < ((int64_t)1 << 31) ? (int64_t)((uint32_t)c / (uint32_t)nc) : c / nc;
    const int t0 = (int)(c - b * nc) * kPer;
    const int64_t row = b * p.dim + d, at = row * p.seqlen + t0;
    // v[i] holds step t0 - 4 + i
    float x[16], dy[12];
    uint32_t id[16];
    const int32_t* idrow = SEQ ? p.seq_idx + b * p.seqlen : nullptr;
    const bool whole = t0 + 8 <= L, more = t0 + 12 <= L, last = t0 + 8 >= L;
    if (whole && (more || last)) {
      load_run<IO, 8>(p.x, at, x + 4);
      load_run<IO, 8>(p.dout, at, dy);
      load_run<IO, 4>(p.x, t0 ? at - 4 : at, x);
      load_run<IO, 4>(p.x, more ? at + 8 : at, x + 12);
      load_run<IO, 4>(p.dout, more ? at + 8 : at, dy + 8);
      if constexpr (SEQ) {
        memcpy(id + 4, idrow + t0, 32);
        memcpy(id, idrow + (t0 ? t0 - 4 : t0), 16);
        memcpy(id + 12, idrow + (more ? t0 + 8 : t0), 16);
      }
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        x[i] = t0 ? x[i] : 0.0f;
        x[12 + i] = more ? x[12 + i] : 0.0f;
        dy[8 + i] = more ? dy[8 + i] : 0.0f;
      }
    } else {
#pragma unroll
      for (int i = 0; i < 16; ++i) {
        const int t = t0 - 4 + i;
        const bool in = t >= 0 && t < L;
        x[i] = in ? load_io<IO>(p.x, at - 4 + i) : 0.0f;
        if constexpr (SEQ) id[i] = in ? (uint32_t)idrow[t] : 0u;
        if (i >= 4) dy[i - 4] = in ? load_io<IO>(p.dout, at - 4 + i) : 0.0f;
      }
    }
    uint32_t first_id = 0, last_id = 0;
    if constexpr (SEQ) {
      first_id = (uint32_t)idrow[0];
      last_id = (uint32_t)idrow[L - 1];
    }
    // the window before the row: steps -1, -2, .. in x[3], x[2], .. of the row's first chunk
    if (W > 1 && t0 == 0 && p.conv_init) {
#pragma unroll
      for (int m = 0; m < W - 1; ++m) x[4 - (W - 1) + m] = p.conv_init[row * (W - 1) + m];
    }
    // input src = t0 - 4 + i reaches step t0 - 4 + j: of the same document (the
    // window belongs to the first)
    auto meets = [&](int i, int j) {
      if constexpr (SEQ) {
        const uint32_t a = t0 - 4 + i < 0 ? first_id : id[i];
        return a == id[j];
      }
      return true;
    };
    float dpre[kPer + W - 1];
#pragma unroll
    for (int e = 0; e < kPer + W - 1; ++e) {
      float pre = bias;
#pragma unroll
      for (int k = 0; k < W; ++k) {
        const int i = 4 + e - (W - 1) + k;
        pre = fmaf(w[k], k == W - 1 || meets(i, 4 + e) ? x[i] : 0.0f, pre);
      }
      float g = dy[e];
      if (p.silu) {
        const float s = sigmoid_f(pre);
        g *= s * fmaf(pre, 1.0f - s, 1.0f);
      }
      dpre[e] = g;
    }
    // Steps behind the row's end have no gradient, whatever their pre is: other
    // weights meet the last inputs there, and it may be infinite where the row's own
    // are not.
    if (t0 + kPer + W - 1 > L) {
#pragma unroll
      for (int e = 0; e < kPer + W - 1; ++e) dpre[e] = t0 + e < L ? dpre[e] : 0.0f;
    }
#pragma unroll
    for (int e = 0; e < kPer; ++e) {
      db += dpre[e];
#pragma unroll
      for (int k = 0; k < W; ++k) {
        const int i = 4 + e - (W - 1) + k;
        dw[k] = fmaf(dpre[e], k == W - 1 || meets(i, 4 + e) ? x[i] : 0.0f, dw[k]);
      }
    }
    float dx[kPer];
#pragma unroll
    for (int e = 0; e < kPer; ++e) {
      float v = 0.0f;
#pragma unroll
      for (int m = 0; m < W; ++m)
        v = fmaf(w[W - 1 - m], m == 0 || meets(4 + e, 4 + e + m) ? dpre[e + m] : 0.0f, v);
      dx[e] = v;
    }
    if constexpr (W > 1) {
      if (p.dconv_final && t0 + kPer > L - (W - 1)) {
#pragma unroll
        for (int e = 0; e < kPer; ++e) {
          const int j = t0 + e - (L - (W - 1));  // entry of conv_final that holds step t0 + e
          if (j >= 0 && j < W - 1 && (!SEQ || id[4 + e] == last_id))
            dx[e] += p.dconv_final[row * (W - 1) + j];
        }
      }
      if (p.dconv_init && t0 == 0) {
#pragma unroll
        for (int m = 0; m < W - 1; ++m) {  // the window's entry m is step m - (W - 1)
          float v = 0.0f;
#pragma unroll
          for (int t = 0; t <= m; ++t)
            if (meets(4 - (W - 1) + m, 4 + t)) v = fmaf(w[m - t], dpre[t], v);
          const int j = m - L;  // a row shorter than the window keeps the entry in conv_final
          if (p.dconv_final && j >= 0 && (!SEQ || last_id == first_id)) v += p.dconv_final[row * (W - 1) + j];
          p.dconv_init[row * (W - 1) + m] = v;
        }
      }
    }
    if (whole) {
      if constexpr (IO == SS_F32) {
        memcpy(static_cast<float*>(p.dx) + at, dx, 32);
      } else {
        uint32_t o[4];
#pragma unroll
        for (int i = 0; i < 4; ++i)
          o[i] = (uint32_t)__builtin_bit_cast(uint16_t, from_f32<IO>(dx[2 * i])) |
                 ((uint32_t)__builtin_bit_cast(uint16_t, from_f32<IO>(dx[2 * i + 1])) << 16);
        memcpy(static_cast<uint16_t*>(p.dx) + at, o, 16);
      }
    } else {
#pragma unroll
      for (int e = 0; e < kPer; ++e)
        if (t0 + e < L) store_io<IO>(p.dx, at + e, dx[e]);
    }
  }

  // sums over the workgroup's threads
  __shared__ float s_sum[4][W + 1];
#pragma unroll
  for (int k = 0; k <= W; ++k) {
    float v = k < W ? dw[k < W ? k : 0] : db;
    v = row_sum(v);
    v += __shfl_xor(v, 16, 64);
    v += __shfl_xor(v, 32, 64);
    if (lane == 0) s_sum[wave][k] = v;
  }
  __syncthreads();
  if (tid <= W) {
    const float v = (s_sum[0][tid] + s_sum[1][tid]) + (s_sum[2][tid] + s_sum[3][tid]);
    if (p.parts > 1) p.ws[((int64_t)part * p.dim + d) * (W + 1) + tid] = v;
    else if (tid < W) p.dw[(int64_t)d * W + tid] = v;
    else if (p.dbias) p.dbias[d] = v;
  }
}

// the parts of every (channel, entry) added in order
template <int W>
__global__ void __launch_bounds__(kBwdThreads) conv1d_bwd_sum_kernel(ConvBwdParams p) {
  const int64_t i = (int64_t)blockIdx.x * kBwdThreads + threadIdx.x, n = p.dim * (W + 1);
  if (i >= n) return;
  float v = 0.0f;
  for (int q = 0; q < p.parts; ++q) v += p.ws[q * n + i];
  const int64_t d = i / (W + 1);
  const int k = (int)(i - d * (W + 1));
  if (k < W) p.dw[d * W + k] = v;
  else if (p.dbias) p.dbias[d] = v;
}

template <int IO, int W>
hipError_t launch_w(const ConvBwdParams& p, hipStream_t st) {
  const dim3 grid((uint32_t)(p.dim * p.parts));
  if (p.seq_idx) hipLaunchKernelGGL((conv1d_bwd_kernel<IO, W, true>), grid, dim3(kBwdThreads), 0, st, p);
  else hipLaunchKernelGGL((conv1d_bwd_kernel<IO, W, false>), grid, dim3(kBwdThreads), 0, st, p);
  const hipError_t e = hipGetLastError();
  if (e != hipSuccess || p.parts == 1) return e;
  hipLaunchKernelGGL((conv1d_bwd_sum_kernel<W>), dim3((uint32_t)((p.dim * (W + 1) + kBwdThreads - 1) / kBwdThreads)),
                     dim3(kBwdThreads), 0, st, p);
  return hipGetLastError();
}
template <int IO>
hipError_t launch_io(const ConvBwdParams& p, hipStream_t st) {
  switch (p.width) {
    case 1: return launch_w<IO, 1>(p, st);
    case 2: return launch_w<IO, 2>(p, st);
    case 3: return launch_w<IO, 3>(p, st);
    default: return launch_w<IO, 4>(p, st);
  }
}

}  // namespace

// units of 256 chunks of 8 steps of one channel
int64_t conv_bwd_units(int64_t batch, int64_t seqlen) {
  return (batch * ((seqlen + kPer - 1) / kPer) + kBwdThreads - 1) / kBwdThreads;
}

hipError_t launch_conv_bwd(const ConvBwdParams& p, hipStream_t st) {
  switch (p.io) {
    case SS_F32: return launch_io<SS_F32>(p, st);
    case SS_F16: return launch_io<SS_F16>(p, st);
    default: return launch_io<SS_BF16>(p, st);
  }
}

}  // namespace ss
