// ss_serve.hip -- the convolution of packed prompts, and a Mamba-2 layer's
// decode step over a pool of state slots (gfx950).
//
// Page "Mamba" (walkthrough), Part IV Stage 2: out[t,d] = silu(bias[d] +
// sum_{k<W} w[d,k] x[t-W+1+k,d]), here with the channels innermost, as the
// input projection writes them, over the packed prompts of a serving batch.
// Page "Mamba" (walkthrough), "Deep dive: Mamba-2 and state-space duality",
// one step of head h (state H[p][n]):
//   H <- exp(Delta A) H + Delta x B^T,  y = (H C + D x) silu(z),
// x, B and C being the convolved channels of the token.
#include "ss_device.h"
#include "ss_internal.h"
#include "ss_packed.h"

namespace ss {
namespace {

// ---- causal conv1d + SiLU of packed prompts ---------------------------------
// A streaming stencil, bound by HBM.  A wave takes a chunk of 16 rows of one
// sequence and 64 times 4 bytes of channels (two 16-bit ones, which need 4-byte
// rows, or one); a lane loads its 16 rows and the W - 1 rows before them at once
// and walks down the rows.  Four bytes a lane, not more: with 16 the weights and
// rows take 142 registers and a quarter of the waves (37 ragged prompts, 16,021
// rows of 5376 fp16 channels: 74 us, 78 with 8 bytes a lane, 86 with 16; fp32
// 139 against 142; one prompt of 2048 rows of 1792 channels 6.0, 7.4 and 10.0
// us), with 2 bytes the large sizes take 75 us; chunks of 8 and 32 rows take 75
// and 76 us.  74 us are 4.75 TB/s.  A workgroup's four waves have
// the same channels of four chunks in a row, so that they share the weights and
// the rows before a chunk in L1.
// The chunk that holds a sequence's first rows reads the slot's window and,
// having read it, writes the new one: no other wave touches these channels of
// the slot, so the update is in place.
constexpr int kLogRows = 4;
constexpr int kRows = 1 << kLogRows;

template <int IO, int VEC>
__device__ __forceinline__ uint32_t load_row(__amdgpu_buffer_rsrc_t r, uint32_t off) {  // the raw bits of VEC channels
  if constexpr (VEC == 1) return bload<IO>(r, off);
  else return __builtin_amdgcn_raw_buffer_load_b32(r, off, 0, 0);
}
template <int IO>
__device__ __forceinline__ float channel(uint32_t a, int e) {
  if constexpr (IO == SS_F32)
    return __uint_as_float(a);
  else
    return bits_f32<IO>((raw_t<IO>)((a >> (16 * e)) & 0xffffu));
}

template <int IO, int W, int VEC>
__global__ void __launch_bounds__(256) conv1d_prompt_kernel(ConvPromptParams p) {
  constexpr int s = (int)io_bytes<IO>();
  const int lane = threadIdx.x % 64;
  const int blocks = ((p.tokens >> kLogRows) + p.nseqs + 3) / 4;  // of the same channels
  const int vb = (int)(blockIdx.x / (uint32_t)blocks);
  const int place = uniform((int)(blockIdx.x - (uint32_t)(vb * blocks)) * 4 + (int)threadIdx.x / 64);
  if (place >= (p.tokens >> kLogRows) + p.nseqs) return;
  const SeqChunk q = find_chunk<kLogRows>(p.cu, p.nseqs, p.tokens, place);
  if (q.chunk < 0 || (q.chunk > 0 && q.chunk * kRows >= q.len)) return;
  const int c0 = (vb * 64 + lane) * VEC;  // first channel of this lane
  if (c0 >= p.dim) return;
  const int row0 = q.begin + q.chunk * kRows;
  const int left = q.len - q.chunk * kRows, rows = left < kRows ? left : kRows;

  // this chunk's rows, and the W - 1 before it inside the sequence; a row past
  // the chunk reads as zeros through the range check
  const auto xv = make_rsrc(static_cast<const char*>(p.x) + row0 * p.x_stride * s,
                            rows > 0 ? (uint32_t)(((rows - 1) * p.x_stride + p.dim) * s) : 0u);
  const uint32_t co = (uint32_t)(c0 * s), rb = (uint32_t)(p.x_stride * s);
  uint32_t cur[kRows];
#pragma unroll
  for (int r = 0; r < kRows; ++r) cur[r] = load_row<IO, VEC>(xv, r < rows ? r * rb + co : kOffNone);

  float w[VEC][W], bias[VEC];
#pragma unroll
  for (int e = 0; e < VEC; ++e) {
    bias[e] = p.bias ? p.bias[c0 + e] : 0.0f;
#pragma unroll
    for (int k = 0; k < W; ++k) w[e][k] = p.w[(int64_t)(c0 + e) * W + k];
  }
  float prev[W > 1 ? W - 1 : 1][VEC];  // the W - 1 inputs before the next row, oldest first
  if constexpr (W > 1) {
    if (q.chunk > 0) {  // all of them inside the sequence (a chunk is longer than a window)
      const auto hv = make_rsrc(static_cast<const char*>(p.x) + (row0 - (W - 1)) * p.x_stride * s,
                                (uint32_t)(((W - 2) * p.x_stride + p.dim) * s));
#pragma unroll
      for (int k = 0; k < W - 1; ++k) {
        const uint32_t a = load_row<IO, VEC>(hv, k * rb + co);
#pragma unroll
        for (int e = 0; e < VEC; ++e) prev[k][e] = channel<IO>(a, e);
      }
    } else {
      const int slot = uniform(slot_of(p.slots, q.seq, p.nslots));
      float* win = p.conv_state + ((int64_t)(slot < 0 ? 0 : slot) * p.dim + c0) * (W - 1);
      const bool carried = slot >= 0 && p.has_state && p.has_state[q.seq] != 0;
#pragma unroll
      for (int k = 0; k < W - 1; ++k)
#pragma unroll
        for (int e = 0; e < VEC; ++e) prev[k][e] = carried ? win[e * (W - 1) + k] : 0.0f;
      if (slot >= 0) {
        // the window behind the sequence's last row: its last W - 1 inputs,
        // of the old window where the sequence is shorter
        const char* xs = static_cast<const char*>(p.x) + (int64_t)q.begin * p.x_stride * s;
#pragma unroll
        for (int k = 0; k < W - 1; ++k) {
          const int r = q.len - (W - 1) + k;  // row of the sequence; below 0: old window entry W - 1 + r
          float v[VEC];
          if (r >= 0) {
            const auto one = make_rsrc(xs + r * p.x_stride * s, (uint32_t)(p.dim * s));
            const uint32_t a = load_row<IO, VEC>(one, co);
#pragma unroll
            for (int e = 0; e < VEC; ++e) v[e] = channel<IO>(a, e);
          } else {
#pragma unroll
            for (int e = 0; e < VEC; ++e) {
              v[e] = 0.0f;
#pragma unroll
              for (int m = 0; m < W - 1; ++m) v[e] = m == W - 1 + r ? prev[m][e] : v[e];
            }
          }
#pragma unroll
          for (int e = 0; e < VEC; ++e) win[e * (W - 1) + k] = v[e];
        }
      }
    }
  }

  // straight through all rows, those past the chunk dropped by the range check: a
  // branch per row would make every wait one for the stores too
  const auto ov = make_rsrc(static_cast<char*>(p.out) + (int64_t)row0 * p.out_stride * s,
                            rows > 0 ? (uint32_t)(((rows - 1) * p.out_stride + p.dim) * s) : 0u);
  const uint32_t ob = (uint32_t)(p.out_stride * s);
#pragma unroll
  for (int r = 0; r < kRows; ++r) {
    float x[VEC], y[VEC];
#pragma unroll
    for (int e = 0; e < VEC; ++e) x[e] = channel<IO>(cur[r], e);
#pragma unroll
    for (int e = 0; e < VEC; ++e) {
      float pre = bias[e];
#pragma unroll
      for (int j = 0; j < W - 1; ++j) pre = fmaf(w[e][j], prev[j][e], pre);
      pre = fmaf(w[e][W - 1], x[e], pre);
      y[e] = p.silu ? pre * sigmoid_f(pre) : pre;
    }
    if constexpr (W > 1) {
#pragma unroll
      for (int e = 0; e < VEC; ++e) {
#pragma unroll
        for (int j = 0; j + 1 < W - 1; ++j) prev[j][e] = prev[j + 1][e];
        prev[W - 2][e] = x[e];
      }
    }
    const uint32_t at = r < rows ? r * ob + co : kOffNone;
    if constexpr (VEC == 1) {
      bstore<IO>(ov, at, y[0]);
    } else {
      const uint32_t o = (uint32_t)__builtin_bit_cast(uint16_t, from_f32<IO>(y[0])) |
                         ((uint32_t)__builtin_bit_cast(uint16_t, from_f32<IO>(y[VEC - 1])) << 16);
      __builtin_amdgcn_raw_buffer_store_b32(o, ov, at, 0, 0);
    }
  }
}

template <int IO, int W, int VEC>
hipError_t launch_conv_prompt_vec(const ConvPromptParams& p, hipStream_t st) {
  const int64_t vecs = ((p.dim + VEC - 1) / VEC + 63) / 64, blocks = ((p.tokens >> kLogRows) + p.nseqs + 3) / 4;
  hipLaunchKernelGGL((conv1d_prompt_kernel<IO, W, VEC>), dim3((uint32_t)(vecs * blocks)), dim3(256), 0, st, p);
  return hipGetLastError();
}
template <int IO, int W>
hipError_t launch_conv_prompt_w(const ConvPromptParams& p, hipStream_t st) {
  if constexpr (IO != SS_F32)
    if (p.pairs) return launch_conv_prompt_vec<IO, W, 2>(p, st);
  return launch_conv_prompt_vec<IO, W, 1>(p, st);
}
template <int IO>
hipError_t launch_conv_prompt_io(const ConvPromptParams& p, hipStream_t st) {
  switch (p.width) {
    case 1: return launch_conv_prompt_w<IO, 1>(p, st);
    case 2: return launch_conv_prompt_w<IO, 2>(p, st);
    case 3: return launch_conv_prompt_w<IO, 3>(p, st);
    default: return launch_conv_prompt_w<IO, 4>(p, st);
  }
}

// ---- decode step of a Mamba-2 layer ---------------------------------------------
// Two kernels.  The heads of a group share B and C, so a head's workgroup
// cannot update their windows while others still read them: the convolution
// (a thread per channel) runs first and leaves the convolved channels in fp32,
// then every (row, head) updates its own state.  fp32 arithmetic throughout.
template <int IO, int W>
__global__ void __launch_bounds__(256) ssd_step_conv_kernel(SsdStepParams p) {
  const int blocks = (p.channels + 255) / 256;
  const int r = (int)(blockIdx.x / (uint32_t)blocks);
  const int c = (int)(blockIdx.x - (uint32_t)(r * blocks)) * 256 + (int)threadIdx.x;
  const int slot = uniform(slot_of(p.slots, r, p.nslots));
  if (slot < 0 || c >= p.channels) return;
  float win[W];
  float* st = p.conv_state + ((int64_t)slot * p.channels + c) * (W - 1);
#pragma unroll
  for (int k = 0; k < W - 1; ++k) win[k] = st[k];
  win[W - 1] = load_io<IO>(p.xbc, (int64_t)r * p.xbc_stride + c);
  float pre = p.conv_bias ? p.conv_bias[c] : 0.0f;
#pragma unroll
  for (int k = 0; k < W; ++k) pre = fmaf(p.conv_w[(int64_t)c * W + k], win[k], pre);
  p.ws_xbc[(int64_t)r * p.channels + c] = silu_f(pre);
#pragma unroll
  for (int k = 0; k < W - 1; ++k) st[k] = win[k + 1];
}

// Workgroup = (row, head): the head's 64 x N state is one contiguous slab,
// read and written once, which is what bounds the kernel (HBM: 61 requests of 24
// heads, state 128: 15.4-17 us, 5.7-6.2 TB/s, part of it from the last level cache; 201
// of 80 heads, state 64: 104 us, 5.2 TB/s).  8 lanes share
// a row p of the state, lane j of them holding the 4 states 4 j + 32 m ..: a
// load instruction covers whole 128-byte lines of 8 rows, every load is issued
// before the first use, and H C is a sum over 8 lanes (three DPP steps).
template <int CTRL>
__device__ __forceinline__ float dpp_add(float v) {
  return v + __int_as_float(__builtin_amdgcn_update_dpp(0, __float_as_int(v), CTRL, 0xf, 0xf, true));
}

template <int IO, int N>
__global__ void __launch_bounds__(256) ssd_step_state_kernel(SsdStepParams p) {
  constexpr int J = N / 32;
  const int tid = threadIdx.x, l8 = tid % 8;
  const int r = (int)(blockIdx.x / (uint32_t)p.nheads);
  const int h = (int)(blockIdx.x - (uint32_t)(r * p.nheads));
  const int slot = uniform(slot_of(p.slots, r, p.nslots));
  if (slot < 0) return;
  float* H = p.state + ((int64_t)slot * p.nheads + h) * (64 * N) + (tid / 8) * N + 4 * l8;
  float4 st[2][J];
#pragma unroll
  for (int q = 0; q < 2; ++q)
#pragma unroll
    for (int j = 0; j < J; ++j) st[q][j] = *reinterpret_cast<const float4*>(H + q * 32 * N + 32 * j);
  const int g = h / (p.nheads / p.ngroups);
  const float* row = p.ws_xbc + (int64_t)r * p.channels;
  const float* Bp = row + p.nheads * 64 + g * N + 4 * l8;
  const float* Cp = Bp + p.ngroups * N;
  float4 b[J], c[J];
#pragma unroll
  for (int j = 0; j < J; ++j) {
    b[j] = *reinterpret_cast<const float4*>(Bp + 32 * j);
    c[j] = *reinterpret_cast<const float4*>(Cp + 32 * j);
  }
  float x[2], zg[2] = {0.0f, 0.0f};
#pragma unroll
  for (int q = 0; q < 2; ++q) {
    const int ch = h * 64 + 32 * q + tid / 8;
    x[q] = row[ch];
    if (p.z) zg[q] = load_io<IO>(p.z, r * p.z_stride + ch);
  }
  const float xd = load_io<IO>(p.dt, r * p.dt_stride + h) + (p.dt_bias ? p.dt_bias[h] : 0.0f);
  const float delta = p.softplus ? softplus_f(xd) : xd;
  const float a = exp2_hw(delta * p.A[h] * kLog2e);
  const float Dh = p.D ? p.D[h] : 0.0f;
#pragma unroll
  for (int q = 0; q < 2; ++q) {
    const float dx = delta * x[q];
    float y = 0.0f;
#pragma unroll
    for (int j = 0; j < J; ++j) {
      float4 v = st[q][j];
      v.x = fmaf(a, v.x, dx * b[j].x);
      v.y = fmaf(a, v.y, dx * b[j].y);
      v.z = fmaf(a, v.z, dx * b[j].z);
      v.w = fmaf(a, v.w, dx * b[j].w);
      *reinterpret_cast<float4*>(H + q * 32 * N + 32 * j) = v;
      y = fmaf(v.x, c[j].x, y);
      y = fmaf(v.y, c[j].y, y);
      y = fmaf(v.z, c[j].z, y);
      y = fmaf(v.w, c[j].w, y);
    }
    y = dpp_add<0xB1>(y);   // quad_perm: lane ^ 1
    y = dpp_add<0x4E>(y);   // quad_perm: lane ^ 2
    y = dpp_add<0x141>(y);  // row_half_mirror: the other quad of the 8 lanes
    y = fmaf(Dh, x[q], y);
    if (p.z) y *= silu_f(zg[q]);
    if (l8 == 0) store_io<IO>(p.y, ((int64_t)r * p.nheads + h) * 64 + 32 * q + tid / 8, y);
  }
}

template <int IO>
hipError_t launch_ssd_step_io(const SsdStepParams& p, hipStream_t st) {
  const dim3 cgrid((uint32_t)((int64_t)p.rows * ((p.channels + 255) / 256)));
  switch (p.width) {
    case 1: hipLaunchKernelGGL((ssd_step_conv_kernel<IO, 1>), cgrid, dim3(256), 0, st, p); break;
    case 2: hipLaunchKernelGGL((ssd_step_conv_kernel<IO, 2>), cgrid, dim3(256), 0, st, p); break;
    case 3: hipLaunchKernelGGL((ssd_step_conv_kernel<IO, 3>), cgrid, dim3(256), 0, st, p); break;
    default: hipLaunchKernelGGL((ssd_step_conv_kernel<IO, 4>), cgrid, dim3(256), 0, st, p); break;
  }
  const hipError_t e = hipGetLastError();
  if (e != hipSuccess) return e;
  const dim3 sgrid((uint32_t)((int64_t)p.rows * p.nheads));
  switch (p.dstate) {
    case 32: hipLaunchKernelGGL((ssd_step_state_kernel<IO, 32>), sgrid, dim3(256), 0, st, p); break;
    case 64: hipLaunchKernelGGL((ssd_step_state_kernel<IO, 64>), sgrid, dim3(256), 0, st, p); break;
    case 96: hipLaunchKernelGGL((ssd_step_state_kernel<IO, 96>), sgrid, dim3(256), 0, st, p); break;
    default: hipLaunchKernelGGL((ssd_step_state_kernel<IO, 128>), sgrid, dim3(256), 0, st, p); break;
  }
  return hipGetLastError();
}

}  // namespace

hipError_t launch_conv_prompt(const ConvPromptParams& p, hipStream_t st) {
  switch (p.io) {
    case SS_F32: return launch_conv_prompt_io<SS_F32>(p, st);
    case SS_F16: return launch_conv_prompt_io<SS_F16>(p, st);
    default: return launch_conv_prompt_io<SS_BF16>(p, st);
  }
}

hipError_t launch_ssd_step(const SsdStepParams& p, hipStream_t st) {
  return p.io == SS_F16 ? launch_ssd_step_io<SS_F16>(p, st) : launch_ssd_step_io<SS_BF16>(p, st);
}

}  // namespace ss
