// ss_norm.hip -- a token's channels normalised in groups, with a gate or an activation (gfx950).
//
// Per row and group of n channels, u = x, or x silu(z) with the gate first:
//   m = sum(u) / n (0 if not centred),  r = (sum((u - m)^2) / n + eps)^-1/2,
//   v = (u - m) r,  o = v w + b,  y = o, silu(o), or o silu(z) with the gate behind.
// Gradients, with do = dy (dsilu(o) or silu(z)) and dv = do w:
//   dw = sum over rows of do v,  db = sum of do,
//   du = r (dv - sum(dv) / n - v sum(dv v) / n)   (no middle term if not centred),
//   dx = du (silu(z) with the gate first),  dz = dy o dsilu(z) or du x dsilu(z).
// All in fp32; the variance is taken about the mean, in a second sum over
// registers, so that a mean far from zero costs no bits.
//
// Bound by HBM.  A group has `lanes` threads (a power of two), each with one vector
// of its channels in registers, so that a row's data are read once; a thread keeps
// its channels, and their w and b, over all the rows that its workgroup walks, which
// is what dw and db are summed over.  Groups of more than 1024 vectors are walked
// by 1024 threads that read the row once for every sum.
#include "ss_device.h"
#include "ss_internal.h"

namespace ss {
namespace {

// VEC elements of the I/O type as floats
template <int IO, int VEC>
struct Vec {
  static constexpr int kBytes = (IO == SS_F32 ? 4 : 2) * VEC;
  template <int N> struct word;
  __device__ __forceinline__ static void load(const void* base, int64_t i, float (&v)[VEC]) {
    if constexpr (VEC == 1) {
      v[0] = load_io<IO>(base, i);
    } else {
      typedef uint32_t W __attribute__((ext_vector_type(kBytes / 4)));
      const W w = *reinterpret_cast<const W*>(static_cast<const char*>(base) + i * (kBytes / VEC));
      if constexpr (IO == SS_F32) {
#pragma unroll
        for (int e = 0; e < VEC; ++e) v[e] = __uint_as_float(w[e]);
      } else {
#pragma unroll
        for (int e = 0; e < VEC / 2; ++e) {
          v[2 * e] = bits_f32<IO>((raw_t<IO>)(w[e] & 0xffffu));
          v[2 * e + 1] = bits_f32<IO>((raw_t<IO>)(w[e] >> 16));
        }
      }
    }
  }
  __device__ __forceinline__ static void store(void* base, int64_t i, const float (&v)[VEC]) {
    if constexpr (VEC == 1) {
      store_io<IO>(base, i, v[0]);
    } else {
      typedef uint32_t W __attribute__((ext_vector_type(kBytes / 4)));
      W w;
      if constexpr (IO == SS_F32) {
#pragma unroll
        for (int e = 0; e < VEC; ++e) w[e] = __float_as_uint(v[e]);
      } else {
#pragma unroll
        for (int e = 0; e < VEC / 2; ++e)
          w[e] = (uint32_t)__builtin_bit_cast(uint16_t, from_f32<IO>(v[2 * e])) |
                 ((uint32_t)__builtin_bit_cast(uint16_t, from_f32<IO>(v[2 * e + 1])) << 16);
      }
      *reinterpret_cast<W*>(static_cast<char*>(base) + i * (kBytes / VEC)) = w;
    }
  }
};
template <int VEC>
__device__ __forceinline__ void load_weights(const float* w, int c, float other, float (&v)[VEC]) {
#pragma unroll
  for (int e = 0; e < VEC; ++e) v[e] = w ? w[c + e] : other;
}

// sums of a and b over the `lanes` threads of a group; `wave_sums` has 2 floats a wave, twice
__device__ __forceinline__ void group_sums(float& a, float& b, int lanes, float* wave_sums, int& turn) {
  for (int off = (lanes < 64 ? lanes : 64) / 2; off > 0; off >>= 1) {
    a += __shfl_xor(a, off, 64);
    b += __shfl_xor(b, off, 64);
  }
  if (lanes <= 64) return;
  const int wave = (int)threadIdx.x / 64, per = lanes / 64, first = wave / per * per;
  float* at = wave_sums + 32 * turn;
  turn ^= 1;  // the other half is written next: one barrier a sum
  if (threadIdx.x % 64 == 0) {
    at[2 * wave] = a;
    at[2 * wave + 1] = b;
  }
  __syncthreads();
  a = b = 0.0f;
  for (int k = 0; k < per; ++k) {
    a += at[2 * (first + k)];
    b += at[2 * (first + k) + 1];
  }
}

// Thread = (row lane, group of the block, vector of the group)
struct NormPlace {
  int lane, slot, group, row_lane;
  bool in;
};
__device__ __forceinline__ NormPlace norm_place(const NormParams& p) {
  NormPlace q;
  q.lane = (int)threadIdx.x % p.lanes;
  q.slot = (int)threadIdx.x / p.lanes;
  q.group = (int)(blockIdx.x % (uint32_t)p.blocks) * p.block_groups + q.slot % p.block_groups;
  q.row_lane = q.slot / p.block_groups;
  q.in = q.group < p.groups && q.row_lane < p.row_lanes;
  return q;
}

template <int IO, int VEC, bool ONE>
__global__ void __launch_bounds__(1024) group_norm_kernel(NormParams p) {
  using V = Vec<IO, VEC>;
  __shared__ float wave_sums[64];
  const NormPlace q = norm_place(p);
  const int nvec = p.size / VEC, c0 = q.group * p.size;
  int turn = 0;
  float w[VEC], b[VEC], x[VEC], z[VEC];
  const bool mine = q.in && q.lane < nvec;
  if (ONE && mine) {
    load_weights<VEC>(p.w, c0 + VEC * q.lane, 1.0f, w);
    load_weights<VEC>(p.b, c0 + VEC * q.lane, 0.0f, b);
  }
  const bool first = p.mode == SS_NORM_GATE_FIRST, behind = p.mode == SS_NORM_GATE;
  const float inv = 1.0f / (float)p.size;
  // a workgroup's threads take the same number of steps: the sums have barriers
  for (int64_t r0 = (int64_t)(blockIdx.x / (uint32_t)p.blocks) * p.row_lanes; r0 < p.rows;
       r0 += (int64_t)p.row_blocks * p.row_lanes) {
    const int64_t r = r0 + q.row_lane;
    const bool in = q.in && r < p.rows;
    auto fetch = [&](int v) {
      V::load(p.x, r * p.x_stride + c0 + VEC * v, x);
      if (first || behind) V::load(p.z, r * p.z_stride + c0 + VEC * v, z);
    };
    auto input = [&](int e) { return first ? x[e] * silu_f(z[e]) : x[e]; };
    const int v_end = in ? nvec : 0;
    float sum = 0.0f, none = 0.0f, mean = 0.0f;
    if (ONE && q.lane < v_end) fetch(q.lane);
    if (p.center) {
      for (int v = q.lane; v < v_end; v += p.lanes) {
        if (!ONE) fetch(v);
#pragma unroll
        for (int e = 0; e < VEC; ++e) sum += input(e);
      }
      group_sums(sum, none, p.lanes, wave_sums, turn);
      mean = sum * inv;
    }
    float sq = 0.0f;
    for (int v = q.lane; v < v_end; v += p.lanes) {
      if (!ONE) fetch(v);
#pragma unroll
      for (int e = 0; e < VEC; ++e) {
        const float d = input(e) - mean;
        sq = fmaf(d, d, sq);
      }
    }
    group_sums(sq, none, p.lanes, wave_sums, turn);
    const float rstd = rsqrtf(sq * inv + p.eps);
    for (int v = q.lane; v < v_end; v += p.lanes) {
      if (!ONE) {
        fetch(v);
        load_weights<VEC>(p.w, c0 + VEC * v, 1.0f, w);
        load_weights<VEC>(p.b, c0 + VEC * v, 0.0f, b);
      }
      float y[VEC];
#pragma unroll
      for (int e = 0; e < VEC; ++e) {
        const float o = fmaf((input(e) - mean) * rstd, w[e], b[e]);
        y[e] = behind ? o * silu_f(z[e]) : p.mode == SS_NORM_SILU ? silu_f(o) : o;
      }
      V::store(p.y, r * p.y_stride + c0 + VEC * v, y);
    }
  }
}

// Gradients.  Every workgroup leaves its sums of dw and db, over the rows it walks, in
// the workspace: (row block, 2, channels).
template <int IO, int VEC, bool ONE>
__global__ void __launch_bounds__(1024) group_norm_bwd_kernel(NormParams p) {
  using V = Vec<IO, VEC>;
  __shared__ float wave_sums[64];
  extern __shared__ float sums[];  // (row lanes, groups of the block, vectors) of dw, then db
  const NormPlace q = norm_place(p);
  const int nvec = p.size / VEC, c0 = q.group * p.size, rb = (int)(blockIdx.x / (uint32_t)p.blocks);
  const int channels = p.groups * p.size;
  float* part = p.ws + (int64_t)rb * 2 * channels + c0;
  int turn = 0;
  float w[VEC], b[VEC], x[VEC], z[VEC], dy[VEC], dw[VEC], db[VEC];
#pragma unroll
  for (int e = 0; e < VEC; ++e) dw[e] = db[e] = 0.0f;
  if (q.in) {
    if (ONE) {
      if (q.lane < nvec) {
        load_weights<VEC>(p.w, c0 + VEC * q.lane, 1.0f, w);
        load_weights<VEC>(p.b, c0 + VEC * q.lane, 0.0f, b);
      }
    } else {
      for (int v = q.lane; v < nvec; v += p.lanes)
#pragma unroll
        for (int e = 0; e < VEC; ++e) part[VEC * v + e] = part[channels + VEC * v + e] = 0.0f;
    }
  }
  const bool first = p.mode == SS_NORM_GATE_FIRST, behind = p.mode == SS_NORM_GATE;
  const float inv = 1.0f / (float)p.size;
  for (int64_t r0 = (int64_t)rb * p.row_lanes; r0 < p.rows; r0 += (int64_t)p.row_blocks * p.row_lanes) {
    const int64_t r = r0 + q.row_lane;
    const bool in = q.in && r < p.rows;
    auto fetch = [&](int v) {
      V::load(p.x, r * p.x_stride + c0 + VEC * v, x);
      if (first || behind) V::load(p.z, r * p.z_stride + c0 + VEC * v, z);
    };
    auto fetch_dy = [&](int v) { V::load(p.dy, r * p.dy_stride + c0 + VEC * v, dy); };
    auto input = [&](int e) { return first ? x[e] * silu_f(z[e]) : x[e]; };
    const int v_end = in ? nvec : 0;
    float sum = 0.0f, none = 0.0f, mean = 0.0f;
    if (ONE && q.lane < v_end) {
      fetch(q.lane);
      fetch_dy(q.lane);
    }
    if (p.center) {
      for (int v = q.lane; v < v_end; v += p.lanes) {
        if (!ONE) fetch(v);
#pragma unroll
        for (int e = 0; e < VEC; ++e) sum += input(e);
      }
      group_sums(sum, none, p.lanes, wave_sums, turn);
      mean = sum * inv;
    }
    float sq = 0.0f;
    for (int v = q.lane; v < v_end; v += p.lanes) {
      if (!ONE) fetch(v);
#pragma unroll
      for (int e = 0; e < VEC; ++e) {
        const float d = input(e) - mean;
        sq = fmaf(d, d, sq);
      }
    }
    group_sums(sq, none, p.lanes, wave_sums, turn);
    const float rstd = rsqrtf(sq * inv + p.eps);
    // do of element e, and o
    auto outer = [&](int e, float v, float& o) {
      o = fmaf(v, w[e], b[e]);
      if (behind) return dy[e] * silu_f(z[e]);
      if (p.mode != SS_NORM_SILU) return dy[e];
      const float s = sigmoid_f(o);
      return dy[e] * (s * fmaf(o, 1.0f - s, 1.0f));
    };
    float s1 = 0.0f, s2 = 0.0f;
    for (int v = q.lane; v < v_end; v += p.lanes) {
      if (!ONE) {
        fetch(v);
        fetch_dy(v);
        load_weights<VEC>(p.w, c0 + VEC * v, 1.0f, w);
        load_weights<VEC>(p.b, c0 + VEC * v, 0.0f, b);
      }
#pragma unroll
      for (int e = 0; e < VEC; ++e) {
        float o;
        const float n = (input(e) - mean) * rstd, d = outer(e, n, o);
        if (ONE) {
          dw[e] = fmaf(d, n, dw[e]);
          db[e] += d;
        } else {
          part[VEC * v + e] += d * n;
          part[channels + VEC * v + e] += d;
        }
        s1 = fmaf(d, w[e], s1);
        s2 = fmaf(d * w[e], n, s2);
      }
    }
    group_sums(s1, s2, p.lanes, wave_sums, turn);
    const float m1 = p.center ? s1 * inv : 0.0f, m2 = s2 * inv;
    for (int v = q.lane; v < v_end; v += p.lanes) {
      if (!ONE) {
        fetch(v);
        fetch_dy(v);
        load_weights<VEC>(p.w, c0 + VEC * v, 1.0f, w);
        load_weights<VEC>(p.b, c0 + VEC * v, 0.0f, b);
      }
      float dx[VEC], dz[VEC];
#pragma unroll
      for (int e = 0; e < VEC; ++e) {
        float o;
        const float n = (input(e) - mean) * rstd, d = outer(e, n, o);
        const float du = rstd * (fmaf(d, w[e], -m1) - n * m2);
        dx[e] = du;
        if (first || behind) {
          const float s = sigmoid_f(z[e]), ds = s * fmaf(z[e], 1.0f - s, 1.0f);
          dz[e] = first ? du * x[e] * ds : dy[e] * o * ds;
          if (first) dx[e] = du * (z[e] * s);
        }
      }
      V::store(p.dx, r * (int64_t)channels + c0 + VEC * v, dx);
      if (first || behind) V::store(p.dz, r * (int64_t)channels + c0 + VEC * v, dz);
    }
  }
  if constexpr (ONE) {  // the row lanes' sums, in their order
    const int per = p.block_groups * p.lanes * VEC, at = (q.row_lane * p.block_groups + q.slot % p.block_groups) * p.lanes * VEC;
    for (int k = 0; k < 2; ++k) {
      __syncthreads();
#pragma unroll
      for (int e = 0; e < VEC; ++e)
        if (q.row_lane < p.row_lanes) sums[at + VEC * q.lane + e] = k ? db[e] : dw[e];
      __syncthreads();
      if (q.in && q.row_lane == 0 && q.lane < nvec) {
#pragma unroll
        for (int e = 0; e < VEC; ++e) {
          float s = 0.0f;
          for (int l = 0; l < p.row_lanes; ++l) s += sums[l * per + at + VEC * q.lane + e];
          part[(int64_t)k * channels + VEC * q.lane + e] = s;
        }
      }
    }
  }
}

// dw and db from the workgroups' sums: 16 channels of 16 row lanes a workgroup
__global__ void __launch_bounds__(256) group_norm_sum_kernel(NormParams p) {
  __shared__ float sums[16][17];
  const int channels = p.groups * p.size, c = (int)blockIdx.x * 16 + (int)threadIdx.x % 16, l = (int)threadIdx.x / 16;
  float s = 0.0f;
  if (c < 2 * channels)
    for (int r = l; r < p.row_blocks; r += 16) s += p.ws[(int64_t)r * 2 * channels + c];
  sums[l][threadIdx.x % 16] = s;
  __syncthreads();
  if (l == 0 && c < 2 * channels) {
    s = 0.0f;
#pragma unroll
    for (int k = 0; k < 16; ++k) s += sums[k][threadIdx.x % 16];
    if (c < channels) {
      if (p.dw) p.dw[c] = s;
    } else if (p.db) {
      p.db[c - channels] = s;
    }
  }
}

template <int IO, int VEC>
hipError_t launch_norm_vec(const NormParams& p, hipStream_t st) {
  const dim3 grid((uint32_t)((int64_t)p.blocks * p.row_blocks)), threads(p.lanes > 256 ? p.lanes : 256);
  const bool one = p.size / VEC <= p.lanes;
  if (!p.dy) {
    if (one) hipLaunchKernelGGL((group_norm_kernel<IO, VEC, true>), grid, threads, 0, st, p);
    else hipLaunchKernelGGL((group_norm_kernel<IO, VEC, false>), grid, threads, 0, st, p);
    return hipGetLastError();
  }
  const uint32_t lds = (uint32_t)(p.row_lanes * p.block_groups * p.lanes * VEC * 4);
  if (one) hipLaunchKernelGGL((group_norm_bwd_kernel<IO, VEC, true>), grid, threads, lds, st, p);
  else hipLaunchKernelGGL((group_norm_bwd_kernel<IO, VEC, false>), grid, threads, 0, st, p);
  const hipError_t e = hipGetLastError();
  if (e != hipSuccess || (!p.dw && !p.db)) return e;
  hipLaunchKernelGGL(group_norm_sum_kernel, dim3((uint32_t)((2 * p.groups * (int64_t)p.size + 15) / 16)), dim3(256), 0, st, p);
  return hipGetLastError();
}

}  // namespace

hipError_t launch_group_norm(const NormParams& p, hipStream_t st) {
  switch (p.io) {
    case SS_F32: return p.vec == 4 ? launch_norm_vec<SS_F32, 4>(p, st) : launch_norm_vec<SS_F32, 1>(p, st);
    case SS_F16:
      return p.vec == 8   ? launch_norm_vec<SS_F16, 8>(p, st)
             : p.vec == 4 ? launch_norm_vec<SS_F16, 4>(p, st)
                          : launch_norm_vec<SS_F16, 1>(p, st);
    default:
      return p.vec == 8   ? launch_norm_vec<SS_BF16, 8>(p, st)
             : p.vec == 4 ? launch_norm_vec<SS_BF16, 4>(p, st)
                          : launch_norm_vec<SS_BF16, 1>(p, st);
  }
}

}  // namespace ss
