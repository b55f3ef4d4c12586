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
// Bound by HBM: 16384 rows of 1536 in bf16, 12 groups, the gate behind, take 26 us forward
// (151 MB) and 54 + 5 us for the gradients (252 MB, 4.7 TB/s); 64 such rows 3.6 us, the
// latency of one load, two sums and a store.  A group has `lanes` threads, each with one
// vector of its channels in registers, so that a row's data are read once, the next
// row's while this one is worked on.  A thread keeps its channels, and their w and b,
// over all the rows that its workgroup walks, which is what dw and db are summed over.
// A kernel for each mode: with the mode as an argument the gradients' kernel branched
// for each element and took 62 us, for it issues as long as it loads.  Groups of more
// than 1024 vectors are walked by 1024 threads, element by element, that read the row
// once for every sum.
#include <type_traits>

#include "ss_device.h"
#include "ss_internal.h"

namespace ss {
namespace {

// VEC elements of the I/O type: as they lie in memory, and as floats
template <int IO, int VEC>
struct Vec {
  static constexpr int kBytes = (IO == SS_F32 ? 4 : 2) * VEC;
  template <int B> struct word { typedef uint32_t T __attribute__((ext_vector_type(B / 4))); };
  using W = typename std::conditional<VEC == 1, word<4>, word<(kBytes < 4 ? 4 : kBytes)>>::type::T;
  __device__ __forceinline__ static W load(const void* base, int64_t i) {
    const char* at = static_cast<const char*>(base) + i * (kBytes / VEC);
    if constexpr (kBytes == 2) {
      W w;
      w[0] = *reinterpret_cast<const uint16_t*>(at);
      return w;
    } else {
      return *reinterpret_cast<const W*>(at);
    }
  }
  __device__ __forceinline__ static float get(W w, int e) {
    if constexpr (IO == SS_F32) return __uint_as_float(w[e]);
    else return bits_f32<IO>((raw_t<IO>)(e & 1 ? w[e / 2] >> 16 : w[e / 2] & 0xffffu));
  }
  __device__ __forceinline__ static void store(void* base, int64_t i, const float (&v)[VEC]) {
    if constexpr (VEC == 1) {
      store_io<IO>(base, i, v[0]);
    } else {
      W w;
      if constexpr (IO == SS_F32) {
#pragma unroll
        for (int e = 0; e < VEC; ++e) w[e] = __float_as_uint(v[e]);
      } else {
#pragma unroll
        for (int e = 0; e < VEC / 2; ++e) {
          w[e] = (uint32_t)__builtin_bit_cast(uint16_t, from_f32<IO>(v[2 * e])) |
                 ((uint32_t)__builtin_bit_cast(uint16_t, from_f32<IO>(v[2 * e + 1])) << 16);
        }
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

// Sums of N values over the `lanes` threads of a group: a power of two up to 64, or whole
// waves.  Within a wave by DPP and row swaps; `waves` holds N floats a wave, twice, in
// turn, so that a sum takes one barrier.
template <int CTRL>
__device__ __forceinline__ float dpp_sum(float v) {
  return v + __int_as_float(__builtin_amdgcn_update_dpp(0, __float_as_int(v), CTRL, 0xf, 0xf, true));
}
__device__ __forceinline__ float lane_sum(float v, int lanes) {
  if (lanes > 1) v = dpp_sum<0xB1>(v);    // quad_perm: lane ^ 1
  if (lanes > 2) v = dpp_sum<0x4E>(v);    // quad_perm: lane ^ 2
  if (lanes > 4) v = dpp_sum<0x141>(v);   // row_half_mirror: the other quad of 8
  if (lanes > 8) v = dpp_sum<0x140>(v);   // row_mirror: the other 8 of 16
  if (lanes > 16) {
    const auto r = __builtin_amdgcn_permlane16_swap(__float_as_uint(v), __float_as_uint(v), false, false);
    v = __uint_as_float(r[0]) + __uint_as_float(r[1]);
  }
  if (lanes > 32) {
    const auto r = __builtin_amdgcn_permlane32_swap(__float_as_uint(v), __float_as_uint(v), false, false);
    v = __uint_as_float(r[0]) + __uint_as_float(r[1]);
  }
  return v;
}
constexpr int kMaxWaves = 16;
template <int N>
__device__ __forceinline__ void group_sums(float (&v)[N], int lanes, float* waves, int& turn) {
#pragma unroll
  for (int i = 0; i < N; ++i) v[i] = lane_sum(v[i], lanes);
  if (lanes <= 64) return;
  const int wave = (int)threadIdx.x / 64, per = lanes / 64, first = wave / per * per;
  float* at = waves + 2 * kMaxWaves * turn;
  turn ^= 1;  // the other half is written next
  if (threadIdx.x % 64 == 0)
#pragma unroll
    for (int i = 0; i < N; ++i) at[N * wave + i] = v[i];
  __syncthreads();
#pragma unroll
  for (int i = 0; i < N; ++i) {
    v[i] = 0.0f;
    for (int k = 0; k < per; ++k) v[i] += at[N * (first + k) + i];
  }
}

// Thread = (row lane, group of the block, vector of the group)
struct NormPlace {
  int lane, slot, group, row_lane, c;
  bool in;
};
__device__ __forceinline__ NormPlace norm_place(const NormParams& p) {
  NormPlace q;
  q.lane = (int)threadIdx.x % p.lanes;
  q.slot = (int)threadIdx.x / p.lanes;
  q.group = (int)(blockIdx.x % (uint32_t)p.blocks) * p.block_groups + q.slot % p.block_groups;
  q.row_lane = q.slot / p.block_groups;
  q.c = q.group * p.size + p.vec * q.lane;
  q.in = q.group < p.groups && q.row_lane < p.row_lanes;
  return q;
}

// A group's mean and 1 / deviation, from its threads' u
template <int VEC>
__device__ __forceinline__ void statistics(const NormParams& p, const float (&u)[VEC], bool mine, float* waves, int& turn,
                                           float& mean, float& rstd) {
  const float inv = 1.0f / (float)p.size;
  mean = 0.0f;
  float s[1] = {0.0f};
  if (p.center) {
#pragma unroll
    for (int e = 0; e < VEC; ++e) s[0] += u[e];
    group_sums(s, p.lanes, waves, turn);
    mean = s[0] * inv;
    s[0] = 0.0f;
  }
  if (mine)
#pragma unroll
    for (int e = 0; e < VEC; ++e) s[0] = fmaf(u[e] - mean, u[e] - mean, s[0]);
  group_sums(s, p.lanes, waves, turn);
  rstd = rsqrtf(fmaf(s[0], inv, p.eps));
}

template <int IO, int VEC, int MODE>
__global__ void __launch_bounds__(1024) group_norm_kernel(NormParams p) {
  using V = Vec<IO, VEC>;
  __shared__ float waves[4 * kMaxWaves];
  const NormPlace q = norm_place(p);
  const bool mine = q.in && q.lane < p.size / VEC;
  constexpr bool first = MODE == SS_NORM_GATE_FIRST, behind = MODE == SS_NORM_GATE;
  int turn = 0;
  float w[VEC], b[VEC];
  if (mine) {
    load_weights<VEC>(p.w, q.c, 1.0f, w);
    load_weights<VEC>(p.b, q.c, 0.0f, b);
  }
  typename V::W xn{}, zn{};
  auto fetch = [&](int64_t r) {
    if (!mine || r >= p.rows) return;
    xn = V::load(p.x, r * p.x_stride + q.c);
    if (first || behind) zn = V::load(p.z, r * p.z_stride + q.c);
  };
  // a workgroup's threads take the same number of steps: the sums may have barriers
  const int64_t step = (int64_t)p.row_blocks * p.row_lanes;
  int64_t r0 = (int64_t)(blockIdx.x / (uint32_t)p.blocks) * p.row_lanes;
  fetch(r0 + q.row_lane);
  for (; r0 < p.rows; r0 += step) {
    const int64_t r = r0 + q.row_lane;
    const typename V::W xw = xn, zw = zn;
    fetch(r + step);
    float u[VEC], mean, rstd;
#pragma unroll
    for (int e = 0; e < VEC; ++e) u[e] = mine ? (first ? V::get(xw, e) * silu_f(V::get(zw, e)) : V::get(xw, e)) : 0.0f;
    statistics<VEC>(p, u, mine, waves, turn, mean, rstd);
    if (!mine || r >= p.rows) continue;
    float y[VEC];
#pragma unroll
    for (int e = 0; e < VEC; ++e) {
      const float o = fmaf((u[e] - mean) * rstd, w[e], b[e]);
      y[e] = behind ? o * silu_f(V::get(zw, e)) : MODE == SS_NORM_SILU ? silu_f(o) : o;
    }
    V::store(p.y, r * p.y_stride + q.c, y);
  }
}

// Gradients of one row's element: do = dy d(y)/d(o)
__device__ __forceinline__ float outer_grad(int mode, float dy, float zs, float o) {
  if (mode == SS_NORM_GATE) return dy * zs;
  if (mode != SS_NORM_SILU) return dy;
  const float s = sigmoid_f(o);
  return dy * (s * fmaf(o, 1.0f - s, 1.0f));
}

// Every workgroup leaves its sums of dw and db, over the rows it walks, in the workspace:
// (row block, 2, channels).
template <int IO, int VEC, int MODE>
__global__ void __launch_bounds__(1024) group_norm_bwd_kernel(NormParams p) {
  using V = Vec<IO, VEC>;
  __shared__ float waves[4 * kMaxWaves];
  extern __shared__ float sums[];  // (row lanes, groups of the block, vectors) of dw, then db
  const NormPlace q = norm_place(p);
  const bool mine = q.in && q.lane < p.size / VEC;
  constexpr bool first = MODE == SS_NORM_GATE_FIRST, gated = first || MODE == SS_NORM_GATE;
  const int channels = p.groups * p.size, rb = (int)(blockIdx.x / (uint32_t)p.blocks);
  const float inv = 1.0f / (float)p.size;
  int turn = 0;
  float w[VEC], b[VEC], dw[VEC], db[VEC];
#pragma unroll
  for (int e = 0; e < VEC; ++e) w[e] = b[e] = dw[e] = db[e] = 0.0f;
  if (mine) {
    load_weights<VEC>(p.w, q.c, 1.0f, w);
    load_weights<VEC>(p.b, q.c, 0.0f, b);
  }
  typename V::W xn{}, zn{}, gn{};
  auto fetch = [&](int64_t r) {
    if (!mine || r >= p.rows) return;
    xn = V::load(p.x, r * p.x_stride + q.c);
    gn = V::load(p.dy, r * p.dy_stride + q.c);
    if (gated) zn = V::load(p.z, r * p.z_stride + q.c);
  };
  const int64_t step = (int64_t)p.row_blocks * p.row_lanes;
  int64_t r0 = (int64_t)rb * p.row_lanes;
  fetch(r0 + q.row_lane);
  for (; r0 < p.rows; r0 += step) {
    const int64_t r = r0 + q.row_lane;
    const typename V::W xw = xn, zw = zn, gw = gn;
    fetch(r + step);
    const bool in = mine && r < p.rows;
    float u[VEC], dn[VEC], mean, rstd, s[2] = {0.0f, 0.0f};
#pragma unroll
    for (int e = 0; e < VEC; ++e) u[e] = in ? (first ? V::get(xw, e) * silu_f(V::get(zw, e)) : V::get(xw, e)) : 0.0f;
    statistics<VEC>(p, u, in, waves, turn, mean, rstd);
#pragma unroll
    for (int e = 0; e < VEC; ++e) {
      const float n = (u[e] - mean) * rstd, o = fmaf(n, w[e], b[e]);
      const float d = in ? outer_grad(MODE, V::get(gw, e), gated ? silu_f(V::get(zw, e)) : 0.0f, o) : 0.0f;
      dw[e] = in ? fmaf(d, n, dw[e]) : dw[e];
      db[e] += d;
      u[e] = n;
      dn[e] = d * w[e];
      s[0] += dn[e];
      s[1] = in ? fmaf(dn[e], n, s[1]) : s[1];
    }
    group_sums(s, p.lanes, waves, turn);
    if (!in) continue;
    const float m1 = p.center ? s[0] * inv : 0.0f, m2 = s[1] * inv;
    float out[VEC];
#pragma unroll
    for (int e = 0; e < VEC; ++e) {
      out[e] = rstd * (dn[e] - m1 - u[e] * m2);
      if (first) dn[e] = out[e];  // du
      if (first) out[e] *= silu_f(V::get(zw, e));
    }
    V::store(p.dx, r * (int64_t)channels + q.c, out);
    if (!gated) continue;
#pragma unroll
    for (int e = 0; e < VEC; ++e) {
      const float z = V::get(zw, e), sg = sigmoid_f(z), ds = sg * fmaf(z, 1.0f - sg, 1.0f);
      out[e] = (first ? dn[e] * V::get(xw, e) : V::get(gw, e) * fmaf(u[e], w[e], b[e])) * ds;
    }
    V::store(p.dz, r * (int64_t)channels + q.c, out);
  }
  // the row lanes' sums, in their order
  const int per = p.block_groups * p.lanes * VEC, at = q.slot * p.lanes * VEC + VEC * q.lane;
  float* part = p.ws + (int64_t)rb * 2 * channels + q.c;
  for (int k = 0; k < 2; ++k) {
    __syncthreads();
    if (q.row_lane < p.row_lanes)
#pragma unroll
      for (int e = 0; e < VEC; ++e) sums[at + e] = k ? db[e] : dw[e];
    __syncthreads();
    if (mine && q.row_lane == 0)
#pragma unroll
      for (int e = 0; e < VEC; ++e) {
        float t = 0.0f;
        for (int l = 0; l < p.row_lanes; ++l) t += sums[l * per + at + e];
        part[(int64_t)k * channels + e] = t;
      }
  }
}

// ---- groups of more than 1024 vectors: a workgroup a group, element by element of the row --------
template <int IO>
__device__ __forceinline__ float big_input(const NormParams& p, int64_t r, int c) {
  const float x = load_io<IO>(p.x, r * p.x_stride + c);
  return p.mode == SS_NORM_GATE_FIRST ? x * silu_f(load_io<IO>(p.z, r * p.z_stride + c)) : x;
}
template <int IO>
__device__ __forceinline__ void big_statistics(const NormParams& p, int64_t r, int c0, float* waves, int& turn, float& mean,
                                               float& rstd) {
  const float inv = 1.0f / (float)p.size;
  float s[1] = {0.0f};
  mean = 0.0f;
  if (p.center) {
    for (int c = threadIdx.x; c < p.size; c += 1024) s[0] += big_input<IO>(p, r, c0 + c);
    group_sums(s, 1024, waves, turn);
    mean = s[0] * inv;
    s[0] = 0.0f;
  }
  for (int c = threadIdx.x; c < p.size; c += 1024) {
    const float d = big_input<IO>(p, r, c0 + c) - mean;
    s[0] = fmaf(d, d, s[0]);
  }
  group_sums(s, 1024, waves, turn);
  rstd = rsqrtf(fmaf(s[0], inv, p.eps));
}
template <int IO>
__global__ void __launch_bounds__(1024) group_norm_big_kernel(NormParams p) {
  __shared__ float waves[4 * kMaxWaves];
  const int c0 = (int)(blockIdx.x % (uint32_t)p.blocks) * p.size;
  int turn = 0;
  for (int64_t r = blockIdx.x / (uint32_t)p.blocks; r < p.rows; r += p.row_blocks) {
    float mean, rstd;
    big_statistics<IO>(p, r, c0, waves, turn, mean, rstd);
    for (int c = c0 + (int)threadIdx.x; c < c0 + p.size; c += 1024) {
      float o = fmaf((big_input<IO>(p, r, c) - mean) * rstd, p.w ? p.w[c] : 1.0f, p.b ? p.b[c] : 0.0f);
      if (p.mode == SS_NORM_GATE) o *= silu_f(load_io<IO>(p.z, r * p.z_stride + c));
      if (p.mode == SS_NORM_SILU) o = silu_f(o);
      store_io<IO>(p.y, r * p.y_stride + c, o);
    }
  }
}
template <int IO>
__global__ void __launch_bounds__(1024) group_norm_big_bwd_kernel(NormParams p) {
  __shared__ float waves[4 * kMaxWaves];
  const int c0 = (int)(blockIdx.x % (uint32_t)p.blocks) * p.size, rb = (int)(blockIdx.x / (uint32_t)p.blocks);
  const int channels = p.groups * p.size;
  const bool first = p.mode == SS_NORM_GATE_FIRST, gated = first || p.mode == SS_NORM_GATE;
  const float inv = 1.0f / (float)p.size;
  float* part = p.ws + (int64_t)rb * 2 * channels;
  int turn = 0;
  for (int c = c0 + (int)threadIdx.x; c < c0 + p.size; c += 1024) part[c] = part[channels + c] = 0.0f;
  for (int64_t r = rb; r < p.rows; r += p.row_blocks) {
    float mean, rstd, s[2] = {0.0f, 0.0f};
    big_statistics<IO>(p, r, c0, waves, turn, mean, rstd);
    auto element = [&](int c, float& n, float& o, float& g) {
      n = (big_input<IO>(p, r, c) - mean) * rstd;
      o = fmaf(n, p.w ? p.w[c] : 1.0f, p.b ? p.b[c] : 0.0f);
      g = outer_grad(p.mode, load_io<IO>(p.dy, r * p.dy_stride + c), gated ? silu_f(load_io<IO>(p.z, r * p.z_stride + c)) : 0.0f, o);
    };
    for (int c = c0 + (int)threadIdx.x; c < c0 + p.size; c += 1024) {
      float n, o, g;
      element(c, n, o, g);
      part[c] += g * n;  // this thread's own
      part[channels + c] += g;
      const float dn = p.w ? g * p.w[c] : g;
      s[0] += dn;
      s[1] = fmaf(dn, n, s[1]);
    }
    group_sums(s, 1024, waves, turn);
    const float m1 = p.center ? s[0] * inv : 0.0f, m2 = s[1] * inv;
    for (int c = c0 + (int)threadIdx.x; c < c0 + p.size; c += 1024) {
      float n, o, g;
      element(c, n, o, g);
      const float du = rstd * ((p.w ? g * p.w[c] : g) - m1 - n * m2);
      float dx = du;
      if (gated) {
        const float z = load_io<IO>(p.z, r * p.z_stride + c), sg = sigmoid_f(z), ds = sg * fmaf(z, 1.0f - sg, 1.0f);
        store_io<IO>(p.dz, r * (int64_t)channels + c,
                     (first ? du * load_io<IO>(p.x, r * p.x_stride + c) : load_io<IO>(p.dy, r * p.dy_stride + c) * o) * ds);
        if (first) dx = du * (z * sg);
      }
      store_io<IO>(p.dx, r * (int64_t)channels + c, dx);
    }
  }
}

// dw and db from the workgroups' sums: 32 channels of 32 row lanes a workgroup, each with 4
// loads at a time (256 sums of 1536 channels: 4.7 us; 1024 sums, one load at a time: 21)
__global__ void __launch_bounds__(1024) group_norm_sum_kernel(NormParams p) {
  __shared__ float sums[32][33];
  const int channels = p.groups * p.size, k = (int)threadIdx.x % 32, c = (int)blockIdx.x * 32 + k, l = (int)threadIdx.x / 32;
  float s[4] = {0.0f, 0.0f, 0.0f, 0.0f};
  if (c < 2 * channels)
    for (int r = l; r < p.row_blocks; r += 128)
#pragma unroll
      for (int i = 0; i < 4; ++i)
        if (r + 32 * i < p.row_blocks) s[i] += p.ws[(int64_t)(r + 32 * i) * 2 * channels + c];
  sums[l][k] = (s[0] + s[1]) + (s[2] + s[3]);
  __syncthreads();
  // the first wave's halves take 16 row lanes each
  if (threadIdx.x >= 64 || c >= 2 * channels) return;
  float t = 0.0f;
#pragma unroll
  for (int i = 0; i < 16; ++i) t += sums[16 * l + i][k];
  t += __shfl_xor(t, 32, 64);
  if (l) return;
  if (c < channels) {
    if (p.dw) p.dw[c] = t;
  } else if (p.db) {
    p.db[c - channels] = t;
  }
}

template <int IO, int VEC, int MODE>
hipError_t launch_norm_mode(const NormParams& p, hipStream_t st) {
  const dim3 grid((uint32_t)((int64_t)p.blocks * p.row_blocks)), threads((uint32_t)p.threads);
  const uint32_t lds = (uint32_t)(p.row_lanes * p.block_groups * p.lanes * VEC * 4);
  if (!p.dy) hipLaunchKernelGGL((group_norm_kernel<IO, VEC, MODE>), grid, threads, 0, st, p);
  else hipLaunchKernelGGL((group_norm_bwd_kernel<IO, VEC, MODE>), grid, threads, lds, st, p);
  return hipGetLastError();
}
template <int IO, int VEC>
hipError_t launch_norm_vec(const NormParams& p, hipStream_t st) {
  switch (p.mode) {
    case SS_NORM_SILU: return launch_norm_mode<IO, VEC, SS_NORM_SILU>(p, st);
    case SS_NORM_GATE: return launch_norm_mode<IO, VEC, SS_NORM_GATE>(p, st);
    case SS_NORM_GATE_FIRST: return launch_norm_mode<IO, VEC, SS_NORM_GATE_FIRST>(p, st);
    default: return launch_norm_mode<IO, VEC, SS_NORM_PLAIN>(p, st);
  }
}
template <int IO>
hipError_t launch_norm_io(const NormParams& p, hipStream_t st) {
  hipError_t e;
  if (p.size / p.vec > 1024) {
    const dim3 grid((uint32_t)((int64_t)p.blocks * p.row_blocks));
    if (!p.dy) hipLaunchKernelGGL((group_norm_big_kernel<IO>), grid, dim3(1024), 0, st, p);
    else hipLaunchKernelGGL((group_norm_big_bwd_kernel<IO>), grid, dim3(1024), 0, st, p);
    e = hipGetLastError();
  } else if (p.vec == (IO == SS_F32 ? 4 : 8)) {
    e = launch_norm_vec<IO, IO == SS_F32 ? 4 : 8>(p, st);
  } else if (IO != SS_F32 && p.vec == 4) {
    e = launch_norm_vec<IO, 4>(p, st);
  } else {
    e = launch_norm_vec<IO, 1>(p, st);
  }
  if (e != hipSuccess || !p.dy || (!p.dw && !p.db)) return e;
  hipLaunchKernelGGL(group_norm_sum_kernel, dim3((uint32_t)((2 * p.groups * (int64_t)p.size + 31) / 32)), dim3(1024), 0, st, p);
  return hipGetLastError();
}

}  // namespace

hipError_t launch_group_norm(const NormParams& p, hipStream_t st) {
  switch (p.io) {
    case SS_F32: return launch_norm_io<SS_F32>(p, st);
    case SS_F16: return launch_norm_io<SS_F16>(p, st);
    default: return launch_norm_io<SS_BF16>(p, st);
  }
}

}  // namespace ss
