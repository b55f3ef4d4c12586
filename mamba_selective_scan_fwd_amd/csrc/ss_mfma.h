// ss_mfma.h -- matrix-core operand helpers shared by the SSD kernels (gfx950).
// Internal to libss.so; not part of the public C ABI.
//
// MFMA: v_mfma_f32_16x16x32_{bf16,f16}, fp32 accumulation.  Operand lane
// layout (checked on the chip): A[m][k] in lane m + 16 (k / 8), element k % 8;
// B[k][n] in lane n + 16 (k / 8), element k % 8; D[m][n] in lane
// n + 16 (m / 4), element m % 4.
#pragma once

#include "ss_device.h"
#include "ss_view.h"

namespace ss {

typedef __bf16 bf16x8 __attribute__((ext_vector_type(8)));
typedef _Float16 f16x8 __attribute__((ext_vector_type(8)));
typedef float f32x4 __attribute__((ext_vector_type(4)));
typedef uint32_t u32x4v __attribute__((ext_vector_type(4)));

template <int IO> struct mfma_t;
template <> struct mfma_t<SS_BF16> {
  using V = bf16x8;
  static __device__ __forceinline__ f32x4 run(V a, V b, f32x4 c) {
    return __builtin_amdgcn_mfma_f32_16x16x32_bf16(a, b, c, 0, 0, 0);
  }
};
template <> struct mfma_t<SS_F16> {
  using V = f16x8;
  static __device__ __forceinline__ f32x4 run(V a, V b, f32x4 c) {
    return __builtin_amdgcn_mfma_f32_16x16x32_f16(a, b, c, 0, 0, 0);
  }
};

// 16-bit storage bits of v in the I/O dtype (round to nearest even)
template <int IO>
__device__ __forceinline__ uint16_t bits16(float v) {
  return __builtin_bit_cast(uint16_t, from_f32<IO>(v));
}
// two values packed low-first into one word of the I/O dtype (one packed
// hardware conversion, round to nearest even)
typedef float f32x2 __attribute__((ext_vector_type(2)));
typedef __bf16 bf16x2 __attribute__((ext_vector_type(2)));
typedef _Float16 f16x2 __attribute__((ext_vector_type(2)));
template <int IO>
__device__ __forceinline__ uint32_t pack2(float lo, float hi) {
  if constexpr (IO == SS_BF16)
    return __builtin_bit_cast(uint32_t, __builtin_convertvector(f32x2{lo, hi}, bf16x2));
  else
    return __builtin_bit_cast(uint32_t, __builtin_convertvector(f32x2{lo, hi}, f16x2));
}
template <int IO>
__device__ __forceinline__ typename mfma_t<IO>::V as_vec(u32x4v w) {
  return __builtin_bit_cast(typename mfma_t<IO>::V, w);
}

__device__ __forceinline__ u32x4v vload16(__amdgpu_buffer_rsrc_t r, uint32_t off) {
  return __builtin_bit_cast(u32x4v, __builtin_amdgcn_raw_buffer_load_b128(r, off, 0, 0));
}
__device__ __forceinline__ uint2 vload8(__amdgpu_buffer_rsrc_t r, uint32_t off) {
  return __builtin_bit_cast(uint2, __builtin_amdgcn_raw_buffer_load_b64(r, off, 0, 0));
}
__device__ __forceinline__ void vstore8(__amdgpu_buffer_rsrc_t r, uint32_t off, uint32_t a, uint32_t b) {
  typedef uint32_t u32x2 __attribute__((ext_vector_type(2)));
  __builtin_amdgcn_raw_buffer_store_b64(u32x2{a, b}, r, off, 0, 0);
}

// Time-major tiles in LDS (row = step, W 16-bit columns, 16-byte chunks of a
// row rotated by (row / 4) so that both the row writes and the transposing
// reads below are free of bank conflicts).  Element offset of (row, col):
template <int W>
__device__ __forceinline__ int tm_off(int row, int col) {
  return row * W + 8 * ((col >> 3) ^ ((row >> 2) & (W / 8 - 1))) + (col & 7);
}
// An MFMA operand fragment whose k axis is time, read from a time-major
// tile with ds_read_b64_tr_b16 (gfx950; lane layout checked on the chip: in
// each group of 16 lanes, lane i receives element i % 4 of the 4-element
// reads of lanes i / 4 + 4q, q = 0..3).  Lane j of group g reads 4 columns
// c0 + 4 (j % 4) .. + 3 of row r0 + 8 g + 4 h + j / 4 (h = 0, 1), so lane i
// ends with column c0 + i at the 8 steps r0 + 8 g .. + 7: A[m = i][k] or
// B[k][n = i] of v_mfma_f32_16x16x32.
typedef short s16x4 __attribute__((ext_vector_type(4)));
typedef short s16x8 __attribute__((ext_vector_type(8)));
// For r0 a multiple of 32 the rotation does not depend on r0, so a lane's
// read address is r0 * W plus a per-lane offset: tm_lane_off gives it (h = 0
// for steps r0 + 8 g .. + 3, h = 1 for the next 4) and tm_frag reads the
// fragment at tile + r0 * W.
template <int W>
__device__ __forceinline__ int tm_lane_off(int c0, int h, int lane) {
  const int j = lane % 16, g = lane / 16;
  return tm_off<W>(8 * g + 4 * h + j / 4, c0 + 4 * (j % 4));
}
__device__ __forceinline__ u32x4v tm_frag(const uint16_t* at, int off_lo, int off_hi) {
  const s16x4 lo = __builtin_amdgcn_ds_read_tr16_b64_v4i16((__attribute__((address_space(3))) s16x4*)(at + off_lo));
  const s16x4 hi = __builtin_amdgcn_ds_read_tr16_b64_v4i16((__attribute__((address_space(3))) s16x4*)(at + off_hi));
  return __builtin_bit_cast(u32x4v, __builtin_shufflevector(lo, hi, 0, 1, 2, 3, 4, 5, 6, 7));
}

// ---- sums over the four 16-lane rows of a wave ---------------------------------
// v_permlane16_swap of a value with itself leaves rows (0, 0, 2, 2) and (1, 1, 3, 3),
// v_permlane32_swap the halves (0, 0) and (1, 1): sums across rows without LDS.
__device__ __forceinline__ void swap_rows(float v, float& even, float& odd) {
  const auto r = __builtin_amdgcn_permlane16_swap(__float_as_uint(v), __float_as_uint(v), false, false);
  even = __uint_as_float(r[0]);
  odd = __uint_as_float(r[1]);
}
__device__ __forceinline__ void swap_halves(float v, float& low, float& high) {
  const auto r = __builtin_amdgcn_permlane32_swap(__float_as_uint(v), __float_as_uint(v), false, false);
  low = __uint_as_float(r[0]);
  high = __uint_as_float(r[1]);
}
__device__ __forceinline__ float quad_sum(float v) {  // of the lanes l % 16 of all rows
  float a, b;
  swap_rows(v, a, b);
  swap_halves(a + b, a, b);
  return a + b;
}
struct QuadSums {
  float before, all;  // the rows before this lane's, and all four
};
__device__ __forceinline__ QuadSums quad_sums(float v) {
  float even, odd, low, high;
  swap_rows(v, even, odd);
  swap_halves(even + odd, low, high);
  return {(threadIdx.x & 16 ? even : 0.0f) + (threadIdx.x & 32 ? low : 0.0f), low + high};
}

// ---- operands as sums of bf16 values -------------------------------------------
// A computed operand v is split into bf16 parts, each the rounding of what the
// parts before it leave: |v - p0 - p1| <= 2^-18 |v|, |v - p0 - p1 - p2| <= 2^-27
// |v|, and multiplied part by part.  Two parts serve what is rounded to 16 bits
// in the end, three what stays in fp32 (states, and the sums of the decays'
// gradients), so that neither shows bf16's error.  bf16 data are one part, fp16
// data two without error (11 bits into 16).  Of two split operands, the
// products of parts i and j with i + j <= 2 (three parts) or <= 1 are formed:
// the rest is below what the split itself leaves.
using BF = mfma_t<SS_BF16>;

// v0, v1 as packed bf16 words hi and lo
__device__ __forceinline__ void split2(float v0, float v1, uint32_t& hi, uint32_t& lo) {
  hi = pack2<SS_BF16>(v0, v1);
  lo = pack2<SS_BF16>(v0 - __uint_as_float(hi << 16), v1 - __uint_as_float(hi & 0xffff0000u));
}
// and as three
__device__ __forceinline__ void split3(float v0, float v1, uint32_t (&w)[3]) {
#pragma unroll
  for (int k = 0; k < 3; ++k) {
    w[k] = pack2<SS_BF16>(v0, v1);
    v0 -= __uint_as_float(w[k] << 16);
    v1 -= __uint_as_float(w[k] & 0xffff0000u);
  }
}
template <int IO>
__device__ __forceinline__ float low16(uint32_t w) { return bits_f32<IO>((raw_t<IO>)(w & 0xffffu)); }
template <int IO>
__device__ __forceinline__ float high16(uint32_t w) { return bits_f32<IO>((raw_t<IO>)(w >> 16)); }
// eight 16-bit values as bf16 hi and lo parts (bf16 input is its own hi)
template <int IO>
__device__ __forceinline__ void split8(u32x4v w, u32x4v& hi, u32x4v& lo) {
#pragma unroll
  for (int q = 0; q < 4; ++q) {
    uint32_t a, b;
    split2(low16<IO>(w[q]), high16<IO>(w[q]), a, b);
    hi[q] = a;
    lo[q] = b;
  }
}
__device__ __forceinline__ bf16x8 bfv(u32x4v w) { return as_vec<SS_BF16>(w); }

// The rows of a chunk of an operand: `at` points at its first row's columns
// (wave-uniform), `cols` bytes a row, rows are `row` bytes apart; rows from
// `rows` on, and in the last one what follows its columns, read as zeros
// through the range check.
__device__ __forceinline__ __amdgpu_buffer_rsrc_t rows_view(const void* at, int64_t row, int rows, int64_t cols) {
  return make_rsrc(at, at ? view_bytes(row, rows, cols) : 0u);
}

// C B^T tiles in operand order: element (i, j) of row tile it = i / 16 and
// k-step kt = j / 32 is float j % 8 of lane i % 16 + 16 ((j % 32) / 8), 8 floats
// a lane, so that a wave reads whole contiguous kilobytes.
__device__ __forceinline__ int64_t cb_at(int it, int kt) { return (int64_t)(it * 8 + kt) * 512; }

}  // namespace ss
