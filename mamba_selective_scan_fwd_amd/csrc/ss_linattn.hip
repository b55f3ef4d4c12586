// ss_linattn.hip -- linear attention with a decay for each head, on MFMA (gfx950).
//
// Per head, with a = exp(log_decay) and the state H[p][n] (dv x dk):
//   H_t = a H_{t-1} + v_t k_t^T,   y_t = scale H_t q_t.
// In a chunk of rows i = 0 .. C-1 that the state E enters:
//   y_i = scale (a^{i+1} E q_i + sum_{j<=i} a^{i-j} (q_i . k_j) v_j)
//   E'  = a^C E + sum_j a^{C-1-j} v_j k_j^T.
// With G_t = dL/dH_t = a G_{t+1} + scale dy_t q_t^T (dfinal behind the last row)
// the gradients are dq_t = scale H_t^T dy_t, dk_t = G_t^T v_t, dv_t = G_t k_t and
// dh0 = a G_0: each is the same walk over the rows with other operands,
//   y : (a, b, c) = (q, k, v)       dq: (dy, v, k)
//   dk: (v, dy, q) from the end     dv: (k, q, dy) from the end
//   out_t = sum_s a^{|t-s|} (a_t . b_s) c_s over the rows s up to t of the walk,
// so that one kernel computes all four, and nothing of the forward is kept.  From
// the end the state that enters a chunk is a G (no decay before the first row,
// one more behind the last), which leaves dh0 behind.
#include "ss_device.h"
#include "ss_internal.h"
#include "ss_mfma.h"
#include "ss_packed.h"

namespace ss {
namespace {

constexpr int kC = 64;  // rows of a chunk
constexpr int kWalkThreads = 256;

// 16-bit tiles of W columns in LDS, 16-byte pieces of a row exchanged by the row:
// the 16 rows of a fragment read (16 or 8 bytes a lane) and the 4 consecutive
// rows of a transposing read (32 bytes each) lie in different banks.
template <int W>
__device__ __forceinline__ int tile_off(int row, int col) {
  static_assert(W == 64 || W == 128, "tile width");
  const int x = W == 128 ? ((row & 3) << 1) | ((row >> 2) & 1) | (((row >> 3) & 1) << 3)
                         : (((row >> 1) & 1) << 1) | ((row >> 2) & 1) | (((row >> 3) & 1) << 2);
  return row * W + 8 * ((col >> 3) ^ x) + (col & 7);
}
__device__ __forceinline__ u32x4v lds16(const uint16_t* at) { return *reinterpret_cast<const u32x4v*>(at); }
__device__ __forceinline__ uint2 lds8(const uint16_t* at) { return *reinterpret_cast<const uint2*>(at); }

// rows row0 .. row0 + 31 (row0 a multiple of 16) of the columns 16 ct .. as an operand whose k axis is the row
template <int W>
__device__ __forceinline__ u32x4v time_frag(const uint16_t* tile, int row0, int ct, int lane) {
  const int j = lane % 16, g = lane / 16, row = 8 * g + j / 4, col = 16 * ct + 4 * (j % 4);
  return tm_frag(tile + row0 * W, tile_off<W>(row, col), tile_off<W>(row + 4, col));
}

// The rows that workgroup place `place` walks.
struct LinRows {
  int seq, begin, len;  // the sequence
  int part;             // of its segments of 2^logq rows; the place is empty if out of range
  int t0, rows;         // the segment's rows, in the walk's order
  bool live, last;
};
__device__ __forceinline__ LinRows lin_rows(const LinParams& p, int place) {
  LinRows r;
  if (p.cu) {
    const SeqChunk q = find_chunk(p.cu, p.nseqs, p.tokens, place, p.logq);
    r.seq = q.seq;
    r.begin = q.begin;
    r.len = q.len;
    r.part = q.chunk;
  } else {
    r.len = p.tokens / p.nseqs;
    const int parts = (int)(((int64_t)r.len + ((int64_t)1 << p.logq) - 1) >> p.logq);
    r.seq = place / parts;
    r.part = place - r.seq * parts;
    r.begin = r.seq * r.len;
  }
  const int64_t t0 = (int64_t)r.part << p.logq;
  r.live = r.part >= 0 && t0 < (r.len > 0 ? r.len : 1);
  r.t0 = r.live ? (int)t0 : 0;
  const int64_t left = r.len - t0, most = (int64_t)1 << p.logq;
  r.rows = r.live ? (int)(left < most ? left : most) : 0;
  r.last = left <= most;
  return r;
}
// A sequence's first state (null: zeros) and where its last one goes (null: nowhere)
__device__ __forceinline__ void lin_states(const LinParams& p, const LinWalk& w, int seq, int h, const float*& init,
                                           float*& fin) {
  int i = seq;
  bool carried = true;
  if (p.pool) {
    i = uniform(slot_of(p.slots, seq, p.nslots));
    carried = p.has_state && uniform(p.has_state[seq]) != 0;
  }
  const int64_t at = ((int64_t)(i < 0 ? 0 : i) * p.heads + h) * (w.dc * w.dout);
  init = i >= 0 && carried && w.init ? w.init + at : nullptr;
  fin = i >= 0 && w.fin ? w.fin + at : nullptr;
}
// element (c, o) of a state in memory: (dv, dk), c being the side that is contracted with a
__device__ __forceinline__ int state_at(const LinWalk& w, int c, int o) { return w.c_inner ? o * w.dc + c : c * w.dout + o; }

// exp(n g) and exp(n g) - 1; n = 0 has no decay, whatever g
__device__ __forceinline__ double lin_power(float g, int n) { return n ? exp((double)n * (double)g) : 1.0; }
__device__ __forceinline__ double lin_power_m1(float g, int n) { return n ? expm1((double)n * (double)g) : 0.0; }

// ---- the walk ----------------------------------------------------------------------
template <int DC, int DO, bool STATE>
struct WalkLds {
  float power[kC + 4];  // a^i
  float decay[2];       // a^rows - 1 of a whole chunk and of the last one
  __attribute__((aligned(16))) uint16_t a[STATE ? 8 : kC * DC];
  __attribute__((aligned(16))) uint16_t b[kC * DC];
  __attribute__((aligned(16))) uint16_t c[kC * DO];
  __attribute__((aligned(16))) uint16_t m[STATE ? 1 : 2][STATE ? 8 : kC * kC];
};

// a 16-bit fragment as bf16 parts: one, or two of fp16 data
template <int IO>
struct Parts {
  bf16x8 hi, lo;
  __device__ __forceinline__ explicit Parts(u32x4v w) {
    if constexpr (IO == SS_BF16) {
      hi = lo = bfv(w);
    } else {
      u32x4v h, l;
      split8<IO>(w, h, l);
      hi = bfv(h);
      lo = bfv(l);
    }
  }
};

template <int IO, int DC, int DO, bool STATE>
__global__ void __launch_bounds__(kWalkThreads, 2) lin_walk_kernel(LinParams p) {
  constexpr int CT = DC / 16, OT = DO / 64;  // state tiles of a wave: all of c, a quarter of o
  constexpr int NB = DC / 32, NO = DO / 32;  // 16-byte pieces of a thread
  constexpr bool kTwo = IO == SS_F16;
  __shared__ WalkLds<DC, DO, STATE> lds;
  const int tid = threadIdx.x, lane = tid % 64, wave = uniform(tid / 64), l16 = lane % 16, g4 = 4 * (lane / 16);
  const int lb = (int)xcd_logical_block();
  const int job = p.job0 + lb % p.njobs, h = lb / p.njobs % p.heads, place = lb / p.njobs / p.heads;
  const LinWalk& w = p.job[job];
  const LinRows q = lin_rows(p, place);
  const int kvh = h / p.share;
  if (!STATE && p.zero_rest && p.cu) {  // rows of no sequence have outputs of zero
    const int lead = seq_row(p.cu, 0, p.tokens), behind = seq_row(p.cu, p.nseqs, p.tokens);
    const int end = behind > lead ? behind : lead;
    for (int r = place; r < lead + p.tokens - end; r += p.places) {
      const int64_t at = ((int64_t)(r < lead ? r : end + r - lead) * p.heads + h) * DO;
      if (tid < DO) {
        if (w.sum) static_cast<float*>(w.out)[at + tid] = 0.0f;
        else static_cast<uint16_t*>(w.out)[at + tid] = 0;
      }
    }
  }
  if (!q.live || (STATE && q.last)) return;
  const float g = p.log_decay[h];
  const int tail = q.rows % kC;
  if (tid < kC + 2) lds.power[tid] = (float)lin_power(g, tid);
  if (tid >= 128 && tid < 130) lds.decay[tid - 128] = (float)lin_power_m1(g, tid == 128 ? kC : tail);
  if constexpr (!STATE)
    for (int k = tid; k < 2 * kC * kC / 8; k += kWalkThreads) reinterpret_cast<u32x4v*>(lds.m)[k] = u32x4v{0, 0, 0, 0};

  // ---- loads of a chunk: rows t .. of the segment, in the walk's order
  const bool rev = w.rev != 0;
  u32x4v ar[STATE ? 1 : NB], br[NB], cr[NO];
  auto load = [&](int t) {
    const int rows = q.rows - t < kC ? q.rows - t : kC;
    const int64_t tok = rev ? (int64_t)q.begin + q.len - (q.t0 + t + rows) : (int64_t)q.begin + q.t0 + t;
    auto view = [&](const void* at, int64_t stride, int head, int cols) {
      return rows_view(static_cast<const char*>(at) + (tok * stride + head * cols) * 2, stride * 2, rows, cols * 2);
    };
    auto off = [&](int row, int64_t stride, int col) {
      return row < rows ? (uint32_t)(rev ? rows - 1 - row : row) * (uint32_t)(stride * 2) + (uint32_t)col * 2u : kOffNone;
    };
    const auto bv = view(w.b, w.b_stride, w.b_kv ? kvh : h, DC);
    const auto cv = view(w.c, w.c_stride, w.c_kv ? kvh : h, DO);
#pragma unroll
    for (int k = 0; k < NB; ++k)
      br[k] = vload16(bv, off(tid / (DC / 8) + k * (2048 / DC), w.b_stride, 8 * (tid % (DC / 8))));
#pragma unroll
    for (int k = 0; k < NO; ++k)
      cr[k] = vload16(cv, off(tid / (DO / 8) + k * (2048 / DO), w.c_stride, 8 * (tid % (DO / 8))));
    if constexpr (!STATE) {
      const auto av = view(w.a, w.a_stride, w.a_kv ? kvh : h, DC);
#pragma unroll
      for (int k = 0; k < NB; ++k)
        ar[k] = vload16(av, off(tid / (DC / 8) + k * (2048 / DC), w.a_stride, 8 * (tid % (DC / 8))));
    }
  };
  load(0);

  // ---- the state that enters
  const float* init;
  float* fin;
  lin_states(p, w, q.seq, h, init, fin);
  const bool several = q.len > q.rows;  // the segments' states are in the workspace
  float* ws = p.ws + (((int64_t)place * p.jobs + job) * p.heads + h) * (DC * DO) + wave * (CT * OT * 256) + lane * 4;
  f32x4 H[CT][OT];  // element r: c = 16 ct + g4 + r, o = 16 (OT wave + ot) + l16
  bool have = !STATE && (several || init);
#pragma unroll
  for (int ct = 0; ct < CT; ++ct)
#pragma unroll
    for (int ot = 0; ot < OT; ++ot) {
      H[ct][ot] = f32x4{0.0f, 0.0f, 0.0f, 0.0f};
      if (!STATE && several) {
        H[ct][ot] = *reinterpret_cast<const f32x4*>(ws + (ct * OT + ot) * 256);
      } else if (have) {
        const float* at = init + state_at(w, 16 * ct + g4, 16 * (OT * wave + ot) + l16);
        if (w.c_inner) {
          H[ct][ot] = *reinterpret_cast<const f32x4*>(at);
        } else {
#pragma unroll
          for (int r = 0; r < 4; ++r) H[ct][ot][r] = at[r * DO];
        }
      }
    }
  __syncthreads();  // the powers are there

  const int later = rev ? 0 : 1;  // the entering state decays before its first row, or behind the last
  // weights of the pairs (row t, row s <= t) of this wave's tiles, of E in row t, and of row s in E'
  float mw[3][4], iw[4], uw[2][8];
  int tile_t[3], tile_s[3];
#pragma unroll
  for (int i = 0; i < 3; ++i) {
    const int n = wave + 4 * i;
    tile_t[i] = n < 1 ? 0 : n < 3 ? 1 : n < 6 ? 2 : n < 10 ? 3 : 4;
    tile_s[i] = n - tile_t[i] * (tile_t[i] + 1) / 2;
#pragma unroll
    for (int r = 0; r < 4; ++r) {
      const int d = 16 * (tile_t[i] - tile_s[i]) + l16 - g4 - r;
      mw[i][r] = d >= 0 && d < kC ? w.m_scale * lds.power[d] : 0.0f;
    }
  }
#pragma unroll
  for (int tt = 0; tt < 4; ++tt) iw[tt] = w.e_scale * lds.power[16 * tt + l16 + later];
  auto set_uw = [&](int rows) {
#pragma unroll
    for (int ks = 0; ks < 2; ++ks)
#pragma unroll
      for (int e = 0; e < 8; ++e) {
        const int n = rows - 32 * ks - 2 * g4 - e - later;  // >= 0 for the rows that are there
        uw[ks][e] = n >= 0 ? w.u_scale * lds.power[n] : 0.0f;
      }
  };
  set_uw(kC);

  for (int t = 0; t < q.rows; t += kC) {
    const int rows = q.rows - t < kC ? q.rows - t : kC;
#pragma unroll
    for (int k = 0; k < NB; ++k) {
      const int at = tile_off<DC>(tid / (DC / 8) + k * (2048 / DC), 8 * (tid % (DC / 8)));
      *reinterpret_cast<u32x4v*>(&lds.b[at]) = br[k];
      if constexpr (!STATE) *reinterpret_cast<u32x4v*>(&lds.a[at]) = ar[k];
    }
#pragma unroll
    for (int k = 0; k < NO; ++k)
      *reinterpret_cast<u32x4v*>(&lds.c[tile_off<DO>(tid / (DO / 8) + k * (2048 / DO), 8 * (tid % (DO / 8)))]) = cr[k];
    __syncthreads();
    if (t + kC < q.rows) load(t + kC);

    f32x4 out[OT][4];  // element r: o = 16 (OT wave + ot) + g4 + r, row 16 tt + l16
    if constexpr (!STATE) {
      // M[t][s] = a^{t-s} (a_t . b_s), a lane with 4 consecutive s of a row t
#pragma unroll
      for (int i = 0; i < 3; ++i) {
        if (tile_t[i] > 3) continue;
        f32x4 acc = f32x4{0.0f, 0.0f, 0.0f, 0.0f};
#pragma unroll
        for (int ks = 0; ks < DC / 32; ++ks) {
          const u32x4v bs = lds16(&lds.b[tile_off<DC>(16 * tile_s[i] + l16, 32 * ks + 2 * g4)]);
          const u32x4v as = lds16(&lds.a[tile_off<DC>(16 * tile_t[i] + l16, 32 * ks + 2 * g4)]);
          acc = mfma_t<IO>::run(as_vec<IO>(bs), as_vec<IO>(as), acc);
        }
        uint32_t h0, h1, l0, l1;
        split2(acc[0] * mw[i][0], acc[1] * mw[i][1], h0, l0);
        split2(acc[2] * mw[i][2], acc[3] * mw[i][3], h1, l1);
        const int at = tile_off<kC>(16 * tile_t[i] + l16, 16 * tile_s[i] + g4);
        *reinterpret_cast<uint2*>(&lds.m[0][at]) = make_uint2(h0, h1);
        *reinterpret_cast<uint2*>(&lds.m[1][at]) = make_uint2(l0, l1);
      }
      // E's part: the accumulators of H are the operand as they lie, its k axis being
      // c = 16 (2 kk) + g4 + 0..3, then 16 (2 kk + 1) + g4 + 0..3; a is read in that order
#pragma unroll
      for (int ot = 0; ot < OT; ++ot)
#pragma unroll
        for (int tt = 0; tt < 4; ++tt) out[ot][tt] = f32x4{0.0f, 0.0f, 0.0f, 0.0f};
      if (have) {
#pragma unroll
        for (int kk = 0; kk < CT / 2; ++kk) {
          u32x4v eh[OT], el[OT];
#pragma unroll
          for (int ot = 0; ot < OT; ++ot)
#pragma unroll
            for (int i = 0; i < 2; ++i)
#pragma unroll
              for (int r = 0; r < 4; r += 2) {
                uint32_t hi, lo;
                split2(H[2 * kk + i][ot][r], H[2 * kk + i][ot][r + 1], hi, lo);
                eh[ot][2 * i + r / 2] = hi;
                el[ot][2 * i + r / 2] = lo;
              }
#pragma unroll
          for (int tt = 0; tt < 4; ++tt) {
            const uint2 a0 = lds8(&lds.a[tile_off<DC>(16 * tt + l16, 32 * kk + g4)]);
            const uint2 a1 = lds8(&lds.a[tile_off<DC>(16 * tt + l16, 32 * kk + 16 + g4)]);
            const Parts<IO> as(u32x4v{a0.x, a0.y, a1.x, a1.y});
#pragma unroll
            for (int ot = 0; ot < OT; ++ot) {
              out[ot][tt] = BF::run(bfv(el[ot]), as.hi, out[ot][tt]);
              if constexpr (kTwo) out[ot][tt] = BF::run(bfv(eh[ot]), as.lo, out[ot][tt]);
              out[ot][tt] = BF::run(bfv(eh[ot]), as.hi, out[ot][tt]);
            }
          }
        }
#pragma unroll
        for (int ot = 0; ot < OT; ++ot)
#pragma unroll
          for (int tt = 0; tt < 4; ++tt) out[ot][tt] *= iw[tt];
      }
      __syncthreads();  // M is there
    }
    u32x4v cf[2][OT];
#pragma unroll
    for (int ks = 0; ks < 2; ++ks)
#pragma unroll
      for (int ot = 0; ot < OT; ++ot) cf[ks][ot] = time_frag<DO>(lds.c, 32 * ks, OT * wave + ot, lane);
    if constexpr (!STATE) {
#pragma unroll
      for (int ks = 0; ks < 2; ++ks) {
        bf16x8 ch[OT], cl[OT];
#pragma unroll
        for (int ot = 0; ot < OT; ++ot) {
          const Parts<IO> cs(cf[ks][ot]);
          ch[ot] = cs.hi;
          cl[ot] = cs.lo;
        }
#pragma unroll
        for (int tt = 2 * ks; tt < 4; ++tt) {
          const int at = tile_off<kC>(16 * tt + l16, 32 * ks + 2 * g4);
          const bf16x8 mh = bfv(lds16(&lds.m[0][at])), ml = bfv(lds16(&lds.m[1][at]));
#pragma unroll
          for (int ot = 0; ot < OT; ++ot) {
            out[ot][tt] = BF::run(ch[ot], ml, out[ot][tt]);
            if constexpr (kTwo) out[ot][tt] = BF::run(cl[ot], mh, out[ot][tt]);
            out[ot][tt] = BF::run(ch[ot], mh, out[ot][tt]);
          }
        }
      }
      // ---- outputs: rows past the segment's last go nowhere
      const int64_t tok = rev ? (int64_t)q.begin + q.len - (q.t0 + t + rows) : (int64_t)q.begin + q.t0 + t;
      const int size = w.sum ? 4 : 2;
      const auto ov = rows_view(static_cast<char*>(w.out) + (tok * p.heads + h) * (DO * size), (int64_t)p.heads * (DO * size),
                                rows, DO * size);
#pragma unroll
      for (int tt = 0; tt < 4; ++tt) {
        const int row = 16 * tt + l16;
        const uint32_t at = row < rows ? (uint32_t)(rev ? rows - 1 - row : row) * (uint32_t)(p.heads * DO) : 0x1ffff000u;
#pragma unroll
        for (int ot = 0; ot < OT; ++ot) {
          const f32x4 v = out[ot][tt];
          const uint32_t col = (uint32_t)(16 * (OT * wave + ot) + g4);
          if (w.sum) __builtin_amdgcn_raw_buffer_store_b128(__builtin_bit_cast(u32x4v, v), ov, (at + col) * 4u, 0, 0);
          else vstore8(ov, (at + col) * 2u, pack2<IO>(v[0], v[1]), pack2<IO>(v[2], v[3]));
        }
      }
    }
    // ---- H <- a^rows H + sum_s a^{rows-1-s} b_s c_s^T
    if (!STATE && t + kC >= q.rows && !(q.last && fin)) break;  // nobody takes it
    if (rows < kC) set_uw(rows);
    if (have) {
      const float d = lds.decay[rows < kC ? 1 : 0];
#pragma unroll
      for (int ct = 0; ct < CT; ++ct)
#pragma unroll
        for (int ot = 0; ot < OT; ++ot)
#pragma unroll
          for (int r = 0; r < 4; ++r) H[ct][ot][r] = fmaf(d, H[ct][ot][r], H[ct][ot][r]);
    }
#pragma unroll
    for (int ks = 0; ks < 2; ++ks) {
      u32x4v part[3][OT];
#pragma unroll
      for (int ot = 0; ot < OT; ++ot)
#pragma unroll
        for (int e = 0; e < 4; ++e) {
          uint32_t v[3];
          split3(low16<IO>(cf[ks][ot][e]) * uw[ks][2 * e], high16<IO>(cf[ks][ot][e]) * uw[ks][2 * e + 1], v);
#pragma unroll
          for (int i = 0; i < 3; ++i) part[i][ot][e] = v[i];
        }
#pragma unroll
      for (int ct = 0; ct < CT; ++ct) {
        const Parts<IO> bs(time_frag<DC>(lds.b, 32 * ks, ct, lane));
#pragma unroll
        for (int ot = 0; ot < OT; ++ot) {
          f32x4 v = H[ct][ot];
          v = BF::run(bs.hi, bfv(part[2][ot]), v);
          if constexpr (kTwo) v = BF::run(bs.lo, bfv(part[1][ot]), v);
          v = BF::run(bs.hi, bfv(part[1][ot]), v);
          if constexpr (kTwo) v = BF::run(bs.lo, bfv(part[0][ot]), v);
          H[ct][ot] = BF::run(bs.hi, bfv(part[0][ot]), v);
        }
      }
    }
    have = true;
    __syncthreads();  // the tiles are used up
  }
#pragma unroll
  for (int ct = 0; ct < CT; ++ct)
#pragma unroll
    for (int ot = 0; ot < OT; ++ot) {
      if constexpr (STATE) {
        *reinterpret_cast<f32x4*>(ws + (ct * OT + ot) * 256) = H[ct][ot];
      } else if (q.last && fin) {
        float* at = fin + state_at(w, 16 * ct + g4, 16 * (OT * wave + ot) + l16);
        if (w.c_inner) {
          *reinterpret_cast<f32x4*>(at) = H[ct][ot];
        } else {
#pragma unroll
          for (int r = 0; r < 4; ++r) at[r * DO] = H[ct][ot][r];
        }
      }
    }
}

// ---- the states between the segments of a sequence ----------------------------------
// Workgroup = (sequence of several segments, head, walk, 1024 elements): E <- the
// sequence's first state; per segment, S <- E in the workspace and E <- decay E + S,
// S being the segment's own state (the last one has none: its walk ends with the
// sequence's).  The first state goes through the workspace too, so that a walk's
// end may overwrite it in the pool while others begin.
__global__ void __launch_bounds__(256) lin_pass_kernel(LinParams p) {
  constexpr int kAhead = 8;
  const int size = p.job[0].dc * p.job[0].dout, parts = size / 1024;
  int i = (int)blockIdx.x;
  const int e4 = i % parts * 256 + (int)threadIdx.x;
  i /= parts;
  const int job = i % p.jobs;
  i /= p.jobs;
  const int h = i % p.heads, s = i / p.heads;
  const LinWalk& w = p.job[job];
  int begin, len, first;
  if (p.cu) {
    begin = uniform(seq_row(p.cu, s, p.tokens));
    len = uniform(seq_row(p.cu, s + 1, p.tokens)) - begin;
    first = (begin >> p.logq) + s;
  } else {
    len = p.tokens / p.nseqs;
    first = s * (int)(((int64_t)len + ((int64_t)1 << p.logq) - 1) >> p.logq);
  }
  if (len <= ((int64_t)1 << p.logq)) return;
  const int n = (int)(((int64_t)len + ((int64_t)1 << p.logq) - 1) >> p.logq);
  const float d = (float)lin_power_m1(p.log_decay[h], 1 << p.logq);
  const float* init;
  float* fin;
  lin_states(p, w, s, h, init, fin);
  f32x4 E = f32x4{0.0f, 0.0f, 0.0f, 0.0f};
  if (init) {
    const int ct_n = w.dc / 16, ot_n = w.dout / 64, tile = e4 / 64, lane = e4 % 64;
    const int ot = tile % ot_n, ct = tile / ot_n % ct_n, wave = tile / ot_n / ct_n;
#pragma unroll
    for (int r = 0; r < 4; ++r)
      E[r] = init[state_at(w, 16 * ct + 4 * (lane / 16) + r, 16 * (ot_n * wave + ot) + lane % 16)];
  }
  const int64_t step = (int64_t)p.jobs * p.heads * size;
  float* ws = p.ws + (((int64_t)first * p.jobs + job) * p.heads + h) * size + 4 * (int64_t)e4;
  f32x4 S[kAhead];
  for (int c = 0; c < n; c += kAhead) {
#pragma unroll
    for (int k = 0; k < kAhead; ++k)
      if (c + k < n - 1) S[k] = *reinterpret_cast<const f32x4*>(ws + (c + k) * step);
#pragma unroll
    for (int k = 0; k < kAhead; ++k) {
      if (c + k < n) *reinterpret_cast<f32x4*>(ws + (c + k) * step) = E;
      if (c + k < n - 1) {
#pragma unroll
        for (int r = 0; r < 4; ++r) E[r] = fmaf(d, E[r], E[r]) + S[k][r];
      }
    }
  }
}

// ---- gradients of a shared key or value: the sum over the heads that share it ---------
// A thread has 4 channels of a row; parts in fp32, (tokens, heads, d).
template <int IO>
__global__ void __launch_bounds__(256) lin_share_kernel(const float* part, void* out, int64_t quads, int share, int d4) {
  const int64_t i = (int64_t)blockIdx.x * 256 + threadIdx.x;
  if (i >= quads) return;
  const f32x4* at = reinterpret_cast<const f32x4*>(part) + i / d4 * d4 * share + i % d4;
  f32x4 sum = at[0];
  for (int k = 1; k < share; ++k) sum += at[(int64_t)k * d4];
  reinterpret_cast<uint2*>(out)[i] = make_uint2(pack2<IO>(sum[0], sum[1]), pack2<IO>(sum[2], sum[3]));
}

// ---- one token of many requests -----------------------------------------------------
// Workgroup = (row, head, J passes over 1024 / dk rows p of the state): dk / 4 lanes
// share a row of H, each with 4 consecutive n, so that a wave reads whole kilobytes;
// all loads are issued before the first use.
template <int IO, int DK, int J>
__global__ void __launch_bounds__(256) lin_step_kernel(LinStepParams p) {
  constexpr int L = DK / 4, R = 256 / L;  // lanes of a state row, rows of a pass
  const int tid = threadIdx.x, l = tid % L;
  const int parts = p.dv / (R * J);
  const int part = (int)(blockIdx.x % (uint32_t)parts), i = (int)(blockIdx.x / (uint32_t)parts);
  const int r = i / p.heads, h = i - r * p.heads;
  const int slot = uniform(slot_of(p.slots, r, p.nslots));
  if (slot < 0) return;
  const int p0 = part * (R * J) + tid / L;
  float* H = p.state + (((int64_t)slot * p.heads + h) * p.dv + p0) * DK + 4 * l;
  f32x4 st[J];
#pragma unroll
  for (int j = 0; j < J; ++j) st[j] = *reinterpret_cast<const f32x4*>(H + j * (R * DK));
  const int kvh = h / p.share;
  float v[J];
#pragma unroll
  for (int j = 0; j < J; ++j) v[j] = load_io<IO>(p.v, r * p.v_stride + kvh * p.dv + p0 + j * R);
  f32x4 k, q;
#pragma unroll
  for (int e = 0; e < 4; ++e) {
    k[e] = load_io<IO>(p.k, r * p.k_stride + kvh * DK + 4 * l + e);
    q[e] = load_io<IO>(p.q, r * p.q_stride + h * DK + 4 * l + e);
  }
  const float d = (float)lin_power_m1(p.log_decay[h], 1);
#pragma unroll
  for (int j = 0; j < J; ++j) {
    float y = 0.0f;
#pragma unroll
    for (int e = 0; e < 4; ++e) {
      const float s = fmaf(v[j], k[e], fmaf(d, st[j][e], st[j][e]));
      st[j][e] = s;
      y = fmaf(s, q[e], y);
    }
    *reinterpret_cast<f32x4*>(H + j * (R * DK)) = st[j];
    y = row_sum(y);
    if constexpr (L == 32) {
      float even, odd;
      swap_rows(y, even, odd);
      y = even + odd;
    }
    if (l == 0) store_io<IO>(p.y, ((int64_t)r * p.heads + h) * p.dv + p0 + j * R, p.scale * y);
  }
}

template <int IO, int DC, int DO>
hipError_t launch_walk(const LinParams& p, hipStream_t st) {
  const dim3 grid((uint32_t)(p.places * p.heads * p.njobs));
  if (p.split) hipLaunchKernelGGL((lin_walk_kernel<IO, DC, DO, true>), grid, dim3(kWalkThreads), 0, st, p);
  else hipLaunchKernelGGL((lin_walk_kernel<IO, DC, DO, false>), grid, dim3(kWalkThreads), 0, st, p);
  return hipGetLastError();
}
template <int IO>
hipError_t launch_walks_io(LinParams p, hipStream_t st) {
  // walks of the same sides share a launch
  for (int j = 0; j < p.jobs; j += p.njobs) {
    p.job0 = j;
    p.njobs = 1;
    while (j + p.njobs < p.jobs && p.job[j + p.njobs].dc == p.job[j].dc && p.job[j + p.njobs].dout == p.job[j].dout)
      ++p.njobs;
    const int dc = p.job[j].dc, dout = p.job[j].dout;
    const hipError_t e = dc == 64 ? (dout == 64 ? launch_walk<IO, 64, 64>(p, st) : launch_walk<IO, 64, 128>(p, st))
                                  : (dout == 64 ? launch_walk<IO, 128, 64>(p, st) : launch_walk<IO, 128, 128>(p, st));
    if (e != hipSuccess) return e;
  }
  return hipSuccess;
}
template <int IO>
hipError_t launch_linattn_io(LinParams p, hipStream_t st) {
  if (p.split) {
    hipError_t e = launch_walks_io<IO>(p, st);
    if (e != hipSuccess) return e;
    const int parts = p.job[0].dc * p.job[0].dout / 1024;
    hipLaunchKernelGGL(lin_pass_kernel, dim3((uint32_t)(p.nseqs * p.heads * p.jobs * parts)), dim3(256), 0, st, p);
    e = hipGetLastError();
    if (e != hipSuccess) return e;
    p.split = 0;
  }
  const hipError_t e = launch_walks_io<IO>(p, st);
  if (e != hipSuccess) return e;
  for (int j = 0; j < p.jobs; ++j)
    if (p.job[j].sum) {
      const int64_t quads = (int64_t)p.tokens * (p.heads / p.share) * p.job[j].dout / 4;
      hipLaunchKernelGGL((lin_share_kernel<IO>), dim3((uint32_t)((quads + 255) / 256)), dim3(256), 0, st,
                         static_cast<const float*>(p.job[j].out), p.job[j].sum, quads, p.share, p.job[j].dout / 4);
      const hipError_t f = hipGetLastError();
      if (f != hipSuccess) return f;
    }
  return hipSuccess;
}

template <int IO, int DK>
hipError_t launch_step_dk(const LinStepParams& p, hipStream_t st) {
  constexpr int R = 1024 / DK;
  const int64_t rows = (int64_t)p.rows * p.heads;
  // a thread's rows of the state: few where the workgroups would not fill the GPU
  if (rows * (p.dv / (4 * R)) >= 4 * device_cus())
    hipLaunchKernelGGL((lin_step_kernel<IO, DK, 4>), dim3((uint32_t)(rows * (p.dv / (4 * R)))), dim3(256), 0, st, p);
  else
    hipLaunchKernelGGL((lin_step_kernel<IO, DK, 1>), dim3((uint32_t)(rows * (p.dv / R))), dim3(256), 0, st, p);
  return hipGetLastError();
}
template <int IO>
hipError_t launch_linattn_step_io(const LinStepParams& p, hipStream_t st) {
  return p.dk == 64 ? launch_step_dk<IO, 64>(p, st) : launch_step_dk<IO, 128>(p, st);
}

}  // namespace

hipError_t launch_linattn(const LinParams& p, hipStream_t st) {
  return p.io == SS_F16 ? launch_linattn_io<SS_F16>(p, st) : launch_linattn_io<SS_BF16>(p, st);
}
hipError_t launch_linattn_step(const LinStepParams& p, hipStream_t st) {
  return p.io == SS_F16 ? launch_linattn_step_io<SS_F16>(p, st) : launch_linattn_step_io<SS_BF16>(p, st);
}

}  // namespace ss
