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
#include <type_traits>

#include "ss_device.h"
#include "ss_internal.h"
#include "ss_mfma.h"
#include "ss_packed.h"

namespace ss {
namespace {

constexpr int kC = 64;  // rows of a chunk
typedef uint32_t u32x2v __attribute__((ext_vector_type(2)));

// 16-bit tiles of W columns in LDS: 4 rows lie together, 64 bytes of each in turn, with the
// 16-byte pieces of these exchanged by the 4 rows' number: piece c of row r is at
//   W 8 (r / 4) + 256 (c' / 4) + 64 (r % 4) + 16 (c' % 4),   c' = c ^ tile_x(r / 4).
// The 16 rows of a fragment read (16 or 8 bytes a lane), in whichever halves they are
// served, and the 4 consecutive rows (32 bytes each) of two of a transposing read's
// lane groups lie in different banks; further columns (of 32) and rows (of 16) are
// immediate offsets.
__device__ __forceinline__ constexpr int tile_x(int four) {  // Gray code of the quarter of 16 rows
  const int q = four & 3;
  return (q >> 1) | (((q ^ (q >> 1)) & 1) << 1);
}
template <int W>
__device__ __forceinline__ constexpr int tile_at(int row, int col) {  // in bytes
  static_assert(W == 64 || W == 128, "tile width");
  const int c = (col >> 3) ^ tile_x(row >> 2);
  return W * 8 * (row >> 2) + 256 * (c >> 2) + 64 * (row & 3) + 16 * (c & 3) + 2 * (col & 7);
}
// LDS by 32-bit address
template <class T>
__device__ __forceinline__ __attribute__((address_space(3))) T* lds_ptr(uint32_t at) {
  return (__attribute__((address_space(3))) T*)(uintptr_t)at;
}
__device__ __forceinline__ uint32_t lds_addr(void* p) { return (uint32_t)(uintptr_t)(__attribute__((address_space(3))) char*)p; }
__device__ __forceinline__ u32x4v lds16(uint32_t at) { return *lds_ptr<u32x4v>(at); }
__device__ __forceinline__ u32x2v lds8(uint32_t at) { return *lds_ptr<u32x2v>(at); }

// Where a lane's fragments lie in a tile:
// rows l16, the columns 32 ks + 8 (lane / 16) ..: row_frag + 256 ks
template <int W>
__device__ __forceinline__ int row_frag(int lane) { return tile_at<W>(lane % 16, 8 * (lane / 16)); }
// rows l16, the columns 16 i + 4 (lane / 16) ..: (quad_frag ^ 32 (i % 2)) + 256 (i / 2)
template <int W>
__device__ __forceinline__ int quad_frag(int lane) { return tile_at<W>(lane % 16, 4 * (lane / 16)); }
// the columns 16 i .. of 32 rows as an operand whose k axis is the row; even and odd: the lane's
// place for even i and for odd i, each the other's for the rows 4 further on
template <int W>
__device__ __forceinline__ int time_frag(int lane) { return tile_at<W>(8 * (lane / 16) + lane % 16 / 4, 4 * (lane % 4)); }
template <int W>
__device__ __forceinline__ u32x4v read_time_frag(uint32_t at, uint32_t next) {
  const s16x4 lo = __builtin_amdgcn_ds_read_tr16_b64_v4i16(lds_ptr<s16x4>(at));
  const s16x4 hi = __builtin_amdgcn_ds_read_tr16_b64_v4i16(lds_ptr<s16x4>(next + W * 8));
  return __builtin_bit_cast(u32x4v, __builtin_shufflevector(lo, hi, 0, 1, 2, 3, 4, 5, 6, 7));
}

// A sequence's rows, and the places of a packed one's chunks, numbered over all of them (an empty one has one)
struct LinSeq {
  int begin, len, first, chunks;
};
__device__ __forceinline__ LinSeq lin_seq_of(int s, int begin, int end) {  // a packed one
  LinSeq q;
  q.begin = uniform(begin);
  end = uniform(end);
  q.len = end > q.begin ? end - q.begin : 0;
  q.first = q.begin / kC + s;
  q.chunks = q.len > 0 ? (q.len + kC - 1) / kC : 1;
  return q;
}
__device__ __forceinline__ LinSeq lin_seq(const LinParams& p, int s) {
  if (p.cu) return lin_seq_of(s, seq_row(p.cu, s, p.tokens), seq_row(p.cu, s + 1, p.tokens));
  const int len = p.tokens / p.nseqs;
  return {s * len, len, 0, (len + kC - 1) / kC};
}
// What pieces of packed sequences share out: the places from the first row's on, of the sequences up to
// the last row, as many to each piece as these take.  (The empty ones behind the last row, which a batch's
// maps have for every request without a prompt, would leave most pieces without a row.)  The launch for
// the states between pieces finds them and leaves them in the workspace, in the place of the state that
// would enter the first piece, for the launches behind it.
struct LinPlaces {
  int seqs;  // sequences before the empty ones behind the last row
  int base;  // the first place
  int span;  // places of a piece
  int row;   // of up to 64 sequences: the lane's first row
};
__device__ __forceinline__ LinPlaces lin_places(const LinParams& p) {
  const int lane = threadIdx.x % 64;
  // a search for the first one that begins at the end, as find_chunk's, its first probes loaded with the ends
  int lo = 0, n = p.nseqs;
  auto probe = [&](int step) { return lane * step < n ? seq_row(p.cu, lo + lane * step, p.tokens) : 0x7fffffff; };
  int step = (n + 63) >> 6, row = probe(step);
  const int rows = row;
  const int first = seq_row(p.cu, 0, p.tokens), last = seq_row(p.cu, p.nseqs, p.tokens);
  const int base = uniform(first) / kC, end = uniform(last);
  for (;;) {
    const int cnt = (int)__builtin_popcountll(__builtin_amdgcn_ballot_w64(row < end));  // <= ceil(n / step): lo stays inside
    if (cnt == 0) break;
    lo += (cnt - 1) * step + 1;
    n -= (cnt - 1) * step + 1;
    n = n < step - 1 ? n : step - 1;
    if (n <= 0) break;
    step = (n + 63) >> 6;
    row = probe(step);
  }
  // never more than span was planned for: end / kC + lo <= tokens / kC + nseqs
  const int used = end / kC + lo - base, span = (used + p.pieces - 1) / p.pieces;
  return {lo, base, span > 2 ? span : 2, rows};
}
__device__ __forceinline__ int32_t* lin_places_at(const LinParams& p) {
  return reinterpret_cast<int32_t*>(p.ws + (int64_t)p.pieces * p.stride * (p.job[0].dc * p.job[0].dout));
}
__device__ __forceinline__ LinPlaces lin_places_found(const LinParams& p) {
  const int lane = threadIdx.x % 64;
  const int32_t* at = lin_places_at(p);
  const int seqs = at[0], base = at[1], span = at[2], row = lane < p.nseqs ? seq_row(p.cu, lane, p.tokens) : 0;
  return {uniform(seqs), uniform(base), uniform(span), row};
}
__device__ __forceinline__ int lin_find(const LinParams& p, const LinPlaces& pl, int place) {  // as find_chunk
  if (p.nseqs > 64) return find_chunk<6>(p.cu, pl.seqs, p.tokens, place).seq;
  const int lane = threadIdx.x % 64;
  const int cnt = (int)__builtin_popcountll(__builtin_amdgcn_ballot_w64(lane < pl.seqs && pl.row / kC + lane <= place));
  return cnt < 1 ? 0 : cnt - 1;
}
// Some of a sequence's chunks, in the walk's order
struct LinRows {
  int seq, begin, len;  // the sequence
  int t0, rows;
  bool last;            // the sequence's last row is among them
  int slot;             // of the piece's states in the workspace
};
__device__ __forceinline__ LinRows lin_rows(const LinSeq& q, int s, int i0, int i1, int slot) {
  const int end = i1 < q.chunks ? i1 * kC : q.len;
  return {s, q.begin, q.len, i0 * kC, end - i0 * kC, i1 >= q.chunks, slot};
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
// A sequence without rows: its first state is its last one
__device__ __forceinline__ void lin_empty(const LinParams& p, const LinWalk& w, int seq, int h) {
  const float* init;
  float* fin;
  lin_states(p, w, seq, h, init, fin);
  if (!fin || fin == init) return;
  for (int i = (int)threadIdx.x; i < w.dc * w.dout / 4; i += (int)blockDim.x)
    reinterpret_cast<f32x4*>(fin)[i] = init ? reinterpret_cast<const f32x4*>(init)[i] : f32x4{0.0f, 0.0f, 0.0f, 0.0f};
}
// element (c, o) of a state in memory: (dv, dk), c being the side that is contracted with a
__device__ __forceinline__ int state_at(const LinWalk& w, int c, int o) { return w.c_inner ? o * w.dc + c : c * w.dout + o; }

// exp(n g), its exponent formed in 64 bits; n = 0 has no decay, whatever g
__device__ __forceinline__ float lin_power(float g, int n) {
  if (n == 0) return 1.0f;
  const double x = (double)n * (double)g * 1.4426950408889634074;
  if (x <= -200.0) return 0.0f;  // below fp32's smallest
  if (!(x < 200.0)) return x > 0.0 ? __builtin_inff() : (float)x;
  const double whole = rint(x);
  return ldexpf(exp2_hw((float)(x - whole)), (int)whole);
}
// H <- exp(n g) H.  A slow decay's own rounding would add up over the chunks that it takes: there the
// factor is exp(n g) - 1, and H <- H + (exp(n g) - 1) H.  That of a fast one would leave a rounding of the
// old H, where only exp(n g) H is left: there it is exp(n g).  The sign bit tells them apart.
__device__ __forceinline__ float lin_decay(float g, int n) {
  const double x = n ? (double)n * (double)g : 0.0;
  if (!(x > -0.25 && x <= 0.0)) return lin_power(g, n);
  double s = 1.0;  // the power series: 0.25^12 / 13! is below 2^-56
#pragma unroll
  for (int k = 12; k > 1; --k) s = fma(s, x * (1.0 / k), 1.0);
  return -fabsf((float)(s * x));
}
__device__ __forceinline__ bool lin_slow(float decay) { return __float_as_int(decay) < 0; }

// ---- the walk ----------------------------------------------------------------------
// Four waves, each with a quarter of the columns o of the outputs and of the state, the
// state as accumulators: what a wave reads of LDS meets two tiles of o (heads of 128).
// Two workgroups share a CU, so that one's products, the other's vector work
// (both halves of the walk take as long) and the reads of LDS go on at once.  A chunk's
// operands come into LDS without registers in between: b, which is in use from a
// chunk's begin to its end, a chunk ahead in one of two buffers; a, once the last
// chunk's is used, for the next; c, which is not needed before the pairs' weights are
// made, at its chunk's begin.  Eight waves with a tile each read LDS twice as often (a layer
// of 8 x 2048 rows, 12 heads of 128 x 128, bf16: 352 us against 335 then); operands through
// registers left one workgroup to a CU (682 against 369).
// Bound by instructions of both kinds that seldom run at once: a chunk of two workgroups takes a CU 12
// thousand cycles, and its 164 matrix and some 720 vector instructions a wave, most of them taking
// fp32 values apart, a SIMD 5.2 and 5.8 thousand (counters: 22 % and 26 % of the time, waves waiting in a
// third of it).  Traced one by one, that layer's walk takes 57 us forward, with 26 and 10 for the states
// between the pieces, and 156, 14 and 7 for the gradients (calls of both together: 250 us, 180 TFLOP/s of
// the formula's operations); fp16, in more parts, 32769 rows of 16 heads of 64 x 128 109, 43 and 12.
constexpr int kWaves = 4, kWalkThreads = 64 * kWaves;
// Weights by number, of rows in E' (0 .. 63), powers of a (64 .. 129) and the decays
// (lin_decay) of a whole chunk and of the last one (160, 161): with M they lie in the columns of
// its first rows that no pair has, so that two workgroups have LDS's 160 KB
constexpr int kPowers = 64, kDecays = 160;
template <int DC, int DO, bool STATE>
struct WalkLds {
  __attribute__((aligned(16))) char m[STATE ? 1024 : 2 * kC * kC * 2];
  __attribute__((aligned(16))) char a[STATE ? 16 : kC * DC * 2];
  __attribute__((aligned(16))) char b[2][kC * DC * 2];
  __attribute__((aligned(16))) char c[STATE ? 2 : 1][kC * DO * 2];
  __device__ __forceinline__ float* weight(int i) {
    return reinterpret_cast<float*>(m + (STATE ? 4 * i : tile_at<kC>(i / 16, 32 + 2 * (i % 16))));
  }
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

// ss_mfma.h's split2 and split3 with a remainder in one instruction: v - p of a pair of bf16 p is a
// dot product with (-1, 0) or (0, -1) onto v, exact as the remainder is (checked on the chip).
// The constants come from registers, for as an inline operand -1 is one of fp32.
struct Remainder {
  uint32_t low, high;
  __device__ __forceinline__ Remainder() {
    asm("s_mov_b32 %0, 0xbf80" : "=s"(low));
    asm("s_mov_b32 %0, 0xbf800000" : "=s"(high));
  }
  __device__ __forceinline__ void take(uint32_t p, float& v0, float& v1) const {
    v0 = __builtin_amdgcn_fdot2_f32_bf16(__builtin_bit_cast(bf16x2, p), __builtin_bit_cast(bf16x2, low), v0, false);
    v1 = __builtin_amdgcn_fdot2_f32_bf16(__builtin_bit_cast(bf16x2, p), __builtin_bit_cast(bf16x2, high), v1, false);
  }
  // The parts of eight values that outlive them, where the builtin overwrites its v: in assembly, with
  // the three cycles that a dot product's result takes to other instructions at the end.  The
  // values may be matrix results: the first parts, made before, have waited for them.
  __device__ __forceinline__ void split8_of(const float (&v)[8], u32x4v& hi, u32x4v& lo) const {
    float r[8];
#pragma unroll
    for (int k = 0; k < 4; ++k) hi[k] = pack2<SS_BF16>(v[2 * k], v[2 * k + 1]);
    asm("v_dot2_f32_bf16 %0, %8, %20, %12\n\tv_dot2_f32_bf16 %1, %8, %21, %13\n\t"
        "v_dot2_f32_bf16 %2, %9, %20, %14\n\tv_dot2_f32_bf16 %3, %9, %21, %15\n\t"
        "v_dot2_f32_bf16 %4, %10, %20, %16\n\tv_dot2_f32_bf16 %5, %10, %21, %17\n\t"
        "v_dot2_f32_bf16 %6, %11, %20, %18\n\tv_dot2_f32_bf16 %7, %11, %21, %19\n\ts_nop 2"
        : "=&v"(r[0]), "=&v"(r[1]), "=&v"(r[2]), "=&v"(r[3]), "=&v"(r[4]), "=&v"(r[5]), "=&v"(r[6]), "=&v"(r[7])
        : "v"(hi[0]), "v"(hi[1]), "v"(hi[2]), "v"(hi[3]), "v"(v[0]), "v"(v[1]), "v"(v[2]), "v"(v[3]), "v"(v[4]), "v"(v[5]),
          "v"(v[6]), "v"(v[7]), "s"(low), "s"(high));
#pragma unroll
    for (int k = 0; k < 4; ++k) lo[k] = pack2<SS_BF16>(r[2 * k], r[2 * k + 1]);
  }
  template <int N>
  __device__ __forceinline__ void split(float v0, float v1, uint32_t (&w)[N]) const {
#pragma unroll
    for (int k = 0; k < N; ++k) {
      w[k] = pack2<SS_BF16>(v0, v1);
      if (k + 1 < N) take(w[k], v0, v1);
    }
  }
};

// v as two fp16 parts, |v - hi - lo| <= 2^-22 |v| where |v| is within a factor of 2^15 of the
// largest that its scale is taken from (2^-38 of that one below).  Every output column o has a
// scale of its own: one that holds an infinity, or far larger values, takes nothing from the others.
__device__ __forceinline__ void split2_f16(float v0, float v1, uint32_t& hi, uint32_t& lo) {
  hi = pack2<SS_F16>(v0, v1);
  lo = pack2<SS_F16>(v0 - low16<SS_F16>(hi), v1 - high16<SS_F16>(hi));
}
// the power of two that takes the largest magnitude of the lanes l16 of all rows to 2^14 .. 2^15, and its inverse
struct Scale {
  float to, from;
};
__device__ __forceinline__ Scale column_scale(float most) {
  float x, y;
  swap_rows(most, x, y);
  swap_halves(fmaxf(x, y), x, y);
  const int e = (int)(__float_as_uint(fmaxf(x, y)) >> 23) & 255;
  const int field = 268 - e < 253 ? 268 - e : 253;
  return {__uint_as_float((uint32_t)field << 23), __uint_as_float((uint32_t)(254 - field) << 23)};
}

// A barrier behind this wave's LDS accesses and its memory accesses but the last AHEAD
// (they end in their order): loads ahead stay in flight through it
template <int AHEAD>
__device__ __forceinline__ void lds_barrier() {
  if constexpr (AHEAD < 0) asm volatile("s_waitcnt lgkmcnt(0)\n\ts_barrier" ::: "memory");
  else asm volatile("s_waitcnt vmcnt(%0) lgkmcnt(0)\n\ts_barrier" ::"n"(AHEAD) : "memory");
}

// 16 bytes a lane from a view (its four words) into LDS at `to` + 16 lane.  In assembly, for the
// compiler would wait for such a load before the next access to LDS that it cannot tell apart
// from its target.  A load keeps its place among the barriers (lds_barrier), which tell both
// the compiler and the waves when LDS changes; between them accesses may pass it, for nobody
// reads its target before the next barrier that waits for memory, or after the last one.
__device__ __forceinline__ void lds_load(u32x4v view, uint32_t to, uint32_t off, int ahead) {
  asm volatile("s_mov_b32 m0, %0\n\ts_nop 0\n\tbuffer_load_dwordx4 %1, %2, %3 offen lds" ::"s"(uniform((int)to)), "v"(off),
               "s"(view), "s"(uniform(ahead)));  // m0 is nobody else's
}

// The rows of a chunk into a tile: a wave's load fills 1 KB of it, 16 bytes a lane in the
// lanes' order, so that the exchange of pieces is made on the memory's side.  In a
// chunk of fewer rows those behind the last one repeat it: no weight but 0 meets
// them, and their outputs go nowhere.
template <int W> constexpr int tile_loads() { return kC * W / 512 / kWaves; }
template <int W>
struct TileLoad {
  static constexpr int kRows = 512 / W, kLoads = tile_loads<W>();  // rows of a load, loads of a wave
  uint32_t whole;  // the offset of this lane's piece of the wave's first load in a whole chunk
  // this lane's row and piece of the wave's first load
  __device__ __forceinline__ static void lane_piece(int wave, int lane, int& row, int& piece) {
    const int in = W == 128 ? lane : lane % 32;
    row = wave * kRows + lane / 4 % 4 + (W == 128 ? 0 : lane / 32 * 4);
    piece = (in / 16 * 4 + in % 4) ^ tile_x(row >> 2);
  }
  __device__ __forceinline__ TileLoad(int wave, int lane, int64_t stride, bool rev) {
    int row, piece;
    lane_piece(wave, lane, row, piece);
    whole = (uint32_t)(rev ? kRows * kWaves - 1 - row : row) * (uint32_t)(stride * 2) + (uint32_t)piece * 16u;
  }
  __device__ __forceinline__ void load(char* tile, const char* at, int64_t stride, int rows, bool rev, int wave, int lane) const {
    const uint64_t base = (uint64_t)(uintptr_t)at;
    const u32x4v v = {(uint32_t)uniform((int)(uint32_t)base), (uint32_t)uniform((int)((base >> 32) & 0xffffu)),
                      (uint32_t)uniform((int)view_bytes(stride * 2, rows, W * 2)), (uint32_t)kRsrcWord3};
    const uint32_t to = lds_addr(tile) + (uint32_t)wave * 1024u;
    if (rows == kC) {
#pragma unroll
      for (int k = 0; k < kLoads; ++k)
        lds_load(v, to + kWaves * 1024 * k, whole, (rev ? kLoads - 1 - k : k) * (kRows * kWaves) * (int)(stride * 2));
      return;
    }
    int row, piece;
    lane_piece(wave, opaque(lane), row, piece);
#pragma unroll
    for (int k = 0; k < kLoads; ++k) {
      const int r = row + k * (kRows * kWaves), in = r < rows ? r : rows - 1;
      lds_load(v, to + kWaves * 1024 * k, (uint32_t)(rev ? rows - 1 - in : in) * (uint32_t)(stride * 2) + (uint32_t)piece * 16u, 0);
    }
  }
};

template <int IO, int DC, int DO, bool STATE, bool FULL>
__device__ __forceinline__ void walk(const LinParams& p, WalkLds<DC, DO, STATE>& lds, int job, int h, const LinRows& q) {
  constexpr int CT = DC / 16, OT = DO / 64;  // tiles of a wave's state: all of c, a quarter of o
  constexpr int kPairs = 3;                  // 16 x 16 tiles of pairs a wave, at the most
  constexpr bool kTwo = IO == SS_F16;
  constexpr int kPlane = kC * kC * 2, kTile = kC * DC * 2;
  const int tid = threadIdx.x, wave = uniform(tid / 64);
  const int lane = tid % 64, l16 = lane % 16, g4 = 4 * (lane / 16);
  const LinWalk& w = p.job[job];
  const int kvh = h / p.share;

  // ---- loads for the chunk that begins at row t of these, in the walk's order
  const bool rev = w.rev != 0;
  auto chunk_rows = [&](int t) { return q.rows - t < kC ? q.rows - t : kC; };
  auto chunk_tok = [&](int t, int rows) {
    return rev ? (int64_t)q.begin + q.len - (q.t0 + t + rows) : (int64_t)q.begin + q.t0 + t;
  };
  auto chunk_at = [&](const void* base, int t, int64_t stride, int head, int cols) {
    return static_cast<const char*>(base) + (chunk_tok(t, chunk_rows(t)) * stride + head * cols) * 2;
  };
  const TileLoad<DC> la(wave, lane, w.a_stride, rev), lb_(wave, lane, w.b_stride, rev);
  const TileLoad<DO> lc(wave, lane, w.c_stride, rev);
  auto load_a = [&](int t) {
    la.load(lds.a, chunk_at(w.a, t, w.a_stride, w.a_kv ? kvh : h, DC), w.a_stride, chunk_rows(t), rev, wave, lane);
  };
  auto load_b = [&](int t, int turn) {
    lb_.load(lds.b[turn], chunk_at(w.b, t, w.b_stride, w.b_kv ? kvh : h, DC), w.b_stride, chunk_rows(t), rev, wave, lane);
  };
  auto load_c = [&](int t, int turn) {
    lc.load(lds.c[turn], chunk_at(w.c, t, w.c_stride, w.c_kv ? kvh : h, DO), w.c_stride, chunk_rows(t), rev, wave, lane);
  };
  load_b(0, 0);
  if constexpr (STATE) load_c(0, 0);
  else load_a(0);

  const float g = p.log_decay[h];
  const int later = rev ? 0 : 1;  // the entering state decays before its first row, or behind the last
  auto set_weights = [&](int rows) {  // of the rows in E'
    if (tid < kC) *lds.weight(tid) = tid < rows ? w.u_scale * lin_power(g, rows - tid - later) : 0.0f;
  };
  set_weights(chunk_rows(0));
  if (tid >= 64 && tid < 64 + kC + 2) *lds.weight(kPowers + tid - 64) = lin_power(g, tid - 64);
  if (tid >= 192 && tid < 194) *lds.weight(kDecays + tid - 192) = lin_decay(g, tid == 192 ? kC : q.rows % kC);
  if constexpr (!STATE) {  // M's 16 x 16 tiles above the diagonal that are read with their neighbours
    if (tid < 128) {
      const int tile = tid / 32 % 2, row = tid / 2 % 16;
      *reinterpret_cast<u32x4v*>(lds.m + tid / 64 * kPlane + tile_at<kC>(32 * tile + row, 16 + 32 * tile + 8 * (tid % 2))) =
          u32x4v{0, 0, 0, 0};
    }
  }

  // ---- the state that enters
  const float* init;
  float* fin;
  lin_states(p, w, q.seq, h, init, fin);
  // a sequence of several pieces: its states between them are in the workspace (LinParams)
  const bool several = q.len > q.rows;
  float* ws = p.ws + (!STATE && q.t0 > 0 ? p.pieces * (int64_t)p.stride + q.slot : q.slot) * (DC * DO) + wave * (CT * OT * 256) + lane * 4;
  f32x4 H[CT][OT];  // element r: c = 16 ct + g4 + r, o = 16 (OT wave + ot) + l16
  bool have = !STATE && (several || init);
  auto each = [&](auto f) {
#pragma unroll
    for (int ct = 0; ct < CT; ++ct)
#pragma unroll
      for (int ot = 0; ot < OT; ++ot) f(ct, ot);
  };
  const int at0 = state_at(w, g4, 16 * OT * wave + l16), at_c1 = state_at(w, 16, 0), at_o1 = state_at(w, 0, 16);
  if (!STATE && several) {
    each([&](int ct, int ot) { H[ct][ot] = *reinterpret_cast<const f32x4*>(ws + (ct * OT + ot) * 256); });
  } else if (have && w.c_inner) {
    each([&](int ct, int ot) { H[ct][ot] = *reinterpret_cast<const f32x4*>(init + at0 + ct * at_c1 + ot * at_o1); });
  } else if (have) {
    each([&](int ct, int ot) {
#pragma unroll
      for (int r = 0; r < 4; ++r) H[ct][ot][r] = init[at0 + ct * at_c1 + ot * at_o1 + r * DO];
    });
  } else {
    each([&](int ct, int ot) { H[ct][ot] = f32x4{0.0f, 0.0f, 0.0f, 0.0f}; });
  }
  lds_barrier<0>();  // the weights and the first chunk are there

  // weights of the pairs (row t, row s <= t) of this wave's tiles and of E in row t
  float mw[kPairs][4], iw[4];
  int tile_t[kPairs], tile_s[kPairs];
  if constexpr (!STATE) {
#pragma unroll
    for (int i = 0; i < kPairs; ++i) {
      const int n = wave + kWaves * i < 10 ? wave + kWaves * i : 9;  // two waves have the last tile too: the same values
      tile_t[i] = n < 1 ? 0 : n < 3 ? 1 : n < 6 ? 2 : 3;
      tile_s[i] = n - tile_t[i] * (tile_t[i] + 1) / 2;
#pragma unroll
      for (int r = 0; r < 4; ++r) {
        const int d = 16 * (tile_t[i] - tile_s[i]) + l16 - g4 - r;
        mw[i][r] = d >= 0 && d < kC ? w.m_scale * *lds.weight(kPowers + d) : 0.0f;
      }
    }
#pragma unroll
    for (int tt = 0; tt < 4; ++tt) iw[tt] = w.e_scale * *lds.weight(kPowers + 16 * tt + l16 + later);
  }
  // the lane's places in the tiles
  const uint32_t at_a = lds_addr(lds.a), at_b = lds_addr(lds.b[0]), at_c = lds_addr(lds.c[0]), at_m = lds_addr(lds.m);
  const uint32_t rows_dc = row_frag<DC>(lane), quad_dc = quad_frag<DC>(lane), time_dc = time_frag<DC>(lane);
  // of c: the wave's first tile of o, and the same one's rows 4 further on (its second tile's are exchanged)
  const uint32_t time_do = time_frag<DO>(lane) ^ (uint32_t)(32 * (OT * wave % 2));
  const uint32_t c_at = at_c + time_do + 256 * (OT * wave / 2), c_next = at_c + (time_do ^ 32u) + 256 * (OT * wave / 2);
  const uint32_t m_rows = at_m + row_frag<kC>(lane), m_quad = quad_frag<kC>(lane);
  const uint32_t row_bytes = (uint32_t)(p.heads * DO) * (w.sum ? 4u : 2u);
  // the lane's columns of an output's row, in bytes
  const uint32_t out_col = (uint32_t)(32 * OT * wave) * (w.sum ? 2u : 1u) +
                           (w.sum || OT == 1 ? (uint32_t)g4 * (w.sum ? 4u : 2u) : (uint32_t)(lane / 16 % 2 * 32 + lane / 32 * 16));
  const uint32_t out_at = (uint32_t)(rev ? kC - 1 - l16 : l16) * row_bytes + out_col;

  const Remainder rem;
  // a chunk; false behind the last
  auto chunk = [&](int t, auto which) {
    constexpr int turn = decltype(which)::value;
    const int rows = chunk_rows(t);
    const bool more = t + kC < q.rows;
    if (STATE && more) {
      load_b(t + kC, turn ^ 1);
      load_c(t + kC, turn ^ 1);
    }
    if (!STATE && t > 0 && rows < kC) set_weights(rows);

    f32x4 out[OT][4];  // element r: o = 16 (OT wave + ot) + g4 + r, row 16 tt + l16
    if constexpr (!STATE) {
      // M[t][s] = a^{t-s} (a_t . b_s), a lane with 4 consecutive s of a row t
      constexpr int KS = DC / 32;
      u32x4v bs[kPairs][KS], as[kPairs][KS];
#pragma unroll
      for (int i = 0; i < kPairs; ++i) {
        const uint32_t b_at = opaque(rows_dc) + at_b + turn * kTile + tile_s[i] * (16 * DC * 2);
        const uint32_t a_at = opaque(rows_dc) + at_a + tile_t[i] * (16 * DC * 2);
#pragma unroll
        for (int ks = 0; ks < KS; ++ks) {
          bs[i][ks] = lds16(b_at + 256 * ks);
          as[i][ks] = lds16(a_at + 256 * ks);
        }
      }
      load_c(t, 0);
      if (more) load_b(t + kC, turn ^ 1);
      f32x4 pair[kPairs];
#pragma unroll
      for (int i = 0; i < kPairs; ++i) pair[i] = f32x4{0.0f, 0.0f, 0.0f, 0.0f};
#pragma unroll
      for (int ks = 0; ks < KS; ++ks)
#pragma unroll
        for (int i = 0; i < kPairs; ++i) pair[i] = mfma_t<IO>::run(as_vec<IO>(bs[i][ks]), as_vec<IO>(as[i][ks]), pair[i]);
#pragma unroll
      for (int i = 0; i < kPairs; ++i) {
        uint32_t m0[2], m1[2];
        rem.split(pair[i][0] * mw[i][0], pair[i][1] * mw[i][1], m0);
        rem.split(pair[i][2] * mw[i][2], pair[i][3] * mw[i][3], m1);
        const uint32_t at = (opaque(m_quad) ^ (uint32_t)(32 * (tile_s[i] % 2))) + at_m + tile_t[i] * (16 * kC * 2) + 256 * (tile_s[i] / 2);
        *lds_ptr<u32x2v>(at) = u32x2v{m0[0], m1[0]};
        *lds_ptr<u32x2v>(at + kPlane) = u32x2v{m0[1], m1[1]};
      }
      // E's part: the accumulators of H are the operand as they lie, its k axis being
      // c = 16 i + g4 + 0..3, then 16 (i + 2) + g4 + 0..3; a is read in that order
#pragma unroll
      for (int ot = 0; ot < OT; ++ot)
#pragma unroll
        for (int tt = 0; tt < 4; ++tt) out[ot][tt] = f32x4{0.0f, 0.0f, 0.0f, 0.0f};
      if (have) {
        const uint32_t even = opaque(quad_dc) + at_a, odd = (opaque(quad_dc) ^ 32u) + at_a;
        Scale sc[OT];
        if constexpr (kTwo) {
#pragma unroll
          for (int ot = 0; ot < OT; ++ot) {
            float most = 0.0f;
#pragma unroll
            for (int ct = 0; ct < CT; ++ct)
#pragma unroll
              for (int r = 0; r < 4; ++r) most = fmaxf(most, fabsf(H[ct][ot][r]));
            sc[ot] = column_scale(most);
          }
        }
#pragma unroll
        for (int kk = 0; kk < CT / 2; ++kk) {
          const int i0 = 4 * (kk / 2) + kk % 2;
          const uint32_t from = (kk % 2 ? odd : even) + 512 * (kk / 2);
          u32x4v eh[OT], el[OT], as[4];
#pragma unroll
          for (int tt = 0; tt < 4; ++tt) {
            const u32x2v a0 = lds8(from + tt * (16 * DC * 2)), a1 = lds8(from + tt * (16 * DC * 2) + 256);
            as[tt] = u32x4v{a0[0], a0[1], a1[0], a1[1]};
          }
#pragma unroll
          for (int ot = 0; ot < OT; ++ot) {
            float v[8];
#pragma unroll
            for (int e = 0; e < 8; ++e) v[e] = kTwo ? H[i0 + e / 4 * 2][ot][e % 4] * sc[ot].to : H[i0 + e / 4 * 2][ot][e % 4];
            if constexpr (kTwo) {
#pragma unroll
              for (int k = 0; k < 4; ++k) {
                uint32_t hi, lo;
                split2_f16(v[2 * k], v[2 * k + 1], hi, lo);
                eh[ot][k] = hi;
                el[ot][k] = lo;
              }
            } else {
              rem.split8_of(v, eh[ot], el[ot]);
            }
          }
#pragma unroll
          for (int ot = 0; ot < OT; ++ot)
#pragma unroll
            for (int tt = 0; tt < 4; ++tt) out[ot][tt] = mfma_t<IO>::run(as_vec<IO>(el[ot]), as_vec<IO>(as[tt]), out[ot][tt]);
#pragma unroll
          for (int ot = 0; ot < OT; ++ot)
#pragma unroll
            for (int tt = 0; tt < 4; ++tt) out[ot][tt] = mfma_t<IO>::run(as_vec<IO>(eh[ot]), as_vec<IO>(as[tt]), out[ot][tt]);
        }
#pragma unroll
        for (int ot = 0; ot < OT; ++ot) {
          if constexpr (kTwo) {  // the lane's four columns' scales, from the lanes that have these as l16
            f32x4 from;
#pragma unroll
            for (int r = 0; r < 4; ++r) from[r] = __shfl(sc[ot].from, g4 + r, 64);
#pragma unroll
            for (int tt = 0; tt < 4; ++tt) out[ot][tt] *= from;
          }
#pragma unroll
          for (int tt = 0; tt < 4; ++tt) out[ot][tt] *= iw[tt];
        }
      }
      // M and c are there; b's next loads, issued behind c's, may be on their way
      if (more) lds_barrier<tile_loads<DC>()>();
      else lds_barrier<0>();
      if (more) load_a(t + kC);
      asm volatile("" ::: "memory");  // the outputs' stores come behind
    }
    u32x4v cf[2][OT];
#pragma unroll
    for (int ks = 0; ks < 2; ++ks)
#pragma unroll
      for (int ot = 0; ot < OT; ++ot) {
        const int at = (STATE ? turn * (kC * DO * 2) : 0) + 32 * ks * (DO * 2);
        cf[ks][ot] = read_time_frag<DO>((ot ? c_next : c_at) + at, (ot ? c_at : c_next) + at);
      }
    if constexpr (!STATE) {
#pragma unroll
      for (int ks = 0; ks < 2; ++ks) {
        bf16x8 mh[4], ml[4], ch[OT], cl[OT];
#pragma unroll
        for (int tt = 2 * ks; tt < 4; ++tt) {
          const uint32_t at = m_rows + tt * (16 * kC * 2) + 256 * ks;
          mh[tt] = bfv(lds16(at));
          ml[tt] = bfv(lds16(at + kPlane));
        }
#pragma unroll
        for (int ot = 0; ot < OT; ++ot) {
          const Parts<IO> cs(cf[ks][ot]);
          ch[ot] = cs.hi;
          cl[ot] = cs.lo;
        }
#pragma unroll
        for (int ot = 0; ot < OT; ++ot)
#pragma unroll
          for (int tt = 2 * ks; tt < 4; ++tt) out[ot][tt] = BF::run(ch[ot], ml[tt], out[ot][tt]);
        if constexpr (kTwo) {
#pragma unroll
          for (int ot = 0; ot < OT; ++ot)
#pragma unroll
            for (int tt = 2 * ks; tt < 4; ++tt) out[ot][tt] = BF::run(cl[ot], mh[tt], out[ot][tt]);
        }
#pragma unroll
        for (int ot = 0; ot < OT; ++ot)
#pragma unroll
          for (int tt = 2 * ks; tt < 4; ++tt) out[ot][tt] = BF::run(ch[ot], mh[tt], out[ot][tt]);
      }
      // ---- outputs: rows past the last go nowhere
      const int size = w.sum ? 4 : 2;
      const auto ov = rows_view(static_cast<char*>(w.out) + (chunk_tok(t, rows) * p.heads + h) * (DO * size), row_bytes, rows, DO * size);
#pragma unroll
      for (int tt = 0; tt < 4; ++tt) {
        uint32_t at = out_at;
        int ahead = (rev ? -16 * tt : 16 * tt) * (int)row_bytes;
        if (rows < kC) {
          const int row = 16 * tt + l16;
          at = row < rows ? (uint32_t)(rev ? rows - 1 - row : row) * row_bytes + out_col : 0x3fffe000u;
          ahead = 0;
        } else if (rev) {
          at += (uint32_t)ahead;
          ahead = 0;
        }
        if (w.sum) {
#pragma unroll
          for (int ot = 0; ot < OT; ++ot)
            __builtin_amdgcn_raw_buffer_store_b128(__builtin_bit_cast(u32x4v, out[ot][tt]), ov, at + 64 * ot, ahead, 0);
        } else if constexpr (OT == 1) {
          const f32x4 v = out[0][tt];
          __builtin_amdgcn_raw_buffer_store_b64(u32x2v{pack2<IO>(v[0], v[1]), pack2<IO>(v[2], v[3])}, ov, at, ahead, 0);
        } else {  // lane groups exchange their halves, so that each has 8 columns of one of the tiles
          const f32x4 v0 = out[0][tt], v1 = out[OT - 1][tt];
          const auto x = __builtin_amdgcn_permlane16_swap(pack2<IO>(v0[0], v0[1]), pack2<IO>(v1[0], v1[1]), false, false);
          const auto y = __builtin_amdgcn_permlane16_swap(pack2<IO>(v0[2], v0[3]), pack2<IO>(v1[2], v1[3]), false, false);
          __builtin_amdgcn_raw_buffer_store_b128(u32x4v{x[0], y[0], x[1], y[1]}, ov, at, ahead, 0);
        }
      }
    }
    // ---- H <- a^rows H + sum_s a^{rows-1-s} b_s c_s^T
    if (!STATE && !more && !(q.last && fin)) return false;  // nobody takes it
    const uint32_t even = opaque(time_dc) + at_b + turn * kTile, odd = (opaque(time_dc) ^ 32u) + at_b + turn * kTile;
    auto b_frag = [&](int ks, int ct) {
      const uint32_t at = 32 * ks * (DC * 2) + 256 * (ct / 2);
      return as_vec<IO>(read_time_frag<DC>((ct % 2 ? odd : even) + at, (ct % 2 ? even : odd) + at));
    };
    // w_s c_s of the rows 32 ks + 2 g4 + 2 e, + 1
    auto weighted = [&](int ks, int e, int ot, float& v0, float& v1) {
      const f32x2 u = *lds_ptr<f32x2>(lds_addr(lds.weight(32 * ks + 2 * g4 + 2 * e)));
      v0 = low16<IO>(cf[ks][ot][e]) * u[0];
      v1 = high16<IO>(cf[ks][ot][e]) * u[1];
    };
    const float d = __int_as_float(uniform(__float_as_int(*lds.weight(kDecays + (rows < kC ? 1 : 0)))));
    auto decay_state = [&]() {
      if (lin_slow(d)) {
        each([&](int ct, int ot) {
#pragma unroll
          for (int r = 0; r < 4; ++r) H[ct][ot][r] = fmaf(d, H[ct][ot][r], H[ct][ot][r]);
        });
      } else {
        each([&](int ct, int ot) { H[ct][ot] *= d; });
      }
    };
    if constexpr (!kTwo) {
      constexpr int kParts = FULL ? 3 : 2;
      decay_state();
#pragma unroll
      for (int ks = 0; ks < 2; ++ks) {
        u32x4v part[OT][kParts];
#pragma unroll
        for (int ot = 0; ot < OT; ++ot)
#pragma unroll
          for (int e = 0; e < 4; ++e) {
            float v0, v1;
            uint32_t v[kParts];
            weighted(ks, e, ot, v0, v1);
            rem.split(v0, v1, v);
#pragma unroll
            for (int i = 0; i < kParts; ++i) part[ot][i][e] = v[i];
          }
#pragma unroll
        for (int c0 = 0; c0 < CT; c0 += 4) {
          typename mfma_t<IO>::V bs[4];
#pragma unroll
          for (int i = 0; i < 4; ++i) bs[i] = b_frag(ks, c0 + i);
#pragma unroll
          for (int j = kParts - 1; j >= 0; --j)
#pragma unroll
            for (int i = 0; i < 4; ++i)
#pragma unroll
              for (int ot = 0; ot < OT; ++ot) H[c0 + i][ot] = mfma_t<IO>::run(bs[i], as_vec<IO>(part[ot][j]), H[c0 + i][ot]);
        }
      }
    } else {
      float wc[2][OT][8];
      Scale sc[OT];
#pragma unroll
      for (int ot = 0; ot < OT; ++ot) {
        float most = 0.0f;
#pragma unroll
        for (int ks = 0; ks < 2; ++ks)
#pragma unroll
          for (int e = 0; e < 4; ++e) {
            weighted(ks, e, ot, wc[ks][ot][2 * e], wc[ks][ot][2 * e + 1]);
            most = fmaxf(most, fmaxf(fabsf(wc[ks][ot][2 * e]), fabsf(wc[ks][ot][2 * e + 1])));
          }
        sc[ot] = column_scale(most);
      }
      u32x4v part[2][OT][2];
#pragma unroll
      for (int ks = 0; ks < 2; ++ks)
#pragma unroll
        for (int ot = 0; ot < OT; ++ot)
#pragma unroll
          for (int e = 0; e < 4; ++e) {
            uint32_t hi, lo;
            split2_f16(wc[ks][ot][2 * e] * sc[ot].to, wc[ks][ot][2 * e + 1] * sc[ot].to, hi, lo);
            part[ks][ot][0][e] = hi;
            part[ks][ot][1][e] = lo;
          }
      decay_state();
#pragma unroll
      for (int c0 = 0; c0 < CT; c0 += 4) {
        f32x4 own[4][OT];  // at their scale
#pragma unroll
        for (int i = 0; i < 4; ++i)
#pragma unroll
          for (int ot = 0; ot < OT; ++ot) own[i][ot] = f32x4{0.0f, 0.0f, 0.0f, 0.0f};
#pragma unroll
        for (int ks = 0; ks < 2; ++ks) {
          typename mfma_t<IO>::V bs[4];
#pragma unroll
          for (int i = 0; i < 4; ++i) bs[i] = b_frag(ks, c0 + i);
#pragma unroll
          for (int j = 1; j >= 0; --j)
#pragma unroll
            for (int i = 0; i < 4; ++i)
#pragma unroll
              for (int ot = 0; ot < OT; ++ot) own[i][ot] = mfma_t<IO>::run(bs[i], as_vec<IO>(part[ks][ot][j]), own[i][ot]);
        }
#pragma unroll
        for (int i = 0; i < 4; ++i)
#pragma unroll
          for (int ot = 0; ot < OT; ++ot)
#pragma unroll
            for (int r = 0; r < 4; ++r)
              H[c0 + i][ot][r] = fmaf(own[i][ot][r], sc[ot].from, H[c0 + i][ot][r]);
      }
    }
    have = true;
    // the next chunk's a and b are there (the outputs' stores, four at the least, issued behind them,
    // may be on their way), and everyone is done with this one
    if (more) lds_barrier<STATE ? 0 : 4>();
    return more;
  };
  for (int t = 0; chunk(t, std::integral_constant<int, 0>{}) && chunk(t + kC, std::integral_constant<int, 1>{}); t += 2 * kC) {
  }
  if constexpr (STATE) {
    each([&](int ct, int ot) { *reinterpret_cast<f32x4*>(ws + (ct * OT + ot) * 256) = H[ct][ot]; });
  } else if (q.last && fin && w.c_inner) {
    each([&](int ct, int ot) { *reinterpret_cast<f32x4*>(fin + at0 + ct * at_c1 + ot * at_o1) = H[ct][ot]; });
  } else if (q.last && fin) {
    each([&](int ct, int ot) {
#pragma unroll
      for (int r = 0; r < 4; ++r) fin[at0 + ct * at_c1 + ot * at_o1 + r * DO] = H[ct][ot][r];
    });
  }
}

// Workgroups: p.whole sequences of a walk each, then p.pieces of p.stride walks each.  A piece is
// `span` chunks of a sequence; or, of packed ones, `span` chunk places, and in them the rest
// of a sequence, whole ones and the begin of another.  For the states between the pieces
// only a piece's last sequence matters, if it goes on behind.
struct LinWork {
  int seq, job, h, piece, slot;  // piece < 0: the whole sequence
};
__device__ __forceinline__ int xcd_logical(int bid, int nb) {  // as xcd_logical_block, among nb workgroups
  const int per = nb / 8, rem = nb % 8, xcd = bid % 8;
  return xcd * per + (xcd < rem ? xcd : rem) + bid / 8;
}
template <bool STATE>
__device__ __forceinline__ LinWork lin_work(const LinParams& p) {
  LinWork k{0, 0, 0, -1, 0};
  const int bid = (int)blockIdx.x, whole = STATE ? 0 : p.whole;
  int u;
  if (bid < whole) {
    u = xcd_logical(bid, whole);
  } else {
    k.slot = xcd_logical(bid - whole, (int)gridDim.x - whole);
    k.piece = k.slot / p.stride;
    u = p.whole + k.slot % p.stride;
  }
  k.job = u % p.jobs;
  u /= p.jobs;
  k.h = u % p.heads;
  k.seq = u / p.heads;  // 0 in pieces of packed sequences
  return k;
}
template <int IO, int DC, int DO, bool STATE, bool FULL>
__device__ __forceinline__ void walk_piece(const LinParams& p, WalkLds<DC, DO, STATE>& lds, const LinWork& k) {
  const bool over = k.piece >= 0 && p.cu;
  const LinPlaces pl = !over ? LinPlaces{p.nseqs, 0, p.span, 0} : STATE ? lin_places(p) : lin_places_found(p);
  const int c0 = pl.base + k.piece * pl.span, c1 = c0 + pl.span;
  if constexpr (STATE) {
    int s = k.seq;
    if (over) {
      if (k.slot == 0 && threadIdx.x < 3) lin_places_at(p)[threadIdx.x] = threadIdx.x == 0 ? pl.seqs : threadIdx.x == 1 ? pl.base : pl.span;
      if (pl.seqs == 0) return;
      s = lin_find(p, pl, c1 - 1);
    }
    const LinSeq q = lin_seq(p, s);
    const int i0 = c0 > q.first ? c0 - q.first : 0, i1 = c1 - q.first;
    if (i1 <= i0 || i1 >= q.chunks) return;
    walk<IO, DC, DO, STATE, FULL>(p, lds, k.job, k.h, lin_rows(q, s, i0, i1, k.slot));
  } else {
    const LinWalk& w = p.job[k.job];
    if (p.zero_rest && p.cu) {  // rows of no sequence have outputs of zero
      const int lead = seq_row(p.cu, 0, p.tokens), behind = seq_row(p.cu, p.nseqs, p.tokens);
      const int end = behind > lead ? behind : lead, tid = threadIdx.x;
      for (int r = k.piece < 0 ? k.seq : k.piece; r < lead + p.tokens - end; r += k.piece < 0 ? p.nseqs : p.pieces) {
        const int64_t at = ((int64_t)(r < lead ? r : end + r - lead) * p.heads + k.h) * DO;
        if (tid < DO) {
          if (w.sum) static_cast<float*>(w.out)[at + tid] = 0.0f;
          else static_cast<uint16_t*>(w.out)[at + tid] = 0;
        }
      }
    }
    int s = k.seq, end = s + 1;
    if (over) {
      // the empty sequences behind the last row, 64 at a time: those whose state is to be written
      for (int s0 = pl.seqs + 64 * k.piece; w.fin && s0 < p.nseqs; s0 += 64 * p.pieces) {
        const int e = s0 + (int)threadIdx.x % 64;
        const bool writes = e < p.nseqs && (!p.pool || (slot_of(p.slots, e, p.nslots) >= 0 && !(p.has_state && p.has_state[e])));
        for (uint64_t left = __builtin_amdgcn_ballot_w64(writes); left; left &= left - 1)
          lin_empty(p, w, s0 + (int)__builtin_ctzll(left), k.h);
      }
      if (pl.seqs == 0) return;
      s = lin_find(p, pl, c0);
      end = pl.span < pl.seqs - s ? s + pl.span : pl.seqs;  // no more sequences than places, whatever the offsets hold
    }
    for (; s < end; ++s) {
      const LinSeq q = lin_seq(p, s);
      int i0 = 0, i1 = q.chunks;
      if (k.piece >= 0) {
        if (q.first >= c1) break;
        i0 = c0 > q.first ? c0 - q.first : 0;
        i1 = i1 < c1 - q.first ? i1 : c1 - q.first;
        if (i0 >= i1) continue;
      }
      if (q.len == 0) {
        lin_empty(p, w, s, k.h);
        continue;
      }
      lds_barrier<-1>();  // everyone is done with the sequence before
      walk<IO, DC, DO, STATE, FULL>(p, lds, k.job, k.h, lin_rows(q, s, i0, i1, k.slot));
    }
  }
}
template <int IO, int DC, int DO, bool STATE, bool FULL>
__global__ void __launch_bounds__(kWalkThreads, 2) lin_walk_kernel(LinParams p) {
  __shared__ WalkLds<DC, DO, STATE> lds;
  walk_piece<IO, DC, DO, STATE, FULL>(p, lds, lin_work<STATE>(p));
}
// The gradients' three walks where dv = DC and dk = DO differ, or where dh0 is asked for: dq's and
// dk's have the states' sides the one way, dv's the other, and dh0 is what dv's ends with; in one
// launch they run beside each other
template <int IO, int DC, int DO, bool STATE, bool FULL>
__global__ void __launch_bounds__(kWalkThreads, 2) lin_walks_kernel(LinParams p) {
  __shared__ union {
    WalkLds<DC, DO, STATE> two;
    WalkLds<DO, DC, STATE> one;
  } lds;
  const LinWork k = lin_work<STATE>(p);
  if (k.job < 2) walk_piece<IO, DC, DO, STATE, false>(p, lds.two, k);
  else walk_piece<IO, DO, DC, STATE, FULL>(p, lds.one, k);
}

// ---- the states between the pieces of a sequence ------------------------------------
// Workgroup = (sequence of several pieces, head, walk, 1024 elements), a packed one found
// among the sequences or, where these are more, as the one that crosses the end of its
// first piece: E <- the sequence's first state; per piece, E to the workspace and E <- decay E + S, S being
// the state of the sequence's rows in the piece (the last one has none: its walk ends
// with the sequence's).  The first state goes through the workspace too, so that a
// walk's end may overwrite it in the pool while others begin.  Bound by memory: the layer's 57
// MB take 10 us; eight states are read ahead.
__global__ void __launch_bounds__(256) lin_pass_kernel(LinParams p) {
  constexpr int kAhead = 8;
  const int size = p.job[0].dc * p.job[0].dout, parts = size / 1024;
  int i = (int)blockIdx.x;
  const int e4 = i % parts * 256 + (int)threadIdx.x;
  i /= parts;
  const int slot = i % p.stride, u = p.whole + slot, job = u % p.jobs, h = u / p.jobs % p.heads;
  const LinWalk& w = p.job[job];
  int s = p.cu ? i / p.stride : u / p.jobs / p.heads, span = p.span;
  LinSeq q;
  if (p.cu) {
    const int begin = seq_row(p.cu, s, p.tokens), next = seq_row(p.cu, s + 1, p.tokens);  // loaded with the places'
    const LinPlaces pl = lin_places_found(p);
    if (pl.seqs == 0) return;
    span = pl.span;
    q = lin_seq_of(s, begin, next);
    const int ends = (s + 1) * span;  // of piece s
    const bool by_end = p.nseqs >= p.pieces;
    if (by_end) {
      s = lin_find(p, pl, pl.base + ends);
      q = lin_seq(p, s);
    }
    q.first -= pl.base;
    if (q.first < 0 || (by_end && (q.first >= ends || q.first < ends - span))) return;
  } else {
    q = lin_seq(p, s);
  }
  // offsets out of order may name places behind the last piece
  const int first = q.first / span, end = (q.first + q.chunks - 1) / span + 1;
  const int n = (end < p.pieces ? end : p.pieces) - first;
  if (n < 2) return;
  const int64_t step = (int64_t)p.stride * size;
  float* own = p.ws + ((int64_t)first * p.stride + slot) * size + 4 * (int64_t)e4;
  float* enter = own + p.pieces * step;
  f32x4 S[kAhead];
  auto load = [&](int c) {
#pragma unroll
    for (int k = 0; k < kAhead; ++k)
      if (c + k < n - 1) S[k] = *reinterpret_cast<const f32x4*>(own + (c + k) * step);
  };
  load(0);  // while the decays are made and the first state comes
  const float g = p.log_decay[h];
  float d = lin_decay(g, ((first + 1) * span - q.first) * kC);  // over the first piece's rows
  const float whole = lin_decay(g, span * kC);
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
  for (int c = 0; c < n; c += kAhead) {
    if (c) load(c);
#pragma unroll
    for (int k = 0; k < kAhead; ++k) {
      if (c + k < n) *reinterpret_cast<f32x4*>((c + k ? enter : own) + (c + k) * step) = E;
      if (c + k < n - 1) {
#pragma unroll
        for (int r = 0; r < 4; ++r) E[r] = fmaf(d, E[r], lin_slow(d) ? E[r] : 0.0f) + S[k][r];
        d = whole;
      }
    }
  }
}

// ---- gradients of shared keys and values: the sums over the heads that share them -----
// A thread has 4 channels of a row of one of them; parts in fp32, (tokens, heads, d).
template <int IO>
__global__ void __launch_bounds__(256) lin_share_kernel(LinParams p) {
  int64_t i = (int64_t)blockIdx.x * 256 + threadIdx.x;
  const int64_t rows = (int64_t)p.tokens * (p.heads / p.share);
  const int dk4 = p.job[1].dout / 4, dv4 = p.job[2].dout / 4;
  const bool second = i >= rows * dk4;
  if (second) i -= rows * dk4;
  const int d4 = second ? dv4 : dk4;
  if (i >= rows * d4) return;
  const LinWalk& w = p.job[second ? 2 : 1];
  const f32x4* at = static_cast<const f32x4*>(w.out) + i / d4 * d4 * p.share + i % d4;
  f32x4 sum = at[0];
  for (int k = 1; k < p.share; ++k) sum += at[(int64_t)k * d4];
  static_cast<uint2*>(w.sum)[i] = make_uint2(pack2<IO>(sum[0], sum[1]), pack2<IO>(sum[2], sum[3]));
}

// ---- one token of many requests -----------------------------------------------------
// Workgroup = (row, head, four passes over 1024 / dk rows p of the state): dk / 4 lanes
// share a row of H, each with 4 consecutive n, so that a wave reads whole kilobytes;
// all loads are issued before the first use.  Bound by HBM (201 rows of 16 heads, 128 x 64, 210 MB of
// states in and out: 32 us, 6.5 TB/s with what the last level cache holds).  Four times as many
// workgroups of one pass are not sooner with few rows either (16 heads of 128 x 128, other states
// every time: one row 3.0 us against 3.2, 2 rows 3.6 and 3.6, 16 rows 10.6 and 10.1, 32 15.1 and 15.1).
template <int IO, int DK>
__global__ void __launch_bounds__(256) lin_step_kernel(LinStepParams p) {
  constexpr int L = DK / 4, R = 256 / L, J = 4;  // lanes of a state row, rows of a pass, passes
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
  const float d = lin_decay(p.log_decay[h], 1);
#pragma unroll
  for (int j = 0; j < J; ++j) {
    float y = 0.0f;
#pragma unroll
    for (int e = 0; e < 4; ++e) {
      const float s = fmaf(v[j], k[e], fmaf(d, st[j][e], lin_slow(d) ? st[j][e] : 0.0f));
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

template <int IO, int DC, int DO, bool FULL>
hipError_t launch_walk(const LinParams& p, hipStream_t st) {
  const dim3 grid((uint32_t)(p.split ? (p.pieces - 1) * p.stride : p.whole + p.pieces * p.stride)), threads(kWalkThreads);
  if constexpr (DC != DO || FULL) {
    if (p.jobs == 3) {
      if (p.split) hipLaunchKernelGGL((lin_walks_kernel<IO, DC, DO, true, FULL>), grid, threads, 0, st, p);
      else hipLaunchKernelGGL((lin_walks_kernel<IO, DC, DO, false, FULL>), grid, threads, 0, st, p);
      return hipGetLastError();
    }
  }
  if (p.split) hipLaunchKernelGGL((lin_walk_kernel<IO, DC, DO, true, FULL>), grid, threads, 0, st, p);
  else hipLaunchKernelGGL((lin_walk_kernel<IO, DC, DO, false, FULL>), grid, threads, 0, st, p);
  return hipGetLastError();
}
// fp16's weighted rows are two parts (split2_f16).  Of bf16's, three keep fp32's error in the last states;
// where a walk leaves none, its outputs are all that shows and two do (8 rows of 2048 tokens, 12 heads of
// 128 x 128, forward and gradients: 242 us against 264 with three): a term is then off by 2^-18, as the
// pairs' weights are.  dq's and dk's walks leave none, so that they are the same with and without dh0; the
// last bit of y (dv) may go by final_state (dh0).
template <int IO, int DC, int DO>
hipError_t launch_walk(const LinParams& p, hipStream_t st) {
  bool full = false;
  for (int j = 0; j < p.jobs; ++j) full = full || p.job[j].fin;
  if constexpr (IO == SS_BF16)
    if (full) return launch_walk<IO, DC, DO, true>(p, st);
  return launch_walk<IO, DC, DO, false>(p, st);
}
template <int IO>
hipError_t launch_walks_io(const LinParams& p, hipStream_t st) {
  const int dc = p.job[0].dc, dout = p.job[0].dout;
  return dc == 64 ? (dout == 64 ? launch_walk<IO, 64, 64>(p, st) : launch_walk<IO, 64, 128>(p, st))
                  : (dout == 64 ? launch_walk<IO, 128, 64>(p, st) : launch_walk<IO, 128, 128>(p, st));
}
template <int IO>
hipError_t launch_linattn_io(LinParams p, hipStream_t st) {
  if (p.split) {
    hipError_t e = launch_walks_io<IO>(p, st);
    if (e != hipSuccess) return e;
    const int parts = p.job[0].dc * p.job[0].dout / 1024;
    const int seqs = !p.cu ? 1 : p.nseqs < p.pieces ? p.nseqs : p.pieces - 1;
    hipLaunchKernelGGL(lin_pass_kernel, dim3((uint32_t)(seqs * p.stride * parts)), dim3(256), 0, st, p);
    e = hipGetLastError();
    if (e != hipSuccess) return e;
    p.split = 0;
  }
  const hipError_t e = launch_walks_io<IO>(p, st);
  if (e != hipSuccess || p.jobs < 3 || !p.job[1].sum) return e;
  const int64_t quads = (int64_t)p.tokens * (p.heads / p.share) * ((p.job[1].dout + p.job[2].dout) / 4);
  hipLaunchKernelGGL((lin_share_kernel<IO>), dim3((uint32_t)((quads + 255) / 256)), dim3(256), 0, st, p);
  return hipGetLastError();
}

template <int IO>
hipError_t launch_linattn_step_io(const LinStepParams& p, hipStream_t st) {
  const dim3 grid((uint32_t)((int64_t)p.rows * p.heads * (p.dk * p.dv / 4096)));
  if (p.dk == 64) hipLaunchKernelGGL((lin_step_kernel<IO, 64>), grid, dim3(256), 0, st, p);
  else hipLaunchKernelGGL((lin_step_kernel<IO, 128>), grid, dim3(256), 0, st, p);
  return hipGetLastError();
}

}  // namespace

hipError_t launch_linattn(const LinParams& p, hipStream_t st) {
  return p.io == SS_F16 ? launch_linattn_io<SS_F16>(p, st) : launch_linattn_io<SS_BF16>(p, st);
}
hipError_t launch_linattn_step(const LinStepParams& p, hipStream_t st) {
  return p.io == SS_F16 ? launch_linattn_step_io<SS_F16>(p, st) : launch_linattn_step_io<SS_BF16>(p, st);
}

}  // namespace ss
