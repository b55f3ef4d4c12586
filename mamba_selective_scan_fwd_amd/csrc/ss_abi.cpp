// ss_abi.cpp -- the C ABI of libss.so: host-side validation and dispatch.
// Every check runs before any HIP call; a failing check returns its status
// and leaves the device untouched.
#include <hip/hip_runtime_api.h>

#include <cstdint>
#include <cstring>

#include "../../include/ss.h"
#include "ss_internal.h"

namespace {

constexpr int64_t kTile = 64;
constexpr int64_t kMaxDstate = 16;
constexpr int64_t kChPerBlock = 16;
// below this many wavefronts a forward splits the time axis into chunks
constexpr int64_t kTargetWaves = 1024;
// the largest grid, in workgroups of up to 512 threads, whose work-item count
// fits the 32-bit grid size of a dispatch
constexpr int64_t kMaxGrid = ((int64_t)1 << 23) - 1;
constexpr int64_t kMaxSeqlen = (int64_t)1 << 24;
constexpr int64_t kConvBwdGroups = 1024;  // workgroups of the convolution's backward, where the sizes allow

bool aligned(const void* ptr) { return ((uintptr_t)ptr & 15u) == 0; }

int64_t elem_size(int32_t io) { return io == SS_F32 ? 4 : 2; }

ss_status check_problem(const ss_problem* p, bool need_seqlen) {
  if (!p) return SS_ERR_NULL_ARG;
  if (p->batch < 1 || p->dim < 1 || p->dstate < 1) return SS_ERR_BAD_SHAPE;
  if (need_seqlen && p->seqlen < 1) return SS_ERR_BAD_SHAPE;
  if (p->dstate > kMaxDstate) return SS_ERR_UNSUPPORTED;
  if (p->io_dtype != SS_F32 && p->io_dtype != SS_F16 && p->io_dtype != SS_BF16) return SS_ERR_BAD_DTYPE;
  // keep every element index far from int64 overflow and every grid within kMaxGrid
  const int64_t lim = (int64_t)1 << 40;
  if (p->batch > lim || p->dim > lim) return SS_ERR_BAD_SHAPE;
  // kernels address a row with 32-bit offsets
  if (need_seqlen && p->seqlen > kMaxSeqlen) return SS_ERR_BAD_SHAPE;
  const double ch = (double)p->batch * (double)p->dim;
  if (ch * (double)(need_seqlen ? p->seqlen : 1) * kMaxDstate > 9.0e18) return SS_ERR_BAD_SHAPE;
  if (ch / kChPerBlock * 2.0 > (double)kMaxGrid) return SS_ERR_BAD_SHAPE;
  return SS_OK;
}

struct FwdPlan {
  int64_t nchunks;
  int64_t chunk_len;
  size_t workspace;
};

// The forward's persistent work queue (problems that do not split time): units
// of kQueueChunk steps of a 16-channel block, for ragged rows or for more row
// blocks than the GPU holds at once.  Workspace: a control block, one flag per
// unit, one carried state per (channel, chunk).
// 2048 steps: a unit hands its state on through memory (a store, a flag and a
// load, each a trip to the memory side), which shorter units pay more often
// (units of 256, 512, 1024, 1536 and 2048 steps measured 0.63, 0.52, 0.47,
// 0.48 and 0.47 ms on the ragged mamba-2.8b workload; 0.71, 0.71, 0.69 and
// 0.69 ms from 512 up on the uniform layer).
constexpr int64_t kQueueChunk = 2048;
constexpr int64_t kQueueMaxRows = 256;
constexpr int64_t kFinalPerCu = 3;  // readout workgroups resident per CU (the headline's launch)
struct QueueLayout {
  int64_t chunks;
  size_t flags, carry, total;  // byte offsets and size
};
size_t align256(size_t v) { return (v + 255) & ~(size_t)255; }
QueueLayout queue_layout(const ss_problem* p) {
  QueueLayout q;
  q.chunks = (p->seqlen + kQueueChunk - 1) / kQueueChunk;
  const int64_t ch_blocks = (p->dim + kChPerBlock - 1) / kChPerBlock;
  q.flags = 256;
  q.carry = q.flags + align256((size_t)(p->batch * ch_blocks * q.chunks) * 4);
  q.total = q.carry + (size_t)(p->batch * p->dim * q.chunks) * 16 * sizeof(float);
  return q;
}

// The time-chunked scan's workspace (one launch): a control block (its second
// word is the error word), then per (channel, chunk, state) the chunk pairs
// (P, S) and per (channel, group but the last, state) the group pairs, one
// 64-bit word each.  Groups hold G chunks, G the least power of two with
// G * G >= K, so that a chunk's entry state composes at most G - 1 chunk
// pairs and K / G group pairs.
struct ChunkLayout {
  int64_t group, ngroups;
  size_t pairs, gpairs, total;  // byte offsets and size
};
ChunkLayout chunk_layout(const ss_problem* p, int64_t nchunks) {
  ChunkLayout c;
  c.group = 1;
  while (c.group * c.group < nchunks) c.group *= 2;
  c.ngroups = (nchunks + c.group - 1) / c.group;
  c.pairs = 256;
  c.gpairs = c.pairs + (size_t)(p->batch * p->dim * nchunks) * 16 * sizeof(uint64_t);
  c.total = c.gpairs + (size_t)(p->batch * p->dim * (c.ngroups - 1)) * 16 * sizeof(uint64_t);
  return c;
}

FwdPlan plan_fwd(const ss_problem* p) {
  FwdPlan pl;
  const int64_t tiles = (p->seqlen + kTile - 1) / kTile;
  const int64_t ch_blocks = (p->dim + kChPerBlock - 1) / kChPerBlock;
  const int64_t waves = p->batch * ch_blocks * 4;
  int64_t k = 1;
  if (waves < kTargetWaves) {
    k = (kTargetWaves + waves - 1) / waves;  // at most kTargetWaves / 4 chunks
    if (k > tiles) k = tiles;
  }
  int64_t tiles_per_chunk = (tiles + k - 1) / k;
  // a time-chunked scan works on both halves of a chunk at once: an even
  // number of tiles per chunk
  if (k > 1) tiles_per_chunk += tiles_per_chunk & 1;
  pl.chunk_len = tiles_per_chunk * kTile;
  pl.nchunks = (p->seqlen + pl.chunk_len - 1) / pl.chunk_len;
  pl.workspace = pl.nchunks > 1 ? chunk_layout(p, pl.nchunks).total : 0;
  return pl;
}

ss_status from_hip(hipError_t e) { return e == hipSuccess ? SS_OK : SS_ERR_HIP; }

// A device buffer as a byte range; a null pointer or zero size is no buffer.
struct Span {
  const void* ptr;
  size_t n;
};
bool share_bytes(const Span& a, const Span& b) {
  if (!a.ptr || !b.ptr || !a.n || !b.n) return false;
  const uintptr_t x = (uintptr_t)a.ptr, y = (uintptr_t)b.ptr;
  return x < y + b.n && y < x + a.n;
}
// True when an output shares a byte with an input (unless it is that input
// itself and inplace[i][j] allows it) or with another output.
template <size_t NI, size_t NO>
bool conflict(const Span (&in)[NI], const Span (&out)[NO], const bool (*inplace)[NI] = nullptr) {
  for (size_t o = 0; o < NO; ++o) {
    for (size_t i = 0; i < NI; ++i)
      if (share_bytes(out[o], in[i]) &&
          !(inplace && inplace[o][i] && out[o].ptr == in[i].ptr && out[o].n == in[i].n))
        return true;
    for (size_t o2 = o + 1; o2 < NO; ++o2)
      if (share_bytes(out[o], out[o2])) return true;
  }
  return false;
}

}  // namespace

extern "C" {

const char* ss_status_str(ss_status s) {
  switch (s) {
    case SS_OK: return "ok";
    case SS_ERR_NULL_ARG: return "ss: a required pointer is NULL (or an optional input/output pair is half given)";
    case SS_ERR_BAD_SHAPE: return "ss: invalid problem size";
    case SS_ERR_BAD_DTYPE: return "ss: io_dtype must be SS_F32, SS_F16 or SS_BF16";
    case SS_ERR_MISALIGNED: return "ss: every tensor pointer must be 16-byte aligned";
    case SS_ERR_UNSUPPORTED:
      return "ss: unsupported request (a size outside the supported set, a workspace missing or too small, or "
             "overlapping buffers)";
    case SS_ERR_HIP: return "ss: HIP launch failed";
  }
  return "ss: unknown status";
}

size_t ss_ckpt_count(const ss_problem* p) {
  if (check_problem(p, true) != SS_OK) return 0;
  return (size_t)(p->batch * p->dim * ((p->seqlen + kTile - 1) / kTile) * p->dstate);
}

size_t ss_fwd_workspace_size(const ss_problem* p) {
  if (check_problem(p, true) != SS_OK) return 0;
  const FwdPlan pl = plan_fwd(p);
  if (pl.nchunks > 1 || p->batch > kQueueMaxRows) return pl.workspace;
  return queue_layout(p).total;
}

size_t ss_fwd_workspace_min(const ss_problem* p) {
  if (check_problem(p, true) != SS_OK) return 0;
  return plan_fwd(p).workspace;
}

ss_status ss_fwd(const ss_problem* p, const void* u, const void* delta, const float* A, const void* Bm,
                 const void* Cm, const float* D, const void* z, const float* delta_bias, const int32_t* lengths,
                 const int32_t* seq_idx, const float* h0, void* y, float* last_state, float* ckpt, void* workspace,
                 size_t workspace_bytes, void* stream) {
  return ss::fwd_checked(p, u, delta, A, Bm, Cm, D, z, delta_bias, lengths, seq_idx, h0, y, last_state, ckpt,
                         workspace, workspace_bytes, stream);
}

}  // extern "C"

namespace ss {

size_t fwd_workspace_bytes(const ss_problem* p) { return ss_fwd_workspace_min(p); }
ss_status fwd_check_problem(const ss_problem* p) { return check_problem(p, true); }

ss_status fwd_checked(const ss_problem* p, const void* u, const void* delta, const float* A, const void* Bm,
                      const void* Cm, const float* D, const void* z, const float* delta_bias, const int32_t* lengths,
                      const int32_t* seq_idx, const float* h0, void* y, float* last_state, float* ckpt,
                      void* workspace, size_t workspace_bytes, void* stream) {
  ss_status s = check_problem(p, true);
  if (s != SS_OK) return s;
  if (!u || !delta || !A || !Bm || !Cm || !y) return SS_ERR_NULL_ARG;
  const void* ptrs[] = {u, delta, A, Bm, Cm, D, z, delta_bias, lengths, seq_idx, h0, y, last_state, ckpt, workspace};
  for (const void* q : ptrs)
    if (q && !aligned(q)) return SS_ERR_MISALIGNED;
  const FwdPlan pl = plan_fwd(p);
  if (pl.workspace > 0 && (!workspace || workspace_bytes < pl.workspace)) return SS_ERR_UNSUPPORTED;
  // the work queue: for ragged rows, or for more 16-channel row blocks than the
  // GPU holds at once when they do not fill its slots evenly; only with a
  // workspace that holds it (without one the same scan runs without the queue)
  bool queue = false;
  const QueueLayout ql = queue_layout(p);
  const int64_t ch_blocks = (p->dim + kChPerBlock - 1) / kChPerBlock;
  const int64_t slots = kFinalPerCu * ss::device_cus();
  if (pl.nchunks == 1 && p->batch <= kQueueMaxRows && workspace && workspace_bytes >= ql.total) {
    const int64_t G = p->batch * ch_blocks;
    queue = lengths != nullptr || (G > slots && G % slots != 0);
  }
  const size_t ws_used = queue ? ql.total : pl.workspace;
  {
    // y may be u, delta or z itself (each wave reads a tile's inputs before it writes the
    // tile's outputs); no other overlap between an output and any buffer
    const size_t io = (size_t)(p->batch * p->dim * p->seqlen) * elem_size(p->io_dtype);
    const size_t bc = (size_t)(p->batch * p->dstate * p->seqlen) * elem_size(p->io_dtype);
    const size_t st = (size_t)(p->batch * p->dim * p->dstate) * sizeof(float);
    const Span in[] = {{u, io}, {delta, io}, {z, io}, {Bm, bc}, {Cm, bc},
                       {A, (size_t)(p->dim * p->dstate) * sizeof(float)}, {D, (size_t)p->dim * sizeof(float)},
                       {delta_bias, (size_t)p->dim * sizeof(float)}, {lengths, (size_t)p->batch * 4},
                       {seq_idx, (size_t)(p->batch * p->seqlen) * 4}, {h0, st}};
    const Span out[] = {{y, io}, {last_state, st}, {ckpt, ss_ckpt_count(p) * sizeof(float)},
                        {ws_used ? workspace : nullptr, ws_used}};
    static const bool inplace[4][11] = {{true, true, true}};
    if (conflict(in, out, inplace)) return SS_ERR_UNSUPPORTED;
  }

  ss::FwdParams k{};
  k.io = p->io_dtype;
  k.softplus = p->delta_softplus != 0;
  k.u = u; k.delta = delta; k.z = z; k.Bm = Bm; k.Cm = Cm;
  k.A = A; k.D = D; k.bias = delta_bias; k.lengths = lengths; k.seq_idx = seq_idx; k.h0 = h0;
  k.y = y; k.last_state = last_state; k.ckpt = ckpt;
  k.batch = p->batch; k.dim = p->dim; k.dstate = p->dstate; k.seqlen = p->seqlen;
  k.chunk_len = pl.chunk_len;
  k.ch_blocks = (p->dim + kChPerBlock - 1) / kChPerBlock;
  k.ckpt_per_row = (p->seqlen + kTile - 1) / kTile;
  k.nchunks = (int32_t)pl.nchunks;
  if (pl.nchunks > 1) {
    const ChunkLayout cl = chunk_layout(p, pl.nchunks);
    char* ws = static_cast<char*>(workspace);
    k.q_ctrl = reinterpret_cast<int32_t*>(ws);
    k.pairs = reinterpret_cast<uint64_t*>(ws + cl.pairs);
    k.gpairs = reinterpret_cast<uint64_t*>(ws + cl.gpairs);
    k.nslots = (int64_t)((cl.total - cl.pairs) / sizeof(uint64_t));
    k.group = (int32_t)cl.group;
    k.ngroups = (int32_t)cl.ngroups;
  }
  if (queue) {
    char* ws = static_cast<char*>(workspace);
    k.q_ctrl = reinterpret_cast<int32_t*>(ws);
    k.q_flags = reinterpret_cast<int32_t*>(ws + ql.flags);
    k.q_carry = reinterpret_cast<float*>(ws + ql.carry);
    k.q_chunks = ql.chunks;
    k.chunk_len = kQueueChunk;
    k.nchunks = (int32_t)ql.chunks;
    const int64_t units = ql.chunks * p->batch * ch_blocks;
    k.q_grid = units < slots ? units : slots;
  }
  return from_hip(ss::launch_fwd(k, pl.nchunks, static_cast<hipStream_t>(stream)));
}

}  // namespace ss

extern "C" {

ss_status ss_fwd_step(const ss_problem* p, const void* u_t, const void* delta_t, const float* A, const void* B_t,
                      const void* C_t, const float* D, const void* z_t, const float* delta_bias,
                      const float* state_in, float* state_out, void* y_t, void* stream) {
  ss_status s = check_problem(p, false);
  if (s != SS_OK) return s;
  if (!u_t || !delta_t || !A || !B_t || !C_t || !state_in || !state_out || !y_t) return SS_ERR_NULL_ARG;
  const void* ptrs[] = {u_t, delta_t, A, B_t, C_t, D, z_t, delta_bias, state_in, state_out, y_t};
  for (const void* q : ptrs)
    if (q && !aligned(q)) return SS_ERR_MISALIGNED;
  // in-place is allowed; a partial overlap of the two state buffers is not
  const uintptr_t a0 = (uintptr_t)state_in, b0 = (uintptr_t)state_out;
  const uintptr_t bytes = (uintptr_t)(p->batch * p->dim * p->dstate) * sizeof(float);
  if (a0 != b0 && a0 < b0 + bytes && b0 < a0 + bytes) return SS_ERR_UNSUPPORTED;

  ss::StepParams k{};
  k.io = p->io_dtype;
  k.softplus = p->delta_softplus != 0;
  k.u = u_t; k.delta = delta_t; k.z = z_t; k.Bt = B_t; k.Ct = C_t;
  k.A = A; k.D = D; k.bias = delta_bias;
  k.state_in = state_in; k.state_out = state_out; k.y = y_t;
  k.batch = p->batch; k.dim = p->dim; k.dstate = p->dstate;
  return from_hip(ss::launch_step(k, static_cast<hipStream_t>(stream)));
}

namespace {
// The backward's own grids: a workgroup per (batch row, 64-step chunk,
// channel block) for the chunk aggregates, one per channel for the carry scan
// (which runs only when there is more than one chunk).
ss_status check_bwd(const ss_problem* p) {
  const ss_status s = check_problem(p, true);
  if (s != SS_OK) return s;
  const double chunks = (double)((p->seqlen + kTile - 1) / kTile);
  const double cblocks = (double)((p->dim + kChPerBlock - 1) / kChPerBlock);
  if ((double)p->batch * chunks * cblocks > (double)kMaxGrid) return SS_ERR_BAD_SHAPE;
  if (chunks > 1 && (double)p->batch * (double)p->dim > (double)kMaxGrid) return SS_ERR_BAD_SHAPE;
  return SS_OK;
}
}  // namespace

size_t ss_bwd_workspace_size(const ss_problem* p) {
  if (check_bwd(p) != SS_OK) return 0;
  const int64_t nchunks = (p->seqlen + kTile - 1) / kTile;
  return (size_t)3 * (size_t)(p->batch * p->dim * nchunks * 16) * sizeof(float);
}

ss_status ss_bwd(const ss_problem* p, const void* u, const void* delta, const float* A, const void* Bm,
                 const void* Cm, const float* D, const void* z, const float* delta_bias, const int32_t* seq_idx,
                 const float* ckpt, const void* dy, const float* dlast, void* du, void* ddelta, void* dz, float* dA,
                 float* dB, float* dC, float* dD, float* dbias, float* dh0, void* workspace, size_t workspace_bytes,
                 void* stream) {
  ss_status s = check_bwd(p);
  if (s != SS_OK) return s;
  if (!u || !delta || !A || !Bm || !Cm || !ckpt || !dy || !du || !ddelta || !dA || !dB || !dC)
    return SS_ERR_NULL_ARG;
  if ((z == nullptr) != (dz == nullptr) || (D == nullptr) != (dD == nullptr) ||
      (delta_bias == nullptr) != (dbias == nullptr))
    return SS_ERR_NULL_ARG;
  const void* ptrs[] = {u, delta, A, Bm, Cm, D, z, delta_bias, seq_idx, ckpt, dy, dlast, du, ddelta, dz, dA, dB, dC,
                        dD, dbias, dh0, workspace};
  for (const void* q : ptrs)
    if (q && !aligned(q)) return SS_ERR_MISALIGNED;
  const size_t need = ss_bwd_workspace_size(p);
  if (!workspace || workspace_bytes < need) return SS_ERR_UNSUPPORTED;
  {
    // no output (or the workspace) shares a byte with any other buffer
    const size_t io = (size_t)(p->batch * p->dim * p->seqlen) * elem_size(p->io_dtype);
    const size_t bc = (size_t)(p->batch * p->dstate * p->seqlen) * elem_size(p->io_dtype);
    const size_t bc32 = (size_t)(p->batch * p->dstate * p->seqlen) * sizeof(float);
    const size_t st = (size_t)(p->batch * p->dim * p->dstate) * sizeof(float);
    const size_t dn = (size_t)(p->dim * p->dstate) * sizeof(float), dv = (size_t)p->dim * sizeof(float);
    const Span in[] = {{u, io}, {delta, io}, {z, io}, {Bm, bc}, {Cm, bc}, {A, dn}, {D, dv}, {delta_bias, dv},
                       {seq_idx, (size_t)(p->batch * p->seqlen) * 4}, {ckpt, ss_ckpt_count(p) * sizeof(float)},
                       {dy, io}, {dlast, st}};
    const Span out[] = {{du, io}, {ddelta, io}, {dz, io}, {dA, dn}, {dB, bc32}, {dC, bc32},
                        {dD, dv}, {dbias, dv}, {dh0, st}, {workspace, need}};
    if (conflict(in, out)) return SS_ERR_UNSUPPORTED;
  }

  ss::BwdParams k{};
  k.io = p->io_dtype;
  k.softplus = p->delta_softplus != 0;
  k.u = u; k.delta = delta; k.z = z; k.Bm = Bm; k.Cm = Cm;
  k.A = A; k.D = D; k.bias = delta_bias; k.ckpt = ckpt; k.dy = dy;
  k.seq_idx = seq_idx; k.dlast = dlast; k.dh0 = dh0;
  k.du = du; k.ddelta = ddelta; k.dz = dz;
  k.dA = dA; k.dB = dB; k.dC = dC; k.dD = dD; k.dbias = dbias;
  k.batch = p->batch; k.dim = p->dim; k.dstate = p->dstate; k.seqlen = p->seqlen;
  k.ch_blocks = (p->dim + kChPerBlock - 1) / kChPerBlock;
  k.nchunks = (p->seqlen + kTile - 1) / kTile;
  const size_t per = (size_t)(p->batch * p->dim * k.nchunks * 16);
  float* ws = static_cast<float*>(workspace);
  k.gcarry = ws;
  k.aggP = ws + per;
  k.aggG = ws + 2 * per;
  return from_hip(ss::launch_bwd(k, static_cast<hipStream_t>(stream)));
}

namespace {
ss_status check_conv(const ss_conv_problem* p, bool need_seqlen) {
  if (!p) return SS_ERR_NULL_ARG;
  if (p->batch < 1 || p->dim < 1) return SS_ERR_BAD_SHAPE;
  if (need_seqlen && (p->seqlen < 1 || p->seqlen > kMaxSeqlen)) return SS_ERR_BAD_SHAPE;
  if (p->io_dtype != SS_F32 && p->io_dtype != SS_F16 && p->io_dtype != SS_BF16) return SS_ERR_BAD_DTYPE;
  if (p->width < 1 || p->width > 4 || p->reserved != 0) return SS_ERR_UNSUPPORTED;
  const int64_t lim = (int64_t)1 << 40;
  if (p->batch > lim || p->dim > lim) return SS_ERR_BAD_SHAPE;
  if (need_seqlen && (double)p->batch * (double)p->dim * (double)ss::conv_tblocks(p->seqlen) > (double)kMaxGrid)
    return SS_ERR_BAD_SHAPE;
  if (!need_seqlen && (double)p->batch * (double)p->dim / 256.0 > (double)kMaxGrid) return SS_ERR_BAD_SHAPE;
  return SS_OK;
}
bool overlaps(const void* a, size_t na, const void* b, size_t nb) {
  const uintptr_t x = (uintptr_t)a, y = (uintptr_t)b;
  return x < y + nb && y < x + na;
}
}  // namespace

ss_status ss_conv1d_fwd(const ss_conv_problem* p, const void* x, const float* w, const float* bias,
                        const int32_t* seq_idx, const float* conv_init, void* out, float* conv_final,
                        void* stream) {
  ss_status s = check_conv(p, true);
  if (s != SS_OK) return s;
  if (!x || !w || !out) return SS_ERR_NULL_ARG;
  const void* ptrs[] = {x, w, bias, seq_idx, conv_init, out, conv_final};
  for (const void* q : ptrs)
    if (q && !aligned(q)) return SS_ERR_MISALIGNED;
  const size_t bytes = (size_t)(p->batch * p->dim * p->seqlen * elem_size(p->io_dtype));
  {
    // no output shares a byte with an input or the other output (the window going out is
    // written by a row's last time block while its first reads the window coming in)
    const size_t win = (size_t)(p->batch * p->dim * (p->width - 1)) * sizeof(float);
    const Span in[] = {{x, bytes}, {w, (size_t)(p->dim * p->width) * sizeof(float)},
                       {bias, (size_t)p->dim * sizeof(float)}, {seq_idx, (size_t)(p->batch * p->seqlen) * 4},
                       {conv_init, win}};
    const Span outs[] = {{out, bytes}, {conv_final, win}};
    if (conflict(in, outs)) return SS_ERR_UNSUPPORTED;
  }
  ss::ConvParams k{};
  k.io = p->io_dtype; k.width = p->width; k.silu = p->silu != 0;
  k.x = x; k.w = w; k.bias = bias; k.seq_idx = seq_idx; k.conv_init = conv_init;
  k.out = out; k.conv_final = conv_final;
  k.batch = p->batch; k.dim = p->dim; k.seqlen = p->seqlen;
  k.tblocks = ss::conv_tblocks(p->seqlen);
  return from_hip(ss::launch_conv(k, static_cast<hipStream_t>(stream)));
}

ss_status ss_conv1d_step(const ss_conv_problem* p, const void* x_t, const float* w, const float* bias,
                         const float* window_in, float* window_out, void* out_t, void* stream) {
  ss_status s = check_conv(p, false);
  if (s != SS_OK) return s;
  if (!x_t || !w || !out_t || ((!window_in || !window_out) && p->width > 1)) return SS_ERR_NULL_ARG;
  const void* ptrs[] = {x_t, w, bias, window_in, window_out, out_t};
  for (const void* q : ptrs)
    if (q && !aligned(q)) return SS_ERR_MISALIGNED;
  const size_t wbytes = (size_t)(p->batch * p->dim * (p->width - 1)) * sizeof(float);
  if (window_in != window_out && wbytes && overlaps(window_in, wbytes, window_out, wbytes)) return SS_ERR_UNSUPPORTED;
  ss::ConvStepParams k{};
  k.io = p->io_dtype; k.width = p->width; k.silu = p->silu != 0;
  k.x = x_t; k.w = w; k.bias = bias; k.window_in = window_in; k.window_out = window_out; k.out = out_t;
  k.batch = p->batch; k.dim = p->dim;
  return from_hip(ss::launch_conv_step(k, static_cast<hipStream_t>(stream)));
}

namespace {
// workgroups per channel of the convolution's backward, each with at least one
// unit of 256 chunks: more than one (and a second kernel that adds their sums)
// only where the channels alone do not fill the GPU (bench branch, 1536
// channels: 38.4 us with one, 42.3 us with three)
int64_t conv_bwd_parts(const ss_conv_problem* p) {
  const int64_t units = ss::conv_bwd_units(p->batch, p->seqlen);
  const int64_t want = (kConvBwdGroups + p->dim - 1) / p->dim;
  return want < units ? want : units;
}
ss_status check_conv_bwd(const ss_conv_problem* p) {
  const ss_status s = check_conv(p, true);
  if (s != SS_OK) return s;
  if (p->dim > kMaxGrid || p->dim * conv_bwd_parts(p) > kMaxGrid) return SS_ERR_BAD_SHAPE;
  return SS_OK;
}
}  // namespace

size_t ss_conv1d_bwd_workspace_size(const ss_conv_problem* p) {
  if (check_conv_bwd(p) != SS_OK) return 0;
  const int64_t parts = conv_bwd_parts(p);
  return parts > 1 ? (size_t)(parts * p->dim * (p->width + 1)) * sizeof(float) : 0;
}

ss_status ss_conv1d_bwd(const ss_conv_problem* p, const void* x, const float* w, const float* bias,
                        const int32_t* seq_idx, const float* conv_init, const void* dout, const float* dconv_final,
                        void* dx, float* dw, float* dbias, float* dconv_init, void* workspace,
                        size_t workspace_bytes, void* stream) {
  const ss_status s = check_conv_bwd(p);
  if (s != SS_OK) return s;
  if (!x || !w || !dout || !dx || !dw || (bias == nullptr) != (dbias == nullptr)) return SS_ERR_NULL_ARG;
  const void* ptrs[] = {x, w, bias, seq_idx, conv_init, dout, dconv_final, dx, dw, dbias, dconv_init, workspace};
  for (const void* q : ptrs)
    if (q && !aligned(q)) return SS_ERR_MISALIGNED;
  const size_t need = ss_conv1d_bwd_workspace_size(p);
  if (need && (!workspace || workspace_bytes < need)) return SS_ERR_UNSUPPORTED;
  {
    const size_t bytes = (size_t)(p->batch * p->dim * p->seqlen * elem_size(p->io_dtype));
    const size_t win = (size_t)(p->batch * p->dim * (p->width - 1)) * sizeof(float);
    const size_t wb = (size_t)(p->dim * p->width) * sizeof(float), vb = (size_t)p->dim * sizeof(float);
    const Span in[] = {{x, bytes}, {w, wb}, {bias, vb}, {seq_idx, (size_t)(p->batch * p->seqlen) * 4},
                       {conv_init, win}, {dout, bytes}, {dconv_final, win}};
    const Span outs[] = {{dx, bytes}, {dw, wb}, {dbias, vb}, {dconv_init, win}, {need ? workspace : nullptr, need}};
    if (conflict(in, outs)) return SS_ERR_UNSUPPORTED;
  }
  ss::ConvBwdParams k{};
  k.io = p->io_dtype; k.width = p->width; k.silu = p->silu != 0; k.parts = (int32_t)conv_bwd_parts(p);
  k.x = x; k.w = w; k.bias = bias; k.seq_idx = seq_idx; k.conv_init = conv_init; k.dout = dout;
  k.dconv_final = dconv_final; k.dx = dx; k.dw = dw; k.dbias = dbias; k.dconv_init = dconv_init;
  k.ws = static_cast<float*>(workspace);
  k.batch = p->batch; k.dim = p->dim; k.seqlen = p->seqlen;
  k.units = ss::conv_bwd_units(p->batch, p->seqlen);
  return from_hip(ss::launch_conv_bwd(k, static_cast<hipStream_t>(stream)));
}

namespace {
constexpr int64_t kSsdChunk = 256;
ss_status check_ssd(const ss_ssd_problem* p) {
  if (!p) return SS_ERR_NULL_ARG;
  if (p->batch < 1 || p->seqlen < 1 || p->nheads < 1 || p->ngroups < 1) return SS_ERR_BAD_SHAPE;
  if (p->io_dtype != SS_F16 && p->io_dtype != SS_BF16) return SS_ERR_BAD_DTYPE;
  if (p->headdim != 64) return SS_ERR_UNSUPPORTED;
  if (p->dstate != 32 && p->dstate != 64 && p->dstate != 96 && p->dstate != 128) return SS_ERR_UNSUPPORTED;
  if (p->nheads % p->ngroups != 0) return SS_ERR_UNSUPPORTED;
  // the kernels address a 256-step chunk of x or z (256 * nheads * 64 * 2
  // bytes) with 32-bit offsets; at most 2^30 bytes
  if (p->nheads > 32768) return SS_ERR_UNSUPPORTED;
  const int64_t lim = (int64_t)1 << 31;
  if (p->batch > lim || p->seqlen > lim || p->nheads > lim) return SS_ERR_BAD_SHAPE;
  const double nchunks = (double)((p->seqlen + kSsdChunk - 1) / kSsdChunk);
  if ((double)p->batch * nchunks * (double)p->nheads > (double)kMaxGrid) return SS_ERR_BAD_SHAPE;
  if ((double)p->batch * (double)p->nheads * (p->dstate / 32) > (double)kMaxGrid) return SS_ERR_BAD_SHAPE;
  if ((double)p->batch * (double)p->seqlen * (double)p->nheads * 64.0 > 9.0e18) return SS_ERR_BAD_SHAPE;
  return SS_OK;
}
size_t ssd_state_elems(const ss_ssd_problem* p) {
  const int64_t nchunks = (p->seqlen + kSsdChunk - 1) / kSsdChunk;
  return (size_t)(p->batch * nchunks * p->nheads) * (size_t)(64 * p->dstate);
}
}  // namespace

size_t ssd_cb_bytes(const ss_ssd_problem* p) {
  const int64_t nchunks = (p->seqlen + kSsdChunk - 1) / kSsdChunk;
  return (size_t)(p->batch * nchunks * p->ngroups) * (size_t)(kSsdChunk * kSsdChunk) * 2;
}

size_t ss_ssd_workspace_size(const ss_ssd_problem* p) {
  if (check_ssd(p) != SS_OK) return 0;
  return align256(ssd_state_elems(p) * 2) + align256(ssd_cb_bytes(p));
}

ss_status ss_ssd_fwd(const ss_ssd_problem* p, const void* x, const void* dt, const float* A, const void* Bm,
                     const void* Cm, const float* D, const void* z, const float* dt_bias, const int32_t* seq_idx,
                     const float* h0, void* y, float* final_state, void* workspace, size_t workspace_bytes,
                     void* stream) {
  ss_status s = check_ssd(p);
  if (s != SS_OK) return s;
  if (!x || !dt || !A || !Bm || !Cm || !y) return SS_ERR_NULL_ARG;
  // a row's document ids are read through one 32-bit range-checked view
  if (seq_idx && p->seqlen > ((int64_t)1 << 29)) return SS_ERR_UNSUPPORTED;
  const void* ptrs[] = {x, dt, A, Bm, Cm, D, z, dt_bias, seq_idx, h0, y, final_state, workspace};
  for (const void* q : ptrs)
    if (q && !aligned(q)) return SS_ERR_MISALIGNED;
  const size_t need = ss_ssd_workspace_size(p);
  if (!workspace || workspace_bytes < need) return SS_ERR_UNSUPPORTED;
  {
    // y may be x or z itself (a workgroup reads its own rows of x and z before it writes
    // them) and final_state may be h0 itself (each element is read and written by one
    // thread); no other overlap between an output or the workspace and an operand
    const size_t xb = (size_t)(p->batch * p->seqlen * p->nheads) * 64 * 2;
    const size_t dtb = (size_t)(p->batch * p->seqlen * p->nheads) * 2;
    const size_t bcb = (size_t)(p->batch * p->seqlen * p->ngroups * p->dstate) * 2;
    const size_t hb = (size_t)(p->batch * p->nheads) * 64 * (size_t)p->dstate * 4;
    const size_t vb = (size_t)p->nheads * 4;
    struct Span { const void* ptr; size_t n; };
    const Span in[] = {{x, xb},       {dt, dtb},      {A, vb},
                       {Bm, bcb},     {Cm, bcb},      {D, vb},
                       {z, xb},       {dt_bias, vb},  {seq_idx, (size_t)(p->batch * p->seqlen) * 4},
                       {h0, hb}};
    for (const Span& r : in) {
      if (!r.ptr) continue;
      if (overlaps(r.ptr, r.n, y, xb) && !(r.ptr == y && (r.ptr == x || r.ptr == z))) return SS_ERR_UNSUPPORTED;
      if (final_state && overlaps(r.ptr, r.n, final_state, hb) && !(r.ptr == final_state && r.ptr == h0))
        return SS_ERR_UNSUPPORTED;
      if (overlaps(r.ptr, r.n, workspace, need)) return SS_ERR_UNSUPPORTED;
    }
    if (final_state && overlaps(final_state, hb, y, xb)) return SS_ERR_UNSUPPORTED;
    if (overlaps(workspace, need, y, xb) || (final_state && overlaps(workspace, need, final_state, hb)))
      return SS_ERR_UNSUPPORTED;
  }
  const size_t e = ssd_state_elems(p);
  ss::SsdParams k{};
  k.io = p->io_dtype; k.softplus = p->dt_softplus != 0;
  k.x = x; k.dt = dt; k.A = A; k.Bm = Bm; k.Cm = Cm; k.D = D; k.z = z; k.dt_bias = dt_bias; k.h0 = h0;
  k.seq_idx = seq_idx;
  k.y = y; k.final_state = final_state;
  char* ws = static_cast<char*>(workspace);
  k.ws_entry = reinterpret_cast<uint16_t*>(ws);
  k.ws_cb = reinterpret_cast<uint16_t*>(ws + align256(e * 2));
  k.batch = p->batch; k.seqlen = p->seqlen; k.nheads = p->nheads; k.ngroups = p->ngroups; k.dstate = p->dstate;
  k.nchunks = (p->seqlen + kSsdChunk - 1) / kSsdChunk;
  return from_hip(ss::launch_ssd(k, static_cast<hipStream_t>(stream)));
}

namespace {
ss_status check_ssd_bwd(const ss_ssd_problem* p) {
  const ss_status s = check_ssd(p);
  if (s != SS_OK) return s;
  const double places = (double)p->batch * (double)((p->seqlen + kSsdChunk - 1) / kSsdChunk);
  // the pass and the pairs share a launch, each rounded up to the XCDs
  if (places * (2.0 * (double)p->nheads + 10.0 * (double)p->ngroups) +
          (double)p->batch * (double)p->nheads * (p->dstate / 16) + 88.0 > (double)kMaxGrid)
    return SS_ERR_BAD_SHAPE;
  return SS_OK;
}
// the workspace of the SSD's backward: one piece after the other, each on a
// 256-byte boundary
struct SsdBwdLayout {
  size_t total = 0;
  size_t take(size_t bytes) {
    const size_t at = total;
    total += align256(bytes);
    return at;
  }
  size_t E, R, decay, dot, cb, bc, delta, cs, cl, from, to, wc, wb, xd, e, r, seg, prow, pcol, S, part;
  size_t x[2], g[3], b[2], c[2];
  SsdBwdLayout(const ss_ssd_problem* p, bool gated);
};
SsdBwdLayout::SsdBwdLayout(const ss_ssd_problem* p, bool gated) {
  const bool f16 = p->io_dtype == SS_F16;
  const size_t places = (size_t)(p->batch * ((p->seqlen + kSsdChunk - 1) / kSsdChunk));
  const size_t ph = places * (size_t)p->nheads, st = ph * (size_t)(64 * p->dstate) * 4, q = ph * 256 * 4;
  const size_t square = places * (size_t)p->ngroups * (256 * 256) * 4;
  const size_t rows = (size_t)(p->batch * p->seqlen);
  const size_t xb = rows * (size_t)p->nheads * 64 * 2, vb = rows * (size_t)(p->ngroups * p->dstate) * 2;
  E = take(st); R = take(st); decay = take(ph * 4); dot = take(ph * (size_t)p->dstate);
  bc = take(square); cb = take(gated ? square : 0);
  delta = take(q); cs = take(q); cl = take(q); from = take(q); to = take(q);
  wc = take(q); wb = take(q); xd = take(q); e = take(2 * q); r = take(2 * q);
  seg = take(places * 256 * 4);
  prow = take(ph * 10 * 64 * 4); pcol = take(ph * 10 * 64 * 4);
  S = take(places * (size_t)p->ngroups * 10 * (64 * 64 * 2) * 4);
  part = take(ph * 3 * 4);
  for (int i = 0; i < 3; ++i) g[i] = take(gated || (f16 && i < 2) ? xb : 0);
  for (int i = 0; i < 2; ++i) {
    x[i] = take(f16 ? xb : 0);
    b[i] = take(f16 ? vb : 0);
    c[i] = take(f16 ? vb : 0);
  }
}
}  // namespace

size_t ss_ssd_bwd_workspace_size(const ss_ssd_problem* p, int32_t gated) {
  if (check_ssd_bwd(p) != SS_OK) return 0;
  return SsdBwdLayout(p, gated != 0).total;
}

ss_status ss_ssd_bwd(const ss_ssd_problem* p, const void* x, const void* dt, const float* A, const void* Bm,
                     const void* Cm, const float* D, const void* z, const float* dt_bias, const int32_t* seq_idx,
                     const float* h0, const void* dy, const float* dfinal, void* dx, void* ddt, float* dA, void* dB,
                     void* dC, float* dD, void* dz, float* ddt_bias, float* dh0, void* workspace,
                     size_t workspace_bytes, void* stream) {
  const ss_status s = check_ssd_bwd(p);
  if (s != SS_OK) return s;
  if (!x || !dt || !A || !Bm || !Cm || !dy || !dx || !ddt || !dA || !dB || !dC) return SS_ERR_NULL_ARG;
  if ((z == nullptr) != (dz == nullptr) || (D == nullptr) != (dD == nullptr) ||
      (dt_bias == nullptr) != (ddt_bias == nullptr))
    return SS_ERR_NULL_ARG;
  const void* ptrs[] = {x, dt, A, Bm, Cm, D, z, dt_bias, seq_idx, h0, dy, dfinal, dx, ddt, dA, dB, dC,
                        dD, dz, ddt_bias, dh0, workspace};
  for (const void* q : ptrs)
    if (q && !aligned(q)) return SS_ERR_MISALIGNED;
  const SsdBwdLayout l(p, z != nullptr);
  if (!workspace || workspace_bytes < l.total) return SS_ERR_UNSUPPORTED;
  {
    const size_t rows = (size_t)(p->batch * p->seqlen);
    const size_t xb = rows * (size_t)p->nheads * 64 * 2, dtb = rows * (size_t)p->nheads * 2;
    const size_t vb = rows * (size_t)(p->ngroups * p->dstate) * 2, nb = (size_t)p->nheads * 4;
    const size_t hb = (size_t)(p->batch * p->nheads) * 64 * (size_t)p->dstate * 4;
    const Span in[] = {{x, xb}, {dt, dtb}, {A, nb}, {Bm, vb}, {Cm, vb}, {D, nb}, {z, xb}, {dt_bias, nb},
                       {seq_idx, rows * 4}, {h0, hb}, {dy, xb}, {dfinal, hb}};
    const Span outs[] = {{dx, xb}, {ddt, dtb}, {dA, nb}, {dB, vb}, {dC, vb}, {dD, nb}, {dz, xb}, {ddt_bias, nb},
                         {dh0, hb}, {workspace, l.total}};
    if (conflict(in, outs)) return SS_ERR_UNSUPPORTED;
  }
  char* ws = static_cast<char*>(workspace);
  auto f32_at = [&](size_t at) { return reinterpret_cast<float*>(ws + at); };
  const bool f16 = p->io_dtype == SS_F16;
  auto planes = [&](int n, const size_t* at, const void* in, const uint16_t** to) {
    if (n == 1) to[0] = static_cast<const uint16_t*>(in);
    else
      for (int i = 0; i < n; ++i) to[i] = reinterpret_cast<const uint16_t*>(ws + at[i]);
  };
  ss::SsdBwdParams k{};
  k.softplus = p->dt_softplus != 0;
  k.x = x; k.dt = dt; k.Bm = Bm; k.Cm = Cm; k.z = z; k.dy = dy; k.A = A; k.D = D; k.dt_bias = dt_bias;
  k.seq_idx = seq_idx; k.h0 = h0; k.dfinal = dfinal;
  k.dx = dx; k.ddt = ddt; k.dB = dB; k.dC = dC; k.dz = dz; k.dA = dA; k.dD = dD; k.ddt_bias = ddt_bias; k.dh0 = dh0;
  const int parts = f16 ? 2 : 1;
  planes(parts, l.x, x, k.xp);
  planes(z ? 3 : parts, l.g, dy, k.gp);
  planes(parts, l.b, Bm, k.bp);
  planes(parts, l.c, Cm, k.cp);
  k.ws_E = f32_at(l.E); k.ws_R = f32_at(l.R); k.ws_decay = f32_at(l.decay); k.ws_dot = f32_at(l.dot);
  k.ws_cb = f32_at(l.cb); k.ws_bc = f32_at(l.bc); k.ws_delta = f32_at(l.delta);
  k.ws_cs = f32_at(l.cs); k.ws_cl = f32_at(l.cl); k.ws_from = f32_at(l.from); k.ws_to = f32_at(l.to);
  k.ws_wc = f32_at(l.wc); k.ws_wb = f32_at(l.wb); k.ws_xd = f32_at(l.xd); k.ws_e = f32_at(l.e); k.ws_r = f32_at(l.r);
  k.ws_seg = reinterpret_cast<int32_t*>(ws + l.seg);
  k.ws_prow = f32_at(l.prow); k.ws_pcol = f32_at(l.pcol); k.ws_S = reinterpret_cast<uint32_t*>(ws + l.S);
  k.ws_part = f32_at(l.part);
  k.batch = p->batch; k.seqlen = p->seqlen;
  k.nheads = (int32_t)p->nheads; k.ngroups = (int32_t)p->ngroups; k.dstate = p->dstate;
  k.nchunks = (int32_t)((p->seqlen + kSsdChunk - 1) / kSsdChunk);
  return from_hip(ss::launch_ssd_bwd(p->io_dtype, k, static_cast<hipStream_t>(stream)));
}

namespace {
constexpr int64_t kMaxTokens = (int64_t)1 << 30;
constexpr int64_t kMaxSeqs = (int64_t)1 << 20;
// the longest row distance: 256 rows of 2-byte elements within 2^30 bytes, the
// kernels' 32-bit offsets inside a chunk
constexpr int64_t kMaxStride = (int64_t)1 << 21;
constexpr int64_t kMaxSlots = ((int64_t)1 << 31) - 1;

bool aligned_to(const void* ptr, int64_t n) { return (uintptr_t)ptr % (uintptr_t)n == 0; }
// bytes from the first element of `rows` strided rows to behind the last one
size_t rows_bytes(int64_t rows, int64_t stride, int64_t row, int64_t elem) {
  return (size_t)(((rows - 1) * stride + row) * elem);
}
ss_status check_packed(int64_t tokens, int64_t nseqs, int64_t nslots) {
  if (tokens < 1 || nseqs < 1 || nslots < 1) return SS_ERR_BAD_SHAPE;
  if (tokens > kMaxTokens || nseqs > kMaxSeqs || nslots > kMaxSlots) return SS_ERR_BAD_SHAPE;
  return SS_OK;
}
ss_status check_conv_prompt(const ss_conv_prompt_problem* p) {
  if (!p) return SS_ERR_NULL_ARG;
  const ss_status s = check_packed(p->tokens, p->nseqs, p->nslots);
  if (s != SS_OK) return s;
  if (p->dim < 1 || p->x_stride < p->dim || p->out_stride < p->dim) return SS_ERR_BAD_SHAPE;
  if (p->dim > kMaxStride || p->x_stride > kMaxStride || p->out_stride > kMaxStride) return SS_ERR_BAD_SHAPE;
  if (p->io_dtype != SS_F32 && p->io_dtype != SS_F16 && p->io_dtype != SS_BF16) return SS_ERR_BAD_DTYPE;
  if (p->width < 1 || p->width > 4 || p->reserved != 0) return SS_ERR_UNSUPPORTED;
  // a workgroup is 64 channels and four chunks of 16 rows at the least
  if (((p->tokens / 16 + p->nseqs + 3) / 4) * ((p->dim + 63) / 64) > kMaxGrid) return SS_ERR_BAD_SHAPE;
  return SS_OK;
}
// the sizes that prompts and steps of the SSD share
ss_status check_ssd_layer(int64_t nheads, int64_t ngroups, int32_t headdim, int32_t dstate, int32_t io_dtype) {
  if (nheads < 1 || ngroups < 1) return SS_ERR_BAD_SHAPE;
  if (io_dtype != SS_F16 && io_dtype != SS_BF16) return SS_ERR_BAD_DTYPE;
  if (headdim != 64) return SS_ERR_UNSUPPORTED;
  if (dstate != 32 && dstate != 64 && dstate != 96 && dstate != 128) return SS_ERR_UNSUPPORTED;
  if (nheads > kMaxStride / 64 || nheads % ngroups != 0) return SS_ERR_UNSUPPORTED;
  return SS_OK;
}
int64_t prompt_chunks(const ss_ssd_prompt_problem* p) { return p->tokens / 256 + p->nseqs; }
ss_status check_prompt(const ss_ssd_prompt_problem* p) {
  if (!p) return SS_ERR_NULL_ARG;
  ss_status s = check_packed(p->tokens, p->nseqs, p->nslots);
  if (s != SS_OK) return s;
  s = check_ssd_layer(p->nheads, p->ngroups, p->headdim, p->dstate, p->io_dtype);
  if (s != SS_OK) return s;
  const int64_t gn = p->ngroups * p->dstate, hp = p->nheads * 64;
  if (p->x_stride < hp || p->b_stride < gn || p->c_stride < gn || p->dt_stride < p->nheads) return SS_ERR_BAD_SHAPE;
  if (p->x_stride > kMaxStride || p->b_stride > kMaxStride || p->c_stride > kMaxStride || p->dt_stride > kMaxStride)
    return SS_ERR_BAD_SHAPE;
  if (p->x_stride % 8 || p->b_stride % 8 || p->c_stride % 8) return SS_ERR_MISALIGNED;
  const int64_t chunks = prompt_chunks(p);
  if (chunks * (p->nheads + 4 * p->ngroups) > kMaxGrid) return SS_ERR_BAD_SHAPE;
  if (p->nseqs * p->nheads * (p->dstate / 16) > kMaxGrid) return SS_ERR_BAD_SHAPE;
  return SS_OK;
}
size_t prompt_state_bytes(const ss_ssd_prompt_problem* p) {
  return align256((size_t)(prompt_chunks(p) * p->nheads) * (size_t)(64 * p->dstate) * 4);
}
size_t prompt_decay_bytes(const ss_ssd_prompt_problem* p) {
  return align256((size_t)(prompt_chunks(p) * p->nheads) * 4);
}
int64_t step_channels(const ss_ssd_step_problem* p) { return p->nheads * 64 + 2 * p->ngroups * p->dstate; }
ss_status check_step_rows(const ss_ssd_step_problem* p) {
  if (!p) return SS_ERR_NULL_ARG;
  if (p->rows < 1 || p->nslots < 1 || p->rows > kMaxSeqs || p->nslots > kMaxSlots) return SS_ERR_BAD_SHAPE;
  const ss_status s = check_ssd_layer(p->nheads, p->ngroups, p->headdim, p->dstate, p->io_dtype);
  if (s != SS_OK) return s;
  if (p->width < 1 || p->width > 4 || p->reserved != 0) return SS_ERR_UNSUPPORTED;
  const int64_t ch = step_channels(p);
  if (p->xbc_stride < ch || p->dt_stride < p->nheads) return SS_ERR_BAD_SHAPE;
  if (p->xbc_stride > kMaxStride || p->dt_stride > kMaxStride) return SS_ERR_BAD_SHAPE;
  if (p->rows * p->nheads > kMaxGrid || p->rows * ((ch + 255) / 256) > kMaxGrid) return SS_ERR_BAD_SHAPE;
  return SS_OK;
}
}  // namespace

ss_status ss_conv1d_prompt(const ss_conv_prompt_problem* p, const void* x, const float* w, const float* bias,
                           const int32_t* cu_seqlens, const int32_t* slots, const int32_t* has_state,
                           float* conv_state, void* out, void* stream) {
  const ss_status s = check_conv_prompt(p);
  if (s != SS_OK) return s;
  if (!x || !w || !cu_seqlens || !out || (!conv_state && p->width > 1)) return SS_ERR_NULL_ARG;
  const int64_t e = elem_size(p->io_dtype);
  if (!aligned_to(x, e) || !aligned_to(out, e)) return SS_ERR_MISALIGNED;
  const void* ptrs[] = {w, bias, cu_seqlens, slots, has_state, conv_state};
  for (const void* q : ptrs)
    if (q && !aligned(q)) return SS_ERR_MISALIGNED;
  if (!slots && p->nslots < p->nseqs) return SS_ERR_UNSUPPORTED;
  {
    const size_t ib = (size_t)p->nseqs * 4;
    const Span in[] = {{x, rows_bytes(p->tokens, p->x_stride, p->dim, e)}, {w, (size_t)(p->dim * p->width) * 4},
                       {bias, (size_t)p->dim * 4}, {cu_seqlens, ib + 4}, {slots, ib}, {has_state, ib}};
    const Span outs[] = {{out, rows_bytes(p->tokens, p->out_stride, p->dim, e)},
                         {conv_state, (size_t)p->nslots * (size_t)(p->dim * (p->width - 1)) * 4}};
    if (conflict(in, outs)) return SS_ERR_UNSUPPORTED;
  }
  ss::ConvPromptParams k{};
  k.io = p->io_dtype; k.width = p->width; k.silu = p->silu != 0;
  k.x = x; k.w = w; k.bias = bias; k.cu = cu_seqlens; k.slots = slots; k.has_state = has_state;
  k.conv_state = conv_state; k.out = out;
  k.x_stride = p->x_stride; k.out_stride = p->out_stride;
  k.tokens = (int32_t)p->tokens; k.nseqs = (int32_t)p->nseqs; k.dim = (int32_t)p->dim; k.nslots = (int32_t)p->nslots;
  k.pairs = e == 2 && aligned_to(x, 4) && aligned_to(out, 4) && p->dim % 2 == 0 && p->x_stride % 2 == 0 &&
            p->out_stride % 2 == 0;
  return from_hip(ss::launch_conv_prompt(k, static_cast<hipStream_t>(stream)));
}

size_t ss_ssd_prompt_workspace_size(const ss_ssd_prompt_problem* p) {
  if (check_prompt(p) != SS_OK) return 0;
  return prompt_state_bytes(p) + prompt_decay_bytes(p) +
         (size_t)(prompt_chunks(p) * p->ngroups) * (size_t)(256 * 256) * 4;
}

ss_status ss_ssd_prompt(const ss_ssd_prompt_problem* p, const void* x, const void* dt, const float* A, const void* Bm,
                        const void* Cm, const float* D, const void* z, const float* dt_bias,
                        const int32_t* cu_seqlens, const int32_t* slots, const int32_t* has_state, float* state,
                        void* y, void* workspace, size_t workspace_bytes, void* stream) {
  const ss_status s = check_prompt(p);
  if (s != SS_OK) return s;
  if (!x || !dt || !A || !Bm || !Cm || !cu_seqlens || !state || !y) return SS_ERR_NULL_ARG;
  const int64_t hp = p->nheads * 64, gn = p->ngroups * p->dstate;
  if (z && (p->z_stride < hp || p->z_stride > kMaxStride)) return SS_ERR_BAD_SHAPE;
  if (z && p->z_stride % 8) return SS_ERR_MISALIGNED;
  const void* ptrs[] = {x, A, Bm, Cm, D, z, dt_bias, cu_seqlens, slots, has_state, state, y, workspace};
  for (const void* q : ptrs)
    if (q && !aligned(q)) return SS_ERR_MISALIGNED;
  if (!aligned_to(dt, 2)) return SS_ERR_MISALIGNED;
  if (!slots && p->nslots < p->nseqs) return SS_ERR_UNSUPPORTED;
  const size_t need = ss_ssd_prompt_workspace_size(p);
  if (!workspace || workspace_bytes < need) return SS_ERR_UNSUPPORTED;
  {
    const size_t ib = (size_t)p->nseqs * 4, vb = (size_t)p->nheads * 4;
    const Span in[] = {{x, rows_bytes(p->tokens, p->x_stride, hp, 2)},
                       {z, rows_bytes(p->tokens, z ? p->z_stride : hp, hp, 2)},
                       {Bm, rows_bytes(p->tokens, p->b_stride, gn, 2)},
                       {Cm, rows_bytes(p->tokens, p->c_stride, gn, 2)},
                       {dt, rows_bytes(p->tokens, p->dt_stride, p->nheads, 2)},
                       {A, vb}, {D, vb}, {dt_bias, vb}, {cu_seqlens, ib + 4}, {slots, ib}, {has_state, ib}};
    const Span outs[] = {{y, (size_t)(p->tokens * hp) * 2},
                         {state, (size_t)p->nslots * (size_t)(hp * p->dstate) * 4},
                         {workspace, need}};
    if (conflict(in, outs)) return SS_ERR_UNSUPPORTED;
  }
  ss::SsdPromptParams k{};
  k.io = p->io_dtype; k.softplus = p->dt_softplus != 0;
  k.x = x; k.dt = dt; k.Bm = Bm; k.Cm = Cm; k.z = z; k.A = A; k.D = D; k.dt_bias = dt_bias;
  k.cu = cu_seqlens; k.slots = slots; k.has_state = has_state; k.state = state; k.y = y;
  char* ws = static_cast<char*>(workspace);
  k.ws_state = reinterpret_cast<float*>(ws);
  k.ws_decay = reinterpret_cast<float*>(ws + prompt_state_bytes(p));
  k.ws_cb = reinterpret_cast<float*>(ws + prompt_state_bytes(p) + prompt_decay_bytes(p));
  k.x_stride = p->x_stride; k.b_stride = p->b_stride; k.c_stride = p->c_stride; k.z_stride = p->z_stride;
  k.dt_stride = p->dt_stride;
  k.tokens = (int32_t)p->tokens; k.nseqs = (int32_t)p->nseqs; k.nslots = (int32_t)p->nslots;
  k.nheads = (int32_t)p->nheads; k.ngroups = (int32_t)p->ngroups; k.dstate = p->dstate;
  k.chunks = (int32_t)prompt_chunks(p);
  return from_hip(ss::launch_ssd_prompt(k, static_cast<hipStream_t>(stream)));
}

size_t ss_ssd_step_workspace_size(const ss_ssd_step_problem* p) {
  if (check_step_rows(p) != SS_OK) return 0;
  return (size_t)(p->rows * step_channels(p)) * 4;
}

ss_status ss_ssd_step(const ss_ssd_step_problem* p, const void* xbc, const void* dt, const float* A,
                      const float* conv_w, const float* conv_bias, const float* D, const void* z,
                      const float* dt_bias, const int32_t* slots, float* conv_state, float* state, void* y,
                      void* workspace, size_t workspace_bytes, void* stream) {
  const ss_status s = check_step_rows(p);
  if (s != SS_OK) return s;
  if (!xbc || !dt || !A || !conv_w || !state || !y || (!conv_state && p->width > 1)) return SS_ERR_NULL_ARG;
  const int64_t hp = p->nheads * 64, ch = step_channels(p);
  if (z && (p->z_stride < hp || p->z_stride > kMaxStride)) return SS_ERR_BAD_SHAPE;
  const void* ptrs[] = {A, conv_w, conv_bias, D, dt_bias, slots, conv_state, state, y, workspace};
  for (const void* q : ptrs)
    if (q && !aligned(q)) return SS_ERR_MISALIGNED;
  if (!aligned_to(xbc, 2) || !aligned_to(dt, 2) || !aligned_to(z, 2)) return SS_ERR_MISALIGNED;
  if (!slots && p->nslots < p->rows) return SS_ERR_UNSUPPORTED;
  const size_t need = ss_ssd_step_workspace_size(p);
  if (!workspace || workspace_bytes < need) return SS_ERR_UNSUPPORTED;
  {
    const size_t vb = (size_t)p->nheads * 4, cb = (size_t)ch * 4;
    const Span in[] = {{xbc, rows_bytes(p->rows, p->xbc_stride, ch, 2)},
                       {dt, rows_bytes(p->rows, p->dt_stride, p->nheads, 2)},
                       {z, rows_bytes(p->rows, z ? p->z_stride : hp, hp, 2)},
                       {A, vb}, {D, vb}, {dt_bias, vb}, {conv_w, cb * p->width}, {conv_bias, cb},
                       {slots, (size_t)p->rows * 4}};
    const Span outs[] = {{y, (size_t)(p->rows * hp) * 2},
                         {conv_state, (size_t)p->nslots * cb * (size_t)(p->width - 1)},
                         {state, (size_t)p->nslots * (size_t)(hp * p->dstate) * 4},
                         {workspace, need}};
    if (conflict(in, outs)) return SS_ERR_UNSUPPORTED;
  }
  ss::SsdStepParams k{};
  k.io = p->io_dtype; k.softplus = p->dt_softplus != 0; k.width = p->width;
  k.xbc = xbc; k.dt = dt; k.z = z; k.A = A; k.D = D; k.dt_bias = dt_bias; k.conv_w = conv_w; k.conv_bias = conv_bias;
  k.slots = slots; k.conv_state = conv_state; k.state = state; k.y = y; k.ws_xbc = static_cast<float*>(workspace);
  k.xbc_stride = p->xbc_stride; k.dt_stride = p->dt_stride; k.z_stride = p->z_stride;
  k.rows = (int32_t)p->rows; k.nslots = (int32_t)p->nslots; k.nheads = (int32_t)p->nheads;
  k.ngroups = (int32_t)p->ngroups; k.dstate = p->dstate; k.channels = (int32_t)ch;
  return from_hip(ss::launch_ssd_step(k, static_cast<hipStream_t>(stream)));
}

ss_status ss_copy_probe(const void* src, void* dst, size_t bytes, void* stream) {
  if (!src || !dst) return SS_ERR_NULL_ARG;
  if (!aligned(src) || !aligned(dst)) return SS_ERR_MISALIGNED;
  if (bytes % 16 != 0 || bytes == 0) return SS_ERR_BAD_SHAPE;
  return from_hip(ss::launch_copy(src, dst, (int64_t)bytes, static_cast<hipStream_t>(stream)));
}

ss_status ss_alu_probe(int32_t kind, int32_t workgroups, int32_t iters, int32_t lds_bytes, int64_t* out,
                       void* stream) {
  if (!out) return SS_ERR_NULL_ARG;
  if (!aligned(out)) return SS_ERR_MISALIGNED;
  if (kind < SS_PROBE_FMA || kind > SS_PROBE_SCAN_STEP) return SS_ERR_UNSUPPORTED;
  if (workgroups < 1 || workgroups > (1 << 20) || iters < 1 || iters > (1 << 20)) return SS_ERR_BAD_SHAPE;
  if (lds_bytes < 0 || lds_bytes > 65536) return SS_ERR_BAD_SHAPE;
  return from_hip(ss::launch_alu_probe(kind, workgroups, iters, lds_bytes, out, static_cast<hipStream_t>(stream)));
}

}  // extern "C"
