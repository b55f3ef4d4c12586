// ss_packed.h -- packed sequences (device side).  Internal to libss.so.
//
// cu holds nseqs + 1 row offsets; sequence s is rows cu[s] .. cu[s + 1] - 1.
// A workgroup takes a chunk of 2^LOGQ rows counted from its sequence's first
// row, so that no chunk holds two sequences.  Sequence s owns the chunk places
// (cu[s] >> LOGQ) + s onwards: from one sequence to the next these grow by at
// least the number of chunks of the first (floor(b / Q) - floor(a / Q) + 1 >=
// ceil((b - a) / Q)), so places never collide, (tokens >> LOGQ) + nseqs places
// hold every batch, and neither the host nor an extra kernel has to see the
// lengths.  Places behind a sequence's last chunk stay empty.
//
// The offsets are clamped to [0, tokens] and every end to its start, so that
// no content of cu makes a kernel leave its buffers.
#pragma once

#include "ss_device.h"

namespace ss {

struct SeqChunk {
  int seq;
  int begin;  // the sequence's first row
  int len;    // its rows
  int chunk;  // the place's chunk of it; the place is empty unless 0 <= chunk * Q < max(len, 1)
};

__device__ __forceinline__ int seq_row(const int32_t* cu, int i, int tokens) {
  const int v = cu[i];
  return v < 0 ? 0 : v > tokens ? tokens : v;
}

// The sequence whose chunk place `place` is (uniform over the wave): a search
// with 64 probes a step, so up to 64 sequences take one load, 4096 two.
template <int LOGQ>
__device__ __forceinline__ SeqChunk find_chunk(const int32_t* cu, int nseqs, int tokens, int place) {
  const int lane = threadIdx.x % 64;
  int lo = 0, n = nseqs;
  while (n > 1) {
    const int step = (n + 63) >> 6, k = lane * step;
    bool le = false;
    if (k < n) le = (seq_row(cu, lo + k, tokens) >> LOGQ) + lo + k <= place;
    int cnt = (int)__builtin_popcountll(__builtin_amdgcn_ballot_w64(le));
    cnt = cnt < 1 ? 1 : cnt;  // cnt <= ceil(n / step): lo stays inside
    lo += (cnt - 1) * step;
    n -= (cnt - 1) * step;
    n = n < step ? n : step;
  }
  SeqChunk q;
  q.seq = uniform(lo);
  q.begin = uniform(seq_row(cu, q.seq, tokens));
  const int end = uniform(seq_row(cu, q.seq + 1, tokens));
  q.len = end > q.begin ? end - q.begin : 0;
  q.chunk = place - ((q.begin >> LOGQ) + q.seq);
  return q;
}

// the slot of sequence or row i, -1 for none (an index outside the pool is none)
__device__ __forceinline__ int slot_of(const int32_t* slots, int i, int nslots) {
  const int v = slots ? slots[i] : i;
  return v >= 0 && v < nslots ? v : -1;
}

}  // namespace ss
