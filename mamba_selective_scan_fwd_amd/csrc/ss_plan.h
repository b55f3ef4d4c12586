// ss_plan.h -- which variant of a kernel a problem takes, by its sizes and the
// GPU's CUs.  Internal to libss.so; plain integers, so that tests can name the
// variant that they reach.
#pragma once

#include <stdint.h>

namespace ss {

// Heads per workgroup: of 1, 2 and 3 the one for which the workgroups' rounds
// over 2 per CU take the least time, a workgroup's being its heads and two
// heads' worth of its own (the weights, V, the first loads).  With 1, 2 and 3: 24
// ragged prompts of 16384 tokens, 24 heads, state 128: 60, 50, 50 us; five prompts
// of 131 tokens: 6.7, 8.4, 10.7 us; one of 32769 tokens, state 64, fp16: 83, 68,
// 68 us (4 spills registers at state 128: 66 us for the first).
inline int state_heads(int64_t chunk_groups, int64_t heads_per_group, int64_t cus) {
  int best = 1;
  int64_t cost = -1;
  for (int hb = 1; hb <= 3; ++hb) {
    const int64_t wgs = chunk_groups * ((heads_per_group + hb - 1) / hb);
    const int64_t c = (wgs + 2 * cus - 1) / (2 * cus) * (hb + 2);
    if (cost < 0 || c <= cost) {
      cost = c;
      best = hb;
    }
  }
  return best;
}

// Chunks' states that the prompts' pass loads ahead: sixteen where a few long
// prompts leave the CUs few workgroups: one prompt of 32769 tokens, 24 heads,
// state 64 (96 workgroups, 129 chunks) takes 20.9 us with 16 against 46.3 us with
// 4 (4.9 and 2.2 TB/s), while 24 ragged prompts of 16384 tokens, state 128 (4608
// workgroups) take 31.8 us against 24.6 us: there the loads behind a prompt's end
// are what is left.
inline int pass_ahead(int64_t workgroups, int64_t chunks, int64_t nseqs, int64_t cus) {
  return workgroups <= 4 * cus && chunks >= 8 * nseqs ? 16 : 4;
}

// Chunk places of 64 rows to a piece in which linear attention walks its sequences, or
// 0: each whole.  `chunks`: the places of all packed sequences, or of each of `runs` of
// one length (the longest of `longest` rows); `walks` of each.  As many pieces as give
// every CU two workgroups at once, none of less than 128 rows, and none of sequences of up to
// 384 rows.  A walk takes 3.5 us a chunk, a split two more launches (12 heads of 128 x 128
// in bf16, whole against segments of 128 rows: 1 sequence of 256 rows 17.5 and 22.7 us, of
// 512 31.6 and 24.1, of 1024 60.1 and 27.5; 4 of 384 24.9 and 32.4, of 1024 61.2 and
// 40.3).  One prompt of 32769 rows with 16 walks: pieces of 448 rows 151 us, 704 139, 1088 (its
// choice: 496 workgroups) 136, 1280 151, whole 1700; a layer's 8 x 2048 rows with 12 walks
// 83 with 384 or 448 (its choice), 89.5 with 256, 118 whole, and with the gradients' 36 walks
// (one piece each) 176 whole, 200 with 512 to 1024.  Pieces of packed sequences go on over
// their ends, for their lengths are not known: 24 ragged prompts of 16384 rows with 12
// walks 113 us, 119 to 132 in pieces that begin with their sequences.  Of sequences of one
// length they do not: the layer's gradients take 208 us in 14 equal pieces a head.
inline int lin_span(int64_t chunks, int64_t runs, int64_t longest, int64_t walks, int64_t cus) {
  if (longest <= 384) return 0;
  const int64_t pieces = 2 * cus / (runs * walks);
  if (pieces < 2) return 0;
  const int64_t span = chunks <= 2 * pieces ? 2 : (chunks + pieces - 1) / pieces;
  return span < chunks ? (int)span : 0;
}

}  // namespace ss
