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

// Rows of the segments in which linear attention walks its sequences (the longest
// of `longest` rows, all of them of `tokens`; `walks` of each), a multiple of 64, or
// kLinWhole where none is split: as many segments as give every CU two workgroups at
// once, none of less than kLinLeast rows, and no sequence of no more than twice these.
constexpr int kLinWhole = 1 << 30, kLinLeast = 128;
inline int lin_segment(int64_t tokens, int64_t nseqs, int64_t longest, int64_t walks, int64_t cus) {
  if (longest <= 2 * kLinLeast) return kLinWhole;
  int64_t rows;
  if (nseqs * longest == tokens) {  // all alike
    const int64_t n = 2 * cus / (nseqs * walks);
    if (n < 2) return kLinWhole;
    rows = (longest + n - 1) / n;
  } else {
    rows = tokens * walks / (2 * cus);
  }
  rows = (rows + 63) / 64 * 64;
  if (rows < kLinLeast) rows = kLinLeast;
  return rows >= longest ? kLinWhole : (int)rows;
}

}  // namespace ss
