// ss_plan.h -- which variant of a kernel a problem takes, by its sizes and the
// GPU's CUs.  Internal to libss.so; plain integers, so that tests can name the
// variant that they reach.
#pragma once

#include <stdint.h>

namespace ss {

// The CUs of plans that sizes alone decide, workspaces among them: those of an MI355X
constexpr int64_t kPlanCus = 256;

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

// How linear attention walks its sequences (`walks` of each, the longest of `longest`
// rows): whole, or cut into pieces of some chunks of 64 rows, as many as give every CU
// two workgroups at once, none of less than 128 rows and none of sequences of up to 384
// rows.  A walk takes 3.6 us a chunk, a cut two more launches (12 heads of 128 x 128 in
// bf16, whole against pieces of 128 rows: 1 sequence of 256 rows 18.5 and 23.7 us, of 512
// 33.1 and 24.5, of 1024 62.6 and 28.7; 4 of 384 26.3 and 31.7, of 512 33.9 and 30.4, of 1024
// 63.3 and 41.6).  One prompt of 32769 rows with 16 walks: pieces of 448 rows 175 us, 704 157,
// 1088 (its choice: 496 workgroups) 144, 1280 157, whole 1794; a layer's 8 x 2048 rows with 12
// walks 83 with 448 (its choice), 86 with 512, 98 with 384, 94 with 256, 122 whole.
// Packed sequences' pieces go on over their ends, for their lengths are not known: 24
// ragged prompts of 16384 rows with 12 walks 113 us, in pieces that began with their
// sequences 119 to 132.
// Of more walks than CUs, all alike, those beyond the last multiple of the CUs would run
// on as long as the others: these alone are cut, one piece for every CU, where they are a
// quarter of the CUs at most and long enough (the layer's gradients, 36 walks: 256 whole
// and 32 in 8 pieces 159 us, all whole 175).  Of 256 and some more forward walks of 128 x 128,
// 24 chunks each, those beyond cut and all whole: 16 more 120 and 141 us, 32 125 and 141, 64
// 135 and 144, 96 151 and 145, 128 167 and 149; 64 chunks: 16 297 and 361, 64 346 and 368, 96 385
// and 376; 16 chunks: 16 84 and 95, 64 97 and 97; 8 chunks: 16 53 and 51, 64 57 and 50.
struct LinCut {
  int whole, span, pieces, stride;  // as in LinParams
};
inline LinCut lin_cut(bool packed, int64_t tokens, int64_t nseqs, int64_t longest, int64_t walks, int64_t cus) {
  const int64_t all = nseqs * walks;
  const LinCut none{(int)all, 1, 0, 1};
  if (longest <= 384) return none;
  const int64_t chunks = packed ? tokens / 64 + nseqs : (longest + 63) / 64;  // of all sequences, or of each
  int64_t cut = packed ? walks : all, n = 2 * cus / cut;
  if (!packed && all > cus) {
    cut = all % cus;
    if (cut == 0 || cut > cus / 4 || chunks < 24) return none;
    n = cus / cut;
  }
  if (n < 2) return none;
  const int64_t span = chunks <= 2 * n ? 2 : (chunks + n - 1) / n;
  if (span >= chunks) return none;
  return {packed ? 0 : (int)(all - cut), (int)span, (int)((chunks + span - 1) / span), (int)cut};
}

}  // namespace ss
