// q8_logits.h -- what the host side of the logits' calls (q8_logits_api.cpp) and
// their kernels (q8_logits.hip: the rules; q8_sample.hip: the draw) share.
#pragma once

#include <stdint.h>

#include <hip/hip_runtime.h>

namespace q8 {

struct LogitRules {
  const int32_t *tokens;        // m x ld_tokens, or null
  int64_t ld_tokens;
  const int32_t *lens;          // m
  const int32_t *prompt_lens;   // m, or null: 0
  const float *repetition, *presence, *frequency;   // m each, or null
  const int32_t *bias_start;    // m + 1, or null
  const int32_t *bias_token;
  const float *bias_value;
  const uint32_t *mask;         // mask_rows x ld_mask words, or null
  int64_t ld_mask;
  const int32_t *mask_row;      // m, or null: row r's is r
  int mask_rows;
  int64_t n_bias;               // entries of bias_token and bias_value
};

struct LogitRulesArgs {
  const float *logits;
  float *out;
  int64_t ld, ld_out;
  int m, V;
  LogitRules r;
};
hipError_t launch_logit_rules(const LogitRulesArgs &a, hipStream_t stream);

// What the draw's launches hand on through the workspace.
struct SliceStat {                            // of a slice of a row
  float top;                                  // its largest logit
  int at;                                     // the lowest index of that
  double exp_sum;                             // of exp(l - top)
  float sum;                                  // of the logits not far below it
  unsigned n;                                 // how many those are
};
struct RowCut {                               // where a row's order is cut
  int bin;                                    // the step of M - l; kSampleBins: nowhere
  unsigned bin_n;                             // tokens in it
  unsigned long long before_n, before_w;      // tokens and weight before it
  unsigned long long total_w;
  unsigned n_cand;
};
struct Candidate {
  float l;
  int i;
};

constexpr int kSampleTile = 1024;             // tokens a wave takes at a time
constexpr int kSampleSlice = 4096;            // tokens of a slice of the statistics
constexpr int kSampleBins = 2048, kSampleCand = 1024;
constexpr int kMaxVocab = 1 << 20;
constexpr int kSampleHeld = 4 * 16 * kSampleTile;   // of a row in a workgroup's registers

// Which rows are drawn by one launch, a workgroup a row, without a workspace: those that
// fit its registers, from half of them on only with rows for a third of the CUs (us, mean
// of the kinds of rows, one launch against slices: 1 x 1000 11 against 23, 1 x 32000 20
// against 25, 256 x 32000 25 against 46, 128 x 65000 38 against 46, 256 x 65000 43 against
// 61; but 1 x 50001 28 against 27, 8 x 50001 mixed 42 against 33, 64 x 65000 mixed 57
// against 49).
constexpr int kSampleHeldRows = 96;
constexpr bool sample_in_one_launch(int64_t m, int64_t V) {
  return V <= kSampleHeld / 2 || (V <= kSampleHeld && m >= kSampleHeldRows);
}

struct SampleArgs {
  const float *logits;
  int64_t ld;
  int m, V;
  const float *temperature, *top_p, *min_p;   // m each, or null: 1, 1, 0
  const int32_t *top_k;                       // m, or null: all
  const double *u;                            // m
  int32_t *token;
  float *logprob;                             // m, or null
  // the workspace
  int slices, parts, row_tiles;               // of a row: statistics, workgroups a pass, tiles
  SliceStat *stats;                           // m x slices
  RowCut *cuts;                               // m
  float *tops;                                // m x row_tiles: a tile's largest logit
  unsigned long long *tiles;                  // m x row_tiles: kept weight
  uint32_t *counts;                           // m x parts x kSampleBins
  unsigned long long *masses;                 // m x parts x kSampleBins
  Candidate *cands;                           // m x kSampleCand
};
hipError_t launch_sample(const SampleArgs &a, hipStream_t stream);

}  // namespace q8
