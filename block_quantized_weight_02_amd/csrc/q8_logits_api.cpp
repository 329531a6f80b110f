// q8_logits_api.cpp -- host side of the logits' calls declared in include/q8gemv.h:
// argument validation before any launch.
#include <hip/hip_runtime.h>

#include <algorithm>

#include "../../include/q8gemv.h"
#include "q8_checks.h"
#include "q8_logits.h"

namespace {

using namespace q8;

static_assert(Q8_MAX_VOCAB == kMaxVocab, "the vocabulary's limit of the ABI and the kernels");

int check_rows(const float *logits, int64_t ld, int64_t m, int64_t V, const char *ld_name) {
  int st;
  if ((st = check_range(m, 1, Q8_MAX_GEMM_ROWS, "m"))) return st;
  if ((st = check_range(V, 1, Q8_MAX_VOCAB, "V"))) return st;
  if (ld < V || ld % 4 || ld > kMaxInt)
    return report_error(Q8_ERR_SHAPE, "%s = %lld: need a multiple of 4, at least %lld", ld_name,
                        (long long)ld, (long long)V);
  return Q8_OK;
}

// Workgroups of a row and pass, at most: of 8 waves, a tile a wave, and not too many for
// one workgroup to sum their histograms.
int64_t most_parts(int64_t tiles) { return std::min<int64_t>((tiles + 7) / 8, 64); }
constexpr int64_t kParts = 1024;           // of all rows together, about

// The workspace of rows drawn in slices, with `parts` workgroups a pass in all: its bytes,
// and with `ws` the places in it.  The products' and attention's counters at its start are
// left alone, so that one workspace serves all.
size_t sample_layout(SampleArgs &a, int64_t rows, int64_t parts, char *ws) {
  const int64_t tiles = (a.V + kSampleTile - 1) / kSampleTile;
  a.slices = (a.V + kSampleSlice - 1) / kSampleSlice;
  a.row_tiles = (int)tiles;
  size_t at = kCounterBytes;
  const auto take = [&](size_t bytes) {
    char *p = ws + at;
    at += (size_t)round_up((int64_t)bytes, 256);
    return ws ? p : nullptr;
  };
  const size_t m = (size_t)rows;
  a.stats = reinterpret_cast<SliceStat *>(take(m * a.slices * sizeof(SliceStat)));
  a.cuts = reinterpret_cast<RowCut *>(take(m * sizeof(RowCut)));
  a.tops = reinterpret_cast<float *>(take(m * tiles * 4));
  a.tiles = reinterpret_cast<unsigned long long *>(take(m * tiles * 8));
  a.counts = reinterpret_cast<uint32_t *>(take((size_t)parts * kSampleBins * 4));
  a.masses = reinterpret_cast<unsigned long long *>(take((size_t)parts * kSampleBins * 8));
  a.cands = reinterpret_cast<Candidate *>(take(m * kSampleCand * sizeof(Candidate)));
  return at;
}

// Bytes that serve every call of up to m rows of up to V logits: of the sliced ones among
// them the most rows and workgroups, and 256 bytes where there are none.
size_t sample_bytes(int64_t m, int64_t V) {
  const int64_t rows = sample_in_one_launch(1, V) ? 0
                       : sample_in_one_launch(m, V) ? kSampleHeldRows - 1 : m;
  if (rows == 0) return kCounterBytes + 256;
  SampleArgs a{};
  a.V = (int)V;
  const int64_t each = most_parts((V + kSampleTile - 1) / kSampleTile);
  return sample_layout(a, rows, std::min(rows * each, std::max(kParts, rows)), nullptr);
}

// A sliced call's places, within sample_bytes(m, V) bytes.
void sample_places(SampleArgs &a, char *ws) {
  // (40 rows of 131072, mixed: 8 each 47 us, 12 46, 16 46, 25 52; 256 rows: 2 each 121, 4
  // 105, 8 99 but all of one kind 83, 85, 93)
  const int64_t tiles = (a.V + kSampleTile - 1) / kSampleTile;
  a.parts = (int)std::min(most_parts(tiles), std::max<int64_t>(1, kParts / a.m));
  sample_layout(a, a.m, (int64_t)a.m * a.parts, ws);
}

}  // namespace

extern "C" {

int q8_logits_rules(const float *logits, int64_t ld, int64_t m, int64_t V,
                    const q8_logit_rules *rules, float *out, int64_t ld_out, hipStream_t stream) {
  int st;
  if ((st = check_rows(logits, ld, m, V, "ld")) || (st = check_rows(out, ld_out, m, V, "ld_out")))
    return st;
  if (!rules) return report_error(Q8_ERR_NULL, "rules is NULL");
  if ((st = check_ptr(logits, "logits")) || (st = check_ptr(out, "out"))) return st;
  if (logits == out && ld != ld_out)
    return report_error(Q8_ERR_SHAPE, "in place ld_out = %lld has to be ld = %lld",
                        (long long)ld_out, (long long)ld);
  LogitRulesArgs a{};
  a.logits = logits;
  a.out = out;
  a.ld = ld;
  a.ld_out = ld_out;
  a.m = (int)m;
  a.V = (int)V;
  LogitRules &r = a.r;
  if (rules->tokens) {
    if ((st = check_ptr(rules->tokens, "tokens")) || (st = check_ptr(rules->lens, "lens")) ||
        (st = check_opt(rules->prompt_lens, "prompt_lens")) ||
        (st = check_range(rules->ld_tokens, 1, kMaxInt, "ld_tokens")) ||
        (st = check_opt(rules->repetition, "repetition")) ||
        (st = check_opt(rules->presence, "presence")) ||
        (st = check_opt(rules->frequency, "frequency")))
      return st;
    r.tokens = rules->tokens;
    r.ld_tokens = rules->ld_tokens;
    r.lens = rules->lens;
    r.prompt_lens = rules->prompt_lens;
    r.repetition = rules->repetition;
    r.presence = rules->presence;
    r.frequency = rules->frequency;
  } else if (rules->repetition || rules->presence || rules->frequency) {
    return report_error(Q8_ERR_NULL, "tokens is NULL and a penalty is given");
  }
  if (rules->bias_start) {
    if ((st = check_ptr(rules->bias_start, "bias_start")) ||
        (st = check_range(rules->bias_entries, 0, kMaxInt, "bias_entries")))
      return st;
    if (rules->bias_entries > 0 && ((st = check_ptr(rules->bias_token, "bias_token")) ||
                                    (st = check_ptr(rules->bias_value, "bias_value"))))
      return st;
    r.bias_start = rules->bias_start;
    r.bias_token = rules->bias_token;
    r.bias_value = rules->bias_value;
    r.n_bias = rules->bias_entries;
  }
  if (rules->mask) {
    if ((st = check_ptr(rules->mask, "mask")) || (st = check_opt(rules->mask_row, "mask_row")) ||
        (st = check_range(rules->ld_mask, (V + 31) / 32, kMaxInt, "ld_mask")) ||
        (st = check_range(rules->mask_rows, rules->mask_row ? 0 : m, kMaxInt, "mask_rows")))
      return st;
    r.mask = rules->mask;
    r.ld_mask = rules->ld_mask;
    r.mask_row = rules->mask_row;
    r.mask_rows = (int)rules->mask_rows;
  }
  return done(launch_logit_rules(a, stream), "logit rules launch");
}

size_t q8_sample_workspace_bytes(int64_t m, int64_t V) {
  if (check_rows(nullptr, (V + 3) / 4 * 4, m, V, "ld")) return 0;
  return sample_bytes(m, V);
}

int q8_sample(const float *logits, int64_t ld, int64_t m, int64_t V, const q8_sampling *sampling,
              int32_t *token, float *logprob, hipStream_t stream, void *workspace, size_t ws_bytes) {
  int st;
  if ((st = check_rows(logits, ld, m, V, "ld"))) return st;
  if (!sampling) return report_error(Q8_ERR_NULL, "sampling is NULL");
  if ((st = check_ptr(logits, "logits")) || (st = check_ptr(token, "token")) ||
      (st = check_opt(logprob, "logprob")) ||
      (st = check_ptr(sampling->u, "u")) ||
      (st = check_opt(sampling->temperature, "temperature")) ||
      (st = check_opt(sampling->top_k, "top_k")) || (st = check_opt(sampling->top_p, "top_p")) ||
      (st = check_opt(sampling->min_p, "min_p")))
    return st;
  SampleArgs a{};
  a.logits = logits;
  a.ld = ld;
  a.m = (int)m;
  a.V = (int)V;
  a.temperature = sampling->temperature;
  a.top_k = sampling->top_k;
  a.top_p = sampling->top_p;
  a.min_p = sampling->min_p;
  a.u = sampling->u;
  a.token = token;
  a.logprob = logprob;
  if ((st = check_workspace(workspace, ws_bytes, sample_bytes(m, V)))) return st;
  if (!sample_in_one_launch(m, V)) sample_places(a, static_cast<char *>(workspace));
  return done(launch_sample(a, stream), "sample launch");
}

}  // extern "C"
