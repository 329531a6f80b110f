// q8_kv.h -- what the cache and attention kernels (q8_kv.hip, q8_attn.hip,
// q8_attn_rows.hip) and their host side (q8_kv_api.cpp) share.  Not installed;
// the public ABI is include/q8gemv.h.
#pragma once

#include <stddef.h>
#include <stdint.h>

#include <hip/hip_runtime_api.h>

#include "../../include/q8gemv.h"

namespace q8 {

// A cache by what the kernels need of it.
struct KvCache {
  char *k, *v;
  int n_pages, heads, dim;
  int page_log2;
  int fmt;
  // bytes of one (page, head) record and of one page
  __host__ __device__ unsigned record() const {
    const unsigned vals = (unsigned)dim << page_log2;
    return fmt == Q8_KV_BF16 ? 2 * vals : vals + vals / 8;
  }
  __host__ __device__ size_t page_bytes() const { return (size_t)record() * heads; }
};

struct HeadsArgs {
  const float *q, *k, *v;
  long long ldq, ldk, ldv;
  int m, q_heads;
  const float *q_norm, *k_norm;
  const double *freqs;
  float eps, attn_factor;
  int rot, layout;
  const int32_t *positions, *slots;
  uint16_t *q_out;
  KvCache cache;
};

// Attention of either form.  row_start null: one row a sequence (m == n).
struct AttnArgs {
  const uint16_t *q;
  int m, n, q_heads, group;     // group: query heads per key/value head
  KvCache cache;
  const int32_t *table;
  long long max_pages;
  const int32_t *lens, *row_start;
  float scale_log2;             // scale * log2(e)
  int window, sinks;
  uint16_t *o;
  int8_t *oq, *oq_view;         // the quantized output (null: none)
  float *oq_scale;
  unsigned *counters;           // arrival counters, zero between calls
  float *partial;
  int chunks;                   // decode: workgroups along the tokens; rows: key splits
};

// Tokens of a tile: one pass of the matrix cores over a head's keys.
constexpr int kKvTile = 32;

// Workgroups a decode launch divides all tokens among, for each (key/value
// head, group of 16 query heads) unit.
int attn_decode_chunks(int64_t units);
size_t attn_decode_partial_bytes(int64_t n, int64_t q_heads, int64_t kv_heads, int64_t dim);
// Key splits of a rows launch.
int attn_rows_splits(int64_t m, int64_t n, int64_t q_heads, int64_t kv_heads, int64_t dim,
                     int fmt);
size_t attn_rows_partial_bytes(int64_t m, int64_t n, int64_t q_heads, int64_t kv_heads,
                               int64_t dim, int fmt);

hipError_t launch_kv_step(const q8_kv_step_args &a, hipStream_t stream);
hipError_t launch_rope_freqs(const q8_rope &r, double *freqs, hipStream_t stream);
hipError_t launch_qkv_heads(const HeadsArgs &a, hipStream_t stream);
hipError_t launch_kv_gather(const KvCache &c, const int32_t *slots, int rows, uint16_t *k_out,
                            uint16_t *v_out, hipStream_t stream);
hipError_t launch_attn_decode(const AttnArgs &a, hipStream_t stream);
hipError_t launch_attn_rows(const AttnArgs &a, hipStream_t stream);

}  // namespace q8
