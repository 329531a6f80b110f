// q8_kv.hip -- the cache's bookkeeping and what writes it: a step's page
// tables, positions and slots (q8_kv_step), the rotary frequencies
// (q8_rope_freqs), head norms with the position rotation and the cache rows
// (q8_qkv_heads), and rows read back (q8_kv_gather).  The formulas, layouts
// and refusals are in include/q8gemv.h.
#include <hip/hip_runtime.h>

#include "q8_device.h"
#include "q8_kv.h"

namespace q8 {
namespace {

using namespace dev;

// ---- a step's tables -----------------------------------------------------------

// Inclusive sum over the workgroup's threads in thread order; *total gets the
// sum of all.  sums: one int per wave.
__device__ __forceinline__ int scan_workgroup(int v, int *sums, int *total) {
  const int lane = threadIdx.x & 63, wave = threadIdx.x >> 6, waves = blockDim.x >> 6;
#pragma unroll
  for (int o = 1; o < 64; o <<= 1) {
    const int u = __shfl_up(v, o);
    if (lane >= o) v += u;
  }
  __syncthreads();                      // sums may still be read from the last scan
  if (lane == 63) sums[wave] = v;
  __syncthreads();
  int before = 0, all = 0;
  for (int w = 0; w < waves; ++w) {
    const int s = sums[w];
    before += w < wave ? s : 0;
    all += s;
  }
  *total = all;
  return v + before;
}

// For each lane's sequence with `pages` > first: put(lane, k, get(lane, k)) for k =
// first .. pages-1, a sequence at a time, the wave's lanes side by side over its
// pages (four sequences at a time measured the same, 10.2 us against 10.1).
template <class Get, class Put>
__device__ __forceinline__ void each_page(int pages, int first, Get get, Put put) {
  const int lane = threadIdx.x & 63;
  unsigned long long some = __ballot(pages > first);
  while (some) {
    const int src = __ffsll(some) - 1, cnt = __shfl(pages, src);
    some &= some - 1;
    for (int k = first; k < cnt; k += 64) {
      const int at = k + lane;
      const int v = get(src, at, at < cnt);
      put(src, at, v, at < cnt);
    }
  }
}

// One workgroup: thread t takes sequences t*E .. t*E+E-1 (E = 1 up to 1024
// sequences, 8 at most), so that two running sums in thread order -- rows and
// returned pages, then needed pages -- give every sequence its place.  It takes
// rows t*R .. t*R+R-1 too (R = 1 or 8): each sequence marks its first row in
// LDS, and a running maximum over the marks gives every row its sequence; the
// rows then go through LDS to be looked up side by side, since neighbours share
// the table's lines.  1024 sequences with 8192 rows: 10.1 us; 13.8 with a search
// in the row starts, 17.0 with each thread's own eight rows looked up.  All lengths are
// read before any is written (lens_out may be lens); the table's and the list's
// new entries are read back after a barrier by the workgroup that wrote them.
// Bound by latency: launch, three dependent loads, the barriers; past 1024
// sequences also by the pages moved, a sequence of the wave's after the other, on
// one CU (2048 sequences of one row 20 us, 8192 32 us).
constexpr int kRefused = -0x7fffffff - 1;

template <int E, int R>
__global__ void __launch_bounds__(1024)
kv_step_kernel(q8_kv_step_args a, int page_log2) {
  extern __shared__ __align__(16) int base[];   // n: a row's position less its row, or kRefused
  __shared__ __align__(16) uint16_t owner[1024 * R];   // at a sequence's first row: its number + 1
  __shared__ int sums[16], marks[16];
  const int n = (int)a.n, m = (int)a.m, most = (int)a.max_pages, cap = (int)a.free_cap;
  const int tid = threadIdx.x;
  const int P1 = (1 << page_log2) - 1;
  const long long longest = (long long)most << page_log2;
#pragma unroll
  for (int k = 0; k < R; ++k) owner[tid * R + k] = 0;
  int len[E], rows[E], held[E];
  bool ended[E];
  int sum_rows = 0, sum_back = 0;
#pragma unroll
  for (int e = 0; e < E; ++e) {
    const int i = tid * E + e;
    const int l = i < n ? a.lens[i] : 0;
    const int w = i < n ? a.new_rows[i] : 0;
    len[e] = (int)min((long long)max(l, 0), longest);
    ended[e] = w < 0;
    rows[e] = min(max(w, 0), m + 1);      // more than m is refused whatever the number
    held[e] = (len[e] >> page_log2) + ((len[e] & P1) != 0);
    sum_rows += rows[e];
    sum_back += ended[e] ? held[e] : 0;
  }
  const int count0 = min(max(a.free_count[0], 0), cap);
  int total_rows, total_back, total_need;
  int row = scan_workgroup(sum_rows, sums, &total_rows) - sum_rows;
  int back = scan_workgroup(sum_back, sums, &total_back) - sum_back;
  const int have = (int)min((long long)count0 + total_back, (long long)cap);

  // needed pages, and who is refused whatever the list holds
  int need[E], row0[E];
  bool barred[E];
  int sum_need = 0;
#pragma unroll
  for (int e = 0; e < E; ++e) {
    row0[e] = row;
    row += rows[e];
    const long long after = (long long)len[e] + rows[e];
    const int pages = (int)((after + P1) >> page_log2);
    barred[e] = tid * E + e < n && !ended[e] &&
                (pages > most || row > m || after > 0x7fffffff);
    need[e] = (ended[e] || barred[e]) ? 0 : pages - held[e];
    sum_need += need[e];
  }
  int upto = scan_workgroup(sum_need, sums, &total_need) - sum_need;
  int taken = 0, refusals = 0;
#pragma unroll
  for (int e = 0; e < E; ++e) {
    const int i = tid * E + e;
    const int first = upto;
    upto += need[e];
    const bool refused = barred[e] || (need[e] > 0 && upto > have);
    if (refused) ++refusals, need[e] = 0;
    taken += need[e];
    if (i < n) {
      base[i] = refused ? kRefused : len[e] - row0[e];
      a.row_start[i] = min(row0[e], m);
      if (rows[e] > 0 && row0[e] < m) owner[row0[e]] = (uint16_t)(i + 1);
      a.lens_out[i] = ended[e] ? 0 : (refused ? len[e] : len[e] + rows[e]);
    }
    // Ended sequences' pages go to the list's end.
    const int at = (int)min((long long)count0 + back, (long long)cap);
    const int gone = ended[e] ? held[e] : 0;
    back += gone;
    each_page(min(gone, cap - at), 0, [&](int src, int k, bool on) Q8_INLINE {
      const long long row = (long long)__shfl(i, src) * most;
      return on ? a.table[row + k] : 0;
    }, [&](int src, int k, int v, bool on) Q8_INLINE {
      const int to = __shfl(at, src);
      if (on) a.free_pages[to + k] = v;
    });
    row0[e] = first;                       // from here: the sequence's first grant
  }
  const int used = min(total_rows, m);
  if (tid == 0) a.row_start[n] = used;
  int all_taken, all_refused;
  (void)scan_workgroup(taken, sums, &all_taken);   // its barriers order the list's new entries
  (void)scan_workgroup(refusals, sums, &all_refused);
  if (tid == 0) {
    a.free_count_out[0] = have - all_taken;
    a.status[0] = all_refused;
    a.status[1] = max(total_need - have, 0);
  }
  // the rows' sequences, but for those that start before the wave's first row
  int seq[R];
#pragma unroll
  for (int k = 0; k < R; ++k) seq[k] = owner[tid * R + k];
#pragma unroll
  for (int k = 1; k < R; ++k) seq[k] = max(seq[k], seq[k - 1]);
  int upto_me = seq[R - 1];
#pragma unroll
  for (int o = 1; o < 64; o <<= 1) upto_me = max(upto_me, __shfl_up(upto_me, o));
  if ((tid & 63) == 63) marks[tid >> 6] = upto_me;
  int before = __shfl_up(upto_me, 1);
  if ((tid & 63) == 0) before = 0;
  // grants, from the list's end
#pragma unroll
  for (int e = 0; e < E; ++e) {
    const int i = tid * E + e;
    int32_t *to = a.table + (long long)i * most + held[e];
    const int32_t *from = a.free_pages + (have - 1 - row0[e]);
    if (need[e] > 0) to[0] = from[0];      // most take one page, if any
    each_page(need[e], 1, [&](int src, int k, bool on) Q8_INLINE {
      const int last = have - 1 - __shfl(row0[e], src);
      return on ? a.free_pages[last - k] : 0;
    }, [&](int src, int k, int v, bool on) Q8_INLINE {
      const long long to = (long long)__shfl(i, src) * most + __shfl(held[e], src);
      if (on) a.table[to + k] = v;
    });
  }
  __syncthreads();
  for (int w = 0; w < tid >> 6; ++w) before = max(before, marks[w]);
#pragma unroll
  for (int k = 0; k < R; ++k) seq[k] = max(seq[k], before);
  if constexpr (R > 1) {      // from here rows side by side: their table entries share lines
#pragma unroll
    for (int k = 0; k < R; ++k) owner[tid * R + k] = (uint16_t)seq[k];
    __syncthreads();
#pragma unroll
    for (int k = 0; k < R; ++k) seq[k] = owner[k * 1024 + tid];
  }
  int pos[R], slot[R];
#pragma unroll
  for (int k = 0; k < R; ++k) {
    const int r = k * 1024 + tid, i = max(seq[k] - 1, 0);
    const int b = r < used ? base[i] : kRefused;
    pos[k] = 0, slot[k] = -1;
    if (b != kRefused) {
      pos[k] = b + r;
      // a page index past what slots can name has none: it must not wrap to another page's
      const int page = a.table[(long long)i * most + (pos[k] >> page_log2)];
      const long long s = ((long long)page << page_log2) + (pos[k] & P1);
      slot[k] = s == (int)s ? (int)s : -1;
    }
  }
#pragma unroll
  for (int k = 0; k < R; ++k)
    if (k * 1024 + tid < m) {
      a.positions[k * 1024 + tid] = pos[k];
      a.slots[k * 1024 + tid] = slot[k];
    }
}

// ---- rotary frequencies ----------------------------------------------------------

__global__ void __launch_bounds__(128) rope_freqs_kernel(q8_rope r, double *__restrict__ freqs) {
  const int p = threadIdx.x, half = r.rot / 2;
  if (p >= half) return;
  const double kTwoPi = 6.283185307179586476925287;
  const double f = pow(r.base, -2.0 * p / r.rot);
  double keep = 1.0;
  if (r.scaling == Q8_ROPE_SCALE_LINEAR) {
    keep = 0.0;
  } else if (r.scaling == Q8_ROPE_SCALE_TURNS) {
    const double t = (double)r.original * f / kTwoPi;
    keep = fmin(fmax((t - r.low) / (r.high - r.low), 0.0), 1.0);
  } else if (r.scaling == Q8_ROPE_SCALE_INDEX) {
    const double d = r.rot / (2.0 * log(r.base));
    const double a = fmax(floor(d * log((double)r.original / (kTwoPi * r.high))), 0.0);
    double b = fmin(ceil(d * log((double)r.original / (kTwoPi * r.low))), (double)r.rot - 1.0);
    b = fmax(b, a + 0.001);
    keep = 1.0 - fmin(fmax((p - a) / (b - a), 0.0), 1.0);
  }
  freqs[p] = f * keep + (keep == 1.0 ? 0.0 : f / r.factor * (1.0 - keep));
}

// ---- head norms, rotation, cache rows ----------------------------------------------

__device__ __forceinline__ uint16_t bf16_bits(float f) {   // nearest even; NaN stays NaN
  return __builtin_bit_cast(uint16_t, (__bf16)f);
}
__device__ __forceinline__ uint2 bf16x4_bits(const float *x) {
  return make_uint2((uint32_t)bf16_bits(x[0]) | (uint32_t)bf16_bits(x[1]) << 16,
                    (uint32_t)bf16_bits(x[2]) | (uint32_t)bf16_bits(x[3]) << 16);
}

// Sum over the LPH lanes of a head, the same in all of them: neighbours, pairs,
// quads and eights through the lane-mirroring forms of an add, the rest by
// shuffles.
template <int CTRL>
__device__ __forceinline__ float dpp(float v) {
  return __int_as_float(__builtin_amdgcn_update_dpp(0, __float_as_int(v), CTRL, 0xf, 0xf, true));
}
template <int LPH>
__device__ __forceinline__ float sum_head(float v) {
  v += dpp<0xB1>(v);    // quad_perm 1 0 3 2
  v += dpp<0x4E>(v);    // quad_perm 2 3 0 1
  v += dpp<0x141>(v);   // row_half_mirror
  v += dpp<0x140>(v);   // row_mirror
#pragma unroll
  for (int o = 16; o < LPH; o <<= 1) v += __shfl_xor(v, o);
  return v;
}
// Maximum over the eight lanes of a block of 32 dims.
__device__ __forceinline__ float max_block(float v) {
  v = fmaxf(v, dpp<0xB1>(v));
  v = fmaxf(v, dpp<0x4E>(v));
  return fmaxf(v, dpp<0x141>(v));
}

// A wave handles one row: 64 / (D/4) heads side by side in a pass, a lane four
// dims of one head (one 16-byte load), `passes` passes.  The four angles' cos
// and sin are the same for all of a row's heads, so they are computed once a
// wave: the angle in turns in fp64 (a position of 2^31 keeps 2^-22 turns),
// reduced to half a turn, then fp32.  The norm's sum and the quantizer's amax
// are lane reductions within the head; the half layout's partner dims sit
// rot/8 lanes away.  Values lie eight tokens to a piece, so a row alone writes
// them two bytes at a time; where the rows of an aligned eight of tokens follow
// each other, as a prompt's do, their eight waves share the value heads out among
// themselves and write whole pieces: 8192 rows of 32 + 8 + 8 heads of 128 in 75 us
// (302 MB, 4.0 TB/s; a large copy reaches 4.8), 99 us with every row for itself;
// Q8_0 93 us (287 MB).
// Loads asked for two to six passes ahead measured no faster (101 .. 107 us).
template <int D, int FMT>
__global__ void __launch_bounds__(512)
qkv_heads_kernel(HeadsArgs a, int passes) {
  constexpr int LPH = D / 4, HPW = 64 / LPH;
  const int lane = threadIdx.x & 63;
  const int r = blockIdx.x * (blockDim.x >> 6) + (threadIdx.x >> 6);
  if (r >= a.m) return;
  const KvCache c = a.cache;
  // The slots of the rows around, in lanes 0 .. 15, its own in lane 7; eight:
  // whether the rows of its aligned eight tokens are all there, in order.
  const int near = r - 7 + (lane & 15);
  const int around = near >= 0 && near < a.m ? a.slots[near] : -1;
  const int slot = __builtin_amdgcn_readlane(around, 7);
  if (slot < 0 || (slot >> c.page_log2) >= c.n_pages) return;
  const unsigned in_order = (unsigned)__ballot(around == slot + near - r);
  const bool eight = (in_order >> (7 - (slot & 7)) & 0xff) == 0xff;
  const int hl = lane / LPH, il = lane % LPH, d0 = il * 4;
  const int P = 1 << c.page_log2, tok = slot & (P - 1);
  const size_t page_at = (size_t)(slot >> c.page_log2) * c.page_bytes();
  const int Ht = a.q_heads + 2 * c.heads;
  const int half = a.rot >> 1;

  float cs[4] = {1.0f, 1.0f, 1.0f, 1.0f}, sn[4] = {0.0f, 0.0f, 0.0f, 0.0f};
  int partner = lane;
  if (a.rot > 0 && d0 < a.rot) {
    const double pos = (double)max(a.positions[r], 0);
    const bool halves = a.layout == Q8_ROPE_HALF;
    const int p0 = halves ? (d0 < half ? d0 : d0 - half) : d0 >> 1;
    float ct[4], st[4];
#pragma unroll
    for (int e = 0; e < 4; ++e) {
      if (e < 2 || halves) {
        const double turns = pos * (a.freqs[p0 + e] * 0.15915494309189533577);
        const float f = (float)(turns - rint(turns));
        sincospif(2.0f * f, &st[e], &ct[e]);
        ct[e] *= a.attn_factor;
        st[e] *= a.attn_factor;
      }
    }
    // y = x cos + (partner) sin with the sign of the partner's term in sin
#pragma unroll
    for (int e = 0; e < 4; ++e) {
      const int t = halves ? e : e >> 1;
      cs[e] = ct[t];
      sn[e] = (halves ? d0 < half : (e & 1) == 0) ? -st[t] : st[t];
    }
    if (halves) partner = lane + (d0 < half ? half / 4 : -(half / 4));
  }
  float wq[4] = {1.0f, 1.0f, 1.0f, 1.0f}, wk[4] = {1.0f, 1.0f, 1.0f, 1.0f};
#pragma unroll
  for (int e = 0; e < 4; ++e) {
    if (a.q_norm) wq[e] = a.q_norm[d0 + e];
    if (a.k_norm) wk[e] = a.k_norm[d0 + e];
  }

  // Value head hv of the eight tokens that the row's is one of: a lane takes one
  // dim of all eight, so that a wave's loads and stores are both consecutive.
  const auto values_of_eight = [&](int hv) Q8_INLINE {
    char *rec = c.v + page_at + (size_t)hv * c.record();
#pragma unroll
    for (int d = lane; d < D; d += 64) {
      const float *src = a.v + (r - (slot & 7)) * a.ldv + (size_t)hv * D + d;
      float x[8];
#pragma unroll
      for (int t = 0; t < 8; ++t) x[t] = src[t * a.ldv];
      const size_t at = (size_t)(tok >> 3) * D + d;
      if constexpr (FMT == Q8_KV_BF16) {
        u32x4_t w;
#pragma unroll
        for (int t = 0; t < 4; ++t)
          w[t] = (uint32_t)bf16_bits(x[2 * t]) | (uint32_t)bf16_bits(x[2 * t + 1]) << 16;
        reinterpret_cast<u32x4_t *>(rec)[at] = w;
      } else {
        float dq[8];
        uint32_t w[2] = {0, 0};
#pragma unroll
        for (int t = 0; t < 8; ++t) {
          float am = max_block(fabsf(x[t]));
          am = fmaxf(am, dpp<0x140>(am));
          dq[t] = q8_scale_of(fmaxf(am, __shfl_xor(am, 16)));
          w[t / 4] |= (uint32_t)(uint8_t)q8_code_of(x[t], dq[t]) << 8 * (t % 4);
        }
        reinterpret_cast<u32x2_t *>(rec)[at] = u32x2_t{w[0], w[1]};
        if ((lane & 31) == 0) {
          f32x4_t *sc = reinterpret_cast<f32x4_t *>(rec + (size_t)D * P) + ((d >> 5) * P + (tok & ~7)) / 4;
          sc[0] = f32x4_t{dq[0], dq[1], dq[2], dq[3]};
          sc[1] = f32x4_t{dq[4], dq[5], dq[6], dq[7]};
        }
      }
    }
  };
  const auto pass = [&](int ps) Q8_INLINE {
    const int h = ps * HPW + hl;
    const bool live = h < Ht;
    const int kind = h < a.q_heads ? 0 : (h < a.q_heads + c.heads ? 1 : 2);
    const int hh = kind == 0 ? h : h - a.q_heads - (kind == 2 ? c.heads : 0);
    const int hv = ps * HPW - a.q_heads - c.heads;       // the pass's first head, among the values'
    if (eight && hv >= 0) {
#pragma unroll
      for (int i = 0; i < HPW; ++i)
        if (hv + i < c.heads && (hv + i) % 8 == (slot & 7)) values_of_eight(hv + i);
      return;
    }
    const float *src = kind == 0 ? a.q + r * a.ldq : (kind == 1 ? a.k + r * a.ldk : a.v + r * a.ldv);
    f32x4_t x4 = {0.0f, 0.0f, 0.0f, 0.0f};
    if (live) x4 = *reinterpret_cast<const f32x4_t *>(src + (size_t)hh * D + d0);
    float x[4] = {x4[0], x4[1], x4[2], x4[3]};
    if (a.q_norm || a.k_norm) {
      const float ss = sum_head<LPH>(x[0] * x[0] + x[1] * x[1] + x[2] * x[2] + x[3] * x[3]);
      const float inv = 1.0f / sqrtf(ss * (1.0f / D) + a.eps);
      const bool normed = (kind == 0 && a.q_norm) || (kind == 1 && a.k_norm);
#pragma unroll
      for (int e = 0; e < 4; ++e)
        if (normed) x[e] = x[e] * inv * (kind == 0 ? wq[e] : wk[e]);
    }
    float y[4];
#pragma unroll
    for (int e = 0; e < 4; ++e) {
      const float mate = a.layout == Q8_ROPE_HALF ? __shfl(x[e], partner) : x[e ^ 1];
      y[e] = x[e] * cs[e] + mate * sn[e];
    }
    if (kind == 2 || d0 >= a.rot) {
#pragma unroll
      for (int e = 0; e < 4; ++e) y[e] = x[e];
    }
    float dq = 0.0f;
    if constexpr (FMT == Q8_KV_Q8_0) {
      const float am = fmaxf(fmaxf(fabsf(y[0]), fabsf(y[1])), fmaxf(fabsf(y[2]), fabsf(y[3])));
      dq = q8_scale_of(max_block(am));
    }
    if (!live) return;
    if (kind == 0) {
      *reinterpret_cast<uint2 *>(a.q_out + ((size_t)r * a.q_heads + h) * D + d0) = bf16x4_bits(y);
      return;
    }
    char *rec = (kind == 1 ? c.k : c.v) + page_at + (size_t)hh * c.record();
    if constexpr (FMT == Q8_KV_BF16) {
      uint16_t *vals = reinterpret_cast<uint16_t *>(rec);
      if (kind == 1) {
        *reinterpret_cast<uint2 *>(vals + ((size_t)(d0 >> 3) * P + tok) * 8 + (d0 & 7)) =
            bf16x4_bits(y);
      } else {
#pragma unroll
        for (int e = 0; e < 4; ++e)
          vals[((size_t)(tok >> 3) * D + d0 + e) * 8 + (tok & 7)] = bf16_bits(y[e]);
      }
    } else {
      int8_t *vals = reinterpret_cast<int8_t *>(rec);
      int8_t q[4];
#pragma unroll
      for (int e = 0; e < 4; ++e) q[e] = q8_code_of(y[e], dq);
      if (kind == 1) {
        const uint32_t w = (uint32_t)(uint8_t)q[0] | (uint32_t)(uint8_t)q[1] << 8 |
                           (uint32_t)(uint8_t)q[2] << 16 | (uint32_t)(uint8_t)q[3] << 24;
        *reinterpret_cast<uint32_t *>(vals + ((size_t)(d0 >> 3) * P + tok) * 8 + (d0 & 7)) = w;
      } else {
#pragma unroll
        for (int e = 0; e < 4; ++e)
          vals[((size_t)(tok >> 3) * D + d0 + e) * 8 + (tok & 7)] = q[e];
      }
      if ((d0 & 31) == 0)
        reinterpret_cast<float *>(vals + (size_t)D * P)[(size_t)(d0 >> 5) * P + tok] = dq;
    }
  };
  const int first = blockIdx.y * passes, end = min(first + passes, (Ht + HPW - 1) / HPW);
  for (int ps = first; ps < end; ++ps) pass(ps);
}

// ---- rows read back -----------------------------------------------------------------

// A thread reads eight dims of one (row, head): one 16-byte piece of the keys,
// eight places of the values.  A launch holds fewer than 2^32 threads, the call
// up to 2^36 pieces, so past kGatherBlocks workgroups a thread takes several.
// 8192 rows of 8 heads of 128: 31 us (67 MB), Q8_0 29 (52 MB), against 14 and 11
// for a copy: bound by the values' reads of two bytes or one at a time.
constexpr long long kGatherBlocks = 1 << 20;

template <int FMT>
__device__ __forceinline__ void gather_piece(const KvCache &c, const int32_t *__restrict__ slots,
                                             uint16_t *__restrict__ k_out,
                                             uint16_t *__restrict__ v_out, int r, int piece) {
  const int D = c.dim;
  const int slot = slots[r];
  const int P = 1 << c.page_log2;
  if (slot < 0 || (slot >> c.page_log2) >= c.n_pages) return;
  const int h = piece / (D / 8), ch = piece % (D / 8);
  const int tok = slot & (P - 1);
  const size_t at = (size_t)(slot >> c.page_log2) * c.page_bytes() + (size_t)h * c.record();
  const size_t out = ((size_t)r * c.heads + h) * D + ch * 8;
#pragma unroll
  for (int which = 0; which < 2; ++which) {
    uint16_t *dst = which ? v_out : k_out;
    if (!dst) continue;
    const char *rec = (which ? c.v : c.k) + at;
    uint16_t y[8];
#pragma unroll
    for (int e = 0; e < 8; ++e) {
      const size_t i = which ? ((size_t)(tok >> 3) * D + ch * 8 + e) * 8 + (tok & 7)
                             : ((size_t)ch * P + tok) * 8 + e;
      if constexpr (FMT == Q8_KV_BF16) {
        y[e] = reinterpret_cast<const uint16_t *>(rec)[i];
      } else {
        const float d = reinterpret_cast<const float *>(rec + (size_t)D * P)[(ch >> 2) * P + tok];
        y[e] = bf16_bits((float)reinterpret_cast<const int8_t *>(rec)[i] * d);
      }
    }
    uint32_t w[4];
#pragma unroll
    for (int e = 0; e < 4; ++e) w[e] = (uint32_t)y[2 * e] | (uint32_t)y[2 * e + 1] << 16;
    *reinterpret_cast<uint4 *>(dst + out) = make_uint4(w[0], w[1], w[2], w[3]);
  }
}

template <int FMT>
__global__ void __launch_bounds__(256)
kv_gather_kernel(KvCache c, const int32_t *__restrict__ slots, int rows,
                 uint16_t *__restrict__ k_out, uint16_t *__restrict__ v_out) {
  const int per_row = c.heads * (c.dim / 8);
  const long long total = (long long)rows * per_row;
  for (long long idx = (long long)blockIdx.x * 256 + threadIdx.x; idx < total;
       idx += (long long)gridDim.x * 256)
    gather_piece<FMT>(c, slots, k_out, v_out, (int)(idx / per_row), (int)(idx % per_row));
}

int log2_of(int v) {
  int l = 0;
  while ((1 << l) < v) ++l;
  return l;
}

}  // namespace

hipError_t launch_kv_step(const q8_kv_step_args &a, hipStream_t stream) {
  const int need = (int)(a.n > a.m ? a.n : a.m);
  const int threads = need >= 1024 ? 1024 : (need + 63) / 64 * 64;
  const size_t lds = (size_t)a.n * 4;
  const int pl = log2_of(a.page);
  if (a.n > threads)
    kv_step_kernel<8, 8><<<1, 1024, lds, stream>>>(a, pl);
  else if (a.m > threads)
    kv_step_kernel<1, 8><<<1, 1024, lds, stream>>>(a, pl);
  else
    kv_step_kernel<1, 1><<<1, threads, lds, stream>>>(a, pl);
  return hipGetLastError();
}

hipError_t launch_rope_freqs(const q8_rope &r, double *freqs, hipStream_t stream) {
  rope_freqs_kernel<<<1, 128, 0, stream>>>(r, freqs);
  return hipGetLastError();
}

hipError_t launch_qkv_heads(const HeadsArgs &a, hipStream_t stream) {
  const int D = a.cache.dim, hpw = 256 / D, heads = a.q_heads + 2 * a.cache.heads;
  const int all = (heads + hpw - 1) / hpw;
  constexpr int waves = 8;
  const int groups = (a.m + waves - 1) / waves;
  // A row's heads are split over as many waves as make 4096 in all, half of what
  // the card holds: 512 rows of 48 heads of 128 take 9.9 us, with 1024 waves 16.0,
  // with 16384 (each computing its row's angles) 13.3.
  int split = 4096 / (groups * waves);
  if (split < 1) split = 1;
  if (split > all) split = all;
  const int passes = (all + split - 1) / split;
  const dim3 grid(groups, (all + passes - 1) / passes);
  const bool q = a.cache.fmt == Q8_KV_Q8_0;
  auto k = D == 64 ? (q ? qkv_heads_kernel<64, 1> : qkv_heads_kernel<64, 0>)
                   : D == 128 ? (q ? qkv_heads_kernel<128, 1> : qkv_heads_kernel<128, 0>)
                              : (q ? qkv_heads_kernel<256, 1> : qkv_heads_kernel<256, 0>);
  k<<<grid, 64 * waves, 0, stream>>>(a, passes);
  return hipGetLastError();
}

hipError_t launch_kv_gather(const KvCache &c, const int32_t *slots, int rows, uint16_t *k_out,
                            uint16_t *v_out, hipStream_t stream) {
  const long long total = (long long)rows * c.heads * (c.dim / 8);
  const long long need = (total + 255) / 256;
  const unsigned blocks = (unsigned)(need < kGatherBlocks ? need : kGatherBlocks);
  auto k = c.fmt == Q8_KV_BF16 ? kv_gather_kernel<0> : kv_gather_kernel<1>;
  k<<<blocks, 256, 0, stream>>>(c, slots, rows, k_out, v_out);
  return hipGetLastError();
}

}  // namespace q8
