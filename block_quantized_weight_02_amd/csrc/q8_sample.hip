// q8_sample.hip -- a token a row from its logits, in one launch: one workgroup of
// 16 waves a row.
//
// With l the row's logits, M the largest, T the temperature, a token's weight is
// w = exp((l - M) / T), and the tokens stand in the order of falling l, lower index
// first among equal ones.  A limit keeps a prefix of that order: top_k its first k;
// top_p the tokens whose predecessors weigh less than p of all the weight; min_p
// those that weigh at least min_p.  The token is the first, by index, at which the
// kept weights' running sum exceeds u times their sum.
//
// Which token that is must not depend on the order of additions: weights are whole
// numbers, w 2^SH rounded, SH = min(51, 62 - log2 V), summed in 64 bits, so every sum
// is exact.  The weight itself is computed in fp64 (exponent in 1/64 octaves, a table
// of 2^(j/64) and four terms of the series: relative error below 1e-13), about twenty
// instructions; it is taken only where a sum needs it.
//
// Passes over the row (from memory once, then from the caches):
//   1. the largest logit with its lowest index, and the mean of the finite ones;
//   2. sum of exp(l - M) for the log-probability; with a limit on the order, counts
//      (and for top_p weights) of 2047 even steps of M - l from 0 to 3/4 of M - mean,
//      which few tokens reach, so that the histogram's LDS additions are few: the
//      rest is one last bin, kept in registers.  Without such a limit, the weights'
//      sum of each tile of 1024 tokens;
//   3. the tokens of the limit's bin become candidates, and the tiles sum what
//      stands before that bin.  Too many candidates: the bin's range of logits (as
//      ordered integers) is divided again, at most three times, down to equal logits,
//      which are counted by index.
// The candidates are ordered by comparing each with all; then the tile that holds
// the drawn weight is walked by one wave.
//
// Bound by the row's first pass at many rows; one row is bound by one CU's issue
// (about 4 us for each 32000 tokens that need weights) and the steps between barriers.
#include <hip/hip_runtime.h>
#include <stdint.h>

#include "q8_logits.h"

namespace q8 {
namespace {

constexpr int kThreads = 1024, kWaves = 16;
constexpr int kBins = 2048;
constexpr int kCand = 1024;
constexpr int kMaxTiles = kMaxVocab / kSampleTile;
constexpr int kVals = 16;                  // tokens of a tile a lane holds

typedef unsigned long long u64;

// Order of a logit as an unsigned integer (larger logit, larger key; -0 as +0).
__device__ __forceinline__ uint32_t key_of(float l) {
  const uint32_t b = __float_as_uint(l + 0.0f);
  return b ^ ((b >> 31) ? 0xffffffffu : 0x80000000u);
}
__device__ __forceinline__ float of_key(uint32_t k) {
  return __uint_as_float(k ^ ((k >> 31) ? 0x80000000u : 0xffffffffu));
}

// A row's weights.  c64: 64 log2(e) / T.
struct Weigher {
  double c64, M;
  float Mf;
  int sh;
  const double *pow;                       // 2^(j/64), in LDS
};
// 2^SH exp((l - M) / T); exactly: w of the largest is 2^SH.
__device__ __forceinline__ double weight_of(const Weigher &w, float l) {
  if (l == w.Mf) return (double)(1ull << w.sh);
  const double t = fmax(((double)l - w.M) * w.c64, -64.0 * 80.0);
  const double magic = 6755399441055744.0;                     // 1.5 * 2^52
  const double k = t + magic;
  const int ki = (int)(uint32_t)__double_as_longlong(k);
  const double r = t - (k - magic);                            // within 1/2 of a step
  // exp(r ln2 / 64): r ln2 / 64 below 0.0055, the first term left out 4e-14
  const double a = 0.010830424696249145, a2 = a * a;
  const double p = fma(r, fma(r, fma(r, fma(r, a2 * a2 / 24, a2 * a / 6), a2 / 2), a), 1.0);
  const double x = ldexp(w.pow[ki & 63] * p, (ki >> 6) + w.sh);
  return l == -INFINITY || !(w.Mf < INFINITY) ? 0.0 : x;
}
__device__ __forceinline__ u64 whole(double x) {               // x <= 2^51, rounded
  return (u64)__double_as_longlong(x + 4503599627370496.0) & 0xfffffffffffffull;
}

__device__ __forceinline__ void load_tile(const float *__restrict__ x, int V, int tile, int lane,
                                          float (&v)[kVals]) {
  const int base = tile * kSampleTile + lane * 4;
#pragma unroll
  for (int j = 0; j < 4; ++j) {
    float4 q = make_float4(-INFINITY, -INFINITY, -INFINITY, -INFINITY);
    const int i = base + j * 256;
    if (i < V) q = *reinterpret_cast<const float4 *>(x + i);   // (the row's stride is whole fours)
    v[4 * j] = q.x;
    v[4 * j + 1] = q.y;
    v[4 * j + 2] = q.z;
    v[4 * j + 3] = q.w;
  }
  if ((tile + 1) * kSampleTile > V) {
#pragma unroll
    for (int j = 0; j < kVals; ++j)
      if (base + (j >> 2) * 256 + (j & 3) >= V) v[j] = -INFINITY;
  }
#pragma unroll
  for (int j = 0; j < kVals; ++j) v[j] = v[j] == v[j] ? v[j] : -INFINITY;   // NaN: no weight
}
__device__ __forceinline__ int index_of(int tile, int lane, int j) {
  return tile * kSampleTile + (j >> 2) * 256 + lane * 4 + (j & 3);
}

__device__ __forceinline__ u64 wave_sum(u64 v) {
#pragma unroll
  for (int o = 32; o > 0; o >>= 1) v += __shfl_xor(v, o);
  return v;
}
__device__ __forceinline__ u64 wave_scan(u64 v, int lane) {    // inclusive
#pragma unroll
  for (int o = 1; o < 64; o <<= 1) {
    const u64 w = __shfl_up(v, o);
    if (lane >= o) v += w;
  }
  return v;
}

struct Lds {
  double pow[64];
  u64 mass[kBins];
  uint32_t count[kBins];
  u64 tile[kMaxTiles];                     // kept weight of a tile
  float cand_l[kCand];
  int cand_i[kCand];
  u64 cand_w[kCand];
  // reductions
  float wmax[kWaves];
  int wi[kWaves];
  double wsum[kWaves];
  uint32_t wn[kWaves];
  u64 wmass[kWaves];
  // the state of the search
  int n_cand;
  int bin;
  u64 before_n, before_w;
  uint32_t bin_n;
  uint32_t kmin, kmax;
  uint32_t cut_key;
  int cut_index;
  int token;
  int pick_tile;
  u64 pick_rest;
};

// Finds, over the histogram, the bin in which the order's cut falls: the first whose
// running count reaches `want_n` or running weight reaches `want_w` (in doubles:
// compared as p * W is).  before_n, before_w: what stands before the histogram's
// range, and on return before the bin.  Leaves s.bin = kBins where none does.
__device__ void find_bin(Lds &s, u64 want_n, double want_w) {
  const int tid = threadIdx.x, lane = tid & 63, wave = tid >> 6;
  // two bins a thread
  const u64 n0 = s.count[2 * tid], n1 = s.count[2 * tid + 1];
  const u64 w0 = s.mass[2 * tid], w1 = s.mass[2 * tid + 1];
  u64 n = wave_scan(n0 + n1, lane), w = wave_scan(w0 + w1, lane);
  if (lane == 63) {
    s.wn[wave] = (uint32_t)n;
    s.wmass[wave] = w;
  }
  if (tid == 0) s.bin = kBins;
  __syncthreads();
  for (int i = 0; i < wave; ++i) {
    n += s.wn[i];
    w += s.wmass[i];
  }
  const u64 bn = s.before_n, bw = s.before_w;
  n += bn;
  w += bw;
  __syncthreads();
  const u64 na = n - n1, wa = w - w1;      // through the thread's first bin
  const u64 np = na - n0, wp = wa - w0;    // before it
  const auto reached = [&](u64 c, u64 m) { return c >= want_n || (double)m >= want_w; };
  // reached is monotone; exactly one bin has it and not the one before (an empty
  // bin never changes it)
  const bool before = tid == 0 ? false : reached(np, wp);
  if (!before && reached(na, wa)) {
    s.bin = 2 * tid;
    s.bin_n = (uint32_t)n0;
    s.before_n = np;
    s.before_w = wp;
  } else if (!before && reached(n, w)) {
    s.bin = 2 * tid + 1;
    s.bin_n = (uint32_t)n1;
    s.before_n = na;
    s.before_w = wa;
  }
  __syncthreads();
}

__device__ void clear_bins(Lds &s) {
  for (int i = threadIdx.x; i < kBins; i += kThreads) {
    s.mass[i] = 0;
    s.count[i] = 0;
  }
}

__global__ void __launch_bounds__(kThreads) sample_kernel(const SampleArgs a) {
  __shared__ Lds s;
  const int row = blockIdx.x, tid = threadIdx.x, lane = tid & 63;
  const int wave = __builtin_amdgcn_readfirstlane(tid >> 6);
  const float *__restrict__ x = a.logits + (size_t)row * a.ld;
  const int V = a.V, tiles = (V + kSampleTile - 1) / kSampleTile;

  // ---- pass 1
  float top = -INFINITY;
  int at = 0x7fffffff;
  float sum = 0.0f;
  uint32_t finite = 0;
  for (int t = wave; t < tiles; t += kWaves) {
    float v[kVals];
    load_tile(x, V, t, lane, v);
#pragma unroll
    for (int j = 0; j < kVals; ++j) {
      if (v[j] > top) {
        top = v[j];
        at = index_of(t, lane, j);
      }
      if (fabsf(v[j]) < INFINITY) {
        sum += v[j];
        ++finite;
      }
    }
  }
  double dsum = sum;
#pragma unroll
  for (int o = 32; o > 0; o >>= 1) {
    const float t2 = __shfl_xor(top, o);
    const int a2 = __shfl_xor(at, o);
    if (t2 > top || (t2 == top && a2 < at)) {
      top = t2;
      at = a2;
    }
    dsum += __shfl_xor(dsum, o);
    finite += __shfl_xor(finite, o);
  }
  if (lane == 0) {
    s.wmax[wave] = top;
    s.wi[wave] = at;
    s.wsum[wave] = dsum;
    s.wn[wave] = finite;
  }
  if (tid < 64) s.pow[tid] = exp2((double)tid / 64.0);
  __syncthreads();
  dsum = 0.0;
  finite = 0;
  top = -INFINITY;
  at = 0x7fffffff;
  for (int i = 0; i < kWaves; ++i) {
    if (s.wmax[i] > top || (s.wmax[i] == top && s.wi[i] < at)) {
      top = s.wmax[i];
      at = s.wi[i];
    }
    dsum += s.wsum[i];
    finite += s.wn[i];
  }
  const float M = top;
  if (M == -INFINITY) {                    // nothing may follow
    if (tid == 0) {
      a.token[row] = -1;
      if (a.logprob) a.logprob[row] = -INFINITY;
    }
    return;
  }

  // ---- the row's limits
  const float T = a.temperature ? a.temperature[row] : 1.0f;
  const bool greedy = !(T > 0.0f);
  const int k_in = a.top_k ? a.top_k[row] : 0;
  const float p_in = a.top_p ? a.top_p[row] : 1.0f;
  const float mp_in = a.min_p ? a.min_p[row] : 0.0f;
  const bool by_k = !greedy && k_in > 0 && k_in < V;
  const bool by_p = !greedy && p_in < 1.0f;
  const double min_p = mp_in > 0.0f ? fmin((double)mp_in, 1.0) : 0.0;
  Weigher w;
  w.c64 = 92.332482616893656878 / (double)(greedy ? 1.0f : T);   // 64 log2(e)
  w.M = M;
  w.Mf = M;
  w.sh = min(51, 62 - (32 - __clz(V)));
  w.pow = s.pow;
  const double min_w = min_p * (double)(1ull << w.sh);
  // below this a token weighs less than min_p without computing it (a margin over
  // the roundings of the bound itself)
  const float min_l = min_p > 0.0 ? (float)((double)M + (double)T * (log(min_p) - 1e-3) -
                                            1e-6 * fabs((double)M)) : -INFINITY;
  const auto kept_weight = [&](float l) -> u64 {     // 0 where min_p leaves the token out
    if (l < min_l) return 0;
    const double d = weight_of(w, l);
    return d < min_w ? 0 : whole(d);
  };
  // 2047 steps over 3/4 of what the largest logit stands above the mean
  const float mean = finite ? (float)(dsum / (double)finite) : 0.0f;
  float step = 2047.0f / (0.75f * (M - mean));
  if (!(step > 0.0f) || !(step < INFINITY) || !(M < INFINITY)) step = 1.0f;
  const auto bin_of = [&](float l) -> int {
    return l == M ? 0 : (int)fminf((M - l) * step, 2047.0f);   // falling l, rising bin
  };

  // ---- pass 2
  const bool cut = by_k || by_p;
  if (cut) clear_bins(s);
  if (tid == 0) {
    s.n_cand = 0;
    s.before_n = 0;
    s.before_w = 0;
    s.cut_key = 0;                         // everything
    s.cut_index = 0x7fffffff;
    s.token = -1;
  }
  __syncthreads();
  float lse = 0.0f;
  u64 rest_w = 0;
  uint32_t rest_n = 0;
  if (a.logprob || !greedy) {
    for (int t = wave; t < tiles; t += kWaves) {
      float v[kVals];
      load_tile(x, V, t, lane, v);
      if (a.logprob) {
#pragma unroll
        for (int j = 0; j < kVals; ++j) lse += v[j] == M ? 1.0f : expf(v[j] - M);
      }
      if (cut) {
        for (int j = 0; j < kVals; ++j) {
          if (v[j] == -INFINITY) continue;
          const u64 wt = by_p ? whole(weight_of(w, v[j])) : 0;
          const int b = bin_of(v[j]);
          if (b == kBins - 1) {
            rest_w += wt;
            ++rest_n;
          } else {
            atomicAdd(&s.count[b], 1u);
            if (by_p) atomicAdd(&s.mass[b], wt);
          }
        }
      } else if (!greedy) {
        u64 wt = 0;
        for (int j = 0; j < kVals; ++j) wt += kept_weight(v[j]);
        wt = wave_sum(wt);
        if (lane == 0) s.tile[t] = wt;
      }
    }
  }
  double dl = lse;
#pragma unroll
  for (int o = 32; o > 0; o >>= 1) dl += __shfl_xor(dl, o);
  __syncthreads();                         // (wsum's readers are done)
  if (lane == 0) s.wsum[wave] = dl;
  if (cut) {
    rest_w = wave_sum(rest_w);
    rest_n = (uint32_t)wave_sum(rest_n);
    if (lane == 0 && rest_n) {
      atomicAdd(&s.count[kBins - 1], rest_n);
      atomicAdd(&s.mass[kBins - 1], rest_w);
    }
  }
  __syncthreads();
  dl = 0.0;
  for (int i = 0; i < kWaves; ++i) dl += s.wsum[i];

  if (!greedy && cut) {
    // ---- where the order is cut
    u64 W = 0;
    if (by_p) {
      u64 part = s.mass[2 * tid] + s.mass[2 * tid + 1];
      part = wave_sum(part);
      if (lane == 0) s.wmass[wave] = part;
      __syncthreads();
      for (int i = 0; i < kWaves; ++i) W += s.wmass[i];
      __syncthreads();
    }
    const u64 want_n = by_k ? (u64)k_in : ~0ull;
    const double want_w = by_p ? (double)p_in * (double)W : INFINITY;
    find_bin(s, want_n, want_w);
    int bin = s.bin;
    // the range of the cut: the tokens of a bin, later of an interval of keys
    uint32_t klo = 0, khi = 0;
    bool keyed = false, equal = false;
    while (bin < kBins && s.bin_n > kCand) {
      if (!keyed) {
        // the bin's smallest and largest key
        if (tid == 0) {
          s.kmin = 0xffffffffu;
          s.kmax = 0;
        }
        __syncthreads();
        uint32_t lo = 0xffffffffu, hi = 0;
        for (int t = wave; t < tiles; t += kWaves) {
          float v[kVals];
          load_tile(x, V, t, lane, v);
          for (int j = 0; j < kVals; ++j)
            if (v[j] != -INFINITY && bin_of(v[j]) == bin) {
              const uint32_t k = key_of(v[j]);
              lo = min(lo, k);
              hi = max(hi, k);
            }
        }
#pragma unroll
        for (int o = 32; o > 0; o >>= 1) {
          lo = min(lo, (uint32_t)__shfl_xor((int)lo, o));
          hi = max(hi, (uint32_t)__shfl_xor((int)hi, o));
        }
        if (lane == 0) {
          atomicMin(&s.kmin, lo);
          atomicMax(&s.kmax, hi);
        }
        __syncthreads();
        klo = s.kmin;
        khi = s.kmax;
        keyed = true;
      }
      if (klo == khi) {
        equal = true;
        break;
      }
      int shift = 0;
      while ((khi - klo) >> shift >= (uint32_t)kBins) ++shift;
      clear_bins(s);
      __syncthreads();
      for (int t = wave; t < tiles; t += kWaves) {
        float v[kVals];
        load_tile(x, V, t, lane, v);
        for (int j = 0; j < kVals; ++j) {
          const uint32_t k = key_of(v[j]);
          if (k < klo || k > khi || v[j] == -INFINITY) continue;
          const uint32_t b = (khi - k) >> shift;
          atomicAdd(&s.count[b], 1u);
          if (by_p) atomicAdd(&s.mass[b], whole(weight_of(w, v[j])));
        }
      }
      __syncthreads();
      find_bin(s, want_n, want_w);
      bin = s.bin;
      if (bin >= kBins) break;             // (the range held the cut: it does not happen)
      khi = khi - ((uint32_t)bin << shift);
      const uint32_t span = (1u << shift) - 1u;
      klo = khi - klo > span ? khi - span : klo;
    }
    const bool cuts = bin < kBins;

    // ---- pass 3: what stands before the range, by tile; its tokens, or how many
    const uint32_t kequal = khi;
    __syncthreads();
    for (int t = wave; t < tiles; t += kWaves) {
      float v[kVals];
      load_tile(x, V, t, lane, v);
      u64 wt = 0;
      uint32_t same = 0;
      for (int j = 0; j < kVals; ++j) {
        if (v[j] == -INFINITY) continue;
        bool first, in;
        if (!cuts) {
          first = true;
          in = false;
        } else if (keyed) {
          const uint32_t k = key_of(v[j]);
          first = k > khi;
          in = k <= khi && k >= klo;
        } else {
          const int b = bin_of(v[j]);
          first = b < bin;
          in = b == bin;
        }
        if (first) wt += kept_weight(v[j]);
        if (in) {
          if (equal) {
            ++same;
          } else {
            const int c = atomicAdd(&s.n_cand, 1);
            if (c < kCand) {
              s.cand_l[c] = v[j];
              s.cand_i[c] = index_of(t, lane, j);
              s.cand_w[c] = whole(weight_of(w, v[j]));
            }
          }
        }
      }
      wt = wave_sum(wt);
      if (equal) same = (uint32_t)wave_sum(same);
      if (lane == 0) {
        s.tile[t] = wt;
        // (equal logits: the histogram's room holds the tiles' counts)
        if (equal) s.count[t] = same;
      }
    }
    __syncthreads();
    if (cuts && !equal) {
      const int n = min(s.n_cand, kCand);
      for (int c = tid; c < n; c += kThreads) {
        const float l = s.cand_l[c];
        const int i = s.cand_i[c];
        u64 rank = s.before_n, mass = s.before_w;
        for (int d = 0; d < n; ++d) {
          const float ld = s.cand_l[d];
          if (ld > l || (ld == l && s.cand_i[d] < i)) {
            ++rank;
            mass += s.cand_w[d];
          }
        }
        const bool keep = rank < want_n && (rank == 0 || (double)mass < want_w);
        const bool next = rank + 1 < want_n && (double)(mass + s.cand_w[c]) < want_w;
        if (keep) {
          const u64 kw = kept_weight(l);
          if (kw) atomicAdd(&s.tile[i / kSampleTile], kw);
          // the last one kept: its successor, if it has one here, is not
          bool last = !next;
          if (next) {
            last = true;
            for (int d = 0; d < n; ++d)
              if (s.cand_l[d] < l || (s.cand_l[d] == l && s.cand_i[d] > i)) {
                last = false;
                break;
              }
          }
          if (last) {
            s.cut_key = key_of(l);
            s.cut_index = i;
          }
        }
      }
    } else if (cuts && equal) {
      // of equal logits the first `take` by index
      if (tid == 0) {
        const u64 each = whole(weight_of(w, of_key(kequal)));
        u64 take = 0;
        if (by_k) take = want_n - s.before_n;
        if (by_p) {
          // tokens j = 0, 1, .. with before_w + j * each < want_w
          const double room = want_w - (double)s.before_w;
          u64 tp = each ? (u64)fmax(ceil(room / (double)each), 0.0) : ~0ull;
          while (tp > 0 && !((double)(s.before_w + (tp - 1) * each) < want_w)) --tp;
          while (each && tp < (u64)V && (double)(s.before_w + tp * each) < want_w) ++tp;
          take = by_k ? (take < tp ? take : tp) : tp;
        }
        if (take == 0 && s.before_n == 0) take = 1;
        const u64 kw = kept_weight(of_key(kequal));
        u64 left = take;
        int edge = -1;
        for (int t = 0; t < tiles && left; ++t) {
          const u64 c = s.count[t] < left ? s.count[t] : left;
          s.tile[t] += kw * c;
          left -= c;
          if (left == 0) edge = t;
        }
        s.cut_key = kequal;
        s.pick_tile = edge;
        s.pick_rest = take;
        // (how many of tile `edge` are kept)
        u64 earlier = 0;
        for (int t = 0; t < edge; ++t) earlier += s.count[t];
        s.before_n = edge < 0 ? 0 : take - earlier;
      }
      __syncthreads();
      const int edge = s.pick_tile;
      const u64 keep = s.before_n;
      if (wave == 0 && edge >= 0) {
        float v[kVals];
        load_tile(x, V, edge, lane, v);
        u64 seen = 0;
        for (int j = 0; j < 4; ++j) {
          u64 mine = 0;
          for (int c = 0; c < 4; ++c) mine += v[4 * j + c] != -INFINITY && key_of(v[4 * j + c]) == kequal;
          u64 n = wave_scan(mine, lane) - mine + seen;
          for (int c = 0; c < 4; ++c)
            if (v[4 * j + c] != -INFINITY && key_of(v[4 * j + c]) == kequal && ++n == keep)
              s.cut_index = index_of(edge, lane, 4 * j + c);
          seen += wave_sum(mine);
        }
      }
    }
    __syncthreads();
  }

  // ---- the draw
  if (!greedy) {
    if (wave == 0) {
      u64 total = 0;
      for (int t = lane; t < tiles; t += 64) total += s.tile[t];
      total = wave_sum(total);
      const double u = a.u[row];
      const double f = floor((u > 0.0 ? u : 0.0) * (double)total);
      u64 target = f < (double)total ? (u64)f : total;
      if (target >= total) target = total - 1;
      // the first tile whose running sum exceeds it
      u64 run = 0;
      int pick = -1;
      for (int t0 = 0; t0 < tiles && pick < 0; t0 += 64) {
        const u64 mine = t0 + lane < tiles ? s.tile[t0 + lane] : 0;
        const u64 upto = wave_scan(mine, lane) + run;
        const u64 over = __ballot(upto > target);
        if (over) {
          const int f0 = __ffsll(over) - 1;
          pick = t0 + f0;
          run = __shfl(upto - mine, f0);
        } else {
          run = __shfl(upto, 63);
        }
      }
      if (pick >= 0) {
        float v[kVals];
        load_tile(x, V, pick, lane, v);
        const uint32_t ck = s.cut_key;
        const int ci = s.cut_index;
        int token = -1;
        for (int j = 0; j < 4 && token < 0; ++j) {
          u64 wt[4], mine = 0;
          for (int c = 0; c < 4; ++c) {
            const float l = v[4 * j + c];
            const uint32_t k = key_of(l);
            const bool in = l != -INFINITY && (k > ck || (k == ck && index_of(pick, lane, 4 * j + c) <= ci));
            wt[c] = in ? kept_weight(l) : 0;
            mine += wt[c];
          }
          const u64 upto = wave_scan(mine, lane) + run;
          const u64 over = __ballot(upto > target);
          if (over) {
            const int f0 = __ffsll(over) - 1;
            u64 r = upto - mine;
            int mine_at = -1;
            for (int c = 0; c < 4 && mine_at < 0; ++c) {
              r += wt[c];
              if (r > target) mine_at = index_of(pick, lane, 4 * j + c);
            }
            token = __shfl(mine_at, f0);
          } else {
            run = __shfl(upto, 63);
          }
        }
        if (lane == 0) s.token = token;
      }
    }
    __syncthreads();
  }
  if (tid == 0) {
    const int token = greedy ? at : s.token;
    a.token[row] = token;
    if (a.logprob) {
      const float l = token >= 0 ? x[token] : M;
      a.logprob[row] = (float)((l == M ? 0.0 : (double)l - (double)M) - log(dl));
    }
  }
}

}  // namespace

hipError_t launch_sample(const SampleArgs &a, hipStream_t stream) {
  (void)hipGetLastError();
  sample_kernel<<<dim3((unsigned)a.m), dim3(kThreads), 0, stream>>>(a);
  return hipGetLastError();
}

}  // namespace q8
