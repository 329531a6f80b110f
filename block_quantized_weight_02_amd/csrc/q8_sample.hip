// q8_sample.hip -- a token a row from its logits.
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
// Five passes:
//   stats    of a slice: its largest logit with the lowest index, sum of exp(l - that),
//            the mean of what is not far below it, and each tile's largest;
//   weights  rows with a limit on the order: counts (for top_p weights too) of 2047 even
//            steps of M - l, in LDS, a slice's histogram written out whole; rows without
//            one: the weights' sum of each tile of 1024 tokens;
//   cut      the slices' histograms summed, and the step in which the order is cut;
//   collect  the tokens of that step as candidates, and the tiles' sums of what stands
//            before it;
//   draw     the candidates ordered by comparing each with all, and the tile that holds
//            the drawn weight walked by one wave.  Where more than 1024 tokens fall into
//            one step, the step's range of logits (as ordered integers) is divided again
//            here, down to equal logits, which are counted by index.
// The steps reach from M to 3/4 of the way to the mean where only top_k cuts (the cut is
// near the top, and few tokens then add to LDS), and as far below the mean as M stands
// above it where top_p does; what lies beyond is one last step, summed in registers.  (A
// cut in that step is divided again by one workgroup: 1 x 131072, top_k 200, 85 us against
// 28 where the largest logit stands 60 above a bulk of deviation 2.5.)
//
// They are five launches with the rows' vocabularies in slices, so that few long rows too
// are worked on by many CUs, or one launch with a workgroup a row, where a row is short
// enough for its registers (sample_in_one_launch has both sides' figures).  Mixed kinds of rows:
// 1 x 32000 17 us, 40 x 50001 36, 256 x 131072 102.  The first pass of those 256 rows, 25
// us, is bound by their 134 MB, with the vector unit busy two thirds of the time; the
// second, 39, by fp64, by additions in LDS and by the rows' unlike work; the collecting one,
// 24, by fp64 and the same; the two with a workgroup a row (6 and 13) by latency, as all of
// them with few rows.  A single row in one launch is bound by its CU's vector unit, busy four
// fifths of the time (top_p 0.9 27 us, top_k 50 19, neither 13).
#include <hip/hip_runtime.h>
#include <stdint.h>

#include "q8_logits.h"

namespace q8 {
namespace {

constexpr int kThreads = 1024, kWaves = 16;   // of a workgroup a row
constexpr int kBins = kSampleBins;
constexpr int kCand = kSampleCand;
constexpr int kMaxTiles = kMaxVocab / kSampleTile;
static_assert(kMaxTiles <= kThreads && kCand <= kThreads && kSampleTile == kThreads,
              "a thread takes a tile's sum, a candidate and a token of the drawn tile");
constexpr int kVals = 16;                  // tokens of a tile a lane holds
static_assert(kSampleHeld == 4 * kWaves * kSampleTile, "the row kernels hold four tiles a wave at most");
constexpr int kStatTiles = kSampleSlice / kSampleTile;   // one a wave

typedef unsigned long long u64;

// Order of a logit as an unsigned integer (larger logit, larger key; -0 as +0).
__device__ __forceinline__ uint32_t key_of(float l) {
  const uint32_t b = __float_as_uint(l + 0.0f);
  return b ^ ((b >> 31) ? 0xffffffffu : 0x80000000u);
}
__device__ __forceinline__ float of_key(uint32_t k) {
  return __uint_as_float(k ^ ((k >> 31) ? 0x80000000u : 0xffffffffu));
}

// 2^(j/64).
__constant__ double kPow[64] = {
    1.0, 1.0108892860517005, 1.0218971486541166, 1.0330248790212284,
    1.0442737824274138, 1.0556451783605572, 1.0671404006768237, 1.0787607977571199,
    1.0905077326652577, 1.1023825833078409, 1.1143867425958924, 1.1265216186082418,
    1.1387886347566916, 1.1511892299529827, 1.1637248587775775, 1.1763969916502812,
    1.189207115002721, 1.2021567314527031, 1.215247359980469, 1.22848053610687,
    1.241857812073484, 1.2553807570246911, 1.2690509571917332, 1.2828700160787783,
    1.2968395546510096, 1.3109612115247644, 1.3252366431597413, 1.3396675240533029,
    1.3542555469368927, 1.3690024229745905, 1.383909881963832, 1.3989796725383112,
    1.4142135623730951, 1.42961333839197, 1.4451808069770467, 1.460917794180647,
    1.4768261459394993, 1.4929077282912648, 1.5091644275934228, 1.5255981507445384,
    1.5422108254079407, 1.5590044002378369, 1.5759808451078865, 1.593142151342267,
    1.6104903319492543, 1.6280274218573478, 1.6457554781539649, 1.6636765803267364,
    1.681792830507429, 1.7001063537185235, 1.7186192981224779, 1.7373338352737062,
    1.7562521603732995, 1.7753764925265212, 1.7947090750031072, 1.8142521755003989,
    1.8340080864093424, 1.8539791250833855, 1.8741676341103, 1.8945759815869656,
    1.9152065613971474, 1.9360617934922943, 1.9571441241754002, 1.9784560263879509};

// A row's weights: 2^SH exp((l - M) / T), exactly 2^SH for the largest.  c64: 64 log2(e)
// / T; sh64: 64 SH, added to the exponent at once.
struct Weigher {
  double c64, M, sh64;
  int sh;
  const double *pow;                       // kPow, in LDS
};
struct Scaled {                            // a weight is power * p
  double power, p;
};
__device__ __forceinline__ Scaled scaled_weight(const Weigher &w, float l) {
  const double t = fmax(fma((double)l - w.M, w.c64, w.sh64), -1024.0);   // (-infinity: 2^-16)
  const double magic = 6755399441055744.0;                     // 1.5 * 2^52
  const double k = t + magic;
  const int ki = (int)(uint32_t)__double_as_longlong(k);
  const double r = t - (k - magic);                            // within 1/2 of a step
  // exp(r ln2 / 64): r ln2 / 64 below 0.0055, the first term left out 4e-14
  const double a = 0.010830424696249145, a2 = a * a;
  const double p = fma(r, fma(r, fma(r, fma(r, a2 * a2 / 24, a2 * a / 6), a2 / 2), a), 1.0);
  return Scaled{ldexp(w.pow[ki & 63], ki >> 6), p};
}
// As a whole number (it is at most 2^51): the sum with 2^52, whose own bits stand above.
__device__ __forceinline__ u64 weight_over(const Scaled &w) {
  return (u64)__double_as_longlong(fma(w.power, w.p, 4503599627370496.0));
}
constexpr u64 kOver = 0x433ull << 52;      // the bits of 2^52
__device__ __forceinline__ u64 weight_of(const Weigher &w, float l) {
  return weight_over(scaled_weight(w, l)) - kOver;
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
// A row whose largest logit is infinite: among 0 (those) and -infinity.
__device__ __forceinline__ void among_infinite(bool infinite, float (&v)[kVals]) {
  if (infinite) {
#pragma unroll
    for (int j = 0; j < kVals; ++j) v[j] = v[j] == INFINITY ? 0.0f : -INFINITY;
  }
}
__device__ __forceinline__ void load_tile(const float *__restrict__ x, int V, int tile, int lane, bool infinite,
                                          float (&v)[kVals]) {
  load_tile(x, V, tile, lane, v);
  among_infinite(infinite, v);
}
__device__ __forceinline__ int index_of(int tile, int lane, int j) {
  return tile * kSampleTile + (j >> 2) * 256 + lane * 4 + (j & 3);
}

// Reductions over the wave by lane moves within the vector unit (a step of a shuffle
// through LDS takes ten times as long, and few rows are bound by latency): rows of 16
// lanes first, then each row's last lane into the rows behind it.
template <int CTRL, int ROWS>
__device__ __forceinline__ u64 moved(u64 v) {                  // 0 where nothing comes
  const int lo = __builtin_amdgcn_update_dpp(0, (int)(uint32_t)v, CTRL, ROWS, 0xf, false);
  const int hi = __builtin_amdgcn_update_dpp(0, (int)(uint32_t)(v >> 32), CTRL, ROWS, 0xf, false);
  return (u64)(uint32_t)hi << 32 | (uint32_t)lo;
}
template <int CTRL, int ROWS>
__device__ __forceinline__ uint32_t moved(uint32_t v) {
  return (uint32_t)__builtin_amdgcn_update_dpp(0, (int)v, CTRL, ROWS, 0xf, false);
}
template <int CTRL, int ROWS>
__device__ __forceinline__ double moved(double v) {
  return __longlong_as_double((long long)moved<CTRL, ROWS>((u64)__double_as_longlong(v)));
}
template <typename T, typename F>
__device__ __forceinline__ T row_scan(T v, F f) {              // of 16 lanes, inclusive
  v = f(v, moved<0x111, 0xf>(v));
  v = f(v, moved<0x112, 0xf>(v));
  v = f(v, moved<0x114, 0xf>(v));
  return f(v, moved<0x118, 0xf>(v));
}
template <typename T, typename F>
__device__ __forceinline__ T wave_scan(T v, F f) {             // inclusive
  v = row_scan(v, f);
  v = f(v, moved<0x142, 0xa>(v));
  return f(v, moved<0x143, 0xc>(v));
}
__device__ __forceinline__ uint32_t of_lane(uint32_t v, int lane) {
  return (uint32_t)__builtin_amdgcn_readlane((int)v, lane);
}
__device__ __forceinline__ u64 of_lane(u64 v, int lane) {
  return (u64)of_lane((uint32_t)(v >> 32), lane) << 32 | of_lane((uint32_t)v, lane);
}
__device__ __forceinline__ double of_lane(double v, int lane) {
  return __longlong_as_double((long long)of_lane((u64)__double_as_longlong(v), lane));
}
struct Add {
  template <typename T>
  __device__ __forceinline__ T operator()(T a, T b) const { return a + b; }
};
template <typename T>
__device__ __forceinline__ T wave_scan(T v) { return wave_scan(v, Add{}); }
template <typename T>
__device__ __forceinline__ T wave_sum(T v) { return of_lane(wave_scan(v, Add{}), 63); }

// A logit and its index as one number: larger logit first, then the lower index.
__device__ __forceinline__ u64 packed(float l, int i) { return (u64)key_of(l) << 32 | (uint32_t)~i; }
__device__ __forceinline__ u64 wave_largest(u64 v) {
  return of_lane(wave_scan(v, [](u64 a, u64 b) { return a > b ? a : b; }), 63);
}

// What the launches hand on about a row.
constexpr float kFar = 60.0f;              // in units of T, below the largest: no weight
struct Params {                            // the row's limits
  float T;
  float far;                               // logits this far below the largest are no part of the mean
  int k;
  float p;
  double min_p;
  bool greedy, by_k, by_p;
};
__device__ __forceinline__ Params params_of(const SampleArgs &a, int row) {
  Params r;
  r.T = a.temperature ? a.temperature[row] : 1.0f;
  r.greedy = !(r.T > 0.0f);
  r.k = a.top_k ? a.top_k[row] : 0;
  r.p = a.top_p ? a.top_p[row] : 1.0f;
  const float mp = a.min_p ? a.min_p[row] : 0.0f;
  r.min_p = mp > 0.0f ? fmin((double)mp, 1.0) : 0.0;
  r.by_k = !r.greedy && r.k > 0 && r.k < a.V;
  r.by_p = !r.greedy && r.p < 1.0f;
  // (top_k's order does not depend on T: at a low one the mean of what can weigh anything
  // lies beside the largest, and the cut behind all the steps that reach to it)
  r.far = kFar * (r.by_p ? r.T : fmaxf(r.T, 1.0f));
  return r;
}

struct Total {                             // the slices' statistics together
  float M;                                 // 0 where the largest is infinite (among_infinite)
  int at;
  float mean;
  bool infinite, none;
};
// By each wave for itself, from the row's slices.
__device__ __forceinline__ Total total_of(const SampleArgs &a, const Params &r, int row, int lane) {
  const SliceStat *st = a.stats + (size_t)row * a.slices;
  u64 best = 0;
  SliceStat mine{};
  for (int i = lane; i < a.slices; i += 64) {
    mine = st[i];
    const u64 v = packed(mine.top, mine.at);
    best = v > best ? v : best;
  }
  best = wave_largest(best);
  const float top = of_key((uint32_t)(best >> 32));
  // (slices of masks of the type's lowest value are no part of the mean)
  const float least = top - r.far;
  double sum = 0.0;
  uint32_t n = 0;
  for (int i = lane; i < a.slices; i += 64) {
    if (a.slices > 64) mine = st[i];
    if (mine.top >= least) {
      sum += mine.sum;
      n += mine.n;
    }
  }
  sum = wave_sum(sum);
  n = wave_sum(n);
  Total t;
  t.infinite = top == INFINITY;
  t.none = top == -INFINITY;
  t.M = t.infinite ? 0.0f : top;
  t.at = (int)~(uint32_t)best;
  t.mean = n && !t.infinite ? (float)(sum / (double)n) : -1.0f;
  return t;
}
// sum exp(l - the largest), by a wave.
__device__ __forceinline__ double exp_sum_of(const SampleArgs &a, int row, int lane) {
  const SliceStat *st = a.stats + (size_t)row * a.slices;
  u64 best = 0;
  for (int i = lane; i < a.slices; i += 64) {
    const u64 v = packed(st[i].top, 0);
    best = v > best ? v : best;
  }
  const float top = of_key((uint32_t)(wave_largest(best) >> 32));
  double e = 0.0;
  for (int i = lane; i < a.slices; i += 64) {
    const SliceStat v = st[i];
    if (v.top > -INFINITY)
      e += v.top == top ? v.exp_sum : v.exp_sum * exp((double)v.top - (double)top);
  }
  return wave_sum(e);
}

// A tile's largest logit, as load_tile gives it.
__device__ __forceinline__ float top_of(const SampleArgs &a, const Total &t, int row, int tile) {
  const float l = a.tops[(size_t)row * a.row_tiles + tile];
  return t.infinite ? (l == INFINITY ? 0.0f : -INFINITY) : l;
}

__device__ __forceinline__ Weigher weigher_of(const SampleArgs &a, const Params &r, float M, const double *pow) {
  Weigher w;
  w.c64 = 92.332482616893656878 / (double)(r.greedy ? 1.0f : r.T);   // 64 log2(e)
  w.M = M;
  w.sh = min(51, 62 - (32 - __clz(a.V)));
  w.sh64 = 64.0 * w.sh;
  w.pow = pow;
  return w;
}
// A token's weight where min_p keeps it, else 0.
struct Keep {
  Weigher w;
  float min_l;                             // below it: out without computing the weight
  double min_w;
  __device__ __forceinline__ Keep(const Weigher &wg, const Params &r) : w(wg) {
    min_w = r.min_p * (double)(1ull << w.sh);
    // (a margin over the roundings of the bound itself)
    min_l = r.min_p > 0.0 ? (float)(w.M + (double)r.T * (log(r.min_p) - 1e-3) - 1e-6 * fabs(w.M)) : -INFINITY;
  }
  __device__ __forceinline__ u64 operator()(float l) const {    // (no min_p: min_w is 0)
    const Scaled d = scaled_weight(w, l);
    return d.power * d.p < min_w ? 0 : weight_over(d) - kOver;
  }
};
// (four at a time: more of their chains at once take registers that no kernel here has)
__device__ __forceinline__ u64 weight_of_tile(const Keep &keep, const float (&v)[kVals]) {
  u64 wt = 0;
  if (keep.min_w > 0.0) {
    bool any = false;
#pragma unroll
    for (int j = 0; j < kVals; ++j) any |= v[j] >= keep.min_l;
    if (!__any(any)) return 0;
#pragma unroll
    for (int j = 0; j < kVals; j += 4) {
      wt += keep(v[j]) + keep(v[j + 1]) + keep(v[j + 2]) + keep(v[j + 3]);
      __builtin_amdgcn_sched_barrier(0);
    }
  } else {
#pragma unroll
    for (int j = 0; j < kVals; j += 4) {
#pragma unroll
      for (int c = 0; c < 4; ++c) wt += weight_over(scaled_weight(keep.w, v[j + c]));
      __builtin_amdgcn_sched_barrier(0);
    }
    wt -= kVals * kOver;                   // (modulo 2^64)
  }
  return wave_sum(wt);
}

// Even steps of M - l: falling l, rising step; the last takes all the rest.
struct Steps {
  float M, per;
  __device__ __forceinline__ Steps(const Total &t, bool by_p) {
    M = t.M;
    per = (float)(kBins - 1) / ((by_p ? 2.0f : 0.75f) * (M - t.mean));
    if (!(per > 0.0f) || !(per < INFINITY)) per = 1.0f;
  }
  __device__ __forceinline__ int operator()(float l) const {
    return (int)fminf((M - l) * per, (float)(kBins - 1));
  }
};

struct Lds {
  double pow[64];
  u64 mass[kBins];
  uint32_t count[kBins];
  u64 tile[kMaxTiles];                     // kept weight of a tile
  u64 cand[kCand], order[kCand];           // packed: key, then the lower index first
  int rank[kCand];
  double log_sum;                          // of exp(l - M)
  int kept;
  uint32_t wn[kWaves];
  u64 wmass[kWaves];
  double wexp[kWaves], wsum[kWaves];
  // the state of the search
  int n_cand;
  int bin;
  u64 before_n, before_w;
  uint32_t bin_n;
  uint32_t kmin, kmax;
  uint32_t cut_key;
  int cut_index;
  int pick_tile;
};

// The n candidates of s.cand in falling order, one a thread (0 past them): each is
// compared with all, `size` (a power of two from 64, at least n) of them by 1024 / size
// threads each.
__device__ u64 sorted(Lds &s, int n, int size) {
  const int tid = threadIdx.x, c = tid & (size - 1), part = tid / size, of = kThreads / size;
  const u64 mine = c < n ? s.cand[c] : 0;
  if (tid < size) s.rank[tid] = 0;
  __syncthreads();
  const int lo = n * part / of, hi = n * (part + 1) / of;
  int above = 0;
#pragma unroll 8
  for (int d = lo; d < hi; ++d) above += s.cand[d] > mine;
  if (c < n) atomicAdd(&s.rank[c], above);
  __syncthreads();
  if (tid < n) s.order[s.rank[tid]] = mine;
  __syncthreads();
  return tid < n ? s.order[tid] : 0;
}

// Of a tile the weight that stands before step `bin`; found(j) of its tokens in it.
// MIN: the row may have min_p; else its test is left out (256 rows of 131072, mixed: 105 ->
// 102 us; a workgroup a row has no registers for both).
template <bool MIN, typename F>
__device__ __forceinline__ u64 collect_kind(const Keep &keep, const Steps &step, int bin, const float (&v)[kVals],
                                            F found) {
  u64 wt = 0;
#pragma unroll
  for (int j = 0; j < kVals; j += 4) {
    int b[4], least = kBins + 1;
#pragma unroll
    for (int c = 0; c < 4; ++c) {
      b[c] = v[j + c] > -INFINITY ? step(v[j + c]) : kBins + 1;
      least = min(least, b[c]);
    }
    if (__any(least <= bin)) {             // (not a branch a token: their chains run side by side)
#pragma unroll
      for (int c = 0; c < 4; ++c) {
        const u64 w = MIN ? keep(v[j + c]) : weight_of(keep.w, v[j + c]);
        wt += b[c] < bin ? w : 0;
        if (b[c] == bin) found(j + c);
      }
    }
  }
  return wave_sum(wt);
}
template <typename F>
__device__ __forceinline__ u64 collect_tile(const Keep &keep, const Steps &step, int bin, const float (&v)[kVals],
                                            F found) {
  return keep.min_w > 0.0 ? collect_kind<true>(keep, step, bin, v, found)
                          : collect_kind<false>(keep, step, bin, v, found);
}

// Of a number each wave has put into LDS: the sum over the waves before this one, and
// over all.
template <typename T>
__device__ __forceinline__ void across_waves(const T *of, int wave, T &before, T &all) {
  const T upto = row_scan(of[threadIdx.x & (kWaves - 1)], Add{});
  all = of_lane(upto, kWaves - 1);
  before = wave ? of_lane(upto, wave - 1) : T(0);
}
static_assert(kWaves == 16, "a row of lanes takes a value of each wave");

// Finds, over the histogram, the bin in which the order's cut falls: the first whose
// running count reaches `want_n` or running weight reaches want_w(the histogram's weight)
// (in doubles: compared as p * W is).  before_n, before_w: what stands before the
// histogram's range, and on return before the bin.  Leaves s.bin = kBins where none does.
// Returns the histogram's weight.
template <typename S, typename F>
__device__ u64 find_bin(S &s, u64 want_n, F want_of) {
  const int tid = threadIdx.x, lane = tid & 63;
  const int wave = __builtin_amdgcn_readfirstlane(tid >> 6);
  // two bins a thread
  const uint32_t n0 = s.count[2 * tid], n1 = s.count[2 * tid + 1];
  const u64 w0 = s.mass[2 * tid], w1 = s.mass[2 * tid + 1];
  const uint32_t ns = wave_scan(n0 + n1);
  const u64 ws = wave_scan(w0 + w1);
  if (lane == 63) {
    s.wn[wave] = ns;
    s.wmass[wave] = ws;
  }
  if (tid == 0) s.bin = kBins;
  const u64 bn = s.before_n, bw = s.before_w;
  __syncthreads();
  uint32_t n_before, n_all;
  u64 w_before, w_all;
  across_waves(s.wn, wave, n_before, n_all);
  across_waves(s.wmass, wave, w_before, w_all);
  const double want_w = want_of(w_all);
  const u64 n = bn + n_before + ns, w = bw + w_before + ws;
  const u64 na = n - n1, wa = w - w1;      // through the thread's first bin
  const u64 np = na - n0, wp = wa - w0;    // before it
  const auto reached = [&](u64 c, u64 m) { return c >= want_n || (double)m >= want_w; };
  // reached is monotone; exactly one bin has it and not the one before (an empty
  // bin never changes it)
  const bool before = tid == 0 ? false : reached(np, wp);
  if (!before && reached(na, wa)) {
    s.bin = 2 * tid;
    s.bin_n = n0;
    s.before_n = np;
    s.before_w = wp;
  } else if (!before && reached(n, w)) {
    s.bin = 2 * tid + 1;
    s.bin_n = n1;
    s.before_n = na;
    s.before_w = wa;
  }
  __syncthreads();
  return w_all;
}

__device__ void clear_bins(Lds &s) {
  for (int i = threadIdx.x; i < kBins; i += kThreads) {
    s.mass[i] = 0;
    s.count[i] = 0;
  }
}

// A tile's tokens into the steps; those of the last step into rest_n and rest_w.  Counts
// where top_k cuts, weights where top_p does.
template <bool K, bool P>
__device__ __forceinline__ void add_kind(const float (&v)[kVals], const Weigher &w, const Steps &step, uint32_t *count,
                                         u64 *mass, uint32_t &rest_n, u64 &rest_w) {
#pragma unroll
  for (int j = 0; j < kVals; j += 4) {
    u64 wt[4];
    if constexpr (P) {
#pragma unroll
      for (int c = 0; c < 4; ++c) wt[c] = weight_of(w, v[j + c]);
    }
#pragma unroll
    for (int c = 0; c < 4; ++c) {
      const int b = step(v[j + c]);
      if (b < kBins - 1) {
        if constexpr (K) atomicAdd(&count[b], 1u);
        if constexpr (P) atomicAdd(&mass[b], wt[c]);
      } else {
        if constexpr (K) rest_n += v[j + c] > -INFINITY;
        if constexpr (P) rest_w += wt[c];  // (0 of -infinity)
      }
    }
    if constexpr (P) __builtin_amdgcn_sched_barrier(0);
  }
}
__device__ __forceinline__ void add_to_steps(const float (&v)[kVals], const Weigher &w, const Steps &step, bool by_k,
                                             bool by_p, uint32_t *count, u64 *mass, uint32_t &rest_n, u64 &rest_w) {
  if (!by_p)
    add_kind<true, false>(v, w, step, count, mass, rest_n, rest_w);
  else if (by_k)
    add_kind<true, true>(v, w, step, count, mass, rest_n, rest_w);
  else
    add_kind<false, true>(v, w, step, count, mass, rest_n, rest_w);
}

// ---- stats ------------------------------------------------------------------------
// What the statistics of a row are for: the index only of greedy rows, the mean only of
// those whose order is cut (all of it for every row: 120 vector instructions a lane's
// four tokens, 30 us for 256 rows of 131072, now 24).
__device__ __forceinline__ float largest_of(const float (&v)[kVals]) {
  float top = v[0];
#pragma unroll
  for (int j = 1; j < kVals; ++j) top = fmaxf(top, v[j]);
  return top;
}
__device__ __forceinline__ int index_in(const float (&v)[kVals], float top, int tile, int lane) {
  int at = 0x7fffffff;
#pragma unroll
  for (int j = kVals - 1; j >= 0; --j) at = v[j] == top ? index_of(tile, lane, j) : at;
  return at;
}
// exp(l - top), summed; top finite, or infinite (then of those alone), or -infinity (0).
// (The terms in fp32, their sum in fp64: beside the largest one's 1 the small ones would
// be rounded to 2^-24, and a log-probability near 0 is their sum.)
__device__ __forceinline__ double exp_sum_in(const float (&v)[kVals], float top) {
  double e = 0.0;
  if (fabsf(top) < INFINITY) {
#pragma unroll
    for (int j = 0; j < kVals; ++j) e += (double)__builtin_amdgcn_exp2f((v[j] - top) * 1.44269504088896f);
  } else if (top > 0.0f) {
#pragma unroll
    for (int j = 0; j < kVals; ++j) e += v[j] == INFINITY ? 1.0 : 0.0;
  }
  return e;
}
// Sum and number of the logits not `far` below `top`.
__device__ __forceinline__ void mean_in(const float (&v)[kVals], float top, float far, float &sum, uint32_t &n) {
  const float least = fmaxf(top - far, -3.402823466e38f);
  if (top == INFINITY) return;
#pragma unroll
  for (int j = 0; j < kVals; ++j) {
    const bool in = v[j] >= least;
    sum += in ? v[j] : 0.0f;
    n += in;
  }
}

__global__ void __launch_bounds__(64 * kStatTiles) sample_stats_kernel(const SampleArgs a) {
  __shared__ u64 wbest[kStatTiles];
  __shared__ double wsum[kStatTiles], wexp[kStatTiles];
  __shared__ uint32_t wn[kStatTiles];
  const int row = blockIdx.y, slice = blockIdx.x, lane = threadIdx.x & 63;
  const int wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
  const int t = slice * kStatTiles + wave;
  float v[kVals];
  load_tile(a.logits + (size_t)row * a.ld, a.V, t, lane, v);
  const Params r = params_of(a, row);
  float top = largest_of(v);
  u64 best = wave_largest(packed(top, r.greedy ? index_in(v, top, t, lane) : 0));
  if (lane == 0) {
    wbest[wave] = best;
    if (t < a.row_tiles) a.tops[(size_t)row * a.row_tiles + t] = of_key((uint32_t)(best >> 32));
  }
  __syncthreads();
#pragma unroll
  for (int i = 0; i < kStatTiles; ++i) best = wbest[i] > best ? wbest[i] : best;
  top = of_key((uint32_t)(best >> 32));
  float sum = 0.0f;
  uint32_t n = 0;
  if (r.by_k || r.by_p) mean_in(v, top, r.far, sum, n);
  const double e = a.logprob ? exp_sum_in(v, top) : 0.0;
  const double ds = wave_sum((double)sum), de = wave_sum(e);
  n = wave_sum(n);
  if (lane == 0) {
    wsum[wave] = ds;
    wexp[wave] = de;
    wn[wave] = n;
  }
  __syncthreads();
  if (threadIdx.x == 0) {
    double d = 0.0, x = 0.0;
    uint32_t c = 0;
    for (int i = 0; i < kStatTiles; ++i) {
      d += wsum[i];
      x += wexp[i];
      c += wn[i];
    }
    a.stats[(size_t)row * a.slices + slice] = SliceStat{top, (int)~(uint32_t)best, x, (float)d, c};
  }
}

// ---- weights ------------------------------------------------------------------------
constexpr int kPassThreads = 512, kPassWaves = kPassThreads / 64;

// The tiles of a workgroup's part of the row.
__device__ __forceinline__ void part_of_row(const SampleArgs &a, int part, int &lo, int &hi) {
  const int tiles = (a.V + kSampleTile - 1) / kSampleTile;
  const int each = (tiles + a.parts - 1) / a.parts;
  lo = min(part * each, tiles);
  hi = min(lo + each, tiles);
}

__global__ void __launch_bounds__(kPassThreads, 4) sample_weights_kernel(const SampleArgs a) {
  __shared__ double pow[64];
  __shared__ u64 mass[kBins];
  __shared__ uint32_t count[kBins];
  const int row = blockIdx.y, tid = threadIdx.x, lane = tid & 63, wave = tid >> 6;
  const float *__restrict__ x = a.logits + (size_t)row * a.ld;
  int lo, hi;
  part_of_row(a, blockIdx.x, lo, hi);
  const Params r = params_of(a, row);
  if (r.greedy) return;
  const bool cut = r.by_k || r.by_p;
  int t = lo + wave;
  float v[kVals];
  // (the first tile's load goes out with the row's statistics)
  if (cut || !(r.min_p > 0.0)) load_tile(x, a.V, t, lane, v);
  const Total tot = total_of(a, r, row, lane);
  if (tot.none) return;
  if (tid < 64) pow[tid] = kPow[tid];
  if (cut)
    for (int i = tid; i < kBins; i += kPassThreads) {
      mass[i] = 0;
      count[i] = 0;
    }
  __syncthreads();
  const Keep keep(weigher_of(a, r, tot.M, pow), r);
  if (!cut) {
    for (; t < hi; t += kPassWaves) {
      u64 wt = 0;
      if (keep.min_w > 0.0) {              // (few tiles hold any: the others are not read)
        if (top_of(a, tot, row, t) >= keep.min_l) {
          load_tile(x, a.V, t, lane, tot.infinite, v);
          wt = weight_of_tile(keep, v);
        }
      } else {
        if (t >= lo + kPassWaves) load_tile(x, a.V, t, lane, v);
        among_infinite(tot.infinite, v);
        wt = weight_of_tile(keep, v);
      }
      if (lane == 0) a.tiles[(size_t)row * a.row_tiles + t] = wt;
    }
    return;
  }
  const Steps step(tot, r.by_p);
  u64 rest_w = 0;
  uint32_t rest_n = 0;
  for (; t < hi; t += kPassWaves) {
    if (t >= lo + kPassWaves) load_tile(x, a.V, t, lane, v);
    among_infinite(tot.infinite, v);
    add_to_steps(v, keep.w, step, r.by_k, r.by_p, count, mass, rest_n, rest_w);
  }
  rest_w = wave_sum(rest_w);
  rest_n = wave_sum(rest_n);
  if (lane == 0) {
    atomicAdd(&count[kBins - 1], rest_n);
    atomicAdd(&mass[kBins - 1], rest_w);
  }
  __syncthreads();
  const size_t at = ((size_t)row * a.parts + blockIdx.x) * kBins;
  for (int i = tid; i < kBins; i += kPassThreads) {
    if (r.by_k) a.counts[at + i] = count[i];
    if (r.by_p) a.masses[at + i] = mass[i];
  }
}

// ---- cut ------------------------------------------------------------------------------
__global__ void __launch_bounds__(kThreads) sample_cut_kernel(const SampleArgs a) {
  __shared__ struct {
    u64 mass[kBins];
    uint32_t count[kBins];
    uint32_t wn[kWaves];
    u64 wmass[kWaves];
    int bin;
    u64 before_n, before_w;
    uint32_t bin_n;
  } s;
  const int row = blockIdx.x, tid = threadIdx.x;
  const Params r = params_of(a, row);
  // (a row of nothing has no histogram: what is found in its place is not used)
  if (!(r.by_k || r.by_p)) return;
  u64 w0 = 0, w1 = 0;
  uint32_t n0 = 0, n1 = 0;
  const size_t at = (size_t)row * a.parts * kBins + 2 * tid;
  if (r.by_k) {                            // (two loops: a branch within one would part its loads)
#pragma unroll 8
    for (int p = 0; p < a.parts; ++p) {
      const uint2 n = *reinterpret_cast<const uint2 *>(a.counts + at + (size_t)p * kBins);
      n0 += n.x;
      n1 += n.y;
    }
  }
  if (r.by_p) {
#pragma unroll 8
    for (int p = 0; p < a.parts; ++p) {
      const ulonglong2 m = *reinterpret_cast<const ulonglong2 *>(a.masses + at + (size_t)p * kBins);
      w0 += m.x;
      w1 += m.y;
    }
  }
  s.mass[2 * tid] = w0;
  s.mass[2 * tid + 1] = w1;
  s.count[2 * tid] = n0;
  s.count[2 * tid + 1] = n1;
  if (tid == 0) {
    s.before_n = 0;
    s.before_w = 0;
  }
  __syncthreads();
  const u64 W = find_bin(s, r.by_k ? (u64)r.k : ~0ull, [&](u64 all) { return r.by_p ? (double)r.p * (double)all : INFINITY; });
  if (tid == 0) {
    RowCut c;
    c.bin = s.bin;
    c.bin_n = s.bin < kBins ? s.bin_n : 0;
    c.before_n = s.before_n;
    c.before_w = s.before_w;
    c.total_w = W;
    c.n_cand = 0;
    a.cuts[row] = c;
  }
}

// ---- collect ----------------------------------------------------------------------------
__global__ void __launch_bounds__(kPassThreads) sample_collect_kernel(const SampleArgs a) {
  __shared__ double pow[64];
  __shared__ Candidate found[kCand];
  __shared__ int n_found;
  __shared__ unsigned place;
  const int row = blockIdx.y, tid = threadIdx.x, lane = tid & 63, wave = tid >> 6;
  const float *__restrict__ x = a.logits + (size_t)row * a.ld;
  int lo, hi;
  part_of_row(a, blockIdx.x, lo, hi);
  const Params r = params_of(a, row);
  if (!(r.by_k || r.by_p)) return;
  const int bin = a.cuts[row].bin;
  const unsigned bin_n = a.cuts[row].bin_n;
  const Total tot = total_of(a, r, row, lane);
  if (tot.none || bin_n > kCand) return;   // (too many: divided again by the draw)
  if (tid < 64) pow[tid] = kPow[tid];
  if (tid == 0) n_found = 0;
  __syncthreads();
  const Keep keep(weigher_of(a, r, tot.M, pow), r);
  const Steps step(tot, r.by_p);
  for (int t = lo + wave; t < hi; t += kPassWaves) {
    u64 wt = 0;
    if (step(top_of(a, tot, row, t)) <= bin) {   // (a tile that holds none of the first is not read)
      float v[kVals];
      load_tile(x, a.V, t, lane, tot.infinite, v);
      wt = collect_tile(keep, step, bin, v, [&](int j) {
        const int c = atomicAdd(&n_found, 1);
        if (c < kCand) found[c] = Candidate{v[j], index_of(t, lane, j)};
      });
    }
    if (lane == 0) a.tiles[(size_t)row * a.row_tiles + t] = wt;
  }
  __syncthreads();
  // (past kCand in all, which only a row without top_k can hold, the draw finds them itself)
  if (tid == 0) place = n_found ? atomicAdd(&a.cuts[row].n_cand, (unsigned)n_found) : 0;
  __syncthreads();
  for (int c = tid; c < min(n_found, kCand); c += kPassThreads)
    if (place + c < kCand) a.cands[(size_t)row * kCand + place + c] = found[c];
}

// ---- draw -------------------------------------------------------------------------------
// The draw of one row.  `again`: step `bin` holds more tokens than s.cand, and neither
// they nor the tiles' sums have been collected; else both are in LDS.  total_w: the
// row's weight in all, for top_p.
__device__ __forceinline__ void draw_row(Lds &s, const SampleArgs &a, const Params &r, const Total &tot,
                                         u64 total_w, int bin, bool again) {
  const int row = blockIdx.x, tid = threadIdx.x, lane = tid & 63;
  const int wave = __builtin_amdgcn_readfirstlane(tid >> 6);
  const float *__restrict__ x = a.logits + (size_t)row * a.ld;
  const int V = a.V, tiles = (V + kSampleTile - 1) / kSampleTile;
  const Weigher w = weigher_of(a, r, tot.M, s.pow);
  const Keep kept_weight(w, r);
  const Steps bin_of(tot, r.by_p);
  const bool by_k = r.by_k, by_p = r.by_p;
  const double u = a.u[row];
  const auto each_tile = [&](auto f) {
    for (int t = wave; t < tiles; t += kWaves) {
      float v[kVals];
      load_tile(x, V, t, lane, tot.infinite, v);
      f(t, v);
    }
  };
  if (tid == 0) {
    s.kept = 0;
    s.cut_key = 0;                         // everything
    s.cut_index = 0x7fffffff;
  }
  __syncthreads();

  if (by_k || by_p) {
    const u64 want_n = by_k ? (u64)r.k : ~0ull;
    const double want_w = by_p ? (double)r.p * (double)total_w : INFINITY;
    bool keyed = false, equal = false;
    uint32_t klo = 0, khi = 0;
    // more than kCand tokens in the step: an interval of keys, divided again
    while (bin < kBins && s.bin_n > kCand) {
      if (!keyed) {
        // the bin's smallest and largest key
        if (tid == 0) {
          s.kmin = 0xffffffffu;
          s.kmax = 0;
        }
        __syncthreads();
        uint32_t lo = 0xffffffffu, hi = 0;
        each_tile([&](int, const float (&v)[kVals]) {
#pragma unroll
          for (int j = 0; j < kVals; ++j)
            if (v[j] != -INFINITY && bin_of(v[j]) == bin) {
              const uint32_t k = key_of(v[j]);
              lo = min(lo, k);
              hi = max(hi, k);
            }
        });
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
      each_tile([&](int, const float (&v)[kVals]) {
#pragma unroll
        for (int j = 0; j < kVals; ++j) {
          const uint32_t k = key_of(v[j]);
          if (k < klo || k > khi || v[j] == -INFINITY) continue;
          const uint32_t b = (khi - k) >> shift;
          atomicAdd(&s.count[b], 1u);
          if (by_p) atomicAdd(&s.mass[b], weight_of(w, v[j]));
        }
      });
      __syncthreads();
      find_bin(s, want_n, [&](u64) { return want_w; });
      bin = s.bin;
      if (bin >= kBins) break;             // (the range held the cut: it does not happen)
      khi = khi - ((uint32_t)bin << shift);
      const uint32_t span = (1u << shift) - 1u;
      klo = khi - klo > span ? khi - span : klo;
    }
    const bool cuts = bin < kBins;

    // what stands before the interval, by tile; its tokens, or how many
    const uint32_t kequal = khi;
    __syncthreads();
    if (again)
      each_tile([&](int t, const float (&v)[kVals]) {
        u64 wt = 0;
        uint32_t same = 0;
#pragma unroll
        for (int j = 0; j < kVals; ++j) {
          if (v[j] == -INFINITY) continue;
          const uint32_t k = key_of(v[j]);
          if (k > khi) {
            wt += kept_weight(v[j]);
          } else if (k >= klo) {
            if (equal) {
              ++same;
            } else {
              const int c = atomicAdd(&s.n_cand, 1);
              if (c < kCand) s.cand[c] = packed(v[j], index_of(t, lane, j));
            }
          }
        }
        wt = wave_sum(wt);
        if (equal) same = wave_sum(same);
        if (lane == 0) {
          s.tile[t] = wt;
          // (equal logits: the histogram's room holds the tiles' counts)
          if (equal) s.count[t] = same;
        }
      });
    __syncthreads();
    if (cuts && !equal) {
      // sorted, a candidate a thread; then those before each are counted and summed
      const int n = min(s.n_cand, kCand);
      int size = 64;
      while (size < n) size *= 2;
      const u64 e = sorted(s, n, size);
      const float l = of_key((uint32_t)(e >> 32));
      const int i = (int)~(uint32_t)e;
      const bool live = tid < n;
      const u64 mine = live ? weight_of(w, l) : 0;
      u64 mass = wave_scan(mine);
      if (lane == 63) s.wmass[wave] = mass;
      __syncthreads();
      u64 earlier, all;
      across_waves(s.wmass, wave, earlier, all);
      mass += s.before_w - mine + earlier;
      const u64 rank = s.before_n + tid;
      const bool keep = live && rank < want_n && (mass == 0 || (double)mass < want_w);
      if (keep) {
        const u64 kw = kept_weight(l);
        if (kw) atomicAdd(&s.tile[i / kSampleTile], kw);
        // (kept ones are a prefix)
        atomicMax(&s.kept, tid + 1);
      }
      __syncthreads();
      if (tid + 1 == s.kept) {
        s.cut_key = (uint32_t)(e >> 32);
        s.cut_index = i;
      }
    } else if (cuts && equal) {
      // of equal logits the first `take` by index
      if (tid == 0) {
        const u64 each = weight_of(w, of_key(kequal));
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
        if (take == 0 && s.before_w == 0) take = 1;
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
        load_tile(x, V, edge, lane, tot.infinite, v);
        u64 seen = 0;
#pragma unroll
        for (int j = 0; j < 4; ++j) {
          u64 mine = 0;
          for (int c = 0; c < 4; ++c) mine += v[4 * j + c] != -INFINITY && key_of(v[4 * j + c]) == kequal;
          u64 n = wave_scan(mine) - mine + seen;
          for (int c = 0; c < 4; ++c)
            if (v[4 * j + c] != -INFINITY && key_of(v[4 * j + c]) == kequal && ++n == keep)
              s.cut_index = index_of(edge, lane, 4 * j + c);
          seen += wave_sum(mine);
        }
      }
    }
    __syncthreads();
  }

  // ---- the token: each wave finds the tile for itself
  u64 total = 0;
  for (int t = lane; t < tiles; t += 64) total += s.tile[t];
  total = wave_sum(total);
  const double f = floor((u > 0.0 ? u : 0.0) * (double)total);
  u64 target = f < (double)total ? (u64)f : total;
  if (target >= total) target = total - 1;
  // the first tile whose running sum exceeds it
  u64 run = 0;
  int pick = -1;
  for (int t0 = 0; t0 < tiles && pick < 0; t0 += 64) {
    const u64 mine = t0 + lane < tiles ? s.tile[t0 + lane] : 0;
    const u64 upto = wave_scan(mine) + run;
    const u64 over = __ballot(upto > target);
    const int f0 = __builtin_amdgcn_readfirstlane(over ? __ffsll(over) - 1 : 63);
    if (over) pick = t0 + f0;
    run = of_lane(over ? upto - mine : upto, f0);
  }
  if (pick < 0) {                          // (the largest logit is always kept: it does not happen)
    if (tid == 0) a.token[row] = -1;
    return;
  }
  // and in it the token: one a thread
  const int i = pick * kSampleTile + tid;
  float l = i < V ? x[i] : -INFINITY;
  l = l == l ? l : -INFINITY;
  if (tot.infinite) l = l == INFINITY ? 0.0f : -INFINITY;
  const uint32_t key = key_of(l), ck = s.cut_key;
  const bool in = l > -INFINITY && (key > ck || (key == ck && i <= s.cut_index));
  const u64 mine = in ? kept_weight(l) : 0;
  const u64 upto = wave_scan(mine);
  if (lane == 63) s.wmass[wave] = upto;
  __syncthreads();
  u64 earlier, all;
  across_waves(s.wmass, wave, earlier, all);
  const u64 end = run + earlier + upto;
  if (end > target && end - mine <= target) {
    a.token[row] = i;
    // (infinite logits stand at 0 here, and M does)
    if (a.logprob) a.logprob[row] = (float)((double)l - (double)tot.M - s.log_sum);
  }
}

// What is not drawn: a row of nothing, and a greedy one.  exp_sum: of exp(l - M).
__device__ __forceinline__ void store_nothing(const SampleArgs &a, int row) {
  a.token[row] = -1;
  if (a.logprob) a.logprob[row] = -INFINITY;
}
__device__ __forceinline__ void store_largest(const SampleArgs &a, int row, const Total &tot, double exp_sum) {
  a.token[row] = tot.at;
  if (a.logprob) a.logprob[row] = (float)-log(exp_sum);
}

__global__ void __launch_bounds__(kThreads) sample_draw_kernel(const SampleArgs a) {
  __shared__ Lds s;
  const int row = blockIdx.x, tid = threadIdx.x, lane = tid & 63;
  const int wave = __builtin_amdgcn_readfirstlane(tid >> 6);
  // (loads of what the passes before have left go out together, also what this kind of
  // row does not use)
  const Params r = params_of(a, row);
  const RowCut rc = a.cuts[row];
  const Candidate c = a.cands[(size_t)row * kCand + tid];
  const u64 tile = tid < a.row_tiles ? a.tiles[(size_t)row * a.row_tiles + tid] : 0;
  const Total tot = total_of(a, r, row, lane);
  if (tot.none) {                          // nothing may follow
    if (tid == 0) store_nothing(a, row);
    return;
  }
  if (r.greedy) {
    if (wave == 0) {
      const double e = a.logprob ? exp_sum_of(a, row, lane) : 1.0;
      if (lane == 0) store_largest(a, row, tot, e);
    }
    return;
  }
  if (tid < 64) s.pow[tid] = kPow[tid];
  const bool cut = r.by_k || r.by_p;
  const unsigned bin_n = max(rc.bin_n, rc.n_cand);   // (without top_k only the latter is counted)
  const bool again = cut && bin_n > kCand;
  const int n = again || !cut ? 0 : (int)rc.n_cand;
  if (tid == 0) {
    s.n_cand = n;
    s.before_n = rc.before_n;
    s.before_w = rc.before_w;
    s.bin_n = bin_n;
  }
  if (a.logprob && wave == kWaves - 1) {
    const double e = log(exp_sum_of(a, row, lane));
    if (lane == 0) s.log_sum = e;
  }
  if (tid < n) s.cand[tid] = packed(c.l, c.i);
  if (tid < a.row_tiles) s.tile[tid] = tile;
  draw_row(s, a, r, tot, rc.total_w, rc.bin, again);
}

// ---- a row's five passes in one workgroup ------------------------------------------------
template <int TW>
struct RowTiles {                          // a wave's tiles, in registers
  int tiles, wave;
  float v[TW][kVals];
  __device__ __forceinline__ RowTiles(const float *x, int V, int wave_, int lane)
      : tiles((V + kSampleTile - 1) / kSampleTile), wave(wave_) {
#pragma unroll
    for (int i = 0; i < TW; ++i) load_tile(x, V, wave + i * kWaves, lane, v[i]);
  }
  __device__ __forceinline__ void settle(bool infinite) {
#pragma unroll
    for (int i = 0; i < TW; ++i) among_infinite(infinite, v[i]);
  }
  template <typename F>
  __device__ __forceinline__ void each(F f) {
#pragma unroll
    for (int i = 0; i < TW; ++i)
      if (wave + i * kWaves < tiles) f(wave + i * kWaves, v[i]);
  }
};

template <int TW>
__global__ void __launch_bounds__(kThreads) sample_row_kernel(const SampleArgs a) {
  __shared__ Lds s;
  const int row = blockIdx.x, tid = threadIdx.x, lane = tid & 63;
  const int wave = __builtin_amdgcn_readfirstlane(tid >> 6);
  RowTiles<TW> held(a.logits + (size_t)row * a.ld, a.V, wave, lane);
  const Params r = params_of(a, row);
  const bool cut = r.by_k || r.by_p;
  if (tid < 64) s.pow[tid] = kPow[tid];
  if (cut) clear_bins(s);
  if (tid == 0) {
    s.n_cand = 0;
    s.before_n = 0;
    s.before_w = 0;
    s.bin_n = 0;
  }

  // the statistics
  u64 best = 0;
  held.each([&](int t, const float (&v)[kVals]) {
    const float top = largest_of(v);
    const u64 b = packed(top, r.greedy ? index_in(v, top, t, lane) : 0);
    best = b > best ? b : best;
  });
  best = wave_largest(best);
  if (lane == 0) s.wmass[wave] = best;
  __syncthreads();
  best = s.wmass[lane & (kWaves - 1)];
  best = wave_largest(best);
  const float top = of_key((uint32_t)(best >> 32));
  Total tot;
  tot.infinite = top == INFINITY;
  tot.none = top == -INFINITY;
  tot.M = tot.infinite ? 0.0f : top;
  tot.at = (int)~(uint32_t)best;
  tot.mean = -1.0f;
  if (tot.none) {
    if (tid == 0) store_nothing(a, row);
    return;
  }
  double exp_sum = 1.0;
  if (cut || a.logprob) {
    double e = 0.0;
    float sum = 0.0f;
    uint32_t n = 0;
    held.each([&](int, const float (&v)[kVals]) {
      if (cut) mean_in(v, top, r.far, sum, n);
      if (a.logprob) e += exp_sum_in(v, top);
    });
    const double de = wave_sum(e), ds = wave_sum((double)sum);
    n = wave_sum(n);
    if (lane == 0) {
      s.wexp[wave] = de;
      s.wsum[wave] = ds;
      s.wn[wave] = n;
    }
    __syncthreads();
    double before, e_all, sum_all;
    uint32_t n_before;
    across_waves(s.wexp, wave, before, e_all);
    across_waves(s.wsum, wave, before, sum_all);
    across_waves(s.wn, wave, n_before, n);
    exp_sum = e_all;
    if (a.logprob && !r.greedy && wave == kWaves - 1) {
      const double l = log(e_all);
      if (lane == 0) s.log_sum = l;
    }
    if (n && !tot.infinite) tot.mean = (float)(sum_all / (double)n);
  }
  if (r.greedy) {
    if (tid == 0) store_largest(a, row, tot, exp_sum);
    return;
  }
  held.settle(tot.infinite);

  const Keep keep(weigher_of(a, r, tot.M, s.pow), r);
  const Steps step(tot, r.by_p);
  u64 total_w = 0;
  int bin = kBins;
  bool again = false;
  if (!cut) {
    held.each([&](int t, const float (&v)[kVals]) {
      const u64 wt = weight_of_tile(keep, v);
      if (lane == 0) s.tile[t] = wt;
    });
  } else {
    uint32_t rest_n = 0;
    u64 rest_w = 0;
    held.each([&](int, const float (&v)[kVals]) {
      add_to_steps(v, keep.w, step, r.by_k, r.by_p, s.count, s.mass, rest_n, rest_w);
    });
    rest_w = wave_sum(rest_w);
    rest_n = wave_sum(rest_n);
    if (lane == 0) {
      atomicAdd(&s.count[kBins - 1], rest_n);
      atomicAdd(&s.mass[kBins - 1], rest_w);
    }
    __syncthreads();
    total_w = find_bin(s, r.by_k ? (u64)r.k : ~0ull, [&](u64 all) { return r.by_p ? (double)r.p * (double)all : INFINITY; });
    bin = s.bin;
    again = bin < kBins && s.bin_n > kCand;
    if (!again) {
      held.each([&](int t, const float (&v)[kVals]) {
        const u64 wt = collect_kind<true>(keep, step, bin, v, [&](int j) {
          const int c = atomicAdd(&s.n_cand, 1);
          if (c < kCand) s.cand[c] = packed(v[j], index_of(t, lane, j));
        });
        if (lane == 0) s.tile[t] = wt;
      });
      if (!r.by_k) {                       // (their counts are not in the histogram)
        __syncthreads();
        again = s.n_cand > kCand;
        __syncthreads();
        if (again && tid == 0) {
          s.bin_n = s.n_cand;
          s.n_cand = 0;
        }
      }
    }
  }
  draw_row(s, a, r, tot, total_w, bin, again);
}

hipError_t launch_slices(const SampleArgs &a, hipStream_t stream) {
  const dim3 slices((unsigned)a.slices, (unsigned)a.m), parts((unsigned)a.parts, (unsigned)a.m), rows((unsigned)a.m);
  sample_stats_kernel<<<slices, 64 * kStatTiles, 0, stream>>>(a);
  sample_weights_kernel<<<parts, kPassThreads, 0, stream>>>(a);
  if (a.top_k || a.top_p) {
    sample_cut_kernel<<<rows, kThreads, 0, stream>>>(a);
    sample_collect_kernel<<<parts, kPassThreads, 0, stream>>>(a);
  }
  sample_draw_kernel<<<rows, kThreads, 0, stream>>>(a);
  return hipGetLastError();
}

}  // namespace

hipError_t launch_sample(const SampleArgs &a, hipStream_t stream) {
  (void)hipGetLastError();
  if (!sample_in_one_launch(a.m, a.V)) return launch_slices(a, stream);
  if (a.V <= kSampleHeld / 4)
    sample_row_kernel<1><<<(unsigned)a.m, kThreads, 0, stream>>>(a);
  else if (a.V <= kSampleHeld / 2)
    sample_row_kernel<2><<<(unsigned)a.m, kThreads, 0, stream>>>(a);
  else
    sample_row_kernel<4><<<(unsigned)a.m, kThreads, 0, stream>>>(a);
  return hipGetLastError();
}

}  // namespace q8
