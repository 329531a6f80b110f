// q8_attn_rows.hip -- attention of chunks of rows over the paged cache
// (q8_attn_rows; the formula and layouts are in include/q8gemv.h).
#include <hip/hip_runtime.h>

#include <type_traits>

#include "q8_attn.h"

namespace q8 {
namespace {

constexpr int kMaxSplits = 16;
constexpr int kMinSplitTiles = 8;       // fewest stages of a split that computes
constexpr int kListGroups = 512;        // 16-token groups whose pages are held in LDS at a time

typedef __attribute__((ext_vector_type(16))) float f32x16_t;

// Waves of a workgroup, 32 columns each: eight (two a SIMD, in turns, below)
// where their registers allow it (not at 256 dims) and the stages need no
// widening.  Over Q8_0 four, of which a CU holds two workgroups that do not wait
// for each other: 128 dims, 3 x 509 rows behind 4096 tokens 153 us, 2048 rows
// 101; with eight 173 and 101 at as many splits, 184 and 112 at twice as many.
template <int D, int FMT> constexpr int kWaves = FMT == Q8_KV_BF16 && D < 256 ? 8 : 4;
template <int D, int FMT> constexpr int kCols = 32 * kWaves<D, FMT>;

// Keys of a stage (what the workgroup loads, and waits for, at a time), and
// the stages in LDS: bf16 computes one while the others load.
template <int D> constexpr int kStageKeys = D == 256 ? 32 : 64;
template <int FMT> constexpr int kSlots = FMT == Q8_KV_BF16 ? 4 : 2;

// LDS bytes of a stage's keys (or values) as bf16 (Q8_0: the codes, exact), and
// of their scales.
template <int D> constexpr int kValBytes = kStageKeys<D> * D * 2;
template <int D, int FMT>
constexpr int kScaleBytes = FMT == Q8_KV_Q8_0 ? kStageKeys<D> * (D / 32) * 4 : 0;

// Floats of a column's row of 64 dims in LDS, on its way out.
constexpr int kOutRow = 68;

struct Block {
  int i;         // sequence
  int block;     // its block of columns
};

__device__ __forceinline__ int rows_of(const AttnArgs &a, int i, int *start) {
  const int s = min(max(a.row_start[i], 0), a.m), e = min(max(a.row_start[i + 1], 0), a.m);
  *start = s;
  return max(e - s, 0);
}

// Block x of all sequences' blocks (i = n past the last).  A wave takes 64
// sequences at a time; every wave finds the same.
__device__ __forceinline__ Block find_block(const AttnArgs &a, int x, int cols) {
  const int lane = threadIdx.x & 63;
  int base = 0;
  for (int b = 0; b < a.n; b += 64) {
    int start;
    const int i = b + lane;
    int incl = i < a.n ? (rows_of(a, i, &start) * a.group + cols - 1) / cols : 0;
#pragma unroll
    for (int o = 1; o < 64; o <<= 1) {
      const int u = __shfl_up(incl, o);
      if (lane >= o) incl += u;
    }
    incl += base;
    const int before = __popcll(__ballot(incl <= x));
    if (before < 64)
      return Block{uni(b + before), uni(x - (before > 0 ? __shfl(incl, before - 1) : base))};
    base = __shfl(incl, 63);
  }
  return Block{a.n, 0};
}

__device__ __forceinline__ float swap_halves(float x) {   // lane l's value in lane l ^ 32
  typedef unsigned u32x2 __attribute__((ext_vector_type(2)));
  const u32x2 r = __builtin_amdgcn_permlane32_swap(__float_as_uint(x), __float_as_uint(x), false, false);
  return __uint_as_float((threadIdx.x & 32) ? r.x : r.y);
}

// Whether any of eight bf16 values is infinite or NaN (exponent all ones).
__device__ __forceinline__ bool not_finite(u32x4_t v) {
  uint32_t odd = 0;
#pragma unroll
  for (int e = 0; e < 4; ++e) odd |= (v[e] & 0x7fff7fffu) + 0x00800080u;
  return (odd & 0x80008000u) != 0;
}

// 16 bytes a lane from memory into LDS at `at` (a scalar) plus 16 times the
// lane, without registers in between; loads_done waits for all but the last N.
// They are written out because the compiler would make every read of LDS wait
// for every such load, the next stages' too.  m0, the load's base in LDS, is a
// register that the compiler sets right before its own uses (here it has none).
__device__ __forceinline__ void load_to_lds(const void *p, unsigned at) {
  asm volatile("s_mov_b32 m0, %1\n\ts_nop 0\n\tglobal_load_lds_dwordx4 %0, off"
               :: "v"(p), "s"(at) : "memory");
}
__device__ __forceinline__ void load_to_lds(const char *base, unsigned off, unsigned at) {
  const uint64_t b = (uint64_t)base;     // one address for the wave, as a scalar
  const uint64_t p = (uint64_t)(unsigned)uni((int)(b >> 32)) << 32 | (unsigned)uni((int)b);
  asm volatile("s_mov_b32 m0, %2\n\ts_nop 0\n\tglobal_load_lds_dwordx4 %0, %1"
               :: "v"(off), "s"(p), "s"(at) : "memory");
}
template <int N>
__device__ __forceinline__ void loads_done() {
  asm volatile("s_waitcnt vmcnt(%0)" :: "n"(N) : "memory");
}

// A barrier that instructions are not moved across.
__device__ __forceinline__ void turn() {
  __builtin_amdgcn_sched_barrier(0);
  __syncthreads();
  __builtin_amdgcn_sched_barrier(0);
}

__host__ __device__ constexpr int record_floats(int cols, int dim) { return cols * dim + 2 * cols; }

// Grid: (blocks of columns x key/value heads, the heads fastest -- eight of
// them put a head's keys in one XCD's L2 --, key splits).  A column is one
// (row, query head of the group) pair, so the group's heads share the keys;
// a wave holds 32 columns, the workgroup's waves share the staged keys and
// values in LDS.  Scores are transposed (32 keys x 32 columns, v_mfma 32x32x16):
// a lane's sixteen scores belong to one column, and with the key fragments'
// rows permuted (row 8a + 4h + e is key 16 (a/2) + 8h + 4 (a%2) + e) they are,
// eight by eight, the value product's operand, so probabilities stay in their
// lane, and the running maximum is a lane's own scalar.  That maximum is only
// raised when a score passes it by 2^8 (kSlack): sums stay far inside fp32, and
// the sums O^T are rescaled once or twice a block instead of at nearly every
// stage.
//
// The matrix cores and the vector unit of a SIMD work at the same time only
// for different waves (or far-apart instructions of one), and a workgroup's
// barriers bring its waves into step.  So with eight waves the two of a SIMD
// take turns (in_turns): waves 0-3 run half a stage before waves 4-7, and
// between two barriers the one half multiplies (a stage's values and the next
// one's keys) while the other turns its scores into probabilities.
//
// Measured on MI355X, 8192 rows of 32 heads over 8, 128 dims, bf16, behind 0
// tokens: 516 us, 1.07 PFLOP/s of 1.3 that a large library product reaches; four
// waves in step with the maximum raised inside the loop took 627, stages through
// registers 658.  Bound by LDS reads: a half's products take 128 KB of
// fragments a turn, 1560 cycles at 85 bytes a clock, against 1470 for the other
// half's probabilities.  Stages of 32 keys took 697 us against 633, waves of 64
// columns spilled.  Q8_0, 3 x 509 rows behind 4096 tokens: 155 us; the codes are
// widened once a stage and each 32 dims' scores scaled, so the vector unit bounds
// it.  256 dims: 2048 rows 164 us, 0.42 PFLOP/s; four waves, one a SIMD, with
// nothing beside their waits, and sums that move between the two halves of the
// register file around each product.
constexpr float kSlack = 8.0f;

template <int D, int FMT>
__global__ void __launch_bounds__((64 * kWaves<D, FMT>), (D == 256 ? 1 : 2))
attn_rows_kernel(AttnArgs a) {
  constexpr int W = kWaves<D, FMT>, kThreads = 64 * W, kBlock = kCols<D, FMT>, SL = kSlots<FMT>;
  constexpr int NB = D / 32, NK = D / 16, KT = kStageKeys<D>, NS = KT / 32;
  constexpr int kVal = kValBytes<D>, kScl = kScaleBytes<D, FMT>;
  constexpr int kElem = FMT == Q8_KV_BF16 ? 16 : 8;        // bytes of eight cached values
  constexpr int kPer = 16 / kElem;                         // eights in a 16-byte piece
  constexpr int kIt = KT * D / 8 / kPer / kThreads;        // a thread's pieces of the keys
  static_assert(kIt * kThreads * kPer * 8 == KT * D, "pieces");
  constexpr int kScales = KT * NB;                         // scales of the keys
  constexpr int kSIt = (kScales + kThreads - 1) / kThreads;
  static_assert(kScales % kThreads == 0 || kSIt == 1, "scales");
  constexpr int kListStages = kListGroups / (KT / 16);
  constexpr bool kTurns = FMT == Q8_KV_BF16 && W == 8;
  extern __shared__ __align__(16) char lds[];              // keys, values, their scales: SL stages each
  __shared__ int pids[kListGroups];
  __shared__ int is_last;
  const int lane = threadIdx.x & 63, wave = uni(threadIdx.x >> 6);
  const int col = lane & 31, hf = lane >> 5;
  const KvCache c = a.cache;
  const int hk = blockIdx.x % c.heads, bx = blockIdx.x / c.heads;
  const int pl = c.page_log2, P = 1 << pl;

  const Block bl = find_block(a, bx, kBlock);
  if (bl.i >= a.n) return;
  int start;
  const int R = uni(rows_of(a, bl.i, &start));
  start = uni(start);
  const int len = uni(clamp_len(a.lens[bl.i], a.max_pages, pl));
  const int ncol = R * a.group;
  // heaviest first: the sequence's last rows see the most tokens
  const int blocks = (ncol + kBlock - 1) / kBlock;
  const int c0 = (blocks - 1 - bl.block) * kBlock, c1 = min(c0 + kBlock, ncol) - 1;
  const int p0 = len - R + c0 / a.group, p1 = len - R + c1 / a.group;
  const Span sp = span_of<KT>(max(p0, 0), p1, a.window, a.sinks);
  const int S = min((int)gridDim.y, max(sp.nt / kMinSplitTiles, 1));
  const int s = blockIdx.y;
  if (s >= S) return;
  const int u0 = (int)((long long)sp.nt * s / S), u1 = (int)((long long)sp.nt * (s + 1) / S);

  // The scale is used as a positive one (so that the largest score stays the
  // largest, and an unseen key's -infinity is one): its sign goes into the
  // queries, and a scale of zero makes them zero.
  const float scale = a.scale_log2 == 0.0f ? 1.0f : fabsf(a.scale_log2);
  const uint32_t flip = a.scale_log2 < 0.0f ? 0x80008000u : 0u;
  const uint32_t keep = a.scale_log2 == 0.0f ? 0u : 0xffffffffu;
  const int mycol = c0 + wave * 32 + col, incol = min(mycol, ncol - 1);
  const int pos = len - R + incol / a.group;
  bf16x8_t q[NK];
#pragma unroll
  for (int k = 0; k < NK; ++k) {
    u32x4_t v = {0u, 0u, 0u, 0u};
    if (mycol < ncol)
      v = *reinterpret_cast<const u32x4_t *>(
          a.q + ((size_t)(start + incol / a.group) * a.q_heads + hk * a.group + incol % a.group) * D +
          16 * k + 8 * hf);
    q[k] = __builtin_bit_cast(bf16x8_t, (v ^ flip) & keep);
  }
  f32x16_t o[NB];
#pragma unroll
  for (int T = 0; T < NB; ++T)
#pragma unroll
    for (int e = 0; e < 16; ++e) o[T][e] = 0.0f;
  float m = kLowest, l = 0.0f;

  const int32_t *trow = a.table + (long long)bl.i * a.max_pages;
  const int last = max(len - 1, 0);
  const size_t head_off = (size_t)hk * c.record();
  const size_t page_bytes = c.page_bytes();
  int base = u0;                           // the first stage whose pages are listed
  auto ids_of = [&](int u) Q8_INLINE { return pids + (u - base) * (KT / 16); };
  auto slot = [&](int u) Q8_INLINE { return (u - base) & (SL - 1); };

  // A stage's 16-byte pieces, thread by thread.  Keys lie as [D/8][KT][8],
  // values as [KT/8][D][8], in the cache's pages and in LDS; a piece is one
  // eight of bf16 values or two of int8 codes.  All of a thread's key pieces are
  // of one key (or pair); a wave's 64 value pieces follow each other within 16
  // tokens, so their page is a scalar.
  static_assert(kThreads * kPer % KT == 0 && (64 * kPer <= D || 64 * kPer % D == 0), "pieces");
  const int tkey = (int)threadIdx.x * kPer % KT, tch = (int)threadIdx.x * kPer / KT;
  auto key_piece = [&](int u) Q8_INLINE {
    return c.k + (size_t)max(ids_of(u)[tkey / 16], 0) * page_bytes + head_off +
           (tch * P + ((sp.tile(u) * KT + tkey) & (P - 1))) * kElem;
  };
  const int key_step = kThreads * kPer / KT * P * kElem;
  auto value_piece = [&](int u, int it) Q8_INLINE {   // the wave's 64 pieces
    const int e = (wave * 64 + it * kThreads) * kPer, vc = e / D;
    return c.v + (size_t)max(uni(ids_of(u)[vc / 2]), 0) * page_bytes + head_off +
           ((((sp.tile(u) * KT + 8 * vc) & (P - 1)) >> 3) * D + e % D) * kElem;
  };
  char *const vals = lds + SL * kVal, *const kscl = lds + 2 * SL * kVal, *const vscl = kscl + SL * kScl;
  // bf16: straight into LDS, 2 kIt loads a stage, from addresses that can be
  // looked up a stage earlier.
  struct Source {
    const char *k, *v[kIt];
  };
  const unsigned lds0 = (unsigned)(size_t)(__attribute__((address_space(3))) char *)lds + wave * 1024;
  auto source = [&](int u) Q8_INLINE {
    Source from;
    from.k = key_piece(u);
#pragma unroll
    for (int it = 0; it < kIt; ++it) from.v[it] = value_piece(u, it);
    return from;
  };
  auto issue_from = [&](const Source &from, int u) Q8_INLINE {
    const unsigned at = lds0 + slot(u) * kVal;
#pragma unroll
    for (int it = 0; it < kIt; ++it) {
      load_to_lds(from.k + (size_t)it * key_step, at + it * kThreads * 16);
      load_to_lds(from.v[it], lane * 16, at + SL * kVal + it * kThreads * 16);
    }
  };
  auto issue = [&](int u) Q8_INLINE { issue_from(source(u), u); };
  // Q8_0: through registers, where the codes are widened.
  u32x4_t rk[kIt], rv[kIt];
  float rks[kSIt], rvs[kSIt];
  const int skey = (int)threadIdx.x % KT, sblk = (int)threadIdx.x / KT;
  auto fetch = [&](int u) Q8_INLINE {
    const char *kp = key_piece(u);
#pragma unroll
    for (int it = 0; it < kIt; ++it) {
      rk[it] = *reinterpret_cast<const u32x4_t *>(kp);
      kp += key_step;
      rv[it] = *reinterpret_cast<const u32x4_t *>(value_piece(u, it) + lane * 16);
    }
    const size_t at = (size_t)max(ids_of(u)[skey / 16], 0) * page_bytes + head_off + (size_t)D * P +
                      (min(sblk, NB - 1) * P + ((sp.tile(u) * KT + skey) & (P - 1))) * 4;
#pragma unroll
    for (int it = 0; it < kSIt; ++it) {
      rks[it] = *reinterpret_cast<const float *>(c.k + at + it * (kThreads / KT) * P * 4);
      rvs[it] = *reinterpret_cast<const float *>(c.v + at + it * (kThreads / KT) * P * 4);
    }
  };
  auto widen = [&](int u) Q8_INLINE {
#pragma unroll
    for (int it = 0; it < kIt; ++it) {
      char *d = lds + slot(u) * kVal + ((int)threadIdx.x + it * kThreads) * kPer * 16;
      *reinterpret_cast<bf16x8_t *>(d) = i8x8_to_bf16(make_uint2(rk[it][0], rk[it][1]));
      *reinterpret_cast<bf16x8_t *>(d + 16) = i8x8_to_bf16(make_uint2(rk[it][2], rk[it][3]));
      d += SL * kVal;
      *reinterpret_cast<bf16x8_t *>(d) = i8x8_to_bf16(make_uint2(rv[it][0], rv[it][1]));
      *reinterpret_cast<bf16x8_t *>(d + 16) = i8x8_to_bf16(make_uint2(rv[it][2], rv[it][3]));
    }
#pragma unroll
    for (int it = 0; it < kSIt; ++it) {
      const int p = (int)threadIdx.x + it * kThreads;
      if (kScales % kThreads == 0 || p < kScales) {
        reinterpret_cast<float *>(kscl + slot(u) * kScl)[p] = rks[it];
        reinterpret_cast<float *>(vscl + slot(u) * kScl)[p] = rvs[it];
      }
    }
  };
  // Whether every column sees all of stage u.
  auto whole = [&](int u) Q8_INLINE {
    const int key0 = sp.tile(u) * KT;
    const int *ids = ids_of(u);
    int pages = ids[0];
#pragma unroll
    for (int g = 1; g < KT / 16; ++g) pages |= ids[g];
    return (key0 + KT - 1 <= p0) & (uni(pages) >= 0) &
           ((a.window <= 0) | (key0 > p1 - a.window) | (key0 + KT <= a.sinks));
  };
  // bf16, a stage that is not whole: the thread's pieces of values of tokens
  // past the sequence or on no page, whose bytes may be anything, become zero.
  // Returns whether a value of the others is infinite or NaN.
  auto clean = [&](int u) Q8_INLINE {
    bool odd = false;
#pragma unroll
    for (int it = 0; it < kIt; ++it) {
      const int piece = here(threadIdx.x) + it * kThreads, vc = piece / D;
      const int left = ids_of(u)[vc / 2] < 0 ? 0 : len - sp.tile(u) * KT - 8 * vc;
      u32x4_t *p = reinterpret_cast<u32x4_t *>(vals + slot(u) * kVal + piece * 16);
      u32x4_t v = *p;
#pragma unroll
      for (int e = 0; e < 4; ++e)
        v[e] &= (left > 2 * e ? 0xffffu : 0u) | (left > 2 * e + 1 ? 0xffff0000u : 0u);
      odd |= not_finite(v);
      if (left < 8) *p = v;
    }
    return odd;
  };

  // row `col` of a key fragment is this key of its 32
  const int fkey = 16 * (col >> 4) + 8 * ((col >> 2) & 1) + 4 * ((col >> 3) & 1) + (col & 3);
  const char *const kfrag = lds + (hf * KT + fkey) * 16, *const vfrag = vals + (hf * D + col) * 16;

  f32x16_t x[NS];           // a stage's scores
  bf16x8_t pb[NS][2];       // bf16: its probabilities
  auto zero_scores = [&]() Q8_INLINE {
#pragma unroll
    for (int n = 0; n < NS; ++n)
#pragma unroll
      for (int e = 0; e < 16; ++e) x[n][e] = 0.0f;
  };
  // The products of a stage's probabilities with its values (steps 0 .. NP-1, vb
  // its value fragments) and of a stage's keys with the queries (the NK * NS after
  // those, kb its key fragments): steps FROM .. TO-1, the fragments read kRead
  // steps ahead.  Each step is fenced: left alone the compiler puts every read
  // right before its product, which then waits for all of LDS's latency.
  constexpr int NP = NS * 2 * NB, kRead = 3;
  auto fragment = [&](int i, const char *vb, const char *kb) Q8_INLINE {
    const int j = i - NP;
    return *reinterpret_cast<const bf16x8_t *>(
        i < NP ? vb + ((i / NB) * 2 * D + 32 * (i % NB)) * 16
               : kb + (2 * (j / NS) * KT + 32 * (j % NS)) * 16);
  };
  auto multiply = [&](auto FROM, auto TO, const char *vb, const char *kb) Q8_INLINE {
    bf16x8_t f[kRead];
    if constexpr (TO > NP) zero_scores();
#pragma unroll
    for (int i = FROM; i < FROM + kRead; ++i) f[i % kRead] = fragment(i, vb, kb);
#pragma unroll
    for (int i = FROM; i < TO; ++i) {
      __builtin_amdgcn_sched_barrier(0);
      const int j = i - NP;
      if (i < NP)
        o[i % NB] = __builtin_amdgcn_mfma_f32_32x32x16_bf16(f[i % kRead], pb[i / (2 * NB)][i / NB % 2], o[i % NB], 0, 0, 0);
      else
        x[j % NS] = __builtin_amdgcn_mfma_f32_32x32x16_bf16(f[i % kRead], q[j / NS], x[j % NS], 0, 0, 0);
      if (i + kRead < TO) f[i % kRead] = fragment(i + kRead, vb, kb);
    }
    __builtin_amdgcn_sched_barrier(0);
  };
  typedef std::integral_constant<int, 0> First;
  typedef std::integral_constant<int, NP> Keys;
  typedef std::integral_constant<int, NP + NK * NS> End;
  auto scores_bf16 = [&](int u) Q8_INLINE { multiply(Keys{}, End{}, nullptr, kfrag + slot(u) * kVal); };
  auto add_values = [&](int u) Q8_INLINE { multiply(First{}, Keys{}, vfrag + slot(u) * kVal, nullptr); };
  auto scores_q8 = [&](int u) Q8_INLINE {   // each 32-dim product times its key's scale
    const char *kb = kfrag + slot(u) * kVal;
    const float *ksc = reinterpret_cast<const float *>(kscl + slot(u) * kScl) + 8 * hf;
    zero_scores();
#pragma unroll
    for (int n = 0; n < NS; ++n)
#pragma unroll
      for (int b = 0; b < NB; ++b) {
        f32x16_t z;
#pragma unroll
        for (int e = 0; e < 16; ++e) z[e] = 0.0f;
#pragma unroll
        for (int k = 2 * b; k < 2 * b + 2; ++k) {
          const bf16x8_t f = *reinterpret_cast<const bf16x8_t *>(kb + (2 * k * KT + 32 * n) * 16);
          z = __builtin_amdgcn_mfma_f32_32x32x16_bf16(f, q[k], z, 0, 0, 0);
        }
#pragma unroll
        for (int h = 0; h < 4; ++h) {
          const f32x4_t w = *reinterpret_cast<const f32x4_t *>(ksc + b * KT + 32 * n + 16 * (h >> 1) + 4 * (h & 1));
#pragma unroll
          for (int e = 0; e < 4; ++e) x[n][4 * h + e] = fmaf(w[e], z[4 * h + e], x[n][4 * h + e]);
        }
      }
  };
  // Bit e of the result: the lane's column sees key 32n + 16 (e/8) + 8 hf + e%8.
  auto seen_keys = [&](int u, int n) Q8_INLINE {
    const int *ids = ids_of(u);
    const int key0 = sp.tile(u) * KT + 32 * n + here(8 * hf), me = here(pos);
    const int from = a.window > 0 ? me - a.window + 1 : 0;
    unsigned seen = 0;
#pragma unroll
    for (int e = 0; e < 16; ++e) {
      const int key = key0 + 16 * (e >> 3) + (e & 7);
      const int stop = ids[2 * n + (e >> 3)] >= 0 ? min(me, len - 1) : -1;
      seen |= (key <= stop) & ((key >= from) | (key < a.sinks)) ? 1u << e : 0u;
    }
    return seen;
  };
  auto hide = [&](int u) Q8_INLINE {       // unseen keys' scores
#pragma unroll
    for (int n = 0; n < NS; ++n) {
      const unsigned seen = seen_keys(u, n);
#pragma unroll
      for (int e = 0; e < 16; ++e) x[n][e] = seen >> e & 1 ? x[n][e] : -__builtin_inff();
    }
  };
  // The largest score, and whether it passes the maximum in some column; raise
  // then raises the maxima to it.  Both loops below leave for it and come back:
  // as a branch inside them it would cost a copy of all sums at every stage.  A
  // column whose own largest does not pass keeps its maximum, so that its
  // roundings do not depend on the columns beside it.
  auto largest = [&]() Q8_INLINE {
    float t[4] = {x[0][0], x[0][1], x[0][2], x[0][3]};
#pragma unroll
    for (int n = 0; n < NS; ++n)
#pragma unroll
      for (int e = 0; e < 16; ++e) t[e & 3] = fmaxf(t[e & 3], x[n][e]);
    const float mx = fmaxf(fmaxf(t[0], t[1]), fmaxf(t[2], t[3]));
    return fmaxf(mx, swap_halves(mx)) * scale;
  };
  auto passes = [&](float mx) Q8_INLINE { return __any(mx > m + kSlack); };
  auto raise = [&](float mx) Q8_INLINE {
    const float mn = mx > m + kSlack ? mx : m;
    const float alpha = exp2_fast(m - mn);
    m = mn;
    l *= alpha;
#pragma unroll
    for (int T = 0; T < NB; ++T) o[T] *= alpha;
  };
  // A score is rounded as the maximum was before they are subtracted, so that the
  // largest one's exponent is 0 (or up to kSlack) however large it is: in one fma
  // the maximum's own rounding stays, from scores of 2^31 on more than an
  // exponent holds, and a row became zeros or NaN (8192 rows 500 us against 513).
  auto exponentials = [&](int n, float *p) Q8_INLINE {
    float ps[4] = {0.0f, 0.0f, 0.0f, 0.0f};
#pragma unroll
    for (int e = 0; e < 16; ++e) {
#pragma clang fp contract(off)
      p[e] = exp2_fast(x[n][e] * scale - m);
      ps[e & 3] += p[e];
    }
    l += (ps[0] + ps[1]) + (ps[2] + ps[3]);
  };
  auto soften = [&]() Q8_INLINE {
#pragma unroll
    for (int n = 0; n < NS; ++n) {
      float p[16];
      exponentials(n, p);
      pb[n][0] = to_bf16x8(p);
      pb[n][1] = to_bf16x8(p + 8);
    }
  };
  // Q8_0: the probabilities take the value scales, for each 32 dims.
  auto add_values_q8 = [&](int u, bool all) Q8_INLINE {
    const char *vb = vfrag + slot(u) * kVal;
    const float *vsc = reinterpret_cast<const float *>(vscl + slot(u) * kScl) + 8 * hf;
#pragma unroll
    for (int n = 0; n < NS; ++n) {
      const unsigned seen = all ? 0xffffu : seen_keys(u, n);
      float p[16];
      exponentials(n, p);
#pragma unroll
      for (int T = 0; T < NB; ++T) {
        float w[16];
#pragma unroll
        for (int h = 0; h < 4; ++h) {
          const f32x4_t s4 = *reinterpret_cast<const f32x4_t *>(vsc + T * KT + 32 * n + 16 * (h >> 1) + 4 * (h & 1));
#pragma unroll
          for (int e = 0; e < 4; ++e) w[4 * h + e] = p[4 * h + e] * s4[e];
        }
        if (!all) {                      // an unseen token's scale may be anything
#pragma unroll
          for (int e = 0; e < 16; ++e) w[e] = seen >> e & 1 ? w[e] : 0.0f;
        }
#pragma unroll
        for (int t = 0; t < 2; ++t) {
          const bf16x8_t f = *reinterpret_cast<const bf16x8_t *>(vb + ((4 * n + 2 * t) * D + 32 * T) * 16);
          o[T] = __builtin_amdgcn_mfma_f32_32x32x16_bf16(f, to_bf16x8(w + 8 * t), o[T], 0, 0, 0);
        }
      }
    }
  };
  // bf16, where some value is infinite or NaN and not every column sees every
  // token: the matrix product would carry it, times zero, into columns that do
  // not see it.  Token by token instead, each column adding those it sees, its
  // probabilities laid out in the place of stage u-1 (its keys' first, then its
  // values': 2 KB a wave) and its sums in memory meanwhile: this part is kept
  // short, not fast.
  auto odd_values = [&](int u) Q8_INLINE {
    static_assert(W * 2048 <= 2 * kVal, "a wave's probabilities");
    constexpr int kInKeys = kVal / 2048;      // waves whose piece is in the keys' place
    char *const scratch = lds + slot(u - 1) * kVal + (wave < kInKeys ? wave : wave - kInKeys) * 2048;
    uint16_t *mine = reinterpret_cast<uint16_t *>(scratch + (wave < kInKeys ? 0 : SL * kVal));
    const int half = here(hf), at = here(col);
    float sums[NB * 16];
#pragma unroll
    for (int T = 0; T < NB; ++T)
#pragma unroll
      for (int e = 0; e < 16; ++e) sums[T * 16 + e] = o[T][e];
#pragma unroll
    for (int n = 0; n < NS; ++n) {
      const unsigned seen = seen_keys(u, n);
      float p[16];
      exponentials(n, p);
#pragma unroll
      for (int e = 0; e < 16; ++e)
        mine[(16 * (e >> 3) + 8 * half + (e & 7)) * 32 + at] =
            seen >> e & 1 ? __builtin_bit_cast(uint16_t, (__bf16)p[e]) : 0xffffu;
      const uint16_t *vp = reinterpret_cast<const uint16_t *>(vals + slot(u) * kVal) + 4 * n * D * 8;
#pragma unroll 1
      for (int k = 0; k < 32; ++k) {
        const uint16_t bits = mine[k * 32 + at];
        const float pk = __uint_as_float((uint32_t)bits << 16);
        if (bits == 0xffffu) continue;
#pragma unroll 1
        for (int i = 0; i < NB * 16; ++i) {
          const int d = 32 * (i >> 4) + 8 * ((i >> 2) & 3) + 4 * half + (i & 3);
          const float v = __uint_as_float((uint32_t)vp[((k >> 3) * D + d) * 8 + (k & 7)] << 16);
          sums[i] = fmaf(pk, v, sums[i]);
        }
      }
    }
#pragma unroll
    for (int T = 0; T < NB; ++T)
#pragma unroll
      for (int e = 0; e < 16; ++e) o[T][e] = sums[T * 16 + e];
  };

  // Stages from .. to-1 one after the other.
  auto in_step = [&](int from, int to) Q8_INLINE {
    int u = from;
    bool all = false, odd = false;
    auto first = [&]() Q8_INLINE {         // stage u's scores
      all = whole(u);
      if constexpr (FMT == Q8_KV_BF16) {
        if (u + SL - 1 <= to) loads_done<(SL - 2) * 2 * kIt>(); else loads_done<0>();
        __syncthreads();       // the stage is there, and the one before has been used
        odd = false;
        if (!all) odd = __syncthreads_or(clean(u));
        if (!odd && u + SL - 1 < to) issue(u + SL - 1);
        scores_bf16(u);
      } else {
        fetch(min(u + 1, to - 1));
        scores_q8(u);
      }
      if (!all) hide(u);
    };
    auto second = [&]() Q8_INLINE {        // its probabilities and values
      if constexpr (FMT == Q8_KV_BF16) {
        if (odd) {
          odd_values(u);
          __syncthreads();
          if (u + SL - 1 < to) issue(u + SL - 1);
        } else {
          soften();
          add_values(u);
        }
      } else {
        add_values_q8(u, all);
        widen(u + 1);
        __syncthreads();
      }
      ++u;
    };
    if constexpr (FMT == Q8_KV_BF16) {
      for (int v = from; v < min(from + SL - 1, to); ++v) issue(v);
    } else {
      fetch(from);
      widen(from);
      __syncthreads();
    }
    while (u < to) {
      float mx;
      if constexpr (kTurns) {  // few stages, those that in_turns leaves: short code
        first();
        mx = largest();
        if (passes(mx)) raise(mx);
        second();
      } else {
        for (;;) {
          first();
          mx = largest();
          if (passes(mx)) break;
          second();
          if (u == to) break;
        }
        if (u == to) break;
        raise(mx);
        second();
      }
    }
    __syncthreads();           // the last stage has been used
  };
  // Stages from .. to-1, all whole, the two halves of the waves in turns: a
  // wave's turns are (values of u-1, scores of u) and (probabilities of u), a
  // barrier after each, and the second half starts one turn later.  A wave waits
  // for its share of stage u+1 at the end of its first turn with u: one turn
  // before any wave reads it.  When a wave takes its second turn with u the
  // stages up to u-2 have been used, so u-2+SL may be loaded in the place of u-2.
  auto in_turns = [&](int from, int to) Q8_INLINE {
    static_assert(FMT != Q8_KV_BF16 || SL == 4, "two stages ahead");
    int u = from;
    Source next;
    auto loaded = [&]() Q8_INLINE {
      __builtin_amdgcn_sched_barrier(0);
      loads_done<0>();
      turn();
      if (u + 2 < to) issue_from(next, u + 2);
      __builtin_amdgcn_sched_barrier(0);
    };
    auto second = [&]() Q8_INLINE {
      next = source(min(u + 3, to - 1));
      soften();
      turn();
      ++u;
    };
    issue(from);
    loads_done<0>();
    if (from + 1 < to) issue(from + 1);
    next = source(min(from + 2, to - 1));
    turn();
    if (wave >= W / 2) turn();
    scores_bf16(u);
    loaded();
    raise(largest());
    second();
    while (u < to) {
      float mx;
      for (;;) {
        multiply(First{}, End{}, vfrag + slot(u - 1) * kVal, kfrag + slot(u) * kVal);
        loaded();
        mx = largest();
        if (passes(mx)) break;
        second();
        if (u == to) break;
      }
      if (u == to) break;
      raise(mx);
      second();
    }
    add_values(to - 1);
    if (wave < W / 2) turn();
    __syncthreads();
  };

  // The stages after the kept first tokens' that every column sees whole (while
  // all their pages are pages): of the last KT tokens' stages those up to p0,
  // and under a window those past where p1's begins.
  const int edge = a.window > 0 ? max((p1 - a.window + KT) / KT, 0) : 0;
  const int whole0 = sp.a + max(edge - sp.t0, 0), whole1 = sp.a - sp.t0 + (p0 + 1) / KT;
  for (; base < u1; base += kListStages) {
    const int end = min(base + kListStages, u1);
    bool lost = false;
    for (int g = threadIdx.x; g < (end - base) * (KT / 16); g += kThreads) {
      const int key = sp.tile(base + g / (KT / 16)) * KT + g % (KT / 16) * 16;
      const int p = trow[min(key, last) >> pl];
      const bool ok = (unsigned)p < (unsigned)c.n_pages;
      pids[g] = ok ? p : -1;
      lost |= !ok;
    }
    lost = __syncthreads_or(lost);
    if constexpr (kTurns) {
      int w0 = min(max(whole0, base), end), w1 = min(max(whole1, w0), end);
      if (lost || w1 - w0 < 3) w0 = w1 = base;
      if (base < w0) in_step(base, w0);
      if (w0 < w1) in_turns(w0, w1);
      if (w1 < end) in_step(w1, end);
    } else {
      in_step(base, end);
    }
  }
  l += swap_halves(l);

  const int units = c.heads, unit = hk;
  constexpr int rec = record_floats(kBlock, D);
  if (S > 1) {
    // this split's sums to the workspace, lane by lane; the last to arrive
    // joins the splits in order
    float *mine = a.partial + ((size_t)(bx * units + unit) * gridDim.y + s) * rec;
    const buf_t out = make_buf(mine, rec * 4);
#pragma unroll
    for (int T = 0; T < NB; ++T)
#pragma unroll
      for (int h = 0; h < 4; ++h)
        buf_st16_sys(out, (((wave * NB + T) * 4 + h) * 64 + lane) * 16,
                     make_float4(o[T][4 * h], o[T][4 * h + 1], o[T][4 * h + 2], o[T][4 * h + 3]));
    const int mat = (kBlock * D + wave * 32 + col) * 4;
    if (hf == 0) {
      __builtin_amdgcn_raw_buffer_store_b32(__float_as_uint(m), out, mat, 0, kBufSys);
      __builtin_amdgcn_raw_buffer_store_b32(__float_as_uint(l), out, mat + kBlock * 4, 0, kBufSys);
    }
    stores_done();
    __syncthreads();
    unsigned *cnt = a.counters + (size_t)bx * units + unit;
    if (threadIdx.x == 0)
      is_last = __hip_atomic_fetch_add(cnt, 1u, __ATOMIC_RELAXED, __HIP_MEMORY_SCOPE_SYSTEM) ==
                (unsigned)(S - 1);
    __syncthreads();
    if (!is_last) return;
    const float *parts = a.partial + (size_t)(bx * units + unit) * gridDim.y * rec;
    const buf_t in = make_buf(parts, (unsigned)((size_t)S * rec * 4));
    m = kLowest;
    for (int r = 0; r < S; ++r)
      m = fmaxf(m, __uint_as_float(__builtin_amdgcn_raw_buffer_load_b32(in, r * rec * 4 + mat, 0, kBufSys)));
    l = 0.0f;
#pragma unroll
    for (int T = 0; T < NB; ++T)
#pragma unroll
      for (int e = 0; e < 16; ++e) o[T][e] = 0.0f;
    for (int r = 0; r < S; ++r) {
      const int rb = r * rec * 4;
      const float rm = __uint_as_float(__builtin_amdgcn_raw_buffer_load_b32(in, rb + mat, 0, kBufSys));
      const float rl = __uint_as_float(__builtin_amdgcn_raw_buffer_load_b32(in, rb + mat + kBlock * 4, 0, kBufSys));
      const float f = exp2_fast(rm - m);
      l += rl * f;
#pragma unroll
      for (int T = 0; T < NB; ++T)
#pragma unroll
        for (int h = 0; h < 4; ++h) {
          const float4 y = buf_ld16_sys(in, rb + (((wave * NB + T) * 4 + h) * 64 + lane) * 16);
          o[T][4 * h] += y.x * f;
          o[T][4 * h + 1] += y.y * f;
          o[T][4 * h + 2] += y.z * f;
          o[T][4 * h + 3] += y.w * f;
        }
    }
    if (threadIdx.x == 0)
      __hip_atomic_store(cnt, 0u, __ATOMIC_RELAXED, __HIP_MEMORY_SCOPE_SYSTEM);
  }

  // divide and write: 64 dims of the wave's columns at a time through LDS, so
  // that eight lanes hold a column's 32-value block
  const float inv = l == 0.0f ? 0.0f : 1.0f / l;
  constexpr int kRowF = kOutRow;
  float *mylds = reinterpret_cast<float *>(lds) + wave * 32 * kRowF;
#pragma unroll
  for (int T2 = 0; T2 < NB; T2 += 2) {
#pragma unroll
    for (int T = T2; T < T2 + 2; ++T)
#pragma unroll
      for (int h = 0; h < 4; ++h)
        *reinterpret_cast<float4 *>(mylds + col * kRowF + 32 * (T - T2) + 8 * h + 4 * hf) = make_float4(
            o[T][4 * h] * inv, o[T][4 * h + 1] * inv, o[T][4 * h + 2] * inv, o[T][4 * h + 3] * inv);
    __builtin_amdgcn_wave_barrier();
#pragma unroll 1
    for (int h = 0; h < 8; ++h) {
      const int cc = h * 4 + (lane >> 4), d = (lane & 15) * 4;
      const int mc = c0 + wave * 32 + cc;
      const float4 y = *reinterpret_cast<const float4 *>(mylds + cc * kRowF + d);
      if (mc < ncol)
        store_out(a, start + mc / a.group, (hk * a.group + mc % a.group) * D + 32 * T2 + d, y);
    }
    __builtin_amdgcn_wave_barrier();
  }
}

template <int D, int FMT>
hipError_t launch(const AttnArgs &a, hipStream_t stream) {
  constexpr int out = kWaves<D, FMT> * 32 * kOutRow * 4;
  constexpr int stages = 2 * kSlots<FMT> * (kValBytes<D> + kScaleBytes<D, FMT>);
  constexpr int lds = stages > out ? stages : out;
  if (lds > 48 * 1024) {
    const hipError_t e =
        hipFuncSetAttribute(reinterpret_cast<const void *>(attn_rows_kernel<D, FMT>),
                            hipFuncAttributeMaxDynamicSharedMemorySize, lds);
    if (e != hipSuccess) return e;
  }
  const unsigned blocks =
      (unsigned)((a.m * (int64_t)a.group + kCols<D, FMT> - 1) / kCols<D, FMT> + a.n);
  attn_rows_kernel<D, FMT><<<dim3(a.cache.heads * blocks, a.chunks), 64 * kWaves<D, FMT>, lds, stream>>>(a);
  return hipGetLastError();
}

int cols_of(int64_t dim, int fmt) {
  return fmt == Q8_KV_BF16 && dim < 256 ? kCols<128, Q8_KV_BF16> : kCols<128, Q8_KV_Q8_0>;
}

int64_t blocks_bound(int64_t m, int64_t n, int64_t group, int cols) {
  return (m * group + cols - 1) / cols + n;
}

}  // namespace

// Key splits: as many as keep the workgroups to one a CU (eight waves), two
// (256 dims) or, over Q8_0, six: there each is short of work for its barriers,
// and a CU holds two at a time.  Measured on MI355X (us; half, one, two, three
// times these): 512 rows behind 4096 tokens 97, 54, 67, 67; 256 dims, 2048 rows
// 164, 164, 163, 230, 512 rows behind 3000 181, 151, 186, 220; Q8_0 (a third, two
// thirds, these, twice), 3 x 509 rows behind 4096 171, 177, 153, 161, 2048 rows
// 110, 110, 101, 104.
// The host knows m and n, not the lengths, so the rule counts every sequence's
// last block as one more, and never gives more than kMaxSplits: one sequence of
// few rows gets half of the workgroups it could use, and of many sequences none
// is split, however long.  32 single rows over contexts of 1000 tokens and one
// of 131072 take 2.8 ms, as the long one's tokens pass through eight workgroups
// (of four such rows, 0.49 ms); all of them in q8_attn_decode 0.1 ms.
int attn_rows_splits(int64_t m, int64_t n, int64_t q_heads, int64_t kv_heads, int64_t dim, int fmt) {
  const int cols = cols_of(dim, fmt), target = dim == 256 ? 512 : fmt == Q8_KV_BF16 ? 256 : 1536;
  const int64_t s = target / (blocks_bound(m, n, q_heads / kv_heads, cols) * kv_heads);
  return (int)(s < 1 ? 1 : (s > kMaxSplits ? kMaxSplits : s));
}

size_t attn_rows_partial_bytes(int64_t m, int64_t n, int64_t q_heads, int64_t kv_heads, int64_t dim,
                               int fmt) {
  const int S = attn_rows_splits(m, n, q_heads, kv_heads, dim, fmt);
  if (S == 1) return 0;
  const int cols = cols_of(dim, fmt);
  return (size_t)blocks_bound(m, n, q_heads / kv_heads, cols) * kv_heads * S *
         record_floats(cols, (int)dim) * 4;
}

hipError_t launch_attn_rows(const AttnArgs &a, hipStream_t stream) {
  const bool q = a.cache.fmt == Q8_KV_Q8_0;
  switch (a.cache.dim) {
    case 64: return q ? launch<64, 1>(a, stream) : launch<64, 0>(a, stream);
    case 128: return q ? launch<128, 1>(a, stream) : launch<128, 0>(a, stream);
    default: return q ? launch<256, 1>(a, stream) : launch<256, 0>(a, stream);
  }
}

}  // namespace q8
