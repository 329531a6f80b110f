// q8_attn_rows.hip -- attention of chunks of rows over the paged cache
// (q8_attn_rows; the formula and layouts are in include/q8gemv.h).
#include <hip/hip_runtime.h>

#include <type_traits>

#include "q8_attn.h"

namespace q8 {
namespace {

constexpr int kWaves = 4;
constexpr int kCols = 32 * kWaves;      // (row, query head) columns of a workgroup
constexpr int kTargetWorkgroups = 512;
constexpr int kMaxSplits = 16;
constexpr int kMinSplitTiles = 8;       // fewest tiles of a split that computes

typedef __attribute__((ext_vector_type(16))) float f32x16_t;

// Keys of a stage: what the workgroup loads, and waits for, at a time.
#ifndef SPV
#define SPV 0
#endif
#if SPV == 0
#define SCHED_PV ;
#elif SPV == 1
#define SCHED_PV read_ahead<NS * NB * 2, 4>();
#else
#define SCHED_PV interleave<NS, NB>();
#endif
#ifndef KTB
#define KTB 64
#define OCC 2
#endif
template <int D, int FMT> constexpr int kStageKeys = D == 256 ? 32 : (FMT == Q8_KV_BF16 ? KTB : 64);
constexpr int kListGroups = 512;        // 16-token groups whose pages are held in LDS at a time

// LDS bytes of one stage: keys and values as bf16 (Q8_0: the codes, exact),
// and their scales.
template <int D, int FMT>
constexpr int stage_bytes() {
  return kStageKeys<D, FMT> * (2 * D * 2 + (FMT == Q8_KV_Q8_0 ? 2 * (D / 32) * 4 : 0));
}

struct Block {
  int i;         // sequence
  int block;     // its block of columns
  int total;     // blocks of all sequences
};

__device__ __forceinline__ int rows_of(const AttnArgs &a, int i, int *start) {
  const int s = min(max(a.row_start[i], 0), a.m), e = min(max(a.row_start[i + 1], 0), a.m);
  *start = s;
  return max(e - s, 0);
}

// Block x of all sequences' blocks (i = n past the last).  A wave takes 64
// sequences at a time; every wave finds the same.
__device__ __forceinline__ Block find_block(const AttnArgs &a, int x) {
  const int lane = threadIdx.x & 63;
  Block r{a.n, 0, 0};
  int base = 0;
  for (int b = 0; b < a.n; b += 64) {
    int start;
    const int i = b + lane;
    int incl = i < a.n ? (rows_of(a, i, &start) * a.group + kCols - 1) / kCols : 0;
#pragma unroll
    for (int o = 1; o < 64; o <<= 1) {
      const int u = __shfl_up(incl, o);
      if (lane >= o) incl += u;
    }
    incl += base;
    const int before = __popcll(__ballot(incl <= x));
    if (before < 64 && r.i == a.n) {
      r.i = b + before;
      r.block = x - (before > 0 ? __shfl(incl, before - 1) : base);
      return r;
    }
    base = __shfl(incl, 63);
  }
  return r;
}

// Schedules a block of N fragment reads and N matrix products: `ahead` reads
// first, then one more with each product.
template <int N, int AHEAD>
__device__ __forceinline__ void read_ahead() {
  __builtin_amdgcn_sched_group_barrier(0x100, AHEAD, 0);
#pragma unroll
  for (int i = 0; i < N - AHEAD; ++i) {
    __builtin_amdgcn_sched_group_barrier(0x8, 1, 0);
    __builtin_amdgcn_sched_group_barrier(0x100, 1, 0);
  }
  __builtin_amdgcn_sched_group_barrier(0x8, AHEAD, 0);
}

template <int NS, int NB>
__device__ __forceinline__ void interleave() {
  __builtin_amdgcn_sched_group_barrier(0x100, 4, 0);
  __builtin_amdgcn_sched_group_barrier(0x2, 56, 0);
#pragma unroll
  for (int i = 0; i < NS * NB * 2; ++i) {
    __builtin_amdgcn_sched_group_barrier(0x8, 1, 0);
    if (i < NS * NB * 2 - 4) __builtin_amdgcn_sched_group_barrier(0x100, 1, 0);
    if (i < (NS - 1) * NB * 2) __builtin_amdgcn_sched_group_barrier(0x2, 56 / (NB * 2), 0);
  }
}

__device__ __forceinline__ float swap_halves(float x) {   // lane l's value in lane l ^ 32
  return __shfl_xor(x, 32);
}

// Whether any of eight bf16 values is infinite or NaN (exponent all ones).
__device__ __forceinline__ bool not_finite(u32x4_t v) {
  uint32_t odd = 0;
#pragma unroll
  for (int e = 0; e < 4; ++e) odd |= (v[e] & 0x7fff7fffu) + 0x00800080u;
  return (odd & 0x80008000u) != 0;
}

// 16 bytes a lane from memory into LDS at `at` (a scalar) plus 16 times the
// lane, without registers in between; loads_done waits for them.  They are
// written out because the compiler would make every read of LDS wait for every
// such load, the next stage's too.
__device__ __forceinline__ void load_to_lds(const void *p, unsigned at) {
  asm volatile("s_mov_b32 m0, %1\n\ts_nop 0\n\tglobal_load_lds_dwordx4 %0, off"
               :: "v"(p), "s"(at) : "memory");
}
__device__ __forceinline__ void loads_done() { asm volatile("s_waitcnt vmcnt(0)" ::: "memory"); }

__host__ __device__ constexpr int record_floats(int dim) { return kCols * dim + 2 * kCols; }

// Grid: (blocks of columns x key/value heads, the heads fastest -- eight of
// them put a head's keys in one XCD's L2 --, key splits).  A column is one
// (row, query head of the group) pair, so the group's heads share the keys;
// a wave holds 32 columns, the workgroup's waves share the staged keys and
// values in LDS (two stages; the next one's loads are in flight, in registers,
// while this one is computed).  Scores are transposed (32 keys x 32 columns,
// v_mfma 32x32x16): a lane's sixteen scores belong to one column, and with the
// key fragments' rows permuted (row 8a + 4h + e is key 16 (a/2) + 8h + 4 (a%2) +
// e) they are, eight by eight, the value product's operand, so probabilities
// stay in their lane, and the running maximum is a lane's own scalar.  That
// maximum is only raised when a score passes it by 2^8 (kSlack): sums stay far
// inside fp32, and the sums O^T are rescaled once or twice a block instead of
// at nearly every stage.
constexpr float kSlack = 8.0f;

template <int D, int FMT>
__global__ void __launch_bounds__(64 * kWaves, D == 256 ? 1 : FMT == Q8_KV_BF16 ? OCC : 2)
attn_rows_kernel(AttnArgs a) {
  constexpr int NB = D / 32, NK = D / 16, KT = kStageKeys<D, FMT>, NS = KT / 32;
  constexpr int kThreads = 64 * kWaves;
  constexpr int kStage = stage_bytes<D, FMT>();
  constexpr int kVal = KT * D * 2;                         // bytes of the staged keys
  constexpr int kElem = FMT == Q8_KV_BF16 ? 16 : 8;        // bytes of eight cached values
  constexpr int kPer = 16 / kElem;                         // eights in a 16-byte piece
  constexpr int kIt = KT * D / 8 / kPer / kThreads;        // a thread's pieces of the keys
  static_assert(kIt * kThreads * kPer * 8 == KT * D, "pieces");
  constexpr int kScales = KT * NB;                         // scales of the keys
  constexpr int kSIt = (kScales + kThreads - 1) / kThreads;
  static_assert(kScales % kThreads == 0 || kSIt == 1, "scales");
  extern __shared__ __align__(16) char lds[];
  __shared__ int pids[kListGroups];
  __shared__ int is_last;
  const int lane = threadIdx.x & 63, wave = uni(threadIdx.x >> 6);
  const int col = lane & 31, hf = lane >> 5;
  const KvCache c = a.cache;
  const int hk = blockIdx.x % c.heads, bx = blockIdx.x / c.heads;
  const int pl = c.page_log2, P = 1 << pl;

  Block bl = find_block(a, bx);
  bl.i = uni(bl.i);
  bl.block = uni(bl.block);
  if (bl.i >= a.n) return;
  int start;
  const int R = uni(rows_of(a, bl.i, &start));
  start = uni(start);
  const int len = uni(clamp_len(a.lens[bl.i], a.max_pages, pl));
  const int ncol = R * a.group;
  // heaviest first: the sequence's last rows see the most tokens
  const int blocks = (ncol + kCols - 1) / kCols;
  const int blk = blocks - 1 - bl.block;
  const int c0 = blk * kCols, c1 = min(c0 + kCols, ncol) - 1;
  const int p0 = len - R + c0 / a.group, p1 = len - R + c1 / a.group;
  const Span sp = span_of<KT>(max(p0, 0), p1, a.window, a.sinks);
  const int S = min((int)gridDim.y, max(sp.nt / kMinSplitTiles, 1));
  const int s = blockIdx.y;
  if (s >= S) return;
  const int u0 = (int)((long long)sp.nt * s / S), u1 = (int)((long long)sp.nt * (s + 1) / S);

  const int mycol = c0 + wave * 32 + col;
  const bool live = mycol < ncol;
  const int j = min(mycol, ncol - 1) / a.group, head = hk * a.group + min(mycol, ncol - 1) % a.group;
  const int pos = len - R + j, row = start + j;

  // The scale is used as a positive one (so that the largest score stays the
  // largest, and an unseen key's -infinity is one): its sign goes into the
  // queries, and a scale of zero makes them zero.
  const float scale = a.scale_log2 == 0.0f ? 1.0f : fabsf(a.scale_log2);
  const uint32_t flip = a.scale_log2 < 0.0f ? 0x80008000u : 0u;
  const uint32_t keep = a.scale_log2 == 0.0f ? 0u : 0xffffffffu;
  bf16x8_t q[NK];
#pragma unroll
  for (int k = 0; k < NK; ++k) {
    uint4 v = make_uint4(0u, 0u, 0u, 0u);
    if (live)
      v = *reinterpret_cast<const uint4 *>(a.q + ((size_t)row * a.q_heads + head) * D + 16 * k + 8 * hf);
    v.x = (v.x ^ flip) & keep;
    v.y = (v.y ^ flip) & keep;
    v.z = (v.z ^ flip) & keep;
    v.w = (v.w ^ flip) & keep;
    q[k] = __builtin_bit_cast(bf16x8_t, v);
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

  // A stage's 16-byte pieces, thread by thread.  Keys lie as [D/8][KT][8],
  // values as [KT/8][D][8], in the cache's pages and in LDS; a piece is one
  // eight of bf16 values or two of int8 codes.  All of a thread's key pieces are
  // of one key (or pair); a wave's 64 value pieces follow each other within 16
  // tokens, so their page is a scalar.
  static_assert(kThreads * kPer % KT == 0 && (64 * kPer <= D || 64 * kPer % D == 0), "pieces");
  const int tkey = (int)threadIdx.x * kPer % KT, tch = (int)threadIdx.x * kPer / KT;
  auto key_piece = [&](int u, int base) {
    const int *ids = pids + (u - base) * (KT / 16);
    return c.k + (size_t)max(ids[tkey / 16], 0) * page_bytes + head_off +
           (tch * P + ((sp.tile(u) * KT + tkey) & (P - 1))) * kElem;
  };
  const int key_step = kThreads * kPer / KT * P * kElem;
  auto value_piece = [&](int u, int base, int it) {
    const int *ids = pids + (u - base) * (KT / 16);
    const int e = (wave * 64 + it * kThreads) * kPer, vc = e / D;
    return c.v + (size_t)max(uni(ids[vc / 2]), 0) * page_bytes + head_off +
           ((((sp.tile(u) * KT + 8 * vc) & (P - 1)) >> 3) * D + e % D) * kElem + lane * 16;
  };
  // bf16: straight into LDS.
  const unsigned lds0 = (unsigned)(size_t)(__attribute__((address_space(3))) char *)lds + wave * 1024;
  auto issue = [&](int u, int base, int buf) {
    const char *kp = key_piece(u, base);
#pragma unroll
    for (int it = 0; it < kIt; ++it) {
      load_to_lds(kp, lds0 + buf * kStage + it * kThreads * 16);
      kp += key_step;
    }
#pragma unroll
    for (int it = 0; it < kIt; ++it)
      load_to_lds(value_piece(u, base, it), lds0 + buf * kStage + kVal + it * kThreads * 16);
  };
  // Q8_0: through registers, where the codes are widened.
  u32x4_t rk[kIt], rv[kIt];
  float rks[kSIt], rvs[kSIt];
  const int skey = (int)threadIdx.x % KT, sblk = (int)threadIdx.x / KT;
  auto fetch = [&](int u, int base) {
    const char *kp = key_piece(u, base);
#pragma unroll
    for (int it = 0; it < kIt; ++it) {
      rk[it] = *reinterpret_cast<const u32x4_t *>(kp);
      kp += key_step;
    }
#pragma unroll
    for (int it = 0; it < kIt; ++it)
      rv[it] = *reinterpret_cast<const u32x4_t *>(value_piece(u, base, it));
    const int *ids = pids + (u - base) * (KT / 16);
    const size_t at = (size_t)max(ids[skey / 16], 0) * page_bytes + head_off + (size_t)D * P +
                      (min(sblk, NB - 1) * P + ((sp.tile(u) * KT + skey) & (P - 1))) * 4;
#pragma unroll
    for (int it = 0; it < kSIt; ++it) {
      rks[it] = *reinterpret_cast<const float *>(c.k + at + it * (kThreads / KT) * P * 4);
      rvs[it] = *reinterpret_cast<const float *>(c.v + at + it * (kThreads / KT) * P * 4);
    }
  };
  auto stage = [&](char *st) {
#pragma unroll
    for (int it = 0; it < kIt; ++it) {
      char *d = st + ((int)threadIdx.x + it * kThreads) * kPer * 16;
      *reinterpret_cast<bf16x8_t *>(d) = i8x8_to_bf16(make_uint2(rk[it][0], rk[it][1]));
      *reinterpret_cast<bf16x8_t *>(d + 16) = i8x8_to_bf16(make_uint2(rk[it][2], rk[it][3]));
      *reinterpret_cast<bf16x8_t *>(d + kVal) = i8x8_to_bf16(make_uint2(rv[it][0], rv[it][1]));
      *reinterpret_cast<bf16x8_t *>(d + kVal + 16) = i8x8_to_bf16(make_uint2(rv[it][2], rv[it][3]));
    }
    float *sc = reinterpret_cast<float *>(st + 2 * kVal);
#pragma unroll
    for (int it = 0; it < kSIt; ++it) {
      const int p = (int)threadIdx.x + it * kThreads;
      if (kScales % kThreads == 0 || p < kScales) {
        sc[p] = rks[it];
        sc[kScales + p] = rvs[it];
      }
    }
  };
  // Whether every column sees all of stage u.
  auto whole = [&](int u, int base) {
    const int key0 = sp.tile(u) * KT;
    const int *ids = pids + (u - base) * (KT / 16);
    int pages = ids[0];
#pragma unroll
    for (int g = 1; g < KT / 16; ++g) pages |= ids[g];
    return (key0 + KT - 1 <= p0) & (uni(pages) >= 0) &
           ((a.window <= 0) | (key0 > p1 - a.window) | (key0 + KT <= a.sinks));
  };
  // bf16, a stage that is not whole: the thread's pieces of values of tokens
  // past the sequence or on no page, whose bytes may be anything, become zero.
  // Returns whether a value of the others is infinite or NaN.
  auto clean = [&](char *st, int u, int base) {
    bool odd = false;
#pragma unroll
    for (int it = 0; it < kIt; ++it) {
      const int piece = here(threadIdx.x) + it * kThreads, vc = piece / D;
      const int left = pids[(u - base) * (KT / 16) + vc / 2] < 0 ? 0 : len - sp.tile(u) * KT - 8 * vc;
      u32x4_t *p = reinterpret_cast<u32x4_t *>(st + kVal + piece * 16);
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

  // One stage.  ODD (bf16): some value is infinite or NaN and not every column
  // sees every token.
  auto compute = [&](auto ODD, const char *st, int u, int base, bool all, char *scratch) {
    const int key0 = sp.tile(u) * KT;
    const char *kb = st + (hf * KT + fkey) * 16, *vb = st + kVal + (hf * D + col) * 16;
    const float *ksc = reinterpret_cast<const float *>(st + 2 * kVal) + 8 * hf, *vsc = ksc + kScales;
    f32x16_t x[NS];
#pragma unroll
    for (int n = 0; n < NS; ++n)
#pragma unroll
      for (int e = 0; e < 16; ++e) x[n][e] = 0.0f;
    if constexpr (FMT == Q8_KV_BF16) {
#pragma unroll
      for (int k = 0; k < NK; ++k)
#pragma unroll
        for (int n = 0; n < NS; ++n) {
          const bf16x8_t f = *reinterpret_cast<const bf16x8_t *>(kb + (2 * k * KT + 32 * n) * 16);
          x[n] = __builtin_amdgcn_mfma_f32_32x32x16_bf16(f, q[k], x[n], 0, 0, 0);
        }
      read_ahead<NK * NS, 4>();
    } else {
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
          for (int g = 0; g < 4; ++g) {
            const float4 w = *reinterpret_cast<const float4 *>(ksc + b * KT + 32 * n + 16 * (g >> 1) + 4 * (g & 1));
            x[n][4 * g] = fmaf(w.x, z[4 * g], x[n][4 * g]);
            x[n][4 * g + 1] = fmaf(w.y, z[4 * g + 1], x[n][4 * g + 1]);
            x[n][4 * g + 2] = fmaf(w.z, z[4 * g + 2], x[n][4 * g + 2]);
            x[n][4 * g + 3] = fmaf(w.w, z[4 * g + 3], x[n][4 * g + 3]);
          }
        }
    }
    // seen[n] bit e: key 32n + 16 (e/8) + 8 hf + e%8 is
    unsigned seen[NS];
#pragma unroll
    for (int n = 0; n < NS; ++n) seen[n] = 0xffffu;
    if (!all) {
      const int *ids = pids + (u - base) * (KT / 16);
      const int h8 = here(8 * hf), me = here(pos), from = a.window > 0 ? me - a.window + 1 : 0;
#pragma unroll
      for (int n = 0; n < NS; ++n) {
        seen[n] = 0;
#pragma unroll
        for (int e = 0; e < 16; ++e) {
          const int key = key0 + 32 * n + 16 * (e >> 3) + h8 + (e & 7);
          const int stop = ids[2 * n + (e >> 3)] >= 0 ? min(me, len - 1) : -1;
          const bool in = (key <= stop) & ((key >= from) | (key < a.sinks));
          seen[n] |= in ? 1u << e : 0u;
          x[n][e] = in ? x[n][e] : -__builtin_inff();
        }
      }
    }
    float mx = x[0][0];
#pragma unroll
    for (int n = 0; n < NS; ++n)
#pragma unroll
      for (int e = 0; e < 16; ++e) mx = fmaxf(mx, x[n][e]);
    mx = fmaxf(mx, swap_halves(mx)) * scale;
    if (__any(mx > m + kSlack)) {
      const float mn = fmaxf(m, mx);
      const float alpha = exp2_fast(m - mn);
      m = mn;
      l *= alpha;
#pragma unroll
      for (int T = 0; T < NB; ++T) o[T] *= alpha;
    }
    float ps[4] = {0.0f, 0.0f, 0.0f, 0.0f};
    if constexpr (ODD) {
      // The matrix product would carry such a value, times zero, into columns
      // that do not see it.  Token by token instead, each column adding those
      // it sees.
      uint16_t *mine = reinterpret_cast<uint16_t *>(scratch) + wave * KT * 32;
      const int half = here(hf), at = here(col);
#pragma unroll
      for (int n = 0; n < NS; ++n)
#pragma unroll
        for (int e = 0; e < 16; ++e) {
          const float p = exp2_fast(fmaf(x[n][e], scale, -m));
          ps[e & 3] += p;
          mine[(32 * n + 16 * (e >> 3) + 8 * half + (e & 7)) * 32 + at] =
              seen[n] >> e & 1 ? __builtin_bit_cast(uint16_t, (__bf16)p) : 0xffffu;
        }
      __syncthreads();
      const uint16_t *vals = reinterpret_cast<const uint16_t *>(st + kVal);
#pragma unroll 1
      for (int k = 0; k < KT; ++k) {
        const uint16_t bits = mine[k * 32 + at];
        const float p = __uint_as_float((uint32_t)bits << 16);
#pragma unroll
        for (int T = 0; T < NB; ++T) {
#pragma unroll
          for (int e = 0; e < 16; ++e) {
            const int d = 32 * T + 8 * (e >> 2) + 4 * half + (e & 3);
            const float v = __uint_as_float((uint32_t)vals[((k >> 3) * D + d) * 8 + (k & 7)] << 16);
            o[T][e] = bits != 0xffffu ? fmaf(p, v, o[T][e]) : o[T][e];
          }
          __builtin_amdgcn_sched_barrier(0);
        }
      }
      __syncthreads();
    } else {
#pragma unroll
      for (int n = 0; n < NS; ++n) {
        float p[16];
#pragma unroll
        for (int e = 0; e < 16; ++e) {
          p[e] = exp2_fast(fmaf(x[n][e], scale, -m));
          ps[e & 3] += p[e];
        }
        if constexpr (FMT == Q8_KV_BF16) {
          const bf16x8_t pb[2] = {to_bf16x8(p), to_bf16x8(p + 8)};
#pragma unroll
          for (int t = 0; t < 2; ++t)
#pragma unroll
            for (int T = 0; T < NB; ++T) {
              const bf16x8_t f = *reinterpret_cast<const bf16x8_t *>(vb + ((4 * n + 2 * t) * D + 32 * T) * 16);
              o[T] = __builtin_amdgcn_mfma_f32_32x32x16_bf16(f, pb[t], o[T], 0, 0, 0);
            }
        } else {
#pragma unroll
          for (int T = 0; T < NB; ++T) {
            float w[16];
#pragma unroll
            for (int g = 0; g < 4; ++g) {
              const float4 s4 = *reinterpret_cast<const float4 *>(vsc + T * KT + 32 * n + 16 * (g >> 1) + 4 * (g & 1));
              w[4 * g] = p[4 * g] * s4.x;
              w[4 * g + 1] = p[4 * g + 1] * s4.y;
              w[4 * g + 2] = p[4 * g + 2] * s4.z;
              w[4 * g + 3] = p[4 * g + 3] * s4.w;
            }
            if (!all) {                  // an unseen token's scale may be anything
#pragma unroll
              for (int e = 0; e < 16; ++e) w[e] = seen[n] >> e & 1 ? w[e] : 0.0f;
            }
#pragma unroll
            for (int t = 0; t < 2; ++t) {
              const bf16x8_t f = *reinterpret_cast<const bf16x8_t *>(vb + ((4 * n + 2 * t) * D + 32 * T) * 16);
              o[T] = __builtin_amdgcn_mfma_f32_32x32x16_bf16(f, to_bf16x8(w + 8 * t), o[T], 0, 0, 0);
            }
          }
        }
      }
      if constexpr (FMT == Q8_KV_BF16) SCHED_PV
    }
    l += (ps[0] + ps[1]) + (ps[2] + ps[3]);
  };

  constexpr int kListStages = kListGroups / (KT / 16);
  for (int base = u0; base < u1; base += kListStages) {
    const int end = min(base + kListStages, u1);
    __syncthreads();                       // the last list is read
    for (int g = threadIdx.x; g < (end - base) * (KT / 16); g += kThreads) {
      const int key = sp.tile(base + g / (KT / 16)) * KT + g % (KT / 16) * 16;
      const int p = trow[min(key, last) >> pl];
      pids[g] = (unsigned)p < (unsigned)c.n_pages ? p : -1;
    }
    __syncthreads();
    if constexpr (FMT == Q8_KV_BF16) {
      issue(base, base, 0);
      for (int u = base; u < end; ++u) {
        const int cur = (u - base) & 1;
        char *st = lds + cur * kStage;
        const bool all = whole(u, base);
        loads_done();
        __syncthreads();     // the stage is in LDS, and the last one has been computed
        bool odd = false;
        if (!all) odd = __syncthreads_or(clean(st, u, base));
        if (!odd && u + 1 < end) issue(u + 1, base, cur ^ 1);
        if (!odd) {
          compute(std::false_type{}, st, u, base, all, nullptr);
        } else {
          compute(std::true_type{}, st, u, base, false, lds + (cur ^ 1) * kStage);
          if (u + 1 < end) issue(u + 1, base, cur ^ 1);
        }
      }
    } else {
      fetch(base, base);
      stage(lds);
      __syncthreads();
      for (int u = base; u < end; ++u) {
        const int cur = (u - base) & 1;
        fetch(min(u + 1, end - 1), base);
        compute(std::false_type{}, lds + cur * kStage, u, base, whole(u, base), nullptr);
        stage(lds + (cur ^ 1) * kStage);
        __syncthreads();
      }
    }
  }
  l += __shfl_xor(l, 32);

  const int units = c.heads, unit = hk;
  const int rec = record_floats(D);
  if (S > 1) {
    // this split's sums to the workspace, lane by lane; the last to arrive
    // joins the splits in order
    float *mine = a.partial + ((size_t)(bx * units + unit) * gridDim.y + s) * rec;
    const buf_t out = make_buf(mine, rec * 4);
#pragma unroll
    for (int T = 0; T < NB; ++T)
#pragma unroll
      for (int g = 0; g < 4; ++g)
        buf_st16_sys(out, (((wave * NB + T) * 4 + g) * 64 + lane) * 16,
                     make_float4(o[T][4 * g], o[T][4 * g + 1], o[T][4 * g + 2], o[T][4 * g + 3]));
    if (hf == 0) {
      float *ml = mine + kCols * D;
      __hip_atomic_store(ml + wave * 32 + col, m, __ATOMIC_RELAXED, __HIP_MEMORY_SCOPE_SYSTEM);
      __hip_atomic_store(ml + kCols + wave * 32 + col, l, __ATOMIC_RELAXED, __HIP_MEMORY_SCOPE_SYSTEM);
    }
    stores_done();
    __syncthreads();
    unsigned *cnt = a.counters + (size_t)bx * units + unit;
    if (threadIdx.x == 0)
      is_last = __hip_atomic_fetch_add(cnt, 1u, __ATOMIC_RELAXED, __HIP_MEMORY_SCOPE_SYSTEM) ==
                (unsigned)(S - 1);
    __syncthreads();
    if (!is_last) return;
    const float *base = a.partial + (size_t)(bx * units + unit) * gridDim.y * rec;
    const buf_t in = make_buf(base, (unsigned)((size_t)S * rec * 4));
    m = kLowest;
    for (int g = 0; g < S; ++g) {
      const unsigned at = (unsigned)g * rec * 4 + (kCols * D + wave * 32 + col) * 4;
      m = fmaxf(m, __builtin_bit_cast(float, __builtin_amdgcn_raw_buffer_load_b32(in, at, 0, kBufSys)));
    }
    l = 0.0f;
#pragma unroll
    for (int T = 0; T < NB; ++T)
#pragma unroll
      for (int e = 0; e < 16; ++e) o[T][e] = 0.0f;
    for (int g = 0; g < S; ++g) {
      const unsigned rb = (unsigned)g * rec * 4;
      const unsigned at = rb + (kCols * D + wave * 32 + col) * 4;
      const float gm = __builtin_bit_cast(float, __builtin_amdgcn_raw_buffer_load_b32(in, at, 0, kBufSys));
      const float gl = __builtin_bit_cast(float, __builtin_amdgcn_raw_buffer_load_b32(in, at + kCols * 4, 0, kBufSys));
      const float f = exp2_fast(gm - m);
      l += gl * f;
#pragma unroll
      for (int T = 0; T < NB; ++T)
#pragma unroll
        for (int gg = 0; gg < 4; ++gg) {
          const float4 y = buf_ld16_sys(in, rb + (((wave * NB + T) * 4 + gg) * 64 + lane) * 16);
          o[T][4 * gg] += y.x * f;
          o[T][4 * gg + 1] += y.y * f;
          o[T][4 * gg + 2] += y.z * f;
          o[T][4 * gg + 3] += y.w * f;
        }
    }
    if (threadIdx.x == 0)
      __hip_atomic_store(cnt, 0u, __ATOMIC_RELAXED, __HIP_MEMORY_SCOPE_SYSTEM);
  }

  // divide and write: 32 dims of the wave's columns at a time through LDS, so
  // that eight lanes hold a column's 32-value block
  const float inv = l == 0.0f ? 0.0f : 1.0f / l;
  __syncthreads();
  constexpr int kRowF = 36;
  float *mylds = reinterpret_cast<float *>(lds) + wave * 32 * kRowF;
#pragma unroll
  for (int T = 0; T < NB; ++T) {
#pragma unroll
    for (int g = 0; g < 4; ++g)
      *reinterpret_cast<float4 *>(mylds + col * kRowF + 8 * g + 4 * hf) =
          make_float4(o[T][4 * g] * inv, o[T][4 * g + 1] * inv, o[T][4 * g + 2] * inv, o[T][4 * g + 3] * inv);
    __builtin_amdgcn_wave_barrier();
#pragma unroll
    for (int g = 0; g < 4; ++g) {
      const int cc = g * 8 + (lane >> 3), d = (lane & 7) * 4;
      const int mc = c0 + wave * 32 + cc;
      const float4 y = *reinterpret_cast<const float4 *>(mylds + cc * kRowF + d);
      if (mc < ncol)
        store_out(a, start + mc / a.group, (hk * a.group + mc % a.group) * D + 32 * T + d, y);
    }
    __builtin_amdgcn_wave_barrier();
  }
}

constexpr int lds_bytes(int stage) {
  const int out = kWaves * 32 * 36 * 4;
  return 2 * stage > out ? 2 * stage : out;
}

template <int D, int FMT>
hipError_t launch(const AttnArgs &a, const dim3 &grid, hipStream_t stream) {
  constexpr int lds = lds_bytes(stage_bytes<D, FMT>());
  if (lds > 64 * 1024) {
    hipError_t e = hipFuncSetAttribute(reinterpret_cast<const void *>(attn_rows_kernel<D, FMT>),
                                       hipFuncAttributeMaxDynamicSharedMemorySize, lds);
    if (e != hipSuccess) return e;
  }
  attn_rows_kernel<D, FMT><<<grid, 64 * kWaves, lds, stream>>>(a);
  return hipGetLastError();
}

int64_t blocks_bound(int64_t m, int64_t n, int64_t group) {
  return (m * group + kCols - 1) / kCols + n;
}

}  // namespace

int attn_rows_splits(int64_t m, int64_t n, int64_t q_heads, int64_t kv_heads) {
  const int64_t wgs = blocks_bound(m, n, q_heads / kv_heads) * kv_heads;
  const int64_t s = kTargetWorkgroups / wgs;
  return (int)(s < 1 ? 1 : (s > kMaxSplits ? kMaxSplits : s));
}

size_t attn_rows_partial_bytes(int64_t m, int64_t n, int64_t q_heads, int64_t kv_heads,
                               int64_t dim) {
  const int S = attn_rows_splits(m, n, q_heads, kv_heads);
  if (S == 1) return 0;
  return (size_t)blocks_bound(m, n, q_heads / kv_heads) * kv_heads * S * record_floats((int)dim) * 4;
}

hipError_t launch_attn_rows(const AttnArgs &a, hipStream_t stream) {
  const dim3 grid(a.cache.heads * (unsigned)blocks_bound(a.m, a.n, a.group), a.chunks);
  const bool q = a.cache.fmt == Q8_KV_Q8_0;
  switch (a.cache.dim) {
    case 64: return q ? launch<64, 1>(a, grid, stream) : launch<64, 0>(a, grid, stream);
    case 128: return q ? launch<128, 1>(a, grid, stream) : launch<128, 0>(a, grid, stream);
    default: return q ? launch<256, 1>(a, grid, stream) : launch<256, 0>(a, grid, stream);
  }
}

}  // namespace q8
