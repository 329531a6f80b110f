// q8_attn_rows.hip -- attention of chunks of rows over the paged cache
// (q8_attn_rows; the formula and layouts are in include/q8gemv.h).
#include <hip/hip_runtime.h>

#include "q8_attn.h"

namespace q8 {
namespace {

constexpr int kWaves = 4;
constexpr int kCols = 32 * kWaves;      // (row, query head) columns of a workgroup
constexpr int kTargetWorkgroups = 512;
constexpr int kMaxSplits = 16;
constexpr int kMinSplitTiles = 8;       // fewest tiles of a split that computes

typedef __attribute__((ext_vector_type(16))) float f32x16_t;

// LDS bytes of one stage: a tile of keys and values, and their scales.
template <int D, int FMT>
constexpr int stage_bytes() {
  return FMT == Q8_KV_BF16 ? 2 * kKvTile * D * 2 : 2 * kKvTile * D + 2 * kKvTile * (D / 32) * 4;
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

__host__ __device__ constexpr int record_floats(int dim) { return kCols * dim + 2 * kCols; }

// Grid: (blocks of columns x key/value heads, the heads fastest -- eight of
// them put a head's keys in one XCD's L2 --, key splits).  A column is one
// (row, query head of the group) pair, so the group's heads share the keys;
// a wave holds 32 columns, the workgroup's waves share the tiles in LDS.
// Scores are transposed (32 keys x 32 columns, v_mfma 32x32x16): a lane's
// sixteen scores belong to one column, and with the key fragments' rows
// permuted (row 8a + 4h + e is key 16 (a/2) + 8h + 4 (a%2) + e) they are, eight
// by eight, the value product's operand, so probabilities stay in their lane.
template <int D, int FMT>
__global__ void __launch_bounds__(64 * kWaves)
attn_rows_kernel(AttnArgs a) {
  constexpr int NB = D / 32, NK = D / 16;
  constexpr int kStage = stage_bytes<D, FMT>();
  constexpr int kValBytes = FMT == Q8_KV_BF16 ? kKvTile * D * 2 : kKvTile * D;
  constexpr int kElem = FMT == Q8_KV_BF16 ? 16 : 8;       // bytes of eight values
  constexpr int kPieces = kValBytes / 16;                  // 16-byte pieces of K (and of V)
  constexpr int kPer = kPieces / (64 * kWaves);            // a thread's
  static_assert(kPieces % (64 * kWaves) == 0 || kPieces < 64 * kWaves, "pieces");
  constexpr int kIt = kPer > 0 ? kPer : 1;
  extern __shared__ __align__(16) char lds[];
  __shared__ int is_last;
  const int lane = threadIdx.x & 63, wave = threadIdx.x >> 6;
  const int col = lane & 31, hf = lane >> 5;
  const KvCache c = a.cache;
  const int hk = blockIdx.x % c.heads, bx = blockIdx.x / c.heads;
  const int pl = c.page_log2, P = 1 << pl;

  const Block bl = find_block(a, bx);
  if (bl.i >= a.n) return;
  int start;
  const int R = rows_of(a, bl.i, &start);
  const int len = clamp_len(a.lens[bl.i], a.max_pages, pl);
  const int ncol = R * a.group;
  // heaviest first: the sequence's last rows see the most tokens
  const int blocks = (ncol + kCols - 1) / kCols;
  const int blk = blocks - 1 - bl.block;
  const int c0 = blk * kCols, c1 = min(c0 + kCols, ncol) - 1;
  const int p0 = len - R + c0 / a.group, p1 = len - R + c1 / a.group;
  const Span sp = span_of(max(p0, 0), p1, a.window, a.sinks);
  const int S = min((int)gridDim.y, max(sp.nt / kMinSplitTiles, 1));
  const int s = blockIdx.y;
  if (s >= S) return;
  const int u0 = (int)((long long)sp.nt * s / S), u1 = (int)((long long)sp.nt * (s + 1) / S);

  const int mycol = c0 + wave * 32 + col;
  const bool live = mycol < ncol;
  const int j = min(mycol, ncol - 1) / a.group, head = hk * a.group + min(mycol, ncol - 1) % a.group;
  const int pos = len - R + j, row = start + j;

  bf16x8_t q[NK];
#pragma unroll
  for (int k = 0; k < NK; ++k) {
    uint4 v = make_uint4(0u, 0u, 0u, 0u);
    if (live)
      v = *reinterpret_cast<const uint4 *>(a.q + ((size_t)row * a.q_heads + head) * D + 16 * k + 8 * hf);
    q[k] = __builtin_bit_cast(bf16x8_t, v);
  }

  f32x16_t o[NB];
#pragma unroll
  for (int T = 0; T < NB; ++T)
#pragma unroll
    for (int e = 0; e < 16; ++e) o[T][e] = 0.0f;
  float m = kLowest, l = 0.0f;

  const int32_t *trow = a.table + (long long)bl.i * a.max_pages;
  const int last_page = max(len - 1, 0) >> pl;
  const size_t head_off = (size_t)hk * c.record();

  // the thread's pieces of a tile, global -> registers -> LDS
  uint4 rk[kIt], rv[kIt];
  float rs[2][(NB * kKvTile + 64 * kWaves - 1) / (64 * kWaves)];
  auto page_of = [&](int key, bool &ok) {
    const int p = trow[min(key >> pl, last_page)];
    ok = (unsigned)p < (unsigned)c.n_pages;
    return ok ? p : 0;
  };
  auto fetch = [&](int u) {
    const int key0 = sp.tile(u) * kKvTile;
#pragma unroll
    for (int it = 0; it < kIt; ++it) {
      const int p = threadIdx.x + it * 64 * kWaves;
      if (kPieces >= 64 * kWaves || p < kPieces) {
        // keys: [D/8][32 keys][kElem]
        const int kk = p * 16 / kElem;                       // (chunk, key) of the piece
        const int key = key0 + kk % kKvTile, ch = kk / kKvTile;
        bool ok;
        const char *rec = c.k + (size_t)page_of(key, ok) * c.page_bytes() + head_off;
        rk[it] = *reinterpret_cast<const uint4 *>(rec + ((size_t)ch * P + (key & (P - 1))) * kElem);
        // values: [4 key chunks][D][kElem]
        const int kv = p * 16 / kElem;
        const int vkey = key0 + kv / D * 8, d = kv % D;
        rec = c.v + (size_t)page_of(vkey, ok) * c.page_bytes() + head_off;
        rv[it] = *reinterpret_cast<const uint4 *>(rec + ((size_t)((vkey & (P - 1)) >> 3) * D + d) * kElem);
      }
    }
    if constexpr (FMT == Q8_KV_Q8_0) {
#pragma unroll
      for (int it = 0; it < (NB * kKvTile + 64 * kWaves - 1) / (64 * kWaves); ++it) {
        const int p = threadIdx.x + it * 64 * kWaves;
        if (p < NB * kKvTile) {
          const int key = key0 + p % kKvTile, b = p / kKvTile;
          bool ok;
          const size_t at = (size_t)page_of(key, ok) * c.page_bytes() + head_off + (size_t)D * P;
          rs[0][it] = reinterpret_cast<const float *>(c.k + at)[b * P + (key & (P - 1))];
          rs[1][it] = reinterpret_cast<const float *>(c.v + at)[b * P + (key & (P - 1))];
        }
      }
    }
  };
  auto stage = [&](char *st) {
#pragma unroll
    for (int it = 0; it < kIt; ++it) {
      const int p = threadIdx.x + it * 64 * kWaves;
      if (kPieces >= 64 * kWaves || p < kPieces) {
        *reinterpret_cast<uint4 *>(st + p * 16) = rk[it];
        *reinterpret_cast<uint4 *>(st + kValBytes + p * 16) = rv[it];
      }
    }
    if constexpr (FMT == Q8_KV_Q8_0) {
      float *sc = reinterpret_cast<float *>(st + 2 * kValBytes);
#pragma unroll
      for (int it = 0; it < (NB * kKvTile + 64 * kWaves - 1) / (64 * kWaves); ++it) {
        const int p = threadIdx.x + it * 64 * kWaves;
        if (p < NB * kKvTile) {
          sc[p] = rs[0][it];
          sc[NB * kKvTile + p] = rs[1][it];
        }
      }
    }
  };
  // row `col` of the key fragment is this key of the tile
  const int fkey = 16 * (col >> 4) + 8 * ((col >> 2) & 1) + 4 * ((col >> 3) & 1) + (col & 3);

  auto compute = [&](const char *st, int u) {
    const int key0 = sp.tile(u) * kKvTile;
    const char *kb = st, *vb = st + kValBytes;
    const float *ksc = reinterpret_cast<const float *>(st + 2 * kValBytes), *vsc = ksc + NB * kKvTile;
    f32x16_t x;
#pragma unroll
    for (int e = 0; e < 16; ++e) x[e] = 0.0f;
    if constexpr (FMT == Q8_KV_BF16) {
#pragma unroll
      for (int k = 0; k < NK; ++k) {
        const uint4 f = *reinterpret_cast<const uint4 *>(kb + ((2 * k + hf) * kKvTile + fkey) * 16);
        x = __builtin_amdgcn_mfma_f32_32x32x16_bf16(__builtin_bit_cast(bf16x8_t, f), q[k], x, 0, 0, 0);
      }
    } else {
#pragma unroll
      for (int b = 0; b < NB; ++b) {
        f32x16_t z;
#pragma unroll
        for (int e = 0; e < 16; ++e) z[e] = 0.0f;
#pragma unroll
        for (int k = 2 * b; k < 2 * b + 2; ++k) {
          const uint2 f = *reinterpret_cast<const uint2 *>(kb + ((2 * k + hf) * kKvTile + fkey) * 8);
          z = __builtin_amdgcn_mfma_f32_32x32x16_bf16(i8x8_to_bf16(f), q[k], z, 0, 0, 0);
        }
#pragma unroll
        for (int g = 0; g < 4; ++g) {
          const float4 w = *reinterpret_cast<const float4 *>(ksc + b * kKvTile + 16 * (g >> 1) + 8 * hf + 4 * (g & 1));
          x[4 * g] = fmaf(w.x, z[4 * g], x[4 * g]);
          x[4 * g + 1] = fmaf(w.y, z[4 * g + 1], x[4 * g + 1]);
          x[4 * g + 2] = fmaf(w.z, z[4 * g + 2], x[4 * g + 2]);
          x[4 * g + 3] = fmaf(w.w, z[4 * g + 3], x[4 * g + 3]);
        }
      }
    }
#pragma unroll
    for (int e = 0; e < 16; ++e) x[e] *= a.scale_log2;
    // bit e: key e of the lane's sixteen (16 (e/8) + 8 hf + e%8) is seen
    const bool inner = key0 + kKvTile - 1 <= p0 &&
                       (a.window <= 0 || key0 > p1 - a.window || key0 + kKvTile <= a.sinks);
    bool ok0, ok1;
    (void)page_of(key0 + 8 * hf, ok0);
    (void)page_of(key0 + 16 + 8 * hf, ok1);
    unsigned seen = 0xffffu;
    unsigned vmask = 0xffffu;     // keys whose values may count for some column
    if (!inner || !__all(ok0 && ok1)) {
      seen = vmask = 0;
#pragma unroll
      for (int e = 0; e < 16; ++e) {
        const int key = key0 + 16 * (e >> 3) + 8 * hf + (e & 7);
        const bool ok = (e < 8 ? ok0 : ok1) && key < len;
        const bool in = ok && key <= pos && (a.window <= 0 || key > pos - a.window || key < a.sinks);
        seen |= in ? 1u << e : 0u;
      }
#pragma unroll
      for (int e = 0; e < 16; ++e)
        if (!(seen >> e & 1)) x[e] = -__builtin_inff();
    }
    (void)vmask;
    float mx = x[0];
#pragma unroll
    for (int e = 1; e < 16; ++e) mx = fmaxf(mx, x[e]);
    mx = fmaxf(mx, __shfl_xor(mx, 32));
    const float mn = fmaxf(m, mx);
    const float alpha = exp2_fast(m - mn);
    m = mn;
    float ps = 0.0f;
#pragma unroll
    for (int e = 0; e < 16; ++e) {
      x[e] = exp2_fast(x[e] - mn);
      ps += x[e];
    }
    l = l * alpha + ps;
    if (__any(alpha != 1.0f)) {
#pragma unroll
      for (int T = 0; T < NB; ++T) o[T] *= alpha;
    }
    if constexpr (FMT == Q8_KV_BF16) {
      float p[16];
#pragma unroll
      for (int e = 0; e < 16; ++e) p[e] = x[e];
      const bf16x8_t pb[2] = {to_bf16x8(p), to_bf16x8(p + 8)};
#pragma unroll
      for (int T = 0; T < NB; ++T)
#pragma unroll
        for (int t = 0; t < 2; ++t) {
          const uint4 f = *reinterpret_cast<const uint4 *>(vb + ((2 * t + hf) * D + 32 * T + col) * 16);
          o[T] = __builtin_amdgcn_mfma_f32_32x32x16_bf16(__builtin_bit_cast(bf16x8_t, f), pb[t], o[T], 0, 0, 0);
        }
    } else {
#pragma unroll
      for (int T = 0; T < NB; ++T) {
        float p[16];
#pragma unroll
        for (int g = 0; g < 4; ++g) {
          const float4 w = *reinterpret_cast<const float4 *>(vsc + T * kKvTile + 16 * (g >> 1) + 8 * hf + 4 * (g & 1));
          p[4 * g] = x[4 * g] * w.x;
          p[4 * g + 1] = x[4 * g + 1] * w.y;
          p[4 * g + 2] = x[4 * g + 2] * w.z;
          p[4 * g + 3] = x[4 * g + 3] * w.w;
        }
        if (seen != 0xffffu) {
#pragma unroll
          for (int e = 0; e < 16; ++e)
            if (!(seen >> e & 1)) p[e] = 0.0f;
        }
#pragma unroll
        for (int t = 0; t < 2; ++t) {
          const uint2 f = *reinterpret_cast<const uint2 *>(vb + ((2 * t + hf) * D + 32 * T + col) * 8);
          o[T] = __builtin_amdgcn_mfma_f32_32x32x16_bf16(i8x8_to_bf16(f), to_bf16x8(p + 8 * t), o[T], 0, 0, 0);
        }
      }
    }
  };

  // Values of tokens past the sequence, or on no page, may hold anything:
  // those of a tile that reaches past the length (or names no page) are
  // zeroed in LDS before they meet a probability of zero.
  auto scrub = [&](char *st, int u) {
    const int key0 = sp.tile(u) * kKvTile;
    if constexpr (FMT == Q8_KV_BF16) {
      bool ok0, ok1;
      (void)page_of(key0, ok0);
      (void)page_of(key0 + 16, ok1);
      if (key0 + kKvTile <= len && ok0 && ok1) return;
      uint16_t *v = reinterpret_cast<uint16_t *>(st + kValBytes);
      for (int e = threadIdx.x; e < kKvTile * D; e += 64 * kWaves) {
        const int k = e / (8 * D) * 8 + e % 8;
        if (key0 + k >= len || !(k < 16 ? ok0 : ok1)) v[e] = 0;
      }
    }
  };

  if (u0 < u1) {
    fetch(u0);
    stage(lds);
    __syncthreads();
    scrub(lds, u0);
    __syncthreads();
    int cur = 0;
    for (int u = u0; u < u1; ++u) {
      if (u + 1 < u1) fetch(u + 1);
      compute(lds + cur * kStage, u);
      if (u + 1 < u1) {
        char *nx = lds + (cur ^ 1) * kStage;
        stage(nx);
        __syncthreads();
        scrub(nx, u + 1);
        __syncthreads();
      }
      cur ^= 1;
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
