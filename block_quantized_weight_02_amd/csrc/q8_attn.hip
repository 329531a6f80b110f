// q8_attn.hip -- attention of one row a sequence over the paged cache
// (q8_attn_decode; the formula and layouts are in include/q8gemv.h).
#include <hip/hip_runtime.h>

#include "q8_attn.h"

namespace q8 {
namespace {

constexpr int kHeadTile = 16;          // query heads of one matrix-core tile
// One workgroup a CU: 1 x 131072 tokens take 85 us, with two 94, with four 133;
// 32 x 8192 67, 72, 86 (8 key/value heads of 128, bf16; more workgroups only add
// pieces to join, since one keeps enough loads on their way).
constexpr int kTargetWorkgroups = 256;
// Fewest tiles of a workgroup's share: 512 tokens take 9.0 us, with eight tiles
// 10.5, with sixteen 12.1.
constexpr int kMinTiles = 4;
constexpr int kListTiles = 256;        // tiles of a share listed in LDS at a time
constexpr int kListSeqs = 64;          // and sequences

__device__ __forceinline__ bf16x8_t as_bf16x8(uint4 v) { return __builtin_bit_cast(bf16x8_t, v); }

// One key/value tile of a wave in registers: lane (i = l%16, c = l/16).
template <int D, int FMT> struct Tile;
template <int D> struct Tile<D, Q8_KV_BF16> {
  uint4 k[D / 32][2];   // block b: keys 2i and 2i+1, dims 32b + 8c ..+7
  uint4 v[D / 16];      // dim 16T + i, keys 8c ..+7
};
template <int D> struct Tile<D, Q8_KV_Q8_0> {
  uint4 k[D / 32];      // block b: dims 32b + 8c ..+7 of keys 2i, then 2i+1
  uint4 v[D / 32];      // keys 8c ..+7 of dims 32T + 2i, then 32T + 2i + 1
  float ks[D / 64];     // the scale of (block, key) = (j / 32, j % 32), j = l + 64r;
  float vs[D / 64];     // they go through LDS to the lanes that need them
};

// A listed tile: its pages (of its two 16-token halves, -1: none), its first
// token, and its sequence's place in the list.
struct Listed {
  int page[2];
  int key0;
  int seq;
};

__device__ __forceinline__ Listed listed(const Listed &t) {   // into scalar registers
  return Listed{{uni(t.page[0]), uni(t.page[1])}, uni(t.key0), 0};
}

// The online softmax of one wave: scores transposed.  A 16x16x32 product of
// (16 keys x 32 dims) with (32 dims x 16 query heads) leaves lane (i, c) with
// keys 4c .. 4c+3 of head i.  The key fragments' rows are interleaved -- row r
// of the first product is key 2r of the 32-key tile, of the second key 2r+1 --
// so the lane's eight scores are keys 8c .. 8c+7, which is exactly the operand
// the value product wants (k = 8c+j, column i): the probabilities never leave
// their lane, and the sums O^T (dims x heads) are rescaled by one factor a lane.
template <int D, int FMT>
struct Wave {
  static constexpr int NB = D / 32, NT = D / 16;
  bf16x8_t q[NB];
  f32x4_t o[NT];
  float m, l;
  Tile<D, FMT> t;

  __device__ __forceinline__ void reset() {
#pragma unroll
    for (int T = 0; T < NT; ++T) o[T] = f32x4_t{0.0f, 0.0f, 0.0f, 0.0f};
    m = kLowest;
    l = 0.0f;
  }

  __device__ __forceinline__ void load_k(const KvCache &c, size_t head_off, const Listed &ti) {
    const int lane = threadIdx.x & 63, i = lane & 15, cc = lane >> 4;
    const int P = 1 << c.page_log2;
    const int kt = (ti.key0 + 2 * i) & (P - 1);
    const int page = max(i < 8 ? ti.page[0] : ti.page[1], 0);
    const char *kr = c.k + (size_t)page * c.page_bytes() + head_off;
    if constexpr (FMT == Q8_KV_BF16) {
      const char *p = kr + (cc * P + kt) * 16;
#pragma unroll
      for (int b = 0; b < NB; ++b) {
        t.k[b][0] = ld_stream16(p + (size_t)b * P * 64);
        t.k[b][1] = ld_stream16(p + (size_t)b * P * 64 + 16);
      }
    } else {
      const char *p = kr + (cc * P + kt) * 8;
#pragma unroll
      for (int b = 0; b < NB; ++b) t.k[b] = ld_stream16(p + (size_t)b * P * 32);
      load_scales(t.ks, c.k, c, head_off, ti);
    }
  }

  __device__ __forceinline__ void load_v(const KvCache &c, size_t head_off, const Listed &ti) {
    const int lane = threadIdx.x & 63, i = lane & 15, cc = lane >> 4;
    const int P = 1 << c.page_log2;
    const int vt = (ti.key0 + 8 * cc) & (P - 1);
    const int page = max(cc < 2 ? ti.page[0] : ti.page[1], 0);
    const char *vr = c.v + (size_t)page * c.page_bytes() + head_off;
    if constexpr (FMT == Q8_KV_BF16) {
      const char *p = vr + ((vt >> 3) * D + i) * 16;
#pragma unroll
      for (int T = 0; T < NT; ++T) t.v[T] = ld_stream16(p + T * 256);
    } else {
      const char *p = vr + ((vt >> 3) * D + 2 * i) * 8;
#pragma unroll
      for (int T = 0; T < NB; ++T) t.v[T] = ld_stream16(p + T * 256);
      load_scales(t.vs, c.v, c, head_off, ti);
    }
  }

  __device__ __forceinline__ static void load_scales(float *s, const char *base, const KvCache &c,
                                                     size_t head_off, const Listed &ti) {
    const int lane = threadIdx.x & 63, P = 1 << c.page_log2, key = lane & 31;
    const int page = max(key < 16 ? ti.page[0] : ti.page[1], 0);
    const float *p = reinterpret_cast<const float *>(base + (size_t)page * c.page_bytes() +
                                                     head_off + (size_t)D * P) +
                     (lane >> 5) * P + ((ti.key0 + key) & (P - 1));
#pragma unroll
    for (int r = 0; r < D / 64; ++r) s[r] = ld_scale4f(p + (size_t)r * 2 * P);
  }

  // Scores of the tile in t.k, as exponents of two.
  __device__ __forceinline__ void scores(float *s, float scale_log2, float *wlds) {
    if constexpr (FMT == Q8_KV_BF16) {
      f32x4_t s0{0.0f, 0.0f, 0.0f, 0.0f}, s1{0.0f, 0.0f, 0.0f, 0.0f};
#pragma unroll
      for (int b = 0; b < NB; ++b) {
        s0 = __builtin_amdgcn_mfma_f32_16x16x32_bf16(as_bf16x8(t.k[b][0]), q[b], s0, 0, 0, 0);
        s1 = __builtin_amdgcn_mfma_f32_16x16x32_bf16(as_bf16x8(t.k[b][1]), q[b], s1, 0, 0, 0);
      }
#pragma unroll
      for (int r = 0; r < 4; ++r) {
        s[2 * r] = s0[r];
        s[2 * r + 1] = s1[r];
      }
    } else {
      const int lane = threadIdx.x & 63, cc = lane >> 4;
#pragma unroll
      for (int r = 0; r < D / 64; ++r) wlds[r * 64 + lane] = t.ks[r];
#pragma unroll
      for (int j = 0; j < 8; ++j) s[j] = 0.0f;
#pragma unroll
      for (int b = 0; b < NB; ++b) {
        const f32x4_t z{0.0f, 0.0f, 0.0f, 0.0f};
        const f32x4_t s0 = __builtin_amdgcn_mfma_f32_16x16x32_bf16(
            i8x8_to_bf16(make_uint2(t.k[b].x, t.k[b].y)), q[b], z, 0, 0, 0);
        const f32x4_t s1 = __builtin_amdgcn_mfma_f32_16x16x32_bf16(
            i8x8_to_bf16(make_uint2(t.k[b].z, t.k[b].w)), q[b], z, 0, 0, 0);
        const float4 a0 = *reinterpret_cast<const float4 *>(wlds + b * 32 + 8 * cc);
        const float4 a1 = *reinterpret_cast<const float4 *>(wlds + b * 32 + 8 * cc + 4);
        const float ks[8] = {a0.x, a0.y, a0.z, a0.w, a1.x, a1.y, a1.z, a1.w};
#pragma unroll
        for (int r = 0; r < 4; ++r) {
          s[2 * r] = fmaf(ks[2 * r], s0[r], s[2 * r]);
          s[2 * r + 1] = fmaf(ks[2 * r + 1], s1[r], s[2 * r + 1]);
        }
      }
    }
#pragma unroll
    for (int j = 0; j < 8; ++j) s[j] *= scale_log2;
  }

  // Softmax step over the scores (s becomes probabilities); unseen keys hold
  // -infinity.  The scores' scaling is not joined with the subtraction here: the
  // largest one's exponent is then 0 however large it is.
  __device__ __forceinline__ void soften(float *s) {
    float mx = fmaxf(fmaxf(fmaxf(s[0], s[1]), fmaxf(s[2], s[3])),
                     fmaxf(fmaxf(s[4], s[5]), fmaxf(s[6], s[7])));
    mx = max_across(mx);
    const float mn = fmaxf(m, mx);
    const float alpha = exp2_fast(m - mn);
    m = mn;
    float ps = 0.0f;
#pragma unroll
    for (int j = 0; j < 8; ++j) {
#pragma clang fp contract(off)
      s[j] = exp2_fast(s[j] - mn);
      ps += s[j];
    }
    l = l * alpha + ps;
    if (__any(alpha != 1.0f)) {
#pragma unroll
      for (int T = 0; T < NT; ++T) o[T] *= alpha;
    }
  }

  // Adds the tile's values.  seen: bit j set if key 8c + j is; all: in every lane.
  __device__ __forceinline__ void values(const float *p, unsigned seen, bool all, float *wlds) {
    if constexpr (FMT == Q8_KV_BF16) {
      const bf16x8_t pb = to_bf16x8(p);
      if (!all) {                        // an unseen key's values may be anything
        const uint32_t keep[4] = {(seen & 1 ? 0xffffu : 0u) | (seen & 2 ? 0xffff0000u : 0u),
                                  (seen & 4 ? 0xffffu : 0u) | (seen & 8 ? 0xffff0000u : 0u),
                                  (seen & 16 ? 0xffffu : 0u) | (seen & 32 ? 0xffff0000u : 0u),
                                  (seen & 64 ? 0xffffu : 0u) | (seen & 128 ? 0xffff0000u : 0u)};
#pragma unroll
        for (int T = 0; T < NT; ++T) {
          t.v[T].x &= keep[0];
          t.v[T].y &= keep[1];
          t.v[T].z &= keep[2];
          t.v[T].w &= keep[3];
        }
      }
#pragma unroll
      for (int T = 0; T < NT; ++T)
        o[T] = __builtin_amdgcn_mfma_f32_16x16x32_bf16(as_bf16x8(t.v[T]), pb, o[T], 0, 0, 0);
    } else {
      const int lane = threadIdx.x & 63, cc = lane >> 4;
      wlds += D;
#pragma unroll
      for (int r = 0; r < D / 64; ++r) wlds[r * 64 + lane] = t.vs[r];
#pragma unroll
      for (int b = 0; b < NB; ++b) {
        const float4 a0 = *reinterpret_cast<const float4 *>(wlds + b * 32 + 8 * cc);
        const float4 a1 = *reinterpret_cast<const float4 *>(wlds + b * 32 + 8 * cc + 4);
        float w[8] = {p[0] * a0.x, p[1] * a0.y, p[2] * a0.z, p[3] * a0.w,
                      p[4] * a1.x, p[5] * a1.y, p[6] * a1.z, p[7] * a1.w};
        if (!all) {                      // nor may its scale count
#pragma unroll
          for (int j = 0; j < 8; ++j)
            if (!(seen >> j & 1)) w[j] = 0.0f;
        }
        const bf16x8_t pb = to_bf16x8(w);
        o[2 * b] = __builtin_amdgcn_mfma_f32_16x16x32_bf16(
            i8x8_to_bf16(make_uint2(t.v[b].x, t.v[b].y)), pb, o[2 * b], 0, 0, 0);
        o[2 * b + 1] = __builtin_amdgcn_mfma_f32_16x16x32_bf16(
            i8x8_to_bf16(make_uint2(t.v[b].z, t.v[b].w)), pb, o[2 * b + 1], 0, 0, 0);
      }
    }
  }

  // The sums of head i to dst[dim].
  __device__ __forceinline__ void store(float *dst) const {
    const int cc = (threadIdx.x & 63) >> 4;
    if constexpr (FMT == Q8_KV_BF16) {   // o[T]: dims 16T + 4c ..+3
#pragma unroll
      for (int T = 0; T < NT; ++T)
        *reinterpret_cast<float4 *>(dst + 16 * T + 4 * cc) =
            make_float4(o[T][0], o[T][1], o[T][2], o[T][3]);
    } else {                             // o[2b], o[2b+1]: even and odd dims of 32b + 8c ..+7
#pragma unroll
      for (int T = 0; T < NT; T += 2) {
        float4 *p = reinterpret_cast<float4 *>(dst + 16 * T + 8 * cc);
        p[0] = make_float4(o[T][0], o[T + 1][0], o[T][1], o[T + 1][1]);
        p[1] = make_float4(o[T][2], o[T + 1][2], o[T][3], o[T + 1][3]);
      }
    }
  }

  __device__ __forceinline__ static float max_across(float x) {   // over the lanes of one head
    typedef unsigned u32x2 __attribute__((ext_vector_type(2)));
    u32x2 r = __builtin_amdgcn_permlane16_swap(__float_as_uint(x), __float_as_uint(x), false, false);
    x = fmaxf(__uint_as_float(r.x), __uint_as_float(r.y));
    r = __builtin_amdgcn_permlane32_swap(__float_as_uint(x), __float_as_uint(x), false, false);
    return fmaxf(__uint_as_float(r.x), __uint_as_float(r.y));
  }
};

__device__ __forceinline__ int tiles_of(const AttnArgs &a, int len) {
  return span_of<kKvTile>(len - 1, len - 1, a.window, a.sinks).nt;
}
__device__ __forceinline__ int len_of(const AttnArgs &a, int i) {
  return i < a.n ? clamp_len(a.lens[i], a.max_pages, a.cache.page_log2) : 0;
}
__device__ __forceinline__ int scan_wave(int v) {   // inclusive sum over the lanes
  const int lane = threadIdx.x & 63;
#pragma unroll
  for (int o = 1; o < 64; o <<= 1) {
    const int u = __shfl_up(v, o);
    if (lane >= o) v += u;
  }
  return v;
}

// Floats of one partial result: up to 16 heads' sums, then their maxima and
// denominators.
__host__ __device__ constexpr int record_floats(int heads, int dim) {
  return heads * dim + 2 * kHeadTile;
}

// Dynamic LDS: the waves' sums (and a join's, in their place), and for Q8_0
// each wave's scales.
template <int D> constexpr int kRowFloats = D + 4;   // 16-byte shifts between heads' rows
template <int D, int FMT, int kWaves>
size_t decode_lds_bytes(int heads) {
  return ((size_t)kWaves * heads * kRowFloats<D> + (FMT == Q8_KV_Q8_0 ? kWaves * 2 * D : 0)) * 4;
}

// Grid: (chunks, units); a unit is one key/value head and up to 16 of its query
// heads.  All sequences' tiles stand in one row and workgroup x takes tiles x*C
// .. (x+1)*C - 1 of it, C the same for all, so that the token streams are
// equally long whatever the lengths; a share may end one sequence and begin
// the next.  The share's tiles are listed in LDS with their pages (no table
// lookup in the stream), wave w takes every kWaves-th: while a tile's scores
// turn into probabilities the next one's keys are in flight, and after its
// values are added the next one's values.  At a sequence's end the waves meet
// in LDS, with the next sequence's first tiles already loading.  A sequence
// that lies in one share is finished there; otherwise its pieces go to the
// workspace and the last workgroup to arrive joins them in order.
template <int D, int FMT, int kWaves>
__global__ void __launch_bounds__(64 * kWaves)
attn_decode_kernel(AttnArgs a) {
  constexpr int kThreads = 64 * kWaves;
  constexpr int NB = D / 32, kRow = kRowFloats<D>, per_head = D / 4;
  extern __shared__ __align__(16) float red[];
  __shared__ float red_m[kWaves][kHeadTile], red_l[kWaves][kHeadTile];
  __shared__ Listed list[kListTiles];
  __shared__ int pre[kListSeqs + 1], slen[kListSeqs];
  __shared__ int sums[Q8_MAX_SEQS / 64];
  __shared__ int is_last;
  const int lane = threadIdx.x & 63, i16 = lane & 15, c4 = lane >> 4;
  const int wave = uni(threadIdx.x >> 6);
  const int units = gridDim.y, unit = blockIdx.y, x = blockIdx.x, chunks = gridDim.x;
  const int tiles_a_head = (a.group + kHeadTile - 1) / kHeadTile;
  const int hk = unit / tiles_a_head, h0 = hk * a.group + (unit % tiles_a_head) * kHeadTile;
  const int heads = min(kHeadTile, a.group - (unit % tiles_a_head) * kHeadTile);
  const int rec = record_floats(min(a.group, kHeadTile), D);
  const KvCache c = a.cache;
  const size_t head_off = (size_t)hk * c.record();
  const int pl = c.page_log2;
  float *wlds = red + (size_t)kWaves * min(a.group, kHeadTile) * kRow + wave * 2 * D;

  // The number of all tiles, the share's size, and the 64 sequences it starts
  // in (w0; before: the tiles of those before them).  list_seqs writes 64
  // sequences' lengths and first tiles.
  auto list_seqs = [&](int w0, int before) {
    const int l = here(threadIdx.x);
    const int len = len_of(a, w0 + l);
    const int incl = scan_wave(tiles_of(a, len));
    if (wave == 0) {
      if (l == 0) pre[0] = before;
      pre[l + 1] = before + incl;
      slen[l] = len;
    }
    return uni(__shfl(incl, 63));
  };
  const int blocks = (a.n + 63) / 64;
  int total = 0, w0 = 0, before = 0;
  if (blocks == 1) {
    if (wave == 0) total = list_seqs(0, 0);
    __syncthreads();
    total = uni(pre[kListSeqs]);
  } else {
    for (int b = wave; b < blocks; b += kWaves) {
      const int s = scan_wave(tiles_of(a, len_of(a, b * 64 + lane)));
      if (lane == 63) sums[b] = s;
    }
    __syncthreads();
    for (int b = 0; b < blocks; ++b) total += uni(sums[b]);
  }
  const int C = max((total + chunks - 1) / chunks, kMinTiles);
  const int x0 = x * C, x1 = min(x0 + C, total);
  if (blocks > 1)
    for (; w0 / 64 < blocks - 1 && before + uni(sums[w0 / 64]) <= x0; w0 += 64)
      before += uni(sums[w0 / 64]);
  bool seqs_listed = blocks == 1;

  Wave<D, FMT> w;
  w.reset();
  auto load_q = [&](int i) {
#pragma unroll
    for (int b = 0; b < NB; ++b) {
      uint4 v = make_uint4(0u, 0u, 0u, 0u);
      if (i16 < heads)
        v = *reinterpret_cast<const uint4 *>(a.q + ((size_t)i * a.q_heads + h0 + i16) * D +
                                             32 * b + 8 * c4);
      w.q[b] = as_bf16x8(v);
    }
  };
  int open = -1;                          // the sequence whose heads (and sums) the waves hold
  bool fresh = true;                      // no sums yet
  for (int tb = x0; tb < x1;) {
    // list 64 sequences from w0, and the share's next tiles among theirs
    if (!seqs_listed) {
      __syncthreads();                    // the last list is read
      if (wave == 0) (void)list_seqs(w0, before);
      __syncthreads();
    }
    seqs_listed = false;
    const int te = min(min(x1, tb + kListTiles), uni(pre[kListSeqs]));
    for (int k0 = wave * 64; k0 < te - tb; k0 += kThreads) {
      // a tile's sequence is the last that starts at or before it: the wave finds
      // that of its first tile, its other tiles are in that one or soon after
      const int l = here(threadIdx.x) & 63, k = k0 + l;
      int lo = __popcll(__ballot(pre[l + 1] <= tb + k0));
      if (k >= te - tb) continue;
      while (pre[lo + 1] <= tb + k) ++lo;
      const int len = slen[lo];
      Listed ti;
      ti.key0 = span_of<kKvTile>(len - 1, len - 1, a.window, a.sinks).tile(tb + k - pre[lo]) * kKvTile;
      ti.seq = lo;
      const int32_t *row = a.table + (long long)(w0 + lo) * a.max_pages;
#pragma unroll
      for (int h = 0; h < 2; ++h) {
        const int p = row[min(ti.key0 + 16 * h, len - 1) >> pl];
        ti.page[h] = (unsigned)p < (unsigned)c.n_pages ? p : -1;
      }
      list[k] = ti;
    }
    __syncthreads();
    const int nk = te - tb;
    int k = wave;
    if (k < nk) {
      w.load_k(c, head_off, listed(list[k]));
      w.load_v(c, head_off, listed(list[k]));
    }

    int j = nk > 0 ? uni(list[0].seq) : kListSeqs;
    for (; j < kListSeqs; ++j) {
      const int s0 = uni(pre[j]), s1 = uni(pre[j + 1]);   // the sequence's tiles of all
      if (s0 >= te) break;
      if (s0 == s1) continue;
      const int i = w0 + j, len = uni(slen[j]), ke = min(s1, te) - tb;
      const int from = a.window > 0 ? len - a.window : 0;   // the window's first token
      if (open != i || fresh) {
        if (open != i) load_q(i);         // else it came while the last one was finished
        open = i;
        fresh = false;
        w.reset();
        // waited for here, so that the stream below waits for its own loads only
#pragma unroll
        for (int b = 0; b < NB; ++b) asm volatile("" : "+v"(w.q[b]));
      }
      for (; k < ke; k += kWaves) {
        const Listed ti = listed(list[k]), tn = listed(list[min(k + kWaves, nk - 1)]);
        float s[8];
        w.scores(s, a.scale_log2, wlds);
        w.load_k(c, head_off, tn);
        const bool all = ((ti.key0 + kKvTile <= len) & ((ti.page[0] | ti.page[1]) >= 0) &
                          ((ti.key0 >= from) | (ti.key0 + kKvTile <= a.sinks)));
        unsigned seen = 0xffu;
        if (!all) {
          seen = 0;
          const int stop = (c4 < 2 ? ti.page[0] : ti.page[1]) >= 0 ? len : 0;
#pragma unroll
          for (int e = 0; e < 8; ++e) {
            const int key = ti.key0 + 8 * c4 + e;
            const bool in = (key < stop) & ((key >= from) | (key < a.sinks));
            seen |= in ? 1u << e : 0u;
            s[e] = in ? s[e] : -__builtin_inff();
          }
        }
        w.soften(s);
        w.values(s, seen, all, wlds);
        w.load_v(c, head_off, tn);
      }
      if (s1 > te && te < x1) break;      // the share's next list goes on with this sequence

      // the waves meet, the next sequence's heads already on their way
      const bool more = ke < nk;
      open = more ? w0 + uni(list[min(ke, nk - 1)].seq) : -1;
      fresh = true;
      if (more) load_q(open);
      float lsum = w.l + __shfl_xor(w.l, 16);
      lsum += __shfl_xor(lsum, 32);
      __syncthreads();                    // the last sequence's sums are read
      if (i16 < heads) {
        w.store(red + (wave * heads + i16) * kRow);
        if (c4 == 0) {
          red_m[wave][i16] = w.m;
          red_l[wave][i16] = lsum;
        }
      }
      __syncthreads();
      const int first = s0 / C, segs = (s1 - 1) / C - first + 1;
      const size_t stride = (size_t)units * rec;
      // this piece's slot x + i is its own: each step along the tiles moves on
      // x or i
      const buf_t out = make_buf(a.partial + ((size_t)(x + i) * units + unit) * rec, rec * 4);
      for (int idx = here(threadIdx.x); idx < heads * per_head; idx += kThreads) {
        const int h = idx / per_head, d = (idx % per_head) * 4;
        float M = red_m[0][h], L = 0.0f;
#pragma unroll
        for (int v = 1; v < kWaves; ++v) M = fmaxf(M, red_m[v][h]);
        float4 y = make_float4(0.0f, 0.0f, 0.0f, 0.0f);
#pragma unroll
        for (int v = 0; v < kWaves; ++v) {
          const float f = exp2_fast(red_m[v][h] - M);
          const float4 z = *reinterpret_cast<const float4 *>(red + (v * heads + h) * kRow + d);
          L += red_l[v][h] * f;
          y.x += z.x * f;
          y.y += z.y * f;
          y.z += z.z * f;
          y.w += z.w * f;
        }
        if (segs == 1) {
          const float inv = L == 0.0f ? 0.0f : 1.0f / L;
          store_out(a, i, (h0 + h) * D + d, make_float4(y.x * inv, y.y * inv, y.z * inv, y.w * inv));
        } else {
          buf_st16_sys(out, (h * D + d) * 4, y);
          if (d == 0) {
            __builtin_amdgcn_raw_buffer_store_b32(__float_as_uint(M), out, (rec - 2 * kHeadTile + h) * 4, 0, kBufSys);
            __builtin_amdgcn_raw_buffer_store_b32(__float_as_uint(L), out, (rec - kHeadTile + h) * 4, 0, kBufSys);
          }
        }
      }
      if (segs == 1) continue;
      stores_done();
      __syncthreads();
      unsigned *cnt = &a.counters[(size_t)i * units + unit];
      if (threadIdx.x == 0)
        is_last = __hip_atomic_fetch_add(cnt, 1u, __ATOMIC_RELAXED, __HIP_MEMORY_SCOPE_SYSTEM) ==
                  (unsigned)(segs - 1);
      __syncthreads();
      if (!is_last) continue;
      // Join: groups of threads take runs of the pieces, then meet in LDS.
      const buf_t in = make_buf(a.partial + ((size_t)(first + i) * units + unit) * rec,
                                (unsigned)(((size_t)(segs - 1) * stride + rec) * 4));
      const unsigned step = (unsigned)(stride * 4);
      const int items = heads * per_head;
      const int groups = max(1, min(kThreads / items, kWaves));
      for (int idx = here(threadIdx.x); idx < items * groups; idx += kThreads) {
        const int g = idx / items, h = idx % items / per_head, d = (idx % per_head) * 4;
        const unsigned at = (h * D + d) * 4, mat = (rec - 2 * kHeadTile + h) * 4;
        const int g0 = segs * g / groups, g1 = segs * (g + 1) / groups;
        float M = kLowest, L = 0.0f;
        float4 y = make_float4(0.0f, 0.0f, 0.0f, 0.0f);
        constexpr int kBatch = 8;
        for (int p0 = g0; p0 < g1; p0 += kBatch) {
          float gm[kBatch], gl[kBatch];
          float4 gy[kBatch];
#pragma unroll
          for (int p = 0; p < kBatch; ++p) {
            const unsigned off = (unsigned)min(p0 + p, g1 - 1) * step;
            gm[p] = __uint_as_float(__builtin_amdgcn_raw_buffer_load_b32(in, off + mat, 0, kBufSys));
            gl[p] = __uint_as_float(__builtin_amdgcn_raw_buffer_load_b32(in, off + mat + kHeadTile * 4, 0, kBufSys));
            gy[p] = buf_ld16_sys(in, off + at);
          }
#pragma unroll
          for (int p = 0; p < kBatch; ++p) {
            if (p0 + p < g1) {
              const float Mn = fmaxf(M, gm[p]);
              const float fo = exp2_fast(M - Mn), fn = exp2_fast(gm[p] - Mn);
              L = L * fo + gl[p] * fn;
              y.x = y.x * fo + gy[p].x * fn;
              y.y = y.y * fo + gy[p].y * fn;
              y.z = y.z * fo + gy[p].z * fn;
              y.w = y.w * fo + gy[p].w * fn;
              M = Mn;
            }
          }
        }
        if (groups == 1) {
          const float inv = L == 0.0f ? 0.0f : 1.0f / L;
          store_out(a, i, (h0 + h) * D + d, make_float4(y.x * inv, y.y * inv, y.z * inv, y.w * inv));
        } else {
          *reinterpret_cast<float4 *>(red + (g * heads + h) * kRow + d) = y;
          if (d == 0) {
            red_m[g][h] = M;
            red_l[g][h] = L;
          }
        }
      }
      if (groups > 1) {
        __syncthreads();
        for (int idx = here(threadIdx.x); idx < items; idx += kThreads) {
          const int h = idx / per_head, d = (idx % per_head) * 4;
          float M = kLowest, L = 0.0f;
          for (int g = 0; g < groups; ++g) M = fmaxf(M, red_m[g][h]);
          float4 y = make_float4(0.0f, 0.0f, 0.0f, 0.0f);
          for (int g = 0; g < groups; ++g) {
            const float f = exp2_fast(red_m[g][h] - M);
            const float4 z = *reinterpret_cast<const float4 *>(red + (g * heads + h) * kRow + d);
            L += red_l[g][h] * f;
            y.x += z.x * f;
            y.y += z.y * f;
            y.z += z.z * f;
            y.w += z.w * f;
          }
          const float inv = L == 0.0f ? 0.0f : 1.0f / L;
          store_out(a, i, (h0 + h) * D + d, make_float4(y.x * inv, y.y * inv, y.z * inv, y.w * inv));
        }
      }
      if (threadIdx.x == 0)
        __hip_atomic_store(cnt, 0u, __ATOMIC_RELAXED, __HIP_MEMORY_SCOPE_SYSTEM);
    }
    tb = te;
    // the next list starts at the sequence that holds tile te
    if (tb < x1) {
      const int jn = min(j, kListSeqs);
      before = pre[jn];
      w0 += jn;
    }
  }

  // sequences without a token: zeros
  for (int i = x; i < a.n; i += chunks) {
    if (tiles_of(a, len_of(a, i)) != 0) continue;
    for (int idx = threadIdx.x; idx < heads * per_head; idx += kThreads)
      store_out(a, i, (h0 + idx / per_head) * D + idx % per_head * 4,
                make_float4(0.0f, 0.0f, 0.0f, 0.0f));
  }
}

// Waves of a workgroup: eight where a tile is short (64 dims) or its codes have
// to be widened, four else, and at 256 dims, where eight waves' registers spill.
// Measured on MI355X (us, eight against four): 64 sequences of 64 dims behind a
// window of 1024 32.4 against 33.5; Q8_0, 16 sequences up to 32768 tokens 96
// against 112; bf16, 128 dims, 1 x 131072 88 against 85.
template <int D, int FMT>
hipError_t launch(const AttnArgs &a, int units, hipStream_t stream) {
  constexpr int kWaves = D == 64 || (FMT == Q8_KV_Q8_0 && D == 128) ? 8 : 4;
  const size_t lds = decode_lds_bytes<D, FMT, kWaves>(a.group < kHeadTile ? a.group : kHeadTile);
  if (lds > 48 * 1024) {
    const hipError_t e = hipFuncSetAttribute(
        reinterpret_cast<const void *>(attn_decode_kernel<D, FMT, kWaves>),
        hipFuncAttributeMaxDynamicSharedMemorySize, (int)lds);
    if (e != hipSuccess) return e;
  }
  attn_decode_kernel<D, FMT, kWaves><<<dim3(a.chunks, units), 64 * kWaves, lds, stream>>>(a);
  return hipGetLastError();
}

}  // namespace

int attn_decode_chunks(int64_t units) {
  const int64_t g = kTargetWorkgroups / units;
  return (int)(g < 1 ? 1 : g);
}

size_t attn_decode_partial_bytes(int64_t n, int64_t q_heads, int64_t kv_heads, int64_t dim) {
  const int64_t group = q_heads / kv_heads;
  const int64_t units = kv_heads * ((group + kHeadTile - 1) / kHeadTile);
  const int64_t chunks = attn_decode_chunks(units);
  return (size_t)(chunks + n) * units *
         record_floats((int)(group < kHeadTile ? group : kHeadTile), (int)dim) * 4;
}

hipError_t launch_attn_decode(const AttnArgs &a, hipStream_t stream) {
  const int units = a.cache.heads * ((a.group + kHeadTile - 1) / kHeadTile);
  const bool q = a.cache.fmt == Q8_KV_Q8_0;
  switch (a.cache.dim) {
    case 64: return q ? launch<64, 1>(a, units, stream) : launch<64, 0>(a, units, stream);
    case 128: return q ? launch<128, 1>(a, units, stream) : launch<128, 0>(a, units, stream);
    default: return q ? launch<256, 1>(a, units, stream) : launch<256, 0>(a, units, stream);
  }
}

}  // namespace q8
