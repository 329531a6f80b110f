// q8_attn.hip -- attention of one row a sequence over the paged cache
// (q8_attn_decode; the formula and layouts are in include/q8gemv.h).
#include <hip/hip_runtime.h>

#include "q8_attn.h"

namespace q8 {
namespace {

constexpr int kWaves = 4;              // waves of a workgroup, each its own tiles
constexpr int kHeadTile = 16;          // query heads of one matrix-core tile
constexpr int kTargetWorkgroups = 512; // two of the 256 CUs' each
constexpr int kMinTiles = kWaves;      // fewest tiles of a workgroup's share

// One key/value tile of a wave in registers.
template <int D, int FMT> struct Tile;
template <int D> struct Tile<D, Q8_KV_BF16> {
  uint4 k[D / 32][2];   // block b: keys 2i and 2i+1, dims 32b + 8c ..+7
  uint4 v[D / 16];      // dim 16T + i, keys 8c ..+7
};
template <int D> struct Tile<D, Q8_KV_Q8_0> {
  uint4 k[D / 32];      // block b: dims 32b + 8c ..+7 of keys 2i, then 2i+1
  uint4 v[D / 32];      // keys 8c ..+7 of dims 32T + 2i, then 32T + 2i + 1
  float4 ks[D / 32][2]; // key scales of keys 8c ..+7
  float4 vs[D / 32][2];
};

__device__ __forceinline__ bf16x8_t as_bf16x8(uint4 v) { return __builtin_bit_cast(bf16x8_t, v); }

// The online softmax of one wave: scores transposed.  A 16x16x32 product of
// (16 keys x 32 dims) with (32 dims x 16 query heads) leaves lane (i = l%16,
// c = l/16) with keys 4c .. 4c+3 of head i.  The key fragments' rows are
// interleaved -- row r of the first product is key 2r of the 32-key tile, of
// the second key 2r+1 -- so the lane's eight scores are keys 8c .. 8c+7, which
// is exactly the operand the value product wants (k = 8c+j, column i): the
// probabilities never leave their lane, and the sums O^T (dims x heads) are
// rescaled by one factor a lane.
template <int D, int FMT>
struct Wave {
  static constexpr int NB = D / 32, NT = D / 16;
  bf16x8_t q[NB];
  f32x4_t o[NT];
  float m, l;

  __device__ __forceinline__ void reset() {
#pragma unroll
    for (int t = 0; t < NT; ++t) o[t] = f32x4_t{0.0f, 0.0f, 0.0f, 0.0f};
    m = kLowest;
    l = 0.0f;
  }

  // kpage, vpage: this lane's pages of the tile (its keys 2i, 2i+1 and 8c ..)
  __device__ __forceinline__ static void load(Tile<D, FMT> &t, const KvCache &c, size_t head_off,
                                              int key0, int kpage, int vpage) {
    const int lane = threadIdx.x & 63, i = lane & 15, cc = lane >> 4;
    const int P = 1 << c.page_log2;
    const int kt = (key0 + 2 * i) & (P - 1), vt = (key0 + 8 * cc) & (P - 1);
    const char *kr = c.k + (size_t)kpage * c.page_bytes() + head_off;
    const char *vr = c.v + (size_t)vpage * c.page_bytes() + head_off;
    if constexpr (FMT == Q8_KV_BF16) {
#pragma unroll
      for (int b = 0; b < NB; ++b) {
        const char *p = kr + ((size_t)((4 * b + cc) * P + kt)) * 16;
        t.k[b][0] = ld_stream16(p);
        t.k[b][1] = ld_stream16(p + 16);
      }
#pragma unroll
      for (int T = 0; T < NT; ++T) t.v[T] = ld_stream16(vr + ((size_t)(vt >> 3) * D + 16 * T + i) * 16);
    } else {
      const float *ks = reinterpret_cast<const float *>(kr + (size_t)D * P);
      const float *vs = reinterpret_cast<const float *>(vr + (size_t)D * P);
      // the key scales are those of the lane's scores: keys 8c .., the value
      // page's tokens
      const float *ksc = reinterpret_cast<const float *>(c.k + (size_t)vpage * c.page_bytes() +
                                                         head_off + (size_t)D * P);
      (void)ks;
#pragma unroll
      for (int b = 0; b < NB; ++b)
        t.k[b] = ld_stream16(kr + ((size_t)((4 * b + cc) * P + kt)) * 8);
#pragma unroll
      for (int b = 0; b < NB; ++b) {
        t.ks[b][0] = ld_scale16f(reinterpret_cast<const float4 *>(ksc + b * P + vt));
        t.ks[b][1] = ld_scale16f(reinterpret_cast<const float4 *>(ksc + b * P + vt + 4));
      }
#pragma unroll
      for (int T = 0; T < NB; ++T)
        t.v[T] = ld_stream16(vr + ((size_t)(vt >> 3) * D + 32 * T + 2 * i) * 8);
#pragma unroll
      for (int b = 0; b < NB; ++b) {
        t.vs[b][0] = ld_scale16f(reinterpret_cast<const float4 *>(vs + b * P + vt));
        t.vs[b][1] = ld_scale16f(reinterpret_cast<const float4 *>(vs + b * P + vt + 4));
      }
    }
  }

  // seen: bit j set if key key0 + 8c + j is seen; all: every lane's are all set
  __device__ __forceinline__ void step(Tile<D, FMT> &t, float scale_log2, unsigned seen, bool all) {
    float s[8];
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
#pragma unroll
      for (int j = 0; j < 8; ++j) s[j] = 0.0f;
#pragma unroll
      for (int b = 0; b < NB; ++b) {
        const f32x4_t z{0.0f, 0.0f, 0.0f, 0.0f};
        const f32x4_t s0 = __builtin_amdgcn_mfma_f32_16x16x32_bf16(
            i8x8_to_bf16(make_uint2(t.k[b].x, t.k[b].y)), q[b], z, 0, 0, 0);
        const f32x4_t s1 = __builtin_amdgcn_mfma_f32_16x16x32_bf16(
            i8x8_to_bf16(make_uint2(t.k[b].z, t.k[b].w)), q[b], z, 0, 0, 0);
        const float ks[8] = {t.ks[b][0].x, t.ks[b][0].y, t.ks[b][0].z, t.ks[b][0].w,
                             t.ks[b][1].x, t.ks[b][1].y, t.ks[b][1].z, t.ks[b][1].w};
#pragma unroll
        for (int r = 0; r < 4; ++r) {
          s[2 * r] = fmaf(ks[2 * r], s0[r], s[2 * r]);
          s[2 * r + 1] = fmaf(ks[2 * r + 1], s1[r], s[2 * r + 1]);
        }
      }
    }
#pragma unroll
    for (int j = 0; j < 8; ++j) s[j] *= scale_log2;
    if (!all) {
      // unseen keys: no score, and no value (their bytes may hold anything)
#pragma unroll
      for (int j = 0; j < 8; ++j)
        if (!(seen >> j & 1)) s[j] = -__builtin_inff();
      if constexpr (FMT == Q8_KV_BF16) {
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
    }
    float mx = fmaxf(fmaxf(fmaxf(s[0], s[1]), fmaxf(s[2], s[3])),
                     fmaxf(fmaxf(s[4], s[5]), fmaxf(s[6], s[7])));
    mx = fmaxf(mx, __shfl_xor(mx, 16));
    mx = fmaxf(mx, __shfl_xor(mx, 32));
    const float mn = fmaxf(m, mx);
    const float alpha = exp2_fast(m - mn);
    m = mn;
    float p[8], ps = 0.0f;
#pragma unroll
    for (int j = 0; j < 8; ++j) {
      p[j] = exp2_fast(s[j] - mn);
      ps += p[j];
    }
    l = l * alpha + ps;
    if (__any(alpha != 1.0f)) {
#pragma unroll
      for (int t2 = 0; t2 < NT; ++t2) o[t2] *= alpha;
    }
    if constexpr (FMT == Q8_KV_BF16) {
      const bf16x8_t pb = to_bf16x8(p);
#pragma unroll
      for (int T = 0; T < NT; ++T)
        o[T] = __builtin_amdgcn_mfma_f32_16x16x32_bf16(as_bf16x8(t.v[T]), pb, o[T], 0, 0, 0);
    } else {
#pragma unroll
      for (int b = 0; b < NB; ++b) {
        const float vs[8] = {t.vs[b][0].x, t.vs[b][0].y, t.vs[b][0].z, t.vs[b][0].w,
                             t.vs[b][1].x, t.vs[b][1].y, t.vs[b][1].z, t.vs[b][1].w};
        float w[8];
#pragma unroll
        for (int j = 0; j < 8; ++j) w[j] = p[j] * vs[j];
        if (!all) {
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
};

// A sequence's place in the launch: its tiles are before .. before + nt of all.
struct Place {
  int i;
  int before;
};

__device__ __forceinline__ int tiles_of(const AttnArgs &a, int i) {
  const int len = clamp_len(a.lens[i], a.max_pages, a.cache.page_log2);
  return span_of(len - 1, len - 1, a.window, a.sinks).nt;
}

// The number of all sequences' tiles, and by all threads alike the sequence
// that holds tile number x * C (n if there is none), C = what fits(total)
// gives.  A wave takes 64 sequences at a time; with more than 64 the blocks'
// sums go through LDS.
__device__ __forceinline__ Place find_place(const AttnArgs &a, int *sums, int x, int chunks,
                                            int *C_out, int *total_out) {
  const int lane = threadIdx.x & 63, wave = threadIdx.x >> 6;
  const int blocks = (a.n + 63) / 64;
  int total = 0, block = 0, base = 0, C, x0;
  if (blocks == 1) {
    const int t = lane < a.n ? tiles_of(a, lane) : 0;
    int incl = t;
#pragma unroll
    for (int o = 1; o < 64; o <<= 1) {
      const int u = __shfl_up(incl, o);
      if (lane >= o) incl += u;
    }
    total = __shfl(incl, 63);
    C = max((total + chunks - 1) / chunks, kMinTiles);
    x0 = x * C;
    const int before = __popcll(__ballot(incl <= x0 && lane < a.n));
    *C_out = C;
    *total_out = total;
    Place p;
    p.i = before;
    p.before = before > 0 ? __shfl(incl, before - 1) : 0;
    return p;
  }
  for (int b = wave; b < blocks; b += kWaves) {
    const int i = b * 64 + lane;
    int t = i < a.n ? tiles_of(a, i) : 0;
#pragma unroll
    for (int o = 32; o > 0; o >>= 1) t += __shfl_xor(t, o);
    if (lane == 0) sums[b] = t;
  }
  __syncthreads();
  for (int b = 0; b < blocks; ++b) total += sums[b];
  C = max((total + chunks - 1) / chunks, kMinTiles);
  x0 = x * C;
  for (block = 0; block < blocks - 1 && base + sums[block] <= x0; ++block) base += sums[block];
  const int i = block * 64 + lane;
  int incl = i < a.n ? tiles_of(a, i) : 0;
#pragma unroll
  for (int o = 1; o < 64; o <<= 1) {
    const int u = __shfl_up(incl, o);
    if (lane >= o) incl += u;
  }
  const int before = __popcll(__ballot(base + incl <= x0 && i < a.n));
  *C_out = C;
  *total_out = total;
  Place p;
  p.i = block * 64 + before;
  p.before = base + (before > 0 ? __shfl(incl, before - 1) : 0);
  return p;
}

// Floats of one partial result: up to 16 heads' sums, then their maxima and
// denominators.
__host__ __device__ constexpr int record_floats(int heads, int dim) {
  return heads * dim + 2 * kHeadTile;
}

// Grid: (chunks, units); a unit is one key/value head and up to 16 of its query
// heads.  All sequences' tiles stand in one row and workgroup x takes tiles x*C
// .. (x+1)*C - 1 of it, C the same for all, so that the token streams are
// equally long whatever the lengths; a share may end one sequence and begin
// the next.  The share's waves take every fourth tile, two tiles in flight
// each (K and V of the next are loaded while this one is computed), and meet
// in LDS.  A sequence that lies in one share is finished there; otherwise its
// pieces go to the workspace and the last workgroup to arrive joins them in
// order.
template <int D, int FMT>
__global__ void __launch_bounds__(64 * kWaves)
attn_decode_kernel(AttnArgs a) {
  constexpr int NB = D / 32, NT = D / 16;
  constexpr int kStride = D + 4;                       // LDS row: 16-byte shifts between heads
  __shared__ float red[(kWaves - 1) * kHeadTile * kStride];
  __shared__ float red_m[kWaves][kHeadTile], red_l[kWaves][kHeadTile];
  __shared__ int sums[Q8_MAX_SEQS / 64];
  __shared__ int is_last;
  const int lane = threadIdx.x & 63, wave = threadIdx.x >> 6, i16 = lane & 15, c4 = lane >> 4;
  const int units = gridDim.y, unit = blockIdx.y, x = blockIdx.x, chunks = gridDim.x;
  const int tiles_a_head = (a.group + kHeadTile - 1) / kHeadTile;
  const int hk = unit / tiles_a_head, h0 = hk * a.group + (unit % tiles_a_head) * kHeadTile;
  const int heads = min(kHeadTile, a.group - (unit % tiles_a_head) * kHeadTile);
  const int rec = record_floats(min(a.group, kHeadTile), D);
  const KvCache c = a.cache;
  const size_t head_off = (size_t)hk * c.record();
  const int pl = c.page_log2;

  int C, total;
  Place pc = find_place(a, sums, x, chunks, &C, &total);
  const int x1 = min((x + 1) * C, total);
  int t = x * C;

  while (t < x1) {
    const int len = clamp_len(a.lens[pc.i], a.max_pages, pl);
    const Span sp = span_of(len - 1, len - 1, a.window, a.sinks);
    if (sp.nt == 0) {
      ++pc.i;
      continue;
    }
    const int s0 = t - pc.before, s1 = min(x1 - pc.before, sp.nt);
    const int32_t *row = a.table + (long long)pc.i * a.max_pages;
    const int last_page = (len - 1) >> pl;

    Wave<D, FMT> w;
    w.reset();
#pragma unroll
    for (int b = 0; b < NB; ++b) {
      uint4 v = make_uint4(0u, 0u, 0u, 0u);
      if (i16 < heads)
        v = *reinterpret_cast<const uint4 *>(a.q + ((size_t)pc.i * a.q_heads + h0 + i16) * D +
                                             32 * b + 8 * c4);
      w.q[b] = as_bf16x8(v);
    }

    Tile<D, FMT> ta, tb;
    bool oka, okb;    // the lane's value page is a page of the cache
    // tile u of the sequence into registers; tiles past the share reload its last
    auto fetch = [&](Tile<D, FMT> &tile, bool &ok, int u) {
      const int key0 = sp.tile(min(u, s1 - 1)) * kKvTile;
      int kp = row[min((key0 + 2 * i16) >> pl, last_page)];
      int vp = row[min((key0 + 8 * c4) >> pl, last_page)];
      ok = (unsigned)vp < (unsigned)c.n_pages;
      if ((unsigned)kp >= (unsigned)c.n_pages) kp = 0;
      if (!ok) vp = 0;
      w.load(tile, c, head_off, key0, kp, vp);
    };
    auto compute = [&](Tile<D, FMT> &tile, bool ok, int u) {
      const int key = sp.tile(u) * kKvTile + 8 * c4;
      unsigned seen = 0;
#pragma unroll
      for (int j = 0; j < 8; ++j) {
        const int k = key + j;
        const bool in = k < len && (a.window <= 0 || k >= len - a.window || k < a.sinks);
        seen |= (in && ok) ? 1u << j : 0u;
      }
      w.step(tile, a.scale_log2, seen, __all(seen == 0xffu));
    };
    int u = s0 + wave;
    if (u < s1) {
      fetch(ta, oka, u);
      for (; u < s1; u += 2 * kWaves) {
        fetch(tb, okb, u + kWaves);
        compute(ta, oka, u);
        if (u + kWaves >= s1) break;
        fetch(ta, oka, u + 2 * kWaves);
        compute(tb, okb, u + kWaves);
      }
    }

    // the waves meet: each scales its sums to the common maximum
    w.l += __shfl_xor(w.l, 16);
    w.l += __shfl_xor(w.l, 32);
    __syncthreads();                       // the last segment's LDS is read
    if (c4 == 0) {
      red_m[wave][i16] = w.m;
      red_l[wave][i16] = w.l;
    }
    __syncthreads();
    float M = red_m[0][i16];
#pragma unroll
    for (int v = 1; v < kWaves; ++v) M = fmaxf(M, red_m[v][i16]);
    const float f = exp2_fast(w.m - M);
#pragma unroll
    for (int T = 0; T < NT; ++T) w.o[T] *= f;
    // (wave, head, dim) in LDS; wave 0's slot is written last, summed in wave order
    auto place = [&](float *dst, int T, bool add) {
      // bf16: T's rows are dims 16T + 4c ..+3.  Q8_0: T = 2b and 2b+1 hold the
      // even and odd dims of 32b + 8c ..+7.
      if constexpr (FMT == Q8_KV_BF16) {
        float4 *p = reinterpret_cast<float4 *>(dst + 16 * T + 4 * c4);
        *p = make_float4(w.o[T][0], w.o[T][1], w.o[T][2], w.o[T][3]);
      } else {
        if (T & 1) return;
        float4 *p = reinterpret_cast<float4 *>(dst + 16 * T + 8 * c4);
        p[0] = make_float4(w.o[T][0], w.o[T + 1][0], w.o[T][1], w.o[T + 1][1]);
        p[1] = make_float4(w.o[T][2], w.o[T + 1][2], w.o[T][3], w.o[T + 1][3]);
      }
      (void)add;
    };
    if (wave > 0 && i16 < heads) {
#pragma unroll
      for (int T = 0; T < NT; ++T) place(red + ((wave - 1) * kHeadTile + i16) * kStride, T, false);
    }
    __syncthreads();
    if (wave == 0 && i16 < heads) {
      // wave 0 adds the others' sums to its own registers and leaves the result
      // in the first slot
#pragma unroll
      for (int T = 0; T < NT; ++T) {
        if constexpr (FMT == Q8_KV_BF16) {
          const int at = i16 * kStride + 16 * T + 4 * c4;
#pragma unroll
          for (int v = 0; v < kWaves - 1; ++v) {
            const float4 y = *reinterpret_cast<const float4 *>(red + v * kHeadTile * kStride + at);
            w.o[T] += f32x4_t{y.x, y.y, y.z, y.w};
          }
        } else if (!(T & 1)) {
          const int at = i16 * kStride + 16 * T + 8 * c4;
#pragma unroll
          for (int v = 0; v < kWaves - 1; ++v) {
            const float4 y0 = *reinterpret_cast<const float4 *>(red + v * kHeadTile * kStride + at);
            const float4 y1 =
                *reinterpret_cast<const float4 *>(red + v * kHeadTile * kStride + at + 4);
            w.o[T] += f32x4_t{y0.x, y0.z, y1.x, y1.z};
            w.o[T + 1] += f32x4_t{y0.y, y0.w, y1.y, y1.w};
          }
        }
        if (FMT == Q8_KV_BF16 || (T & 1)) place(red + i16 * kStride, FMT == Q8_KV_BF16 ? T : T - 1, true);
      }
    }
    __syncthreads();

    const int first = pc.before / C, segs = (pc.before + sp.nt - 1) / C - first + 1;
    const int per_head = D / 4;
    if (segs == 1) {
      for (int idx = threadIdx.x; idx < heads * per_head; idx += 64 * kWaves) {
        const int h = idx / per_head, d = (idx % per_head) * 4;
        float Mh = red_m[0][h], L = 0.0f;
#pragma unroll
        for (int v = 1; v < kWaves; ++v) Mh = fmaxf(Mh, red_m[v][h]);
#pragma unroll
        for (int v = 0; v < kWaves; ++v) L += red_l[v][h] * exp2_fast(red_m[v][h] - Mh);
        const float inv = L == 0.0f ? 0.0f : 1.0f / L;
        const float4 y = *reinterpret_cast<const float4 *>(red + h * kStride + d);
        store_out(a, pc.i, (h0 + h) * D + d, make_float4(y.x * inv, y.y * inv, y.z * inv, y.w * inv));
      }
    } else {
      // this piece to the workspace, at slot x + i (unique: each step along
      // the tiles moves on x or i)
      const size_t stride = (size_t)units * rec;
      float *mine = a.partial + ((size_t)(x + pc.i) * units + unit) * rec;
      const buf_t out = make_buf(mine, rec * 4);
      for (int idx = threadIdx.x; idx < heads * per_head; idx += 64 * kWaves) {
        const int h = idx / per_head, d = (idx % per_head) * 4;
        buf_st16_sys(out, (h * D + d) * 4, *reinterpret_cast<const float4 *>(red + h * kStride + d));
      }
      if (threadIdx.x < heads) {
        const int h = threadIdx.x;
        float Mh = red_m[0][h], L = 0.0f;
        for (int v = 1; v < kWaves; ++v) Mh = fmaxf(Mh, red_m[v][h]);
        for (int v = 0; v < kWaves; ++v) L += red_l[v][h] * exp2_fast(red_m[v][h] - Mh);
        float *ml = mine + (rec - 2 * kHeadTile);
        __hip_atomic_store(ml + h, Mh, __ATOMIC_RELAXED, __HIP_MEMORY_SCOPE_SYSTEM);
        __hip_atomic_store(ml + kHeadTile + h, L, __ATOMIC_RELAXED, __HIP_MEMORY_SCOPE_SYSTEM);
      }
      stores_done();
      __syncthreads();
      if (threadIdx.x == 0)
        is_last = __hip_atomic_fetch_add(&a.counters[pc.i * units + unit], 1u, __ATOMIC_RELAXED,
                                         __HIP_MEMORY_SCOPE_SYSTEM) == (unsigned)(segs - 1);
      __syncthreads();
      if (is_last) {
        const float *base = a.partial + ((size_t)(first + pc.i) * units + unit) * rec;
        const buf_t in = make_buf(base, (unsigned)(((size_t)(segs - 1) * stride + rec) * 4));
        const unsigned step = (unsigned)(stride * 4);
        for (int idx = threadIdx.x; idx < heads * per_head; idx += 64 * kWaves) {
          const int h = idx / per_head, d = (idx % per_head) * 4;
          const unsigned at = (h * D + d) * 4, mat = (rec - 2 * kHeadTile + h) * 4;
          float Mh = kLowest, L = 0.0f;
          float4 y = make_float4(0.0f, 0.0f, 0.0f, 0.0f);
          constexpr int kBatch = 8;
          for (int g0 = 0; g0 < segs; g0 += kBatch) {
            float gm[kBatch], gl[kBatch];
            float4 gy[kBatch];
#pragma unroll
            for (int g = 0; g < kBatch; ++g) {
              const unsigned off = (unsigned)min(g0 + g, segs - 1) * step;
              gm[g] = __builtin_bit_cast(float, __builtin_amdgcn_raw_buffer_load_b32(in, off + mat, 0, kBufSys));
              gl[g] = __builtin_bit_cast(float, __builtin_amdgcn_raw_buffer_load_b32(in, off + mat + kHeadTile * 4, 0, kBufSys));
              gy[g] = buf_ld16_sys(in, off + at);
            }
#pragma unroll
            for (int g = 0; g < kBatch; ++g) {
              if (g0 + g < segs) {
                const float Mn = fmaxf(Mh, gm[g]);
                const float fo = exp2_fast(Mh - Mn), fn = exp2_fast(gm[g] - Mn);
                L = L * fo + gl[g] * fn;
                y.x = y.x * fo + gy[g].x * fn;
                y.y = y.y * fo + gy[g].y * fn;
                y.z = y.z * fo + gy[g].z * fn;
                y.w = y.w * fo + gy[g].w * fn;
                Mh = Mn;
              }
            }
          }
          const float inv = L == 0.0f ? 0.0f : 1.0f / L;
          store_out(a, pc.i, (h0 + h) * D + d,
                    make_float4(y.x * inv, y.y * inv, y.z * inv, y.w * inv));
        }
        if (threadIdx.x == 0)
          __hip_atomic_store(&a.counters[pc.i * units + unit], 0u, __ATOMIC_RELAXED,
                             __HIP_MEMORY_SCOPE_SYSTEM);
      }
    }
    t = pc.before + s1;
    if (s1 == sp.nt) {
      pc.before += sp.nt;
      ++pc.i;
    }
  }

  // sequences without a token: zeros
  for (int i = x; i < a.n; i += chunks) {
    if (tiles_of(a, i) != 0) continue;
    for (int idx = threadIdx.x; idx < heads * (D / 4); idx += 64 * kWaves)
      store_out(a, i, (h0 + idx / (D / 4)) * D + idx % (D / 4) * 4, make_float4(0.0f, 0.0f, 0.0f, 0.0f));
  }
}

}  // namespace

int attn_decode_chunks(int64_t n, int64_t units) {
  (void)n;
  const int64_t g = kTargetWorkgroups / units;
  return (int)(g < 1 ? 1 : g);
}

size_t attn_decode_partial_bytes(int64_t n, int64_t q_heads, int64_t kv_heads, int64_t dim) {
  const int64_t group = q_heads / kv_heads;
  const int64_t units = kv_heads * ((group + kHeadTile - 1) / kHeadTile);
  const int64_t chunks = attn_decode_chunks(n, units);
  return (size_t)(chunks + n) * units *
         record_floats((int)(group < kHeadTile ? group : kHeadTile), (int)dim) * 4;
}

hipError_t launch_attn_decode(const AttnArgs &a, hipStream_t stream) {
  const int units = a.cache.heads * ((a.group + kHeadTile - 1) / kHeadTile);
  const dim3 grid(a.chunks, units);
  const bool q = a.cache.fmt == Q8_KV_Q8_0;
  auto k = a.cache.dim == 64
               ? (q ? attn_decode_kernel<64, 1> : attn_decode_kernel<64, 0>)
               : a.cache.dim == 128 ? (q ? attn_decode_kernel<128, 1> : attn_decode_kernel<128, 0>)
                                    : (q ? attn_decode_kernel<256, 1> : attn_decode_kernel<256, 0>);
  k<<<grid, 64 * kWaves, 0, stream>>>(a);
  return hipGetLastError();
}

}  // namespace q8
