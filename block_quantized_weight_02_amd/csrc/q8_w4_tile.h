// q8_w4_tile.h -- the product over a 4-bit weight for few rows, and the gated pair:
// one workgroup per column tile and K split, its waves splitting K.  Included by
// the two sources that instantiate it (q8_w4_bf16.hip, q8_w4_q8.hip).
//
// y[r,n] = sum_j s[j,n] sum_{k in group j} x[r,k] (u[k,n] - z[j,n]).
//
// Bound by the weight's bytes (half a byte a value), so the vector unit's work a
// value has to stay below what the stream leaves it: at 6.5 TB/s a SIMD has 1700
// cycles for a stage of 64 columns x 128 rows, 34 a wave-wide instruction per row
// group of 16.  What keeps it there:
//   * bf16: u becomes the bf16 number 16 + u by a shift and an and-or for two
//     values (u in the mantissa's upper four bits), exactly.  The surplus is
//     taken out by the matrix core itself: its accumulator starts at -(16 + 8)
//     sum x, which one more product with a constant operand gives for all columns
//     at once; with zero points at -(16 + z) sum x, one multiplication a value and
//     group.  A group's sum is at most 31/4 times larger than without the
//     surplus, and so is its fp32 rounding (relative error against 64 bits
//     2e-7..1e-6 at K = 1024..16384, that of the plain fp32 product).
//   * Q8_0 activations: u is an int8 operand as it is, the accumulator starts at
//     -z sum x, all exact; the activation's bytes take the nibbles' order.
//   * a group's blocks chain in one accumulator and are scaled once.
//   * activation row 4 e + q sits in operand row 4 q + e, so that with up to 4 rows
//     only the first of a lane's four results counts, and is scaled.
// A wave has two stages in flight, taking turns in two register sets; the waves'
// carries meet in LDS, the splits' through finish_tile.
#pragma once

#include <hip/hip_runtime.h>
#include <stdint.h>

#include <type_traits>

#include "q8_device.h"
#include "q8_internal.h"
#include "q8_product.h"
#include "q8_w4.h"

namespace q8 {
namespace {

using namespace dev;

// A 16-bit scale's value.
__device__ __forceinline__ float w4_scale(uint32_t bits, bool bf16) {
  return bf16 ? __uint_as_float(bits << 16)
              : (float)__builtin_bit_cast(_Float16, (unsigned short)bits);
}
__device__ __forceinline__ void w4_scales4(uint2 v, int bf16, float (&f)[4]) {
  if (bf16) {
    f[0] = bf16_lo(v.x);
    f[1] = bf16_hi(v.x);
    f[2] = bf16_lo(v.y);
    f[3] = bf16_hi(v.y);
  } else {
    f[0] = w4_scale(v.x & 0xffffu, false);
    f[1] = w4_scale(v.x >> 16, false);
    f[2] = w4_scale(v.y & 0xffffu, false);
    f[3] = w4_scale(v.y >> 16, false);
  }
}

// Eight nibbles -> the bf16 numbers 16 + u, in row order.
__device__ __forceinline__ bf16x8_t w4_bf16(uint32_t w) {
  const uint32_t p0 = ((w << 3) & 0x00780078u) | 0x41804180u;
  const uint32_t p1 = ((w >> 1) & 0x00780078u) | 0x41804180u;
  const uint32_t p2 = ((w >> 5) & 0x00780078u) | 0x41804180u;
  const uint32_t p3 = ((w >> 9) & 0x00780078u) | 0x41804180u;
  return __builtin_bit_cast(bf16x8_t, make_uint4(p0, p1, p2, p3));
}
// Eight nibbles -> int8, rows 0,4,1,5 and 2,6,3,7.
__device__ __forceinline__ long w4_i8(uint32_t w) {
  return __builtin_bit_cast(long, make_uint2(w & 0x0f0f0f0fu, (w >> 4) & 0x0f0f0f0fu));
}

// Rows of carries that a wave keeps.
constexpr int w4_rows(int RG, int EL) { return RG == 1 ? 4 * EL : 16 * RG; }
// Waves a weight whose carries still stand apart when the tile is finished: its
// W/NW waves, halved until all of them fit 32 KiB.
constexpr int w4_final_waves(int W, int NW, int rows) {
  int n = W / NW;
  while (n > 1 && n * NW * rows * 256 > 32 * 1024) n /= 2;
  return n;
}
constexpr int w4_lds_bytes(int W, int NW, int rows) {
  const int n = w4_final_waves(W, NW, rows), first = W / NW / 2;
  return (n < W / NW && first > n ? first : n) * NW * rows * 256;
}

template <int ACT, int W, int RG, int EL, int GB, bool ZEROS, bool PAIR>
__global__ void __launch_bounds__(64 * W) w4_tile_kernel(const W4Args a) {
  constexpr bool kQ8 = ACT == kActQ8;
  constexpr int MR = w4_rows(RG, EL);
  constexpr int NW = PAIR ? 2 : 1;
  constexpr int WK = W / NW;                 // waves that split a weight's K range
  constexpr int QB = RG > 1 ? 2 : 4;         // blocks a stage (more rows: their operands fill the registers)
  constexpr int CH = GB < QB ? GB : QB;      // of them, blocks that share a scale
  constexpr int NS = QB / CH;                // scales a stage and column
  __shared__ __attribute__((aligned(16))) char lds[w4_lds_bytes(W, NW, MR)];
  float *red = reinterpret_cast<float *>(lds);

  const int lane = threadIdx.x & 63;
  const int q = lane >> 4, i = lane & 15;
  const int wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
  const int sel = PAIR ? wave / WK : 0, wk = PAIR ? wave % WK : wave;
  const int t = blockIdx.x, s = blockIdx.y;
  const int r0 = blockIdx.z * MR;
  const int mz = min(a.m - r0, MR);
  // a split is whole quads of blocks
  int b_lo, b_hi;
  {
    const int quads = (a.NB + 3) / 4;
    split_range(s, quads / a.split_k, quads % a.split_k, b_lo, b_hi);
    b_lo *= 4;
    b_hi = min(b_hi * 4, a.NB);
  }

  const W4 w = PAIR && sel ? a.w_u : a.w;
  constexpr int kGroupRows = GB * 32;
  const unsigned groups = (unsigned)w4_groups((int64_t)a.NB * 32, kGroupRows);
  const buf_t wr = make_buf(w.values + (size_t)t * a.NB * kW4Chunk, (unsigned)a.NB * kW4Chunk);
  const buf_t sr = make_buf(w.scales + (size_t)t * groups * 128, groups * 128u);
  const buf_t zr = ZEROS ? make_buf(w.zeros + (size_t)t * groups * 64, groups * 64u) : wr;
  const unsigned lw = (unsigned)lane * 16u;

  // operand row i of a group holds the activation's row 4 (i % 4) + i / 4; rows
  // past the chunk load its first row, and their results are never read
  const int ri = 4 * (i & 3) + (i >> 2);
  unsigned xoff[RG];
  const buf_t xr = kQ8 ? make_buf(static_cast<const char *>(a.x) + a.act_view_off,
                                  (unsigned)a.m * (unsigned)a.K)
                       : make_buf(static_cast<const char *>(a.x) + (size_t)r0 * a.K * 2,
                                  (unsigned)mz * (unsigned)a.K * 2u);
#pragma unroll
  for (int rg = 0; rg < RG; ++rg) {
    const int r = 16 * rg + ri < mz ? 16 * rg + ri : 0;
    xoff[rg] = kQ8 ? (unsigned)(r0 + r) * 32u + (unsigned)q * 8u
                   : (unsigned)r * (unsigned)a.K * 2u + (unsigned)q * 16u;
  }
  // int8: the scales of the rows whose results the lane holds
  const buf_t dr = kQ8 ? make_buf(static_cast<const char *>(a.x) + a.act_scale_off,
                                  (unsigned)a.m * (unsigned)a.NB * 4u) : xr;
  unsigned doff[RG][EL];
  if constexpr (kQ8) {
#pragma unroll
    for (int rg = 0; rg < RG; ++rg)
#pragma unroll
      for (int e = 0; e < EL; ++e) {
        const int r = min(16 * rg + 4 * e + q, mz - 1);
        doff[rg][e] = (unsigned)(r0 + r) * (unsigned)a.NB * 4u;
      }
  }

  struct Stage {
    uint4 v[QB];
    uint2 sc[NS];
    uint32_t z[NS];
    uint4 xa[QB][RG];                  // int8: .xy
    float dx[kQ8 ? RG : 1][kQ8 ? EL : 1][QB];
  };
  auto load = [&](Stage &st, int bv) Q8_INLINE {
    const int b = __builtin_amdgcn_readfirstlane(bv);
#pragma unroll
    for (int u = 0; u < QB; ++u) st.v[u] = buf_ld16(wr, lw, (unsigned)(b + u) * kW4Chunk);
    if constexpr (NS >= 2) {           // two groups a load
#pragma unroll
      for (int p = 0; p < NS / 2; ++p) {
        const unsigned pair = (unsigned)(b / GB / 2 + p);
        const u32x4_t v = __builtin_amdgcn_raw_buffer_load_b128(sr, (unsigned)i * 16u, pair * 256u, 0);
        st.sc[2 * p] = make_uint2(v.x, v.y);
        st.sc[2 * p + 1] = make_uint2(v.z, v.w);
        if constexpr (ZEROS) {
          const u32x2_t zz = __builtin_amdgcn_raw_buffer_load_b64(zr, (unsigned)i * 8u, pair * 128u, 0);
          st.z[2 * p] = zz.x;
          st.z[2 * p + 1] = zz.y;
        }
      }
    } else {
      const unsigned j = (unsigned)(b / GB);
      const unsigned at = GB == 4 ? j * 128u : (j >> 1) * 256u + (j & 1u) * 8u;
      const u32x2_t v = __builtin_amdgcn_raw_buffer_load_b64(sr, (unsigned)i * (GB == 4 ? 8u : 16u), at, 0);
      st.sc[0] = make_uint2(v.x, v.y);
      if constexpr (ZEROS)
        st.z[0] = __builtin_amdgcn_raw_buffer_load_b32(zr, (unsigned)i * (GB == 4 ? 4u : 8u), at / 2u, 0);
    }
#pragma unroll
    for (int u = 0; u < QB; ++u)
#pragma unroll
      for (int rg = 0; rg < RG; ++rg) {
        if constexpr (kQ8) {
          const u32x2_t v = __builtin_amdgcn_raw_buffer_load_b64(
              xr, xoff[rg], (unsigned)(b + u) * (unsigned)a.m * 32u, 0);
          st.xa[u][rg] = make_uint4(v.x, v.y, 0u, 0u);
        } else {
          const u32x4_t v = __builtin_amdgcn_raw_buffer_load_b128(xr, xoff[rg], (unsigned)(b + u) * 64u, 0);
          st.xa[u][rg] = make_uint4(v.x, v.y, v.z, v.w);
        }
      }
    if constexpr (kQ8) {
#pragma unroll
      for (int rg = 0; rg < RG; ++rg)
#pragma unroll
        for (int e = 0; e < EL; ++e)
#pragma unroll
          for (int u = 0; u < QB; ++u)
            st.dx[rg][e][u] = buf_ld4f(dr, doff[rg][e], (unsigned)(b + u) * 4u);
    }
  };

  f32x4_t acc[RG][4];
#pragma unroll
  for (int rg = 0; rg < RG; ++rg)
#pragma unroll
    for (int g = 0; g < 4; ++g) acc[rg][g] = f32x4_t{0.0f, 0.0f, 0.0f, 0.0f};

  // WHOLE: all of the stage's blocks are the range's (else the first nb)
  auto compute = [&](auto whole, const Stage &st, int nb) Q8_INLINE {
    constexpr bool WHOLE = decltype(whole)::value;
#pragma unroll
    for (int n = 0; n < NS; ++n) {
      if (!WHOLE && n * CH >= nb) break;
      float sc[4];
      w4_scales4(st.sc[n], a.scale_bf16, sc);
      if constexpr (kQ8) {
        float tt[RG][4][EL];
#pragma unroll
        for (int c = 0; c < CH; ++c) {
          const int u = n * CH + c;
          if (!WHOLE && u >= nb) break;
          const uint32_t wd[4] = {st.v[u].x, st.v[u].y, st.v[u].z, st.v[u].w};
#pragma unroll
          for (int rg = 0; rg < RG; ++rg) {
            const uint32_t x0 = st.xa[u][rg].x, x1 = st.xa[u][rg].y;
            const long xv = __builtin_bit_cast(
                long, make_uint2(__builtin_amdgcn_perm(x1, x0, 0x05010400u),
                                 __builtin_amdgcn_perm(x1, x0, 0x07030602u)));
            const long cst = ZEROS ? 0x0101010101010101l : (long)0xf8f8f8f8f8f8f8f8ul;
            const i32x4_t X = __builtin_amdgcn_mfma_i32_16x16x32_i8(xv, cst, i32x4_t{0, 0, 0, 0}, 0, 0, 0);
#pragma unroll
            for (int g = 0; g < 4; ++g) {
              i32x4_t C = X;
              if constexpr (ZEROS) {
                const int z = -(int)((st.z[n] >> (8 * g)) & 0xffu);
#pragma unroll
                for (int e = 0; e < EL; ++e) C[e] = __mul24(X[e], z);
              }
              const i32x4_t D = __builtin_amdgcn_mfma_i32_16x16x32_i8(xv, w4_i8(wd[g]), C, 0, 0, 0);
#pragma unroll
              for (int e = 0; e < EL; ++e) {
                const float d = (float)D[e], dx = st.dx[rg][e][u];
                if constexpr (CH == 1)
                  acc[rg][g][e] = fmaf(dx * sc[g], d, acc[rg][g][e]);
                else
                  tt[rg][g][e] = c == 0 ? dx * d : fmaf(dx, d, tt[rg][g][e]);
              }
            }
          }
        }
        if constexpr (CH > 1) {
#pragma unroll
          for (int rg = 0; rg < RG; ++rg)
#pragma unroll
            for (int g = 0; g < 4; ++g)
#pragma unroll
              for (int e = 0; e < EL; ++e) acc[rg][g][e] = fmaf(sc[g], tt[rg][g][e], acc[rg][g][e]);
        }
      } else {
        // -24 (16 + the 8 that u stands above), or 1 where zero points are given
        const uint32_t cw = ZEROS ? 0x3f803f80u : 0xc1c0c1c0u;
        const bf16x8_t cst = __builtin_bit_cast(bf16x8_t, make_uint4(cw, cw, cw, cw));
        f32x4_t D[RG][4];
#pragma unroll
        for (int rg = 0; rg < RG; ++rg) {
          f32x4_t X = {0.0f, 0.0f, 0.0f, 0.0f};
#pragma unroll
          for (int c = 0; c < CH; ++c) {
            if (!WHOLE && n * CH + c >= nb) break;
            X = __builtin_amdgcn_mfma_f32_16x16x32_bf16(
                __builtin_bit_cast(bf16x8_t, st.xa[n * CH + c][rg]), cst, X, 0, 0, 0);
          }
#pragma unroll
          for (int g = 0; g < 4; ++g) {
            D[rg][g] = X;
            if constexpr (ZEROS) {
              const float z = -16.0f - (float)((st.z[n] >> (8 * g)) & 0xffu);
#pragma unroll
              for (int e = 0; e < EL; ++e) D[rg][g][e] = z * X[e];
            }
          }
        }
#pragma unroll
        for (int c = 0; c < CH; ++c) {
          const int u = n * CH + c;
          if (!WHOLE && u >= nb) break;
          const uint32_t wd[4] = {st.v[u].x, st.v[u].y, st.v[u].z, st.v[u].w};
#pragma unroll
          for (int g = 0; g < 4; ++g) {
            const bf16x8_t bw = w4_bf16(wd[g]);
#pragma unroll
            for (int rg = 0; rg < RG; ++rg)
              D[rg][g] = __builtin_amdgcn_mfma_f32_16x16x32_bf16(
                  __builtin_bit_cast(bf16x8_t, st.xa[u][rg]), bw, D[rg][g], 0, 0, 0);
          }
        }
#pragma unroll
        for (int rg = 0; rg < RG; ++rg)
#pragma unroll
          for (int g = 0; g < 4; ++g)
#pragma unroll
            for (int e = 0; e < EL; ++e) acc[rg][g][e] = fmaf(sc[g], D[rg][g][e], acc[rg][g][e]);
      }
    }
  };
  auto step = [&](const Stage &st, int b) Q8_INLINE {
    if (b + QB <= b_hi)
      compute(std::true_type{}, st, QB);
    else
      compute(std::false_type{}, st, b_hi - b);
  };

  {
    Stage A, B;
    constexpr int stride = WK * QB;
    int b = b_lo + QB * wk;
    if (b < b_hi) {
      load(A, b);
      while (true) {
        if (b + stride >= b_hi) {
          step(A, b);
          break;
        }
        load(B, b + stride);
        compute(std::true_type{}, A, QB);
        b += stride;
        if (b + stride >= b_hi) {
          step(B, b);
          break;
        }
        load(A, b + stride);
        compute(std::true_type{}, B, QB);
        b += stride;
      }
    }
  }

  // the waves' carries: halved until the rest fits, then side by side in LDS
  constexpr int WF = w4_final_waves(W, NW, MR);
  static_assert(EL == 4 || WF == WK, "halving moves all four of a lane's results");
#pragma unroll
  for (int half = WK / 2; half >= WF; half /= 2) {
    if (wk >= half && wk < 2 * half) {
      float *rw = red + (size_t)(sel * half + wk - half) * MR * 64;
#pragma unroll
      for (int rg = 0; rg < RG; ++rg)
#pragma unroll
        for (int g = 0; g < 4; ++g)
          *reinterpret_cast<f32x4_t *>(rw + (rg * 4 + g) * 256 + lane * 4) = acc[rg][g];
    }
    __syncthreads();
    if (wk < half) {
      const float *rw = red + (size_t)(sel * half + wk) * MR * 64;
#pragma unroll
      for (int rg = 0; rg < RG; ++rg)
#pragma unroll
        for (int g = 0; g < 4; ++g)
          acc[rg][g] += *reinterpret_cast<const f32x4_t *>(rw + (rg * 4 + g) * 256 + lane * 4);
    }
    __syncthreads();
  }
  if (wk < WF) {
    float *rw = red + (size_t)(sel * WF + wk) * MR * 64;
#pragma unroll
    for (int rg = 0; rg < RG; ++rg)
#pragma unroll
      for (int g = 0; g < 4; ++g)
#pragma unroll
        for (int e = 0; e < EL; ++e) rw[(16 * rg + 4 * e + q) * 64 + 16 * g + i] = acc[rg][g][e];
  }
  __syncthreads();
  // the chunk's rows of the outputs (a launch of several chunks has one split and
  // no residual)
  Epi ep = a.ep;
  if (ep.yq) {
    ep.yq += (size_t)r0 * a.Npad;
    ep.yq_scale += (size_t)r0 * (a.Npad / 32);
    ep.yq_view += (size_t)r0 * 32;
    ep.view_rows = a.m;
  }
  const TileOut out{a.y + (size_t)r0 * a.Npad, a.Npad, (size_t)t * kTile, (size_t)t * kTile, a.Npad,
                    (unsigned)t};
  if constexpr (PAIR)
    finish_pair_tile<MR, 2 * WF, 64 * W>(red, out, a.partial, a.counters, mz, s, a.split_k, ep);
  else
    finish_tile<MR, WF, false, 64 * W>(red, out, a.partial, a.counters, mz, s, a.split_k, 0, ep);
}

template <int ACT, int W, int RG, int EL, int GB, bool ZEROS, bool PAIR>
hipError_t launch_w4_k(const W4Args &a, hipStream_t stream) {
  const unsigned chunks = (unsigned)((a.m + w4_rows(RG, EL) - 1) / w4_rows(RG, EL));
  (void)hipGetLastError();
  w4_tile_kernel<ACT, W, RG, EL, GB, ZEROS, PAIR>
      <<<dim3((unsigned)a.T, (unsigned)a.split_k, chunks), dim3(64 * W), 0, stream>>>(a);
  return hipGetLastError();
}

template <int ACT, int W, int RG, int EL, bool PAIR>
hipError_t launch_w4_g(const W4Args &a, hipStream_t stream) {
  const bool z = a.w.zeros != nullptr;
  switch (a.group) {
    case 32: return z ? launch_w4_k<ACT, W, RG, EL, 1, true, PAIR>(a, stream)
                      : launch_w4_k<ACT, W, RG, EL, 1, false, PAIR>(a, stream);
    case 64: return z ? launch_w4_k<ACT, W, RG, EL, 2, true, PAIR>(a, stream)
                      : launch_w4_k<ACT, W, RG, EL, 2, false, PAIR>(a, stream);
    case 128: return z ? launch_w4_k<ACT, W, RG, EL, 4, true, PAIR>(a, stream)
                       : launch_w4_k<ACT, W, RG, EL, 4, false, PAIR>(a, stream);
    default: return hipErrorInvalidValue;
  }
}

template <int ACT>
hipError_t launch_w4_tile(int rows, bool pair, const W4Args &a, hipStream_t stream) {
  // more rows than a workgroup covers: chunks, without splits or a residual
  if (a.m > rows && (a.split_k != 1 || a.ep.residual)) return hipErrorInvalidValue;
  switch (rows) {
    case 4: return pair ? launch_w4_g<ACT, 8, 1, 1, true>(a, stream)
                        : launch_w4_g<ACT, 8, 1, 1, false>(a, stream);
    case 16: return pair ? launch_w4_g<ACT, 8, 1, 4, true>(a, stream)
                         : launch_w4_g<ACT, 8, 1, 4, false>(a, stream);
    case 32: return pair ? launch_w4_g<ACT, 8, 2, 4, true>(a, stream)
                         : launch_w4_g<ACT, 8, 2, 4, false>(a, stream);
    case 64: return pair ? launch_w4_g<ACT, 4, 4, 4, true>(a, stream)
                         : launch_w4_g<ACT, 4, 4, 4, false>(a, stream);
    default: return hipErrorInvalidValue;
  }
}

}  // namespace
}  // namespace q8
