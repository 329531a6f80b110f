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
//   * a stage's blocks of a group chain in one accumulator and are scaled once.
//   * activation row 4 e + q sits in operand row 4 q + e, so that with up to 4 rows
//     only the first of a lane's four results counts, and is scaled; with Q8_0
//     activations, whose results are each converted and scaled twice a block, of 8 or 24
//     rows the first two of the last row group's (m = 24, K 5120, N 32001: 30.3 -> 27.6
//     us, a pair of 8 rows, K 4096, N 14336, 17.3 -> 15.3; bf16 gains 2 %).
// A wave has two stages in flight, taking turns: the weight's in two register sets, the
// activation's rows (and Q8_0 scales) loaded straight into two places in LDS of the
// wave's own, so that the registers hold weight alone and no wave waits for another.
// The waves' carries meet in LDS, the splits' through finish_tile.
//
// Measured, calls back to back: m = 1, K = 4096, N = 14336 8.1 us, N = 32000 13.5 (68 MB,
// 5.0 TB/s); m = 16, N = 14336, zero points 9.1 (31 MB; a plain read 4.9): the launch, the
// first loads' latency and the join stand beside the stream.  Q8_0, groups of 32, m = 32, K
// = 5120, N = 32001 31..34 (92 MB; a plain read 14): the vector unit is busy half of the
// cycles (three instructions a result and block, conversion and two scales; with zero
// points four), the matrix unit an eighth, and the two waves that the registers leave a
// SIMD wait for each other's chains of them.
#pragma once

#include <hip/hip_runtime.h>
#include <stdint.h>

#include <atomic>
#include <type_traits>

#include "q8_device.h"
#include "q8_internal.h"
#include "q8_product.h"
#include "q8_w4.h"
#include "q8_w4_device.h"

namespace q8 {
namespace {

using namespace dev;

// Eight nibbles -> the bf16 numbers 16 + u, in row order.  The constants are held in
// registers that the compiler does not look into: written out, each would be a literal,
// and the and-or two instructions.
struct Bf16Consts {
  uint32_t nibble = 0x00780078u, sixteen = 0x41804180u;
  __device__ Bf16Consts() { asm("" : "+s"(nibble), "+v"(sixteen)); }
};
__device__ __forceinline__ bf16x8_t w4_bf16(uint32_t w, const Bf16Consts &k) {
  return __builtin_bit_cast(bf16x8_t, make_uint4(((w << 3) & k.nibble) | k.sixteen, ((w >> 1) & k.nibble) | k.sixteen,
                                                 ((w >> 5) & k.nibble) | k.sixteen, ((w >> 9) & k.nibble) | k.sixteen));
}
// Eight nibbles -> int8, rows 0,4,1,5 and 2,6,3,7.
__device__ __forceinline__ long w4_i8(uint32_t w) {
  return __builtin_bit_cast(long, make_uint2(w & 0x0f0f0f0fu, (w >> 4) & 0x0f0f0f0fu));
}

// Rows of carries that a wave keeps.
constexpr int w4_rows(int RG, int EL) { return RG == 1 ? 4 * EL : 16 * RG; }
// Waves whose carries still stand apart when the NT tiles are finished: W, halved until
// all of them fit 32 KiB; and the LDS that they (and the halves before) take.
constexpr int w4_final_waves(int W, int NT, int rows) {
  int n = W;
  while (n > 1 && n * NT * rows * 256 > 32 * 1024) n /= 2;
  return n;
}
constexpr int w4_carry_bytes(int W, int NT, int rows) {
  const int n = w4_final_waves(W, NT, rows);
  return (n < W ? W / 2 : W) * NT * rows * 256;
}

// Blocks a stage, and the bytes of LDS that a stage's activation takes.
constexpr int w4_stage_blocks(int RG, int NT) { return RG * NT > 1 ? 2 : 4; }
constexpr int w4_slot_x(int ACT, int RG, int EL, int NT) {
  return EL < 4 ? 1024 : RG * w4_stage_blocks(RG, NT) * (ACT == kActQ8 ? 512 : 1024);
}
constexpr int w4_slot(int ACT, int RG, int EL, int NT) {
  return w4_slot_x(ACT, RG, EL, NT) + (ACT == kActQ8 ? RG * 256 : 0);
}
constexpr int w4_lds(int ACT, int W, int RG, int EL, int NT) {
  const int stages = 2 * W * w4_slot(ACT, RG, EL, NT), carries = w4_carry_bytes(W, NT, w4_rows(RG, EL));
  return stages > carries ? stages : carries;
}

// Waves a SIMD that the registers are kept to: four (128 registers) where the carries and
// stages fit, else two.
constexpr int w4_waves_per_simd(int ACT, int RG, int EL, int NT, int GB) {
  return EL < 4 || (RG * NT == 1 && !(ACT == kActQ8 && GB == 4)) ? 4 : 2;
}

// NT: column tiles a wave covers, sharing its activation stage: the pair's two weights'
// (PAIR), or two of one weight side by side.
template <int ACT, int W, int RG, int EL, int LE, int NT, int GB, bool ZEROS, bool PAIR>
__global__ void __launch_bounds__(64 * W, w4_waves_per_simd(ACT, RG, EL, NT, GB)) w4_tile_kernel(const W4Args a) {
  constexpr bool kQ8 = ACT == kActQ8;
  constexpr int MR = w4_rows(RG, EL);
  // results of a lane that count: of the last row group LE
  const auto el = [](int rg) Q8_INLINE { return rg == RG - 1 ? LE : EL; };
  static_assert(!PAIR || NT == 2, "the pair's tiles of both weights");
  constexpr int QB = w4_stage_blocks(RG, NT);
  constexpr int CH = GB < QB ? GB : QB;      // of them, blocks that share a scale
  constexpr int NS = QB / CH;                // scales a stage and column
  constexpr int kSlotX = w4_slot_x(ACT, RG, EL, NT), kSlot = w4_slot(ACT, RG, EL, NT);
  extern __shared__ __attribute__((aligned(16))) char lds[];
  float *const red = reinterpret_cast<float *>(lds);

  const int lane = threadIdx.x & 63;
  const int q = lane >> 4, i = lane & 15;
  const int wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
  const int s = blockIdx.y;
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

  // the wave's tiles (past the weight's last: that one again, not stored)
  const unsigned groups = (unsigned)w4_groups((int64_t)a.NB * 32, GB * 32);
  const unsigned lw = (unsigned)lane * 16u;
  buf_t wr[NT], sr[NT], zr[NT];
  int tile[NT];
#pragma unroll
  for (int k = 0; k < NT; ++k) {
    const W4 &w = PAIR && k ? a.w_u : a.w;
    tile[k] = PAIR ? (int)blockIdx.x : NT * (int)blockIdx.x + k;
    const size_t t = (size_t)min(tile[k], a.T - 1);
    wr[k] = make_buf(w.values + t * a.NB * kW4Chunk, (unsigned)a.NB * kW4Chunk);
    sr[k] = make_buf(w.scales + t * groups * 128, groups * 128u);
    zr[k] = ZEROS ? make_buf(w.zeros + t * groups * 64, groups * 64u) : wr[k];
  }

  // ---- the activation's stages.  Operand row o of a row group holds the activation's
  // row 4 (o % 4) + o / 4 (with 4 rows in all, LDS holds just these); rows past the chunk
  // load its last one, and their results are never read; blocks past K load the last.
  const auto row_of = [&](int rg, int o) { return r0 + min(16 * rg + 4 * (o & 3) + (o >> 2), mz - 1); };
  char *const mine = lds + (size_t)wave * 2 * kSlot;
  const unsigned mine_at = __builtin_amdgcn_readfirstlane(lds_offset(mine));
  const char *const xb = static_cast<const char *>(a.x) + (kQ8 ? a.act_view_off : 0u);
  const char *const db = static_cast<const char *>(a.x) + a.act_scale_off;
  // A load takes two blocks (4 rows: the whole stage): of 8 rows of bf16, whole cache
  // lines of 128 bytes (a load of 16 rows' 64 bytes reads every line twice: m = 32, N =
  // 32001, loads alone 28 us), or of 16 rows of Q8_0 codes, which lie side by side.
  constexpr int kRowLoads = EL < 4 ? 1 : kQ8 ? RG : 2 * RG;
  unsigned xoff[kRowLoads], doff[kQ8 ? RG : 1];
  const unsigned xstep = kQ8 ? (unsigned)a.m * 32u : 64u;
  int xu;                // the lane's block within a load
  if constexpr (kQ8) {
    xu = EL < 4 ? (lane >> 3) & 3 : lane >> 5;
#pragma unroll
    for (int k = 0; k < kRowLoads; ++k) {
      const int o = EL < 4 ? (lane >> 1) & 3 : (lane & 31) >> 1;
      const int r = EL < 4 ? r0 + min(o, mz - 1) : row_of(k, o);
      xoff[k] = (unsigned)r * 32u + (unsigned)(lane & 1) * 16u;
    }
  } else if constexpr (EL < 4) {
    // [block][row][4 parts of 16 bytes], part p of row o at place p ^ (o / 2)
    const int o = (lane & 15) >> 2;
    xu = lane >> 4;
    xoff[0] = (unsigned)min(o, mz - 1) * (unsigned)a.K * 2u + (unsigned)(((lane & 3) ^ (o >> 1)) * 16);
  } else {
    // [row][8 parts of two blocks], part p of row o at place p ^ (o / 2): the operand
    // reads (16 rows' part p) spread over all LDS banks
    const int part = (lane & 7) ^ (lane >> 4);       // (rows 8 .. 15: ^ 4 more, below)
    xu = part >> 2;
#pragma unroll
    for (int k = 0; k < kRowLoads; ++k)
      xoff[k] = (unsigned)(row_of(k >> 1, 8 * (k & 1) + (lane >> 3)) - r0) * (unsigned)a.K * 2u + (unsigned)(part & 3) * 16u;
  }
  if constexpr (kQ8) {
#pragma unroll
    for (int rg = 0; rg < RG; ++rg) doff[rg] = (unsigned)row_of(rg, lane & 15) * (unsigned)a.NB * 4u;
  }
  const char *const xrow = kQ8 ? xb : xb + (size_t)r0 * a.K * 2;
  const auto fetch = [&](int b, int slot) Q8_INLINE {
    const unsigned at = mine_at + (unsigned)slot * kSlot;
    const int last = a.NB - 1;
    if constexpr (EL < 4) {
      load_to_lds16(xrow, (unsigned)min(b + xu, last) * xstep + xoff[0], at);
    } else if constexpr (kQ8) {
#pragma unroll
      for (int j = 0; j < QB / 2; ++j) {
        const unsigned bo = (unsigned)min(b + 2 * j + xu, last) * xstep;
#pragma unroll
        for (int rg = 0; rg < RG; ++rg) load_to_lds16(xrow, bo + xoff[rg], at + (j * RG + rg) * 1024);
      }
    } else {
#pragma unroll
      for (int j = 0; j < QB / 2; ++j) {
        // rows 8 .. 15 have the two blocks' places the other way round
        const unsigned bo[2] = {(unsigned)min(b + 2 * j + xu, last) * 64u,
                                (unsigned)min(b + 2 * j + (xu ^ 1), last) * 64u};
#pragma unroll
        for (int k = 0; k < kRowLoads; ++k)
          load_to_lds16(xrow, bo[k & 1] + xoff[k], at + (j * kRowLoads + k) * 1024);
      }
    }
    if constexpr (kQ8) {
      const unsigned bo = (unsigned)min(b + (lane >> 4) % QB, last) * 4u;
#pragma unroll
      for (int rg = 0; rg < RG; ++rg) load_to_lds4(db, doff[rg] + bo, at + kSlotX + rg * 256);
    }
  };
  // loads that a stage surely issues: what may be left when the one before is computed
  constexpr int kFetch = (EL < 4 ? 1 : kQ8 ? RG * QB / 2 : RG * QB) + (kQ8 ? RG : 0);
  constexpr int kStageLoads = kFetch + NT * QB;

  struct Weight {
    uint4 v[QB];
    uint2 sc[NS];
    uint32_t z[NS];
  };
  struct Stage {
    Weight w[NT];
  };
  auto load = [&](Stage &st, int bv, int slot) Q8_INLINE {
    const int b = __builtin_amdgcn_readfirstlane(bv), last = a.NB - 1;
    // (past K the last block and pair of groups again, and not used: a resource's extent
    // need not bound an access by its uniform offset)
    __builtin_amdgcn_s_waitcnt(0xc07f);   // lgkmcnt(0): the slot's last reads have returned
    fetch(b, slot);
#pragma unroll
    for (int k = 0; k < NT; ++k) {
      Weight &w = st.w[k];
#pragma unroll
      for (int u = 0; u < QB; ++u) w.v[u] = buf_ld16(wr[k], lw, (unsigned)min(b + u, last) * kW4Chunk);
      if constexpr (NS >= 2) {           // two groups a load
#pragma unroll
        for (int p = 0; p < NS / 2; ++p) {
          const unsigned pair = (unsigned)min(b / GB / 2 + p, (int)groups / 2 - 1);
          const u32x4_t v = __builtin_amdgcn_raw_buffer_load_b128(sr[k], (unsigned)i * 16u, pair * 256u, 0);
          w.sc[2 * p] = make_uint2(v.x, v.y);
          w.sc[2 * p + 1] = make_uint2(v.z, v.w);
          if constexpr (ZEROS) {
            const u32x2_t zz = __builtin_amdgcn_raw_buffer_load_b64(zr[k], (unsigned)i * 8u, pair * 128u, 0);
            w.z[2 * p] = zz.x;
            w.z[2 * p + 1] = zz.y;
          }
        }
      } else {
        const unsigned j = (unsigned)(b / GB);
        const unsigned at = GB == 4 ? j * 128u : (j >> 1) * 256u + (j & 1u) * 8u;
        const u32x2_t v = __builtin_amdgcn_raw_buffer_load_b64(sr[k], (unsigned)i * (GB == 4 ? 8u : 16u), at, 0);
        w.sc[0] = make_uint2(v.x, v.y);
        if constexpr (ZEROS)
          w.z[0] = __builtin_amdgcn_raw_buffer_load_b32(zr[k], (unsigned)i * (GB == 4 ? 4u : 8u), at / 2u, 0);
      }
    }
  };

  float acc[NT][RG][4][EL];
#pragma unroll
  for (int k = 0; k < NT; ++k)
#pragma unroll
    for (int rg = 0; rg < RG; ++rg)
#pragma unroll
      for (int g = 0; g < 4; ++g)
#pragma unroll
        for (int e = 0; e < EL; ++e) acc[k][rg][g][e] = 0.0f;

  const Bf16Consts consts;
  // the lane's operand bytes of block u, row group rg of a stage
  const int xlane = kQ8 ? (EL < 4 ? (i >> 2) * 32 + q * 8 : i * 32 + q * 8)
                        : (EL < 4 ? (i >> 2) * 64 + ((q ^ (i >> 3)) * 16) : i * 128 + ((q ^ (i >> 1)) * 16));
  const auto x_at = [&](const char *slot, int u, int rg) Q8_INLINE {
    if constexpr (EL < 4) return slot + u * (kQ8 ? 128 : 256) + xlane;
    else if constexpr (kQ8) return slot + ((u >> 1) * RG + rg) * 1024 + (u & 1) * 512 + xlane;
    else return slot + ((u >> 1) * RG + rg) * 2048 + (xlane ^ (u & 1) * 64);
  };
  // WHOLE: all of the stage's blocks are the range's (else the first nb)
  auto compute = [&](auto whole, const Stage &st, int slot, int nb) Q8_INLINE {
    constexpr bool WHOLE = decltype(whole)::value;
    const char *const xs = mine + slot * kSlot;
#pragma unroll
    for (int n = 0; n < NS; ++n) {
      if (!WHOLE && n * CH >= nb) break;
      float sc[NT][4];
#pragma unroll
      for (int k = 0; k < NT; ++k) w4_scales4(st.w[k].sc[n], a.scale_bf16 ? ~0u : 0u, sc[k]);
      if constexpr (kQ8) {
        float tt[NT][RG][4][EL];
#pragma unroll
        for (int c = 0; c < CH; ++c) {
          const int u = n * CH + c;
          if (!WHOLE && u >= nb) break;
#pragma unroll
          for (int rg = 0; rg < RG; ++rg) {
            const uint2 xw = *reinterpret_cast<const uint2 *>(x_at(xs, u, rg));
            const long xv = __builtin_bit_cast(
                long, make_uint2(__builtin_amdgcn_perm(xw.y, xw.x, 0x05010400u),
                                 __builtin_amdgcn_perm(xw.y, xw.x, 0x07030602u)));
            // scales of rows 4e + q: places 4q + e
            const float *dp = reinterpret_cast<const float *>(xs + kSlotX + rg * 256) + u * 16 + 4 * q;
            float dx[EL];
            if constexpr (EL == 4) {
              const float4 v = *reinterpret_cast<const float4 *>(dp);
              dx[0] = v.x; dx[1] = v.y; dx[2] = v.z; dx[3] = v.w;
            } else {
#pragma unroll
              for (int e = 0; e < el(rg); ++e) dx[e] = dp[e];
            }
            // -8 sum x, or -sum x where zero points multiply it
            const long cst = ZEROS ? -1l : (long)0xf8f8f8f8f8f8f8f8ul;
            const i32x4_t X = __builtin_amdgcn_mfma_i32_16x16x32_i8(xv, cst, i32x4_t{0, 0, 0, 0}, 0, 0, 0);
#pragma unroll
            for (int k = 0; k < NT; ++k) {
              const uint4 v = st.w[k].v[u];
              const uint32_t wd[4] = {v.x, v.y, v.z, v.w};
#pragma unroll
              for (int g = 0; g < 4; ++g) {
                i32x4_t C = X;
                if constexpr (ZEROS) {
                  const int z = (int)((st.w[k].z[n] >> (8 * g)) & 0xffu);
#pragma unroll
                  for (int e = 0; e < el(rg); ++e) C[e] = __mul24(X[e], z);
                }
                const i32x4_t D = __builtin_amdgcn_mfma_i32_16x16x32_i8(xv, w4_i8(wd[g]), C, 0, 0, 0);
#pragma unroll
                for (int e = 0; e < el(rg); ++e) {
                  const float d = (float)D[e];
                  if constexpr (CH == 1)
                    acc[k][rg][g][e] = fmaf(dx[e] * sc[k][g], d, acc[k][rg][g][e]);
                  else
                    tt[k][rg][g][e] = c == 0 ? dx[e] * d : fmaf(dx[e], d, tt[k][rg][g][e]);
                }
              }
            }
          }
        }
        if constexpr (CH > 1) {
#pragma unroll
          for (int k = 0; k < NT; ++k)
#pragma unroll
            for (int rg = 0; rg < RG; ++rg)
#pragma unroll
              for (int g = 0; g < 4; ++g)
#pragma unroll
                for (int e = 0; e < el(rg); ++e)
                  acc[k][rg][g][e] = fmaf(sc[k][g], tt[k][rg][g][e], acc[k][rg][g][e]);
        }
      } else {
        // -24 (16 + the 8 that u stands above), or 1 where zero points are given
        const uint32_t cw = ZEROS ? 0x3f803f80u : 0xc1c0c1c0u;
        const bf16x8_t cst = __builtin_bit_cast(bf16x8_t, make_uint4(cw, cw, cw, cw));
        bf16x8_t xv[CH][RG];
        f32x4_t X[RG];
#pragma unroll
        for (int c = 0; c < CH; ++c)
#pragma unroll
          for (int rg = 0; rg < RG; ++rg)
            xv[c][rg] = *reinterpret_cast<const bf16x8_t *>(x_at(xs, n * CH + c, rg));
#pragma unroll
        for (int rg = 0; rg < RG; ++rg) {
          X[rg] = f32x4_t{0.0f, 0.0f, 0.0f, 0.0f};
#pragma unroll
          for (int c = 0; c < CH; ++c) {
            if (!WHOLE && n * CH + c >= nb) break;
            X[rg] = __builtin_amdgcn_mfma_f32_16x16x32_bf16(xv[c][rg], cst, X[rg], 0, 0, 0);
          }
        }
#pragma unroll
        for (int k = 0; k < NT; ++k) {
          f32x4_t D[RG][4];
#pragma unroll
          for (int rg = 0; rg < RG; ++rg)
#pragma unroll
            for (int g = 0; g < 4; ++g) {
              D[rg][g] = X[rg];
              if constexpr (ZEROS) {
                const float z = -16.0f - (float)((st.w[k].z[n] >> (8 * g)) & 0xffu);
#pragma unroll
                for (int e = 0; e < el(rg); ++e) D[rg][g][e] = z * X[rg][e];
              }
            }
#pragma unroll
          for (int c = 0; c < CH; ++c) {
            const int u = n * CH + c;
            if (!WHOLE && u >= nb) break;
            const uint4 v = st.w[k].v[u];
            const uint32_t wd[4] = {v.x, v.y, v.z, v.w};
#pragma unroll
            for (int g = 0; g < 4; ++g) {
              const bf16x8_t bw = w4_bf16(wd[g], consts);
#pragma unroll
              for (int rg = 0; rg < RG; ++rg)
                D[rg][g] = __builtin_amdgcn_mfma_f32_16x16x32_bf16(xv[c][rg], bw, D[rg][g], 0, 0, 0);
            }
          }
#pragma unroll
          for (int rg = 0; rg < RG; ++rg)
#pragma unroll
            for (int g = 0; g < 4; ++g)
#pragma unroll
              for (int e = 0; e < el(rg); ++e)
                acc[k][rg][g][e] = fmaf(sc[k][g], D[rg][g][e], acc[k][rg][g][e]);
        }
      }
      // (the sums are taken here: left to the loop's end, a stage's products fill the
      // registers)
#pragma unroll
      for (int k = 0; k < NT; ++k)
#pragma unroll
        for (int rg = 0; rg < RG; ++rg)
#pragma unroll
          for (int g = 0; g < 4; ++g)
#pragma unroll
            for (int e = 0; e < el(rg); ++e) asm volatile("" : "+v"(acc[k][rg][g][e]));
      __builtin_amdgcn_sched_barrier(0);
    }
  };

  {
    // stages n of this wave, two in flight; only the last may be cut short
    Stage A, B;
    constexpr int stride = W * QB;
    int b = b_lo + QB * wave;
    int n = (b_hi - b + stride - 1) / stride;
    if (n > 0) load(A, b, 0);
    for (; n > 2; n -= 2, b += 2 * stride) {
      load(B, b + stride, 1);
      loads_left<kStageLoads>();
      compute(std::true_type{}, A, 0, QB);
      load(A, b + 2 * stride, 0);
      loads_left<kStageLoads>();
      compute(std::true_type{}, B, 1, QB);
    }
    if (n == 2) {
      load(B, b + stride, 1);
      loads_left<kStageLoads>();
      compute(std::true_type{}, A, 0, QB);
      loads_left<0>();
      compute(std::false_type{}, B, 1, min(QB, b_hi - b - stride));
    } else if (n == 1) {
      loads_left<0>();
      compute(std::false_type{}, A, 0, min(QB, b_hi - b));
    }
  }
  __syncthreads();       // the stages' room is the carries' now

  // the waves' carries: halved until the rest fits, then side by side in LDS
  constexpr int WF = w4_final_waves(W, NT, MR);
#pragma unroll
  for (int half = W / 2; half >= WF; half /= 2) {
    float *rw = red + (size_t)(wave & (half - 1)) * NT * MR * 64;
    if (wave >= half && wave < 2 * half) {
#pragma unroll
      for (int k = 0; k < NT; ++k)
#pragma unroll
        for (int rg = 0; rg < RG; ++rg)
#pragma unroll
          for (int g = 0; g < 4; ++g)
#pragma unroll
            for (int e = 0; e < el(rg); ++e)
              rw[(((k * RG + rg) * 4 + g) * EL + e) * 64 + lane] = acc[k][rg][g][e];
    }
    __syncthreads();
    if (wave < half) {
#pragma unroll
      for (int k = 0; k < NT; ++k)
#pragma unroll
        for (int rg = 0; rg < RG; ++rg)
#pragma unroll
          for (int g = 0; g < 4; ++g)
#pragma unroll
            for (int e = 0; e < el(rg); ++e)
              acc[k][rg][g][e] += rw[(((k * RG + rg) * 4 + g) * EL + e) * 64 + lane];
    }
    __syncthreads();
  }
  if (wave < WF) {
#pragma unroll
    for (int k = 0; k < NT; ++k) {
      float *rw = red + (size_t)(k * WF + wave) * MR * 64;
#pragma unroll
      for (int rg = 0; rg < RG; ++rg)
#pragma unroll
        for (int g = 0; g < 4; ++g)
#pragma unroll
          for (int e = 0; e < el(rg); ++e) rw[(16 * rg + 4 * e + q) * 64 + 16 * g + i] = acc[k][rg][g][e];
    }
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
  const auto out = [&](int t) {
    return TileOut{a.y + (size_t)r0 * a.Npad, a.Npad, (size_t)t * kTile, (size_t)t * kTile, a.Npad, (unsigned)t};
  };
  if constexpr (PAIR) {
    finish_pair_tile<MR, 2 * WF, 64 * W>(red, out(tile[0]), a.partial, a.counters, mz, s, a.split_k, ep);
  } else {
    finish_tile<MR, WF, false, 64 * W>(red, out(tile[0]), a.partial, a.counters, mz, s, a.split_k, 0, ep);
    if constexpr (NT == 2)               // (two tiles a wave are not split: finish_tile does not return early)
      if (tile[1] < a.T)
        finish_tile<MR, WF, false, 64 * W>(red + WF * MR * 64, out(tile[1]), a.partial, a.counters, mz, s,
                                           a.split_k, 0, ep);
  }
}

// Instances that the host side's plans reach.  Not sixteen waves with Q8_0 rows above four
// and groups of 128 (they leave it 128 registers, fewer than it has in use), nor two tiles of
// one weight for 24 Q8_0 rows without zero points or with groups of 32.
template <int ACT, int W, int RG, int EL, int LE, int NT, int GB, bool ZEROS, bool PAIR>
constexpr bool w4_reached() {
  if (ACT != kActQ8 || EL < 4) return true;
  if (W == 16) return GB != 4;
  return !(RG == 2 && LE == 2 && NT == 2 && !PAIR) || (ZEROS && GB > 1);
}

template <int ACT, int W, int RG, int EL, int LE, int NT, int GB, bool ZEROS, bool PAIR>
hipError_t launch_w4_k(const W4Args &a, hipStream_t stream) {
  if constexpr (!w4_reached<ACT, W, RG, EL, LE, NT, GB, ZEROS, PAIR>()) {
    return hipErrorInvalidValue;
  } else {
    constexpr int MR = w4_rows(RG, EL), lds = w4_lds(ACT, W, RG, EL, NT);
    const auto kern = w4_tile_kernel<ACT, W, RG, EL, LE, NT, GB, ZEROS, PAIR>;
    if constexpr (lds > 64 * 1024) {
      // once a device: dynamic LDS above the default 64 KiB
      static std::atomic<uint64_t> granted{0};
      int dev = 0;
      hipError_t e = hipGetDevice(&dev);
      if (e != hipSuccess) return e;
      const uint64_t bit = 1ull << (dev & 63);
      if (dev > 63 || !(granted.load(std::memory_order_relaxed) & bit)) {
        e = hipFuncSetAttribute(reinterpret_cast<const void *>(kern),
                                hipFuncAttributeMaxDynamicSharedMemorySize, lds);
        if (e != hipSuccess) return e;
        granted.fetch_or(bit, std::memory_order_relaxed);
      }
    }
    const unsigned chunks = (unsigned)((a.m + MR - 1) / MR);
    (void)hipGetLastError();
    const unsigned units = PAIR ? (unsigned)a.T : (unsigned)((a.T + NT - 1) / NT);
    kern<<<dim3(units, (unsigned)a.split_k, chunks), dim3(64 * W), lds, stream>>>(a);
    return hipGetLastError();
  }
}

template <int ACT, int W, int RG, int EL, int LE, int NT, bool PAIR>
hipError_t launch_w4_g(const W4Args &a, hipStream_t stream) {
  const bool z = a.w.zeros != nullptr;
  switch (a.group) {
    case 32: return z ? launch_w4_k<ACT, W, RG, EL, LE, NT, 1, true, PAIR>(a, stream)
                      : launch_w4_k<ACT, W, RG, EL, LE, NT, 1, false, PAIR>(a, stream);
    case 64: return z ? launch_w4_k<ACT, W, RG, EL, LE, NT, 2, true, PAIR>(a, stream)
                      : launch_w4_k<ACT, W, RG, EL, LE, NT, 2, false, PAIR>(a, stream);
    case 128: return z ? launch_w4_k<ACT, W, RG, EL, LE, NT, 4, true, PAIR>(a, stream)
                       : launch_w4_k<ACT, W, RG, EL, LE, NT, 4, false, PAIR>(a, stream);
    default: return hipErrorInvalidValue;
  }
}

template <int ACT>
hipError_t launch_w4_tile(const W4Plan &p, bool pair, const W4Args &a, hipStream_t stream) {
  // more rows than a workgroup covers: chunks, without splits or a residual; two tiles
  // of one weight: without splits
  if (a.m > p.rows && (a.split_k != 1 || a.ep.residual)) return hipErrorInvalidValue;
  if (!pair && p.tiles == 2 && a.split_k != 1) return hipErrorInvalidValue;
  const int key = p.rows * 1000 + p.waves * 10 + p.tiles;
  if constexpr (ACT == kActQ8) {
    switch (pair ? -key : key) {
      case 8081: return launch_w4_g<ACT, 8, 1, 4, 2, 1, false>(a, stream);
      case 24081: return launch_w4_g<ACT, 8, 2, 4, 2, 1, false>(a, stream);
      case 24082: return launch_w4_g<ACT, 8, 2, 4, 2, 2, false>(a, stream);
      case -8082: return launch_w4_g<ACT, 8, 1, 4, 2, 2, true>(a, stream);
      case -24082: return launch_w4_g<ACT, 8, 2, 4, 2, 2, true>(a, stream);
    }
  }
  switch (pair ? -key : key) {
    case 4081: return launch_w4_g<ACT, 8, 1, 1, 1, 1, false>(a, stream);
    case 4161: return launch_w4_g<ACT, 16, 1, 1, 1, 1, false>(a, stream);
    case 16081: return launch_w4_g<ACT, 8, 1, 4, 4, 1, false>(a, stream);
    case 16161: return launch_w4_g<ACT, 16, 1, 4, 4, 1, false>(a, stream);
    case 32081: return launch_w4_g<ACT, 8, 2, 4, 4, 1, false>(a, stream);
    case 32082: return launch_w4_g<ACT, 8, 2, 4, 4, 2, false>(a, stream);
    case 64081: return launch_w4_g<ACT, 8, 4, 4, 4, 1, false>(a, stream);
    case -4162: return launch_w4_g<ACT, 16, 1, 1, 1, 2, true>(a, stream);
    case -16082: return launch_w4_g<ACT, 8, 1, 4, 4, 2, true>(a, stream);
    case -32082: return launch_w4_g<ACT, 8, 2, 4, 4, 2, true>(a, stream);
    default: return hipErrorInvalidValue;
  }
}

}  // namespace
}  // namespace q8
