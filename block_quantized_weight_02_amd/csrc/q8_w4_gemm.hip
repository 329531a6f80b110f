// q8_w4_gemm.hip -- the product over a 4-bit weight for many activation rows, and the
// gated pair: a matrix-core GEMM over the packed weight (q8_w4.h).
//
//   * a workgroup of 4 waves owns 128 rows x 256 columns (the pair: 128 of each
//     weight), each wave 128 rows x one 64-column tile: 8 row groups x 4 column groups
//     of 16x16x32 products;
//   * the packed weight is the matrix product's operand order, so a wave loads its
//     tile's dwords straight into registers (one 16-byte load a block) and turns them
//     into bf16 there, once for its 128 rows: u - 8 (with zero points u - z), exact, in
//     1/16ths by the 4-bit conversion, two values in 3.5 instructions (5.5).  The
//     sums are 16ths too, until they are stored (16 times a scale could pass fp32's range);
//   * the activation rows of two blocks are staged in LDS, double buffered: bf16 rows
//     loaded straight into LDS, Q8_0 codes widened to bf16 on the way (exact: their
//     products' sums are then the same exact integers, in fp32), with their scales;
//   * a group's blocks within a stage chain in one accumulator and are scaled once:
//     one FMA a result and group (Q8_0 activations: one more a block for theirs);
//   * workgroups are numbered so that each XCD walks a contiguous range of (column
//     block, row block) with the row block fastest: the row blocks that read one
//     weight tile run together, and its L2 serves the tile to all of them.
//
// Measured: 2048 rows, K = 4096, N = 14336, groups of 128, 215..225 us (1070..1120
// TFLOP/s; the large bf16 library product reaches 1325, 181 us); 8192 rows 854 (1127).  The
// matrix unit is busy 47 % of the time, the vector unit 65 %, and the LDS reads of the
// activation's operands (128 rows for 64 columns a wave) hold both up: without them 159 us.
// More columns a wave would halve them, but their sums do not fit the registers.
#include <hip/hip_runtime.h>
#include <stdint.h>

#include <type_traits>

#include "q8_device.h"
#include "q8_product.h"
#include "q8_w4.h"
#include "q8_w4_device.h"

namespace q8 {
namespace {

using namespace dev;

constexpr int kThreads = 256;
constexpr int kRows = 128;                 // rows a workgroup
constexpr int kCB = 2;                     // blocks a stage
constexpr int kRG = kRows / 16;
constexpr int kA = kCB * kRows * 64;       // staged activation bytes (bf16)
constexpr int kDx = kCB * kRows * 4;       // staged activation scales (Q8_0)

// Within one row's 64 staged bytes of a block, 16-byte part p is at place
// p ^ (row / 2 % 4): the operand read (lane (q, i): part q of row i) and the staging
// writes spread over all LDS banks.
__device__ __forceinline__ int a_place(int r, int p) { return (p ^ ((r >> 1) & 3)) * 16; }

// Eight nibbles -> bf16 (u - 8) / 16, plus `add` where there are zero points
// ((8 - z) / 16: then (u - z) / 16).
template <bool ZEROS>
__device__ __forceinline__ bf16x8_t w4_signed(uint32_t w, float add) {
  // rows 0,4,1,5 are the bytes of lo, 2,6,3,7 those of hi
  const uint32_t lo = w ^ 0x88888888u;
  uint32_t hi;
  asm("v_lshrrev_b32 %0, 4, %1" : "=v"(hi) : "v"(lo));   // (one shift for four conversions)
  float f[8];
#pragma unroll
  for (int b = 0; b < 4; ++b) {
    const int r = (b >> 1) + 4 * (b & 1);
    f[r] = __builtin_amdgcn_cvt_off_f32_i4((int)(lo >> (8 * b) & 0xffu));
    f[r + 2] = __builtin_amdgcn_cvt_off_f32_i4((int)(hi >> (8 * b) & 0xffu));
  }
  if constexpr (ZEROS) {
#pragma unroll
    for (int r = 0; r < 8; ++r) f[r] += add;
  }
  uint32_t p[4];
#pragma unroll
  for (int e = 0; e < 4; ++e)
    p[e] = __builtin_amdgcn_perm(__float_as_uint(f[2 * e + 1]), __float_as_uint(f[2 * e]), 0x07060302u);
  return __builtin_bit_cast(bf16x8_t, make_uint4(p[0], p[1], p[2], p[3]));
}

// z of one output element of the pair.
__device__ __forceinline__ float pair_value(const Epi &ep, int col, float g, float u) {
  if (col >= ep.N) return 0.0f;
  if (ep.bias) g += ep.bias[col];
  if (ep.bias_u) u += ep.bias_u[col];
  return silu(g) * u;
}

template <int ACT, int GB, bool ZEROS, bool PAIR>
__global__ void __launch_bounds__(kThreads, 2)
w4_gemm_kernel(const W4Args a, int MB, int NBN) {
  constexpr bool kQ8 = ACT == kActQ8;
  constexpr int CH = GB < kCB ? GB : kCB;
  constexpr int NS = kCB / CH;
  constexpr int kStage = kA + (kQ8 ? kDx : 0);
  __shared__ __attribute__((aligned(16))) char lds[2 * kStage];

  const int G = MB * NBN, bid = (int)blockIdx.x;
  const int logical = G % 8 == 0 ? bid % 8 * (G / 8) + bid / 8 : bid;
  const int row0 = logical % MB * kRows, nb = logical / MB;

  const int tid = threadIdx.x, lane = tid & 63;
  const int q = lane >> 4, i = lane & 15;
  const int wave = __builtin_amdgcn_readfirstlane(tid >> 6);
  const int sel = PAIR ? wave >> 1 : 0;
  const int t = PAIR ? 2 * nb + (wave & 1) : 4 * nb + wave;   // this wave's tile
  const int tc = min(t, a.T - 1);          // (past the last: loads of the last, no stores)
  const W4 w = PAIR && sel ? a.w_u : a.w;
  const unsigned groups = (unsigned)w4_groups((int64_t)a.NB * 32, GB * 32);
  const buf_t wr = make_buf(w.values + (size_t)tc * a.NB * kW4Chunk, (unsigned)a.NB * kW4Chunk);
  const buf_t sr = make_buf(w.scales + (size_t)tc * groups * 128, groups * 128u);
  const buf_t zr = ZEROS ? make_buf(w.zeros + (size_t)tc * groups * 64, groups * 64u) : wr;

  // ---- the activation's stages
  // bf16: a wave loads 16 rows x 64 bytes at a time straight into LDS, lane L place
  // L % 4 of row L / 4; 4 such pieces a wave and stage.  Rows past m: the last row.
  constexpr int kPieces = kA / 1024 / 4;
  const unsigned lds0 = lds_offset(lds);
  unsigned aoff[kQ8 ? 1 : kPieces];
  const char *abase = static_cast<const char *>(a.x) + (size_t)row0 * a.K * (kQ8 ? 1 : 2);
  if constexpr (!kQ8) {
#pragma unroll
    for (int k = 0; k < kPieces; ++k) {
      const int piece = k * 4 + wave, cb = piece / kRG, r = piece % kRG * 16 + (lane >> 2);
      const unsigned rc = (unsigned)(min(row0 + r, a.m - 1) - row0);
      aoff[k] = rc * (unsigned)a.K * 2u + (unsigned)cb * 64u + (unsigned)(((lane & 3) ^ ((r >> 1) & 3)) * 16);
    }
  }
  // Q8_0: thread tid takes 16 codes (half a block) of row tid / 2, both blocks; and
  // the scale of block tid / 128 of row tid % 128
  const int qrow = tid >> 1, qhalf = tid & 1;
  const unsigned qoff = (unsigned)(min(row0 + qrow, a.m - 1) - row0) * (unsigned)a.K + (unsigned)qhalf * 16u;
  const float *dxp = reinterpret_cast<const float *>(static_cast<const char *>(a.x) + a.act_scale_off) +
                     (size_t)min(row0 + (tid & 127), a.m - 1) * a.NB;
  u32x4_t qv[kCB];
  float qd = 0.0f;
  const auto fetch = [&](int b0, int buf) Q8_INLINE {
    if constexpr (kQ8) {
#pragma unroll
      for (int cb = 0; cb < kCB; ++cb)
        qv[cb] = *reinterpret_cast<const u32x4_t *>(abase + (size_t)min(b0 + cb, a.NB - 1) * 32 + qoff);
      qd = dxp[min(b0 + (tid >> 7), a.NB - 1)];
    } else {
      // (the second block of a last odd stage is read from the first: never used)
      const int step = b0 + 1 < a.NB ? 0 : 64;
      const char *base = abase + (size_t)b0 * 64;
#pragma unroll
      for (int k = 0; k < kPieces; ++k) {
        const int piece = k * 4 + wave;
        load_to_lds16(base, aoff[k] - (piece >= kRG ? (unsigned)step : 0u),
                    lds0 + (unsigned)(buf * kStage + piece * 1024));
      }
    }
  };
  const auto put = [&](int buf) Q8_INLINE {      // Q8_0: the fetched codes into LDS
    if constexpr (kQ8) {
      char *d = lds + buf * kStage;
#pragma unroll
      for (int cb = 0; cb < kCB; ++cb) {
#pragma unroll
        for (int h = 0; h < 2; ++h)
          *reinterpret_cast<bf16x8_t *>(d + (cb * kRows + qrow) * 64 + a_place(qrow, 2 * qhalf + h)) =
              i8x8_to_bf16(make_uint2(qv[cb][2 * h], qv[cb][2 * h + 1]));
      }
      reinterpret_cast<float *>(d + kA)[tid] = qd;
    }
  };

  // ---- the weight's stages
  struct Weight {
    uint4 v[kCB];
    uint2 sc[NS];
    uint32_t z[NS];
  };
  const auto load = [&](Weight &st, int b) Q8_INLINE {
#pragma unroll
    for (int u = 0; u < kCB; ++u) {
      // (past K the last block again: a resource's extent need not bound an access by its
      // uniform offset)
      const unsigned at = (unsigned)(u ? min(b + u, a.NB - 1) : b) * kW4Chunk;
      const u32x4_t v = __builtin_amdgcn_raw_buffer_load_b128(wr, (unsigned)lane * 16u, at, 0);
      st.v[u] = make_uint4(v.x, v.y, v.z, v.w);
    }
    if constexpr (NS == 2) {
      const unsigned pair = (unsigned)(b / 2);
      const u32x4_t v = __builtin_amdgcn_raw_buffer_load_b128(sr, (unsigned)i * 16u, pair * 256u, 0);
      st.sc[0] = make_uint2(v.x, v.y);
      st.sc[1] = make_uint2(v.z, v.w);
      if constexpr (ZEROS) {
        const u32x2_t z = __builtin_amdgcn_raw_buffer_load_b64(zr, (unsigned)i * 8u, pair * 128u, 0);
        st.z[0] = z.x;
        st.z[1] = z.y;
      }
    } else {
      const unsigned j = (unsigned)(b / GB);
      const unsigned at = GB == 4 ? j * 128u : (j >> 1) * 256u + (j & 1u) * 8u;
      const u32x2_t v = __builtin_amdgcn_raw_buffer_load_b64(sr, (unsigned)i * (GB == 4 ? 8u : 16u), at, 0);
      st.sc[0] = make_uint2(v.x, v.y);
      if constexpr (ZEROS)
        st.z[0] = __builtin_amdgcn_raw_buffer_load_b32(zr, (unsigned)i * (GB == 4 ? 4u : 8u), at / 2u, 0);
    }
  };

  f32x4_t acc[kRG][4];
#pragma unroll
  for (int rg = 0; rg < kRG; ++rg)
#pragma unroll
    for (int g = 0; g < 4; ++g) acc[rg][g] = f32x4_t{0.0f, 0.0f, 0.0f, 0.0f};

  const int a_lane = i * 64 + a_place(i, q);
  const auto compute = [&](auto whole, const Weight &st, int buf, int nb_live) Q8_INLINE {
    constexpr bool WHOLE = decltype(whole)::value;   // both blocks are the weight's
    const char *As = lds + buf * kStage;
#pragma unroll
    for (int n = 0; n < NS; ++n) {
      float sc[4];
      w4_scales4(st.sc[n], a.scale_bf16 ? ~0u : 0u, sc);
      bf16x8_t bw[CH][4];
#pragma unroll
      for (int c = 0; c < CH; ++c) {
        const uint4 v = st.v[n * CH + c];
        const uint32_t wd[4] = {v.x, v.y, v.z, v.w};
#pragma unroll
        for (int g = 0; g < 4; ++g) {
          const float add = ZEROS ? 0.5f - (float)(st.z[n] >> (8 * g) & 0xffu) * 0.0625f : 0.0f;
          bw[c][g] = w4_signed<ZEROS>(wd[g], add);
        }
      }
      // the second block of a last odd stage: no part of a chained group (a group of
      // its own has the scale 0); its rows are the first block's again
      if (!WHOLE && CH == 2 && nb_live < kCB) {
#pragma unroll
        for (int g = 0; g < 4; ++g) bw[CH - 1][g] = __builtin_bit_cast(bf16x8_t, make_uint4(0, 0, 0, 0));
      }
      // a row group's products are issued while the one before is scaled; its operand
      // rows are read a row group ahead
      f32x4_t D[2][4], dx[2][CH];
      bf16x8_t av[2][CH];
      const auto read = [&](int rg) Q8_INLINE {
#pragma unroll
        for (int c = 0; c < CH; ++c) {
          av[rg & 1][c] = *reinterpret_cast<const bf16x8_t *>(As + ((n * CH + c) * kRows + rg * 16) * 64 + a_lane);
          if constexpr (kQ8)
            dx[rg & 1][c] = *reinterpret_cast<const f32x4_t *>(
                As + kA + ((n * CH + c) * kRows + rg * 16 + 4 * q) * 4);
        }
      };
      const auto scale = [&](int rg) Q8_INLINE {
#pragma unroll
        for (int g = 0; g < 4; ++g)
#pragma unroll
          for (int e = 0; e < 4; ++e) acc[rg][g][e] = fmaf(sc[g], D[rg & 1][g][e], acc[rg][g][e]);
        // (the sums are taken here: moved to the loop's end, the products wait in memory)
#pragma unroll
        for (int g = 0; g < 4; ++g) asm volatile("" : "+v"(acc[rg][g]));
      };
      read(0);
      // products before other waves' conversions: the SIMD's two waves then take turns
      // (2048 rows, K 4096, N 14336: 249 -> 222 us)
      __builtin_amdgcn_s_setprio(1);
#pragma unroll
      for (int rg = 0; rg < kRG; ++rg) {
        const int p = rg & 1;
        if constexpr (kQ8) {
          // the codes' sums are scaled by their rows' scales block by block
#pragma unroll
          for (int c = 0; c < CH; ++c) {
            f32x4_t d[4];
#pragma unroll
            for (int g = 0; g < 4; ++g)
              d[g] = __builtin_amdgcn_mfma_f32_16x16x32_bf16(av[p][c], bw[c][g], f32x4_t{0.0f, 0.0f, 0.0f, 0.0f}, 0, 0, 0);
            if (c == 0 && rg + 1 < kRG) read(rg + 1);
            if (c == 0 && rg > 0) scale(rg - 1);
#pragma unroll
            for (int g = 0; g < 4; ++g)
#pragma unroll
              for (int e = 0; e < 4; ++e)
                D[p][g][e] = c == 0 ? dx[p][c][e] * d[g][e] : fmaf(dx[p][c][e], d[g][e], D[p][g][e]);
          }
        } else {
#pragma unroll
          for (int c = 0; c < CH; ++c)
#pragma unroll
            for (int g = 0; g < 4; ++g)
              D[p][g] = __builtin_amdgcn_mfma_f32_16x16x32_bf16(
                  av[p][c], bw[c][g], c == 0 ? f32x4_t{0.0f, 0.0f, 0.0f, 0.0f} : D[p][g], 0, 0, 0);
          if (rg + 1 < kRG) read(rg + 1);
          if (rg > 0) scale(rg - 1);
        }
        if constexpr (!kQ8 && CH == 2) {
          // operand reads first, then two FMAs behind each matrix instruction
          if (rg + 1 < kRG) __builtin_amdgcn_sched_group_barrier(0x100, CH, 0);
#pragma unroll
          for (int k = 0; k < 8; ++k) {
            __builtin_amdgcn_sched_group_barrier(0x008, 1, 0);
            __builtin_amdgcn_sched_group_barrier(0x002, 2, 0);
          }
        }
        __builtin_amdgcn_sched_barrier(0);
      }
      __builtin_amdgcn_s_setprio(0);
      scale(kRG - 1);
    }
  };

  // ---- the stages in turn: while one is computed the next one's loads are in flight
  const auto ready = [&]() Q8_INLINE {           // this wave's loads have landed, then everyone's
    __builtin_amdgcn_s_waitcnt(0x0070);          // vmcnt(0) lgkmcnt(0)
    __builtin_amdgcn_sched_barrier(0);
    __syncthreads();
  };
  const int NC = (a.NB + kCB - 1) / kCB;
  Weight wa, wb;
  fetch(0, 0);
  load(wa, 0);
  put(0);
  for (int c = 0; c + 1 < NC; ++c) {
    ready();
    fetch((c + 1) * kCB, (c + 1) & 1);
    load(wb, (c + 1) * kCB);
    compute(std::true_type{}, wa, c & 1, kCB);
    put((c + 1) & 1);
    wa = wb;
  }
  ready();
  compute(std::false_type{}, wa, (NC - 1) & 1, a.NB - (NC - 1) * kCB);

  // ---- the outputs
#pragma unroll
  for (int rg = 0; rg < kRG; ++rg)
#pragma unroll
    for (int g = 0; g < 4; ++g) acc[rg][g] *= 16.0f;
  const Epi &ep = a.ep;
  if constexpr (!PAIR) {
    if (t >= a.T) return;
#pragma unroll
    for (int rg = 0; rg < kRG; ++rg)
#pragma unroll
      for (int e = 0; e < 4; ++e) {
        const int r = row0 + 16 * rg + 4 * q + e;
        if (r < a.m) {
#pragma unroll
          for (int g = 0; g < 4; ++g) {
            const int col = t * kTile + 16 * g + i;
            a.y[(size_t)r * a.Npad + col] = col < ep.N ? acc[rg][g][e] : 0.0f;
          }
        }
      }
  } else {
    // the two waves of a tile exchange halves of their rows, two row groups a round:
    // the gate's wave finishes rows 0..63, the up weight's rows 64..127
    float *x = reinterpret_cast<float *>(lds);   // [wave][2][16 rows][64 columns], lane-major
#pragma unroll
    for (int round = 0; round < 2; ++round) {
      __syncthreads();
#pragma unroll
      for (int k = 0; k < 2; ++k)
#pragma unroll
        for (int g = 0; g < 4; ++g) {
          f32x4_t *d = reinterpret_cast<f32x4_t *>(x + ((wave * 2 + k) * 4 + g) * 256 + lane * 4);
          if (sel)
            *d = acc[2 * round + k][g];
          else
            *d = acc[4 + 2 * round + k][g];
        }
      __syncthreads();
#pragma unroll
      for (int k = 0; k < 2; ++k) {
        f32x4_t z[4];
#pragma unroll
        for (int g = 0; g < 4; ++g) {
          const f32x4_t other = *reinterpret_cast<const f32x4_t *>(x + (((wave ^ 2) * 2 + k) * 4 + g) * 256 + lane * 4);
          const int col = tc * kTile + 16 * g + i;
#pragma unroll
          for (int e = 0; e < 4; ++e) {
            if (sel)
              z[g][e] = pair_value(ep, col, other[e], acc[4 + 2 * round + k][g][e]);
            else
              z[g][e] = pair_value(ep, col, acc[2 * round + k][g][e], other[e]);
          }
        }
        const int rg = (sel ? 4 : 0) + 2 * round + k;
#pragma unroll
        for (int e = 0; e < 4; ++e) {
          const int r = row0 + 16 * rg + 4 * q + e;
          const bool live = r < a.m && t < a.T;
          if (live && ep.write_y) {
#pragma unroll
            for (int g = 0; g < 4; ++g) a.y[(size_t)r * a.Npad + t * kTile + 16 * g + i] = z[g][e];
          }
          if (ep.yq) {
#pragma unroll
            for (int h = 0; h < 2; ++h) {         // 32 columns: column groups 2h and 2h + 1
              float top = fmaxf(fabsf(z[2 * h][e]), fabsf(z[2 * h + 1][e]));
#pragma unroll
              for (int o = 8; o > 0; o >>= 1) top = fmaxf(top, __shfl_xor(top, o, 16));
              if (live) {
                const float d = q8_scale_of(top);
                const size_t block = (size_t)t * 2 + h;
#pragma unroll
                for (int g = 0; g < 2; ++g) {
                  const int8_t code = q8_code_of(z[2 * h + g][e], d);
                  ep.yq[(size_t)r * a.Npad + block * 32 + 16 * g + i] = code;
                  ep.yq_view[(block * a.m + r) * 32 + 16 * g + i] = code;
                }
                if (i == 0) ep.yq_scale[(size_t)r * (a.Npad / 32) + block] = d;
              }
            }
          }
        }
      }
    }
  }
}

template <int ACT, bool PAIR>
hipError_t launch_g(const W4Args &a, hipStream_t stream) {
  const int MB = (a.m + kRows - 1) / kRows, per = PAIR ? 2 : 4, NBN = (a.T + per - 1) / per;
  const dim3 grid((unsigned)(MB * NBN)), block(kThreads);
  (void)hipGetLastError();
  const bool z = a.w.zeros != nullptr;
  switch (a.group) {
    case 32:
      if (z) w4_gemm_kernel<ACT, 1, true, PAIR><<<grid, block, 0, stream>>>(a, MB, NBN);
      else w4_gemm_kernel<ACT, 1, false, PAIR><<<grid, block, 0, stream>>>(a, MB, NBN);
      break;
    case 64:
      if (z) w4_gemm_kernel<ACT, 2, true, PAIR><<<grid, block, 0, stream>>>(a, MB, NBN);
      else w4_gemm_kernel<ACT, 2, false, PAIR><<<grid, block, 0, stream>>>(a, MB, NBN);
      break;
    case 128:
      if (z) w4_gemm_kernel<ACT, 4, true, PAIR><<<grid, block, 0, stream>>>(a, MB, NBN);
      else w4_gemm_kernel<ACT, 4, false, PAIR><<<grid, block, 0, stream>>>(a, MB, NBN);
      break;
    default: return hipErrorInvalidValue;
  }
  return hipGetLastError();
}

}  // namespace

hipError_t launch_w4_gemm(int act, bool pair, const W4Args &a, hipStream_t stream) {
  if (act == kActBf16) return pair ? launch_g<kActBf16, true>(a, stream) : launch_g<kActBf16, false>(a, stream);
  return pair ? launch_g<kActQ8, true>(a, stream) : launch_g<kActQ8, false>(a, stream);
}

}  // namespace q8
