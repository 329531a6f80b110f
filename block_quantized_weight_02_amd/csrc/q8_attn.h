// q8_attn.h -- device parts that the two attention kernels share: which tiles
// of a sequence a row range sees, page lookups, and the output's store.
#pragma once

#include <hip/hip_runtime.h>

#include "q8_device.h"
#include "q8_kv.h"

namespace q8 {
namespace {

using namespace dev;

// Where a running maximum starts: finite, and no finite score is below it.
constexpr float kLowest = -3.402823466e38f;

// A value all lanes hold alike, in a scalar register.
__device__ __forceinline__ int uni(int v) { return __builtin_amdgcn_readfirstlane(v); }

// A value made opaque where it is used: what is computed from it stays there
// rather than being kept in registers across the token stream.
__device__ __forceinline__ int here(int v) {
  asm volatile("" : "+v"(v));
  return v;
}

// The tiles of KT tokens that rows at positions p0 .. p1 of a sequence
// see: tiles 0 .. a-1 (the first tokens kept under a window), then t0 .. up to
// p1's.  Tile u of the nt is tile u (u < a) or u - a + t0.
struct Span {
  int a, t0, nt;
  __device__ __forceinline__ int tile(int u) const { return u < a ? u : u - a + t0; }
};
template <int KT>
__device__ __forceinline__ Span span_of(int p0, int p1, int window, int sinks) {
  Span s;
  const int lo = (window > 0 && p0 >= window) ? p0 - window + 1 : 0;
  s.t0 = lo / KT;
  s.a = (int)(((long long)min(sinks, lo) + KT - 1) / KT);
  if (s.a >= s.t0) s.a = s.t0 = 0;
  s.nt = p1 < 0 ? 0 : s.a + p1 / KT + 1 - s.t0;
  return s;
}

__device__ __forceinline__ int clamp_len(int len, long long max_pages, int page_log2) {
  return (int)min((long long)max(len, 0), max_pages << page_log2);
}

// Four fp32 values of output row r, columns col .. col+3 (col a multiple of
// 4): bf16 and/or the quantized form.  Called by whole groups of eight lanes
// that hold a 32-column block.
__device__ __forceinline__ void store_out(const AttnArgs &a, int r, int col, float4 v) {
  const int K = a.q_heads * a.cache.dim;
  if (a.o) {
    const uint32_t lo = (uint32_t)__builtin_bit_cast(uint16_t, (__bf16)v.x) |
                        (uint32_t)__builtin_bit_cast(uint16_t, (__bf16)v.y) << 16;
    const uint32_t hi = (uint32_t)__builtin_bit_cast(uint16_t, (__bf16)v.z) |
                        (uint32_t)__builtin_bit_cast(uint16_t, (__bf16)v.w) << 16;
    *reinterpret_cast<uint2 *>(a.o + (size_t)r * K + col) = make_uint2(lo, hi);
  }
  if (a.oq) {
    float am = fmaxf(fmaxf(fabsf(v.x), fabsf(v.y)), fmaxf(fabsf(v.z), fabsf(v.w)));
#pragma unroll
    for (int o = 4; o > 0; o >>= 1) am = fmaxf(am, __shfl_xor(am, o));
    const float d = q8_scale_of(am);
    const uint32_t w = (uint32_t)(uint8_t)q8_code_of(v.x, d) |
                       (uint32_t)(uint8_t)q8_code_of(v.y, d) << 8 |
                       (uint32_t)(uint8_t)q8_code_of(v.z, d) << 16 |
                       (uint32_t)(uint8_t)q8_code_of(v.w, d) << 24;
    *reinterpret_cast<uint32_t *>(a.oq + (size_t)r * K + col) = w;
    *reinterpret_cast<uint32_t *>(a.oq_view + ((size_t)(col >> 5) * a.m + r) * 32 + (col & 31)) = w;
    if ((col & 31) == 0) a.oq_scale[(size_t)r * (K >> 5) + (col >> 5)] = d;
  }
}

// Eight fp32 -> eight bf16, nearest even.
__device__ __forceinline__ bf16x8_t to_bf16x8(const float *f) {
  bf16x8_t v;
#pragma unroll
  for (int e = 0; e < 8; ++e) v[e] = (__bf16)f[e];
  return v;
}

__device__ __forceinline__ float exp2_fast(float x) { return __builtin_amdgcn_exp2f(x); }

// Waits for the thread's own stores, so that a following arrival count is not
// seen before them (as in finish_tile, whose protocol the joins share).
__device__ __forceinline__ void stores_done() {
  __atomic_signal_fence(__ATOMIC_SEQ_CST);
  __builtin_amdgcn_s_waitcnt(0);
  __atomic_signal_fence(__ATOMIC_SEQ_CST);
}

}  // namespace
}  // namespace q8
