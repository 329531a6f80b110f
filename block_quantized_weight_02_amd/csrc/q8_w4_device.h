// q8_w4_device.h -- device pieces that the 4-bit weight's kernels share.
#pragma once

#include <hip/hip_runtime.h>
#include <stdint.h>

namespace q8 {
namespace {

// A lane's four scales.  `bf16`: all ones where they are bf16, else 0: both conversions
// and a blend, since a branch would end the straight line that a stage is scheduled in.
__device__ __forceinline__ void w4_scales4(uint2 v, uint32_t bf16, float (&f)[4]) {
  const uint32_t bits[4] = {v.x & 0xffffu, v.x >> 16, v.y & 0xffffu, v.y >> 16};
  const uint32_t high[4] = {v.x << 16, v.x & 0xffff0000u, v.y << 16, v.y & 0xffff0000u};
#pragma unroll
  for (int g = 0; g < 4; ++g) {
    const float h = (float)__builtin_bit_cast(_Float16, (unsigned short)bits[g]);
    f[g] = __uint_as_float((bf16 & high[g]) | (~bf16 & __float_as_uint(h)));
  }
}

// 16 (4) bytes a lane straight into LDS at `at` + 16 (4) lane; base and `at` are the
// wave's.  Written out because the compiler would make every read of LDS wait for every
// such load, the next stages' too; loads_left waits for all but the last N.  m0, the
// load's base in LDS, is a register that the compiler sets right before its own uses.
__device__ __forceinline__ const char *wave_ptr(const char *p) {
  const uint64_t b = (uint64_t)p;
  const unsigned lo = __builtin_amdgcn_readfirstlane((unsigned)b);
  const unsigned hi = __builtin_amdgcn_readfirstlane((unsigned)(b >> 32));
  return reinterpret_cast<const char *>((uint64_t)hi << 32 | lo);
}
__device__ __forceinline__ void load_to_lds16(const char *base, unsigned off, unsigned at) {
  asm volatile("s_mov_b32 m0, %2\n\ts_nop 0\n\tglobal_load_lds_dwordx4 %0, %1"
               ::"v"(off), "s"(wave_ptr(base)), "s"(at) : "memory");
}
__device__ __forceinline__ void load_to_lds4(const char *base, unsigned off, unsigned at) {
  asm volatile("s_mov_b32 m0, %2\n\ts_nop 0\n\tglobal_load_lds_dword %0, %1"
               ::"v"(off), "s"(wave_ptr(base)), "s"(at) : "memory");
}
template <int N>
__device__ __forceinline__ void loads_left() {
  asm volatile("s_waitcnt vmcnt(%0)" ::"n"(N) : "memory");
}

// Byte offset of an object in LDS.
__device__ __forceinline__ unsigned lds_offset(const char *p) {
  return (unsigned)(size_t)(__attribute__((address_space(3))) const char *)p;
}

}  // namespace
}  // namespace q8
