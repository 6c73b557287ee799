// Device helpers of the 8-bit activation checkpoints.
#pragma once
#include <cuda_bf16.h>
#include <cstdint>

namespace muon {

// 2^(byte - 127) in bf16 in both halves; byte 0 is zero, byte 255 infinity.
__device__ __forceinline__ uint32_t act8_scale2(uint32_t byte) { return (byte << 7) | (byte << 23); }

// Four int8 to bf16, times the scales of elements 0, 1 and 2, 3. Low 7 bits under the exponent
// of 128 give 128 + low7, the sign bit there gives 128 or 256; their difference is the value,
// and both steps are exact.
__device__ __forceinline__ void act8_restore4(uint32_t w, uint32_t s01, uint32_t s23, uint32_t* lo, uint32_t* hi) {
  const uint32_t v = w & 0x7F7F7F7Fu, g = w & 0x80808080u, m = 0x43434343u;
  const uint32_t a0 = __byte_perm(v, m, 0x4140), a1 = __byte_perm(v, m, 0x4342);
  const uint32_t c0 = __byte_perm(g, m, 0x4140), c1 = __byte_perm(g, m, 0x4342);
  auto bf2 = [](uint32_t x) { return *reinterpret_cast<const __nv_bfloat162*>(&x); };
  const __nv_bfloat162 r0 = __hmul2(__hsub2(bf2(a0), bf2(c0)), bf2(s01));
  const __nv_bfloat162 r1 = __hmul2(__hsub2(bf2(a1), bf2(c1)), bf2(s23));
  *lo = *reinterpret_cast<const uint32_t*>(&r0);
  *hi = *reinterpret_cast<const uint32_t*>(&r1);
}

}  // namespace muon
