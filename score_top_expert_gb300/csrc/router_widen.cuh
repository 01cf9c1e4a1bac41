// 8-bit integers as fp16, for the products on the 16-bit tensor cores, and their scales.
#pragma once

#include <cuda_fp16.h>
#include <stdint.h>

namespace moe_router {

// Two signed bytes of u (offset by 128) as fp16: 1024 + byte by placing it in the low
// mantissa bits, then 1152 less; both exact.
__device__ __forceinline__ uint32_t widen_two(uint32_t u, uint32_t select) {
  const uint32_t v = __byte_perm(u, 0x64646464u, select);
  const uint32_t offset = 0x64806480u;
  const __half2 d = __hsub2(*reinterpret_cast<const __half2*>(&v),
                            *reinterpret_cast<const __half2*>(&offset));
  return *reinterpret_cast<const uint32_t*>(&d);
}

// Eight signed bytes in order.
__device__ __forceinline__ uint4 widen_eight(uint32_t a, uint32_t b) {
  a ^= 0x80808080u;
  b ^= 0x80808080u;
  return make_uint4(widen_two(a, 0x4140), widen_two(a, 0x4342), widen_two(b, 0x4140),
                    widen_two(b, 0x4342));
}

// A sum of integers with its output channel's and its row's scale, in both 8-bit kernels.  One
// after the other: the product of the scales alone may be subnormal or infinite where the output
// is an ordinary number (a row of 2^-126, the quantiser's smallest).  The channel's first: it is
// a parameter of ordinary size, while a row's may lie anywhere, and the sum is a whole number.
__device__ __forceinline__ float scaled_sum(float sum, float channel, float row) {
  return sum * channel * row;
}

}  // namespace moe_router
