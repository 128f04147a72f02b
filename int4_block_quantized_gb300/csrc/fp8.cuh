// fp8.cuh -- FP8 (e4m3) tensors with a scale for each block of 128, shared by
// the quantisers and the reader (fp8.cu).
#pragma once

#include "mx.cuh"

namespace qmoe {

// Bits of the largest magnitude of 16 values; NaN and infinity order above
// every finite one.
__device__ __forceinline__ uint32_t fp8_max16(const float (&v)[16]) {
  float m = 0.f;
#pragma unroll
  for (int j = 0; j < 16; j += 2)
    asm("max.NaN.f32 %0, %0, %1, %2;" : "+f"(m) : "f"(fabsf(v[j])), "f"(fabsf(v[j + 1])));
  return __float_as_uint(m);
}
// The same over the eight neighbouring lanes that share a block (all of them
// call this).
__device__ __forceinline__ uint32_t fp8_group_max(uint32_t m) {
  const uint32_t mask = 0xffu << (threadIdx.x & 24);
#pragma unroll
  for (int o = 1; o < 8; o <<= 1) m = max(m, __shfl_xor_sync(mask, m, o));
  return m;
}

// A block's scale and codes, from the bits of its largest magnitude.  A block
// with a NaN or an infinity has a NaN scale and zero codes.
struct Fp8Block {
  float scale, inv;
  bool finite;
  __device__ __forceinline__ explicit Fp8Block(uint32_t max_bits) {
    finite = max_bits < 0x7f800000u;
    const float a = fmaxf(finite ? __uint_as_float(max_bits) : 1.f, 0x1p-100f);
    scale = finite ? __fdiv_rn(a, 448.f) : __uint_as_float(0x7fffffffu);
    inv = __fdiv_rn(448.f, a);
  }
  // v * inv cut towards zero, its last bit set where the cut was not exact
  __device__ __forceinline__ float odd(float v) const {
    const float t = __fmul_rz(v, inv);
    return __uint_as_float(__float_as_uint(t) | (__fmaf_rn(v, inv, -t) != 0.f ? 1u : 0u));
  }
  __device__ __forceinline__ uint4 codes16(const float (&v)[16]) const {
    uint32_t c[4];
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      c[i] = mx_e4m3x4(odd(v[4 * i]), odd(v[4 * i + 1]), odd(v[4 * i + 2]), odd(v[4 * i + 3]));
      if (!finite) c[i] = 0u;
    }
    return make_uint4(c[0], c[1], c[2], c[3]);
  }
};

}  // namespace qmoe
