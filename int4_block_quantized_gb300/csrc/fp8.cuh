// fp8.cuh -- FP8 (e4m3) tensors with a scale for each block of 128, shared by
// the quantisers and the reader (fp8.cu).
#pragma once

#include "mx.cuh"

namespace qmoe {

// Sixteen elements of fp16, bf16 or fp32 as they lie in memory, and the bits (as
// fp32) of their largest magnitude: magnitudes order as integers, NaN and
// infinity above every finite one, 16-bit ones two at a time.
template <typename T>
struct Sixteen {
  uint32_t w[sizeof(T) / 2][8];
  __device__ __forceinline__ void load(const void* base, size_t i) {
#pragma unroll
    for (uint32_t q = 0; q < sizeof(T) / 2; ++q) load32(static_cast<const uint8_t*>(base) + i * sizeof(T) + 32 * q, w[q]);
  }
  __device__ __forceinline__ void clear() {
#pragma unroll
    for (uint32_t q = 0; q < sizeof(T) / 2; ++q)
#pragma unroll
      for (int j = 0; j < 8; ++j) w[q][j] = 0;
  }
  // in the elements' own format, two of them where they have 16 bits
  __device__ __forceinline__ uint32_t max_raw() const {
    uint32_t m = 0;
#pragma unroll
    for (uint32_t q = 0; q < sizeof(T) / 2; ++q)
#pragma unroll
      for (int j = 0; j < 8; j += 2) {
        if constexpr (sizeof(T) == 4) m = __vimax3_u32(m, w[q][j] & 0x7fffffffu, w[q][j + 1] & 0x7fffffffu);
        else m = __vimax3_u16x2(m, w[q][j] & 0x7fff7fffu, w[q][j + 1] & 0x7fff7fffu);
      }
    return m;
  }
  static __device__ __forceinline__ uint32_t max_bits(uint32_t raw) {
    if constexpr (sizeof(T) == 4) return raw;
    else return __float_as_uint(Half<T>::to_float((uint16_t)max(raw & 0xffffu, raw >> 16)));
  }
  // the lowest of them where one is below zero (its bits are then the largest, but
  // for a NaN's), else some other, as fp32
  __device__ __forceinline__ float lowest() const {
    uint32_t m = 0;
#pragma unroll
    for (uint32_t q = 0; q < sizeof(T) / 2; ++q)
#pragma unroll
      for (int j = 0; j < 8; j += 2) {
        if constexpr (sizeof(T) == 4) m = __vimax3_u32(m, w[q][j], w[q][j + 1]);
        else m = __vimax3_u16x2(m, w[q][j], w[q][j + 1]);
      }
    if constexpr (sizeof(T) == 4) return __uint_as_float(m);
    else return Half<T>::to_float((uint16_t)max(m & 0xffffu, m >> 16));
  }
  __device__ __forceinline__ void values(float (&v)[16]) const {
#pragma unroll
    for (int j = 0; j < 8; ++j) {
      if constexpr (sizeof(T) == 4) {
        v[j] = __uint_as_float(w[0][j]);
        v[8 + j] = __uint_as_float(w[1][j]);
      } else {
        v[2 * j] = Half<T>::to_float((uint16_t)(w[0][j] & 0xffffu));
        v[2 * j + 1] = Half<T>::to_float((uint16_t)(w[0][j] >> 16));
      }
    }
  }
};
// the same bits of 16 values
__device__ __forceinline__ uint32_t fp8_max16(const float (&v)[16]) {
  uint32_t m = 0;
#pragma unroll
  for (int j = 0; j < 16; j += 2)
    m = __vimax3_u32(m, __float_as_uint(v[j]) & 0x7fffffffu, __float_as_uint(v[j + 1]) & 0x7fffffffu);
  return m;
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
  // v * inv cut towards zero, its last bit set where the cut was not exact (the
  // rest is then no zero, nor is its sign bit alone set)
  __device__ __forceinline__ f2 odd(float x, float y) const {
    f2 t, e;
    asm("{\n .reg .b64 v, i, t;\n mov.b64 v, {%2, %3};\n mov.b64 i, {%4, %4};\n mul.rz.f32x2 t, v, i;\n"
        " mov.b64 {%0, %1}, t;\n}"
        : "=f"(t.x), "=f"(t.y)
        : "f"(x), "f"(y), "f"(inv));
    e = ffma2(make_float2(x, y), make_float2(-inv, -inv), t);
    return make_float2(__uint_as_float(__float_as_uint(t.x) | min(__float_as_uint(e.x), 1u)),
                       __uint_as_float(__float_as_uint(t.y) | min(__float_as_uint(e.y), 1u)));
  }
  __device__ __forceinline__ uint4 codes16(const float (&v)[16]) const {
    uint32_t c[4];
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      const f2 a = odd(v[4 * i], v[4 * i + 1]), b = odd(v[4 * i + 2], v[4 * i + 3]);
      c[i] = mx_e4m3x4(a.x, a.y, b.x, b.y);
    }
    return finite ? make_uint4(c[0], c[1], c[2], c[3]) : make_uint4(0, 0, 0, 0);
  }
};

}  // namespace qmoe
