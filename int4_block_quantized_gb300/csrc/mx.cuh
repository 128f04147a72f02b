// mx.cuh -- microscaled (MX) formats, shared by the quantisers, the reader
// and the product: the scale-tile index, e8m0 scales, e4m3 / e2m1 codes.
//
// A block is 32 consecutive elements of a row with one scale X = 2^(s - 127),
// s one byte (255: NaN).  A code is an e4m3 byte (MXFP8) or an e2m1 nibble
// (MXFP4, even k in the low nibble); an element is code * X.
#pragma once

#include <type_traits>

#include "common.cuh"

namespace qmoe {

constexpr int kMxfp8 = 0, kMxfp4 = 1;  // QMOE_MXFP8, QMOE_MXFP4

// Scales are kept in tiles of 128 rows x 4 blocks, 512 bytes each: the order
// in which a tensor-core product's scale operand lies in tensor memory (lane
// r % 32, column r / 32, four blocks to a 32-bit word), so a tile goes there
// as one contiguous copy.
__host__ __device__ __forceinline__ size_t mx_scale_index(int r, int b, int kt) {
  return ((size_t)(r >> 7) * kt + (b >> 2)) * 512 + (r & 31) * 16 + ((r >> 5) & 3) * 4 + (b & 3);
}

__device__ __forceinline__ float mx_scale(uint32_t s) {
  // 2^-127 is subnormal in fp32
  return __uint_as_float(s == 255u ? 0x7fffffffu : (s ? s << 23 : 0x00400000u));
}

// Scale byte of a block from the bits of its largest magnitude (the OCP rule
// floor(log2 max) - emax, emax = 8 for e4m3 and 2 for e2m1).  The biased fp32
// exponent is floor(log2) + 127; below fp32's normal range the clamp to
// 2^-127 decides.  NaN and infinity order above every finite magnitude.
template <int FMT>
__device__ __forceinline__ uint32_t mx_scale_byte(uint32_t amax_bits) {
  if (amax_bits >= 0x7f800000u) return 255u;
  const int s = (int)(amax_bits >> 23) - (FMT == kMxfp8 ? 8 : 2);
  return s > 0 ? (uint32_t)s : 0u;
}
// 1 / X, exact: s <= 254 - emax, so the exponent stays normal
__device__ __forceinline__ float mx_inv_scale(uint32_t s) { return __uint_as_float((254u - s) << 23); }

// Four e4m3 codes of four scaled values, round to nearest even, saturating.
__device__ __forceinline__ uint32_t mx_e4m3x4(float a, float b, float c, float d) {
  uint16_t lo, hi;
  asm("cvt.rn.satfinite.e4m3x2.f32 %0, %2, %1;" : "=h"(lo) : "f"(a), "f"(b));
  asm("cvt.rn.satfinite.e4m3x2.f32 %0, %2, %1;" : "=h"(hi) : "f"(c), "f"(d));
  return (uint32_t)lo | ((uint32_t)hi << 16);
}
// Eight e2m1 codes of eight scaled values, likewise; element j in nibble j.
__device__ __forceinline__ uint32_t mx_e2m1x8(const float* v) {
  uint32_t r;
  asm("{\n .reg .b8 b0, b1, b2, b3;\n"
      " cvt.rn.satfinite.e2m1x2.f32 b0, %2, %1;\n"
      " cvt.rn.satfinite.e2m1x2.f32 b1, %4, %3;\n"
      " cvt.rn.satfinite.e2m1x2.f32 b2, %6, %5;\n"
      " cvt.rn.satfinite.e2m1x2.f32 b3, %8, %7;\n"
      " mov.b32 %0, {b0, b1, b2, b3};\n}"
      : "=r"(r)
      : "f"(v[0]), "f"(v[1]), "f"(v[2]), "f"(v[3]), "f"(v[4]), "f"(v[5]), "f"(v[6]), "f"(v[7]));
  return r;
}
// Eight e2m1 codes to fp32 (exact; fp16 holds every e2m1 value).
__device__ __forceinline__ void mx_from_e2m1x8(uint32_t w, float* v) {
  uint32_t h[4];
  asm("{\n .reg .b8 b0, b1, b2, b3;\n mov.b32 {b0, b1, b2, b3}, %4;\n"
      " cvt.rn.f16x2.e2m1x2 %0, b0;\n cvt.rn.f16x2.e2m1x2 %1, b1;\n"
      " cvt.rn.f16x2.e2m1x2 %2, b2;\n cvt.rn.f16x2.e2m1x2 %3, b3;\n}"
      : "=r"(h[0]), "=r"(h[1]), "=r"(h[2]), "=r"(h[3])
      : "r"(w));
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    const float2 f = __half22float2(*reinterpret_cast<__half2*>(&h[i]));
    v[2 * i] = f.x;
    v[2 * i + 1] = f.y;
  }
}
// Four e4m3 codes to fp32 (exact; the NaN code gives NaN).
__device__ __forceinline__ void mx_from_e4m3x4(uint32_t w, float* v) {
  uint32_t h[2];
  asm("cvt.rn.f16x2.e4m3x2 %0, %1;" : "=r"(h[0]) : "h"((uint16_t)(w & 0xffffu)));
  asm("cvt.rn.f16x2.e4m3x2 %0, %1;" : "=r"(h[1]) : "h"((uint16_t)(w >> 16)));
#pragma unroll
  for (int i = 0; i < 2; ++i) {
    const float2 f = __half22float2(*reinterpret_cast<__half2*>(&h[i]));
    v[2 * i] = f.x;
    v[2 * i + 1] = f.y;
  }
}

// 32 bytes: one access on a 32-byte boundary (a whole sector; two 16-byte
// stores would reach L2 as two half sectors), else two of 16.
__device__ __forceinline__ void load32(const void* p, uint32_t (&w)[8]) {
  if ((reinterpret_cast<uintptr_t>(p) & 31) == 0) {
    asm volatile("ld.global.v8.b32 {%0, %1, %2, %3, %4, %5, %6, %7}, [%8];"
                 : "=r"(w[0]), "=r"(w[1]), "=r"(w[2]), "=r"(w[3]), "=r"(w[4]), "=r"(w[5]), "=r"(w[6]), "=r"(w[7])
                 : "l"(p)
                 : "memory");
  } else {
    const uint4 a = static_cast<const uint4*>(p)[0], b = static_cast<const uint4*>(p)[1];
    w[0] = a.x, w[1] = a.y, w[2] = a.z, w[3] = a.w, w[4] = b.x, w[5] = b.y, w[6] = b.z, w[7] = b.w;
  }
}
__device__ __forceinline__ void store32(void* p, const uint32_t (&w)[8]) {
  if ((reinterpret_cast<uintptr_t>(p) & 31) == 0) {
    asm volatile("st.global.v8.b32 [%8], {%0, %1, %2, %3, %4, %5, %6, %7};" ::"r"(w[0]), "r"(w[1]), "r"(w[2]), "r"(w[3]),
                 "r"(w[4]), "r"(w[5]), "r"(w[6]), "r"(w[7]), "l"(p)
                 : "memory");
  } else {
    static_cast<uint4*>(p)[0] = make_uint4(w[0], w[1], w[2], w[3]);
    static_cast<uint4*>(p)[1] = make_uint4(w[4], w[5], w[6], w[7]);
  }
}

// Sixteen elements of fp16, bf16 or fp32 at element i (a multiple of 16).
template <typename T>
__device__ __forceinline__ void load16(const void* base, size_t i, float (&v)[16]) {
  const uint8_t* p = static_cast<const uint8_t*>(base) + i * sizeof(T);
  uint32_t w[8];
  if constexpr (sizeof(T) == 4) {
#pragma unroll
    for (int q = 0; q < 2; ++q) {
      load32(p + 32 * q, w);
#pragma unroll
      for (int j = 0; j < 8; ++j) v[q * 8 + j] = __uint_as_float(w[j]);
    }
  } else {
    load32(p, w);
#pragma unroll
    for (int j = 0; j < 8; ++j) {
      v[2 * j] = Half<T>::to_float((uint16_t)(w[j] & 0xffffu));
      v[2 * j + 1] = Half<T>::to_float((uint16_t)(w[j] >> 16));
    }
  }
}
// sixteen values rounded to a 16-bit type
template <typename T>
__device__ __forceinline__ void pack16(const float (&v)[16], uint32_t (&w)[8]) {
#pragma unroll
  for (int j = 0; j < 8; ++j) {
    if constexpr (std::is_same<T, __nv_bfloat16>::value) {
      const __nv_bfloat162 h = __floats2bfloat162_rn(v[2 * j], v[2 * j + 1]);
      w[j] = *reinterpret_cast<const uint32_t*>(&h);
    } else {
      const __half2 h = __floats2half2_rn(v[2 * j], v[2 * j + 1]);
      w[j] = *reinterpret_cast<const uint32_t*>(&h);
    }
  }
}
template <typename T>
__device__ __forceinline__ void store16(void* base, size_t i, const float (&v)[16]) {
  uint8_t* p = static_cast<uint8_t*>(base) + i * sizeof(T);
  uint32_t w[8];
  if constexpr (sizeof(T) == 4) {
#pragma unroll
    for (int q = 0; q < 2; ++q) {
#pragma unroll
      for (int j = 0; j < 8; ++j) w[j] = __float_as_uint(v[q * 8 + j]);
      store32(p + 32 * q, w);
    }
  } else {
    pack16<T>(v, w);
    store32(p, w);
  }
}

// Rows of `per_row` units walked with a fixed stride: one 32-bit division at
// the start and at the stride, none per step (a 64-bit one cost the reader a
// quarter of its time).
struct RowWalk {
  uint32_t per_row, dr, du, r, u;
  __device__ __forceinline__ RowWalk(uint32_t start, uint32_t stride, uint32_t per_row_)
      : per_row(per_row_), dr(stride / per_row_), r(start / per_row_) {
    du = stride - dr * per_row;
    u = start - r * per_row;
  }
  __device__ __forceinline__ void next() {
    r += dr;
    u += du;
    if (u >= per_row) {
      u -= per_row;
      ++r;
    }
  }
};

// Half a block per thread, the other half in the neighbouring lane (lane ^
// 1).  Both lanes of a pair call these.
__device__ __forceinline__ uint32_t mx_pair_mask() { return 3u << (threadIdx.x & 30); }
// The largest magnitude of the block, as bits; NaN where the block has one.
__device__ __forceinline__ uint32_t mx_block_max(const float (&v)[16]) {
  float m = 0.f;
#pragma unroll
  for (int j = 0; j < 16; j += 2)
    asm("max.NaN.f32 %0, %0, %1, %2;" : "+f"(m) : "f"(fabsf(v[j])), "f"(fabsf(v[j + 1])));
  const uint32_t b = __float_as_uint(m);
  return max(b, __shfl_xor_sync(mx_pair_mask(), b, 1));
}
// Codes of sixteen values times `scale`.
template <int FMT>
struct MxCodes {
  uint32_t w[FMT == kMxfp8 ? 4 : 2];
  __device__ __forceinline__ void set(const float (&v)[16], float scale) {
    float u[8];
#pragma unroll
    for (int h = 0; h < 2; ++h) {
#pragma unroll
      for (int j = 0; j < 8; ++j) u[j] = v[8 * h + j] * scale;
      if constexpr (FMT == kMxfp8) {
        w[2 * h] = mx_e4m3x4(u[0], u[1], u[2], u[3]);
        w[2 * h + 1] = mx_e4m3x4(u[4], u[5], u[6], u[7]);
      } else {
        w[h] = mx_e2m1x8(u);
      }
    }
  }
  __device__ __forceinline__ bool same(const MxCodes& o) const {
    uint32_t d = 0;
#pragma unroll
    for (uint32_t i = 0; i < sizeof(w) / 4; ++i) d |= w[i] ^ o.w[i];
    return d == 0;
  }
  // at element i; `keep` = false: zeros (a block with a NaN or infinity)
  __device__ __forceinline__ void store(uint8_t* codes, size_t i, bool keep) const {
    if constexpr (FMT == kMxfp8)
      *reinterpret_cast<uint4*>(codes + i) = keep ? make_uint4(w[0], w[1], w[2], w[3]) : make_uint4(0, 0, 0, 0);
    else
      *reinterpret_cast<uint2*>(codes + i / 2) = keep ? make_uint2(w[0], w[1]) : make_uint2(0, 0);
  }
};
// scale byte of the block (returned) and codes
template <int FMT>
__device__ __forceinline__ uint32_t mx_encode16(const float (&v)[16], uint8_t* codes, size_t i) {
  const uint32_t s = mx_scale_byte<FMT>(mx_block_max(v));
  MxCodes<FMT> c;
  c.set(v, mx_inv_scale(s == 255u ? 127u : s));
  c.store(codes, i, s != 255u);
  return s;
}

// Zeroes of the scale tiles' padding, split over n_threads threads: the rows
// M .. a multiple of 128 (words), and in the rows below M the blocks K / 32 ..
// a multiple of 4 (bytes).
__host__ __device__ __forceinline__ uint32_t mx_padding_words(int M, int K) {
  return (uint32_t)(-M & 127) * (uint32_t)((K + 127) / 128);
}
__device__ __forceinline__ void mx_zero_rows(uint8_t* scales, int M, int K, uint32_t thread, uint32_t n_threads) {
  const int kt = (K + 127) / 128;
  const uint32_t words = mx_padding_words(M, K), rows = (uint32_t)(-M & 127);
  for (uint32_t i = thread; i < words; i += n_threads)  // along the rows: neighbours in a tile
    *reinterpret_cast<uint32_t*>(scales + mx_scale_index(M + (int)(i % rows), 4 * (int)(i / rows), kt)) = 0u;
}
__device__ __forceinline__ void mx_zero_padding(uint8_t* scales, int M, int K, uint32_t thread, uint32_t n_threads) {
  const int nb = K / 32, kt = (K + 127) / 128;
  mx_zero_rows(scales, M, K, thread, n_threads);
  if (nb & 3)
    for (uint32_t r = thread; r < (uint32_t)M; r += n_threads)
      for (int b = nb; b < 4 * kt; ++b) scales[mx_scale_index((int)r, b, kt)] = 0;
}

}  // namespace qmoe
