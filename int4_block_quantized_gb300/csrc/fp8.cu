// fp8.cu -- FP8 tensors with a scale for each block of 128: quantisation of
// activations (a row's 128 columns share a scale; in token order, or written to
// the places that the experts' order gives; of SwiGLU's output) and of weights
// (128 x 128 elements share one), and the reader.
//
//   a = max(2^-100, largest magnitude of the block)
//   scale = RN(a / 448), code = RN_e4m3(v * RN(448 / a)), value = code * scale
//
// The product v * RN(448 / a) is rounded once, to the code: it is first cut to
// fp32 towards zero with its last bit set where something was cut off ("round to
// odd"), which no border between codes can be mistaken for.  Rounding it to fp32
// in between would move the elements whose fp32 product happens to be such a
// border: one in a million.
#include "fp8.cuh"
#include "launch.h"

namespace qmoe {

static dim3 fp8_grid(size_t work) {
  const size_t cap = (size_t)device_sm_count() * 32;
  const size_t b = (work + 255) / 256;
  return dim3((unsigned)(b < 1 ? 1 : b > cap ? cap : b));
}

// -------------------------------------------------------------- activations
// Eight lanes take a block, 16 elements each (a row's last block may have
// fewer: its other lanes bring zeros).  With places, a token is quantised once
// and written to each of its k rows.  Bound by HBM and, nearly as much, by its
// eleven instructions an element: 8192 x 4096 bf16 in 17.7 us, 5.7 TB/s.
template <typename T, bool PLACES>
__global__ void __launch_bounds__(256) fp8_rows_kernel(const void* __restrict__ x, int M, int K,
                                                       const int32_t* __restrict__ pos, int k,
                                                       uint8_t* __restrict__ codes, float* __restrict__ scales) {
  pdl_wait();
  const uint32_t nb = (uint32_t)(K + 127) / 128, rows = PLACES ? (uint32_t)M * k : (uint32_t)M;
  for (RowWalk w(blockIdx.x * 256 + threadIdx.x, gridDim.x * 256, nb * 8); w.r < (uint32_t)M; w.next()) {
    const bool in = 16 * w.u < (uint32_t)K;
    Sixteen<T> raw;
    if (in) raw.load(x, (size_t)w.r * K + 16 * w.u);
    else raw.clear();
    const Fp8Block b(fp8_group_max(Sixteen<T>::max_bits(raw.max_raw())));
    float v[16];
    raw.values(v);
    const uint4 c = b.codes16(v);
    if (!PLACES) {
      if (in) *reinterpret_cast<uint4*>(codes + (size_t)w.r * K + 16 * w.u) = c;
      if (!(w.u & 7)) scales[(size_t)w.r * nb + w.u / 8] = b.scale;
    } else {
      for (int j0 = 0; j0 < k; j0 += 4) {
        uint32_t p[4];
#pragma unroll
        for (int j = 0; j < 4; ++j) p[j] = j0 + j < k ? (uint32_t)pos[(size_t)w.r * k + j0 + j] : ~0u;
#pragma unroll
        for (int j = 0; j < 4; ++j) {
          if (p[j] >= rows) continue;  // this assignment goes nowhere
          if (in) *reinterpret_cast<uint4*>(codes + (size_t)p[j] * K + 16 * w.u) = c;
          if (!(w.u & 7)) scales[(size_t)p[j] * nb + w.u / 8] = b.scale;
        }
      }
    }
  }
}

// silu(g) * u of h [M, 2 I] (gate, then up), in fp32, quantised as above.  Bound by
// instructions, the exponential's and the quantiser's: 8192 x 1408 bf16 in 13.9 us,
// 4.2 TB/s (a tenth less with an exponential that loses accuracy far from 0).
//
// Below kDeepGate exp(-g) comes near the end of fp32, and its reciprocal is no
// normal number any more.  1 + exp(g) is 1 there, and g exp(g) u is computed as
// g exp(g + 96) (u 2^-64) (2^64 exp(-96)), whose factors and products are normal
// numbers for every u that leaves a code (g + 96 is exact down to -192; what is
// further below is no code for any u).  Such gates are rare, and a thread asks once
// whether it has one among its 16.  What it does then is a function of its own:
// unrolled in place it takes registers of everybody (bf16 7 to 16 % slower than without
// it; so, 3, and fp16 8).
constexpr float kDeepGate = -87.f;
__device__ __forceinline__ float fp8_swiglu(float g, float u) {
  float r;  // (a rounded quotient takes eight instructions more)
  asm("rcp.approx.ftz.f32 %0, %1;" : "=f"(r) : "f"(1.f + expf(-g)));
  return u * (g * r);
}
__device__ __forceinline__ float fp8_swiglu_deep(float g, float u) {
  return g * expf(g + 96.f) * (u * 0x1p-64f) * 3.7467047e-23f;
}
// v's elements with such gates; h from the first of the 16 gates on
template <typename T>
__device__ __noinline__ void fp8_swiglu_deep16(const void* h, size_t at, int I, float* v) {
  float g[16], u[16];
  load16<T>(h, at, g);
  load16<T>(h, at + I, u);
#pragma unroll
  for (int j = 0; j < 16; ++j)
    if (g[j] < kDeepGate) v[j] = fp8_swiglu_deep(g[j], u[j]);
}
template <typename T>
__global__ void __launch_bounds__(256) fp8_swiglu_kernel(const void* __restrict__ h, int M, int I,
                                                         uint8_t* __restrict__ codes, float* __restrict__ scales) {
  pdl_wait();
  const uint32_t nb = (uint32_t)(I + 127) / 128;
  for (RowWalk w(blockIdx.x * 256 + threadIdx.x, gridDim.x * 256, nb * 8); w.r < (uint32_t)M; w.next()) {
    const bool in = 16 * w.u < (uint32_t)I;
    float v[16] = {};
    if (in) {
      const size_t at = (size_t)w.r * 2 * I + 16 * w.u;
      float g[16];
      Sixteen<T> gate;
      gate.load(h, at);
      load16<T>(h, at + I, v);
      gate.values(g);
      const bool deep = !(gate.lowest() >= kDeepGate);
#pragma unroll
      for (int j = 0; j < 16; ++j) v[j] = fp8_swiglu(g[j], v[j]);
      if (deep) {
        float t[16];
#pragma unroll
        for (int j = 0; j < 16; ++j) t[j] = v[j];
        fp8_swiglu_deep16<T>(h, at, I, t);
#pragma unroll
        for (int j = 0; j < 16; ++j) v[j] = t[j];
      }
    }
    const Fp8Block b(fp8_group_max(fp8_max16(v)));
    const uint4 c = b.codes16(v);
    if (in) *reinterpret_cast<uint4*>(codes + (size_t)w.r * I + 16 * w.u) = c;
    if (!(w.u & 7)) scales[(size_t)w.r * nb + w.u / 8] = b.scale;
  }
}

// ------------------------------------------------------------------ weights
// One CTA per 128 x 128 block: a thread takes 16 columns of four rows, which it
// keeps as they came until the block's maximum is known.  Five CTAs an SM, so that
// others load while one reduces or writes (three: 91 us, four: 84).  Bound by HBM:
// 60 x 1408 x 2048 fp16 in 77 us, 6.8 TB/s.
template <typename T>
__global__ void __launch_bounds__(256, sizeof(T) == 4 ? 2 : 5) fp8_weights_kernel(const void* __restrict__ w, int N, int K,
                                                          uint8_t* __restrict__ codes, float* __restrict__ scales) {
  pdl_wait();
  const uint32_t nb = (uint32_t)(K + 127) / 128, rb = (uint32_t)(N + 127) / 128;
  const uint32_t b = blockIdx.x % nb, q = blockIdx.x / nb, r = q % rb, e = q / rb;
  const uint32_t col = b * 128 + (threadIdx.x & 7) * 16, row = r * 128 + threadIdx.x / 8;
  const size_t at = ((size_t)e * N + row) * K + col;
  Sixteen<T> raw[4];
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    if (col < (uint32_t)K && row + 32 * i < (uint32_t)N) raw[i].load(w, at + (size_t)32 * i * K);
    else raw[i].clear();
  }
  uint32_t m = 0;
#pragma unroll
  for (int i = 0; i < 4; ++i) m = max(m, Sixteen<T>::max_bits(raw[i].max_raw()));
  m = __reduce_max_sync(0xffffffffu, m);
  __shared__ uint32_t part[8];
  if ((threadIdx.x & 31) == 0) part[threadIdx.x / 32] = m;
  __syncthreads();
#pragma unroll
  for (int i = 0; i < 8; ++i) m = max(m, part[i]);
  const Fp8Block blk(m);
#pragma unroll
  for (int i = 0; i < 4; ++i)
    if (col < (uint32_t)K && row + 32 * i < (uint32_t)N) {
      float v[16];
      raw[i].values(v);
      *reinterpret_cast<uint4*>(codes + at + (size_t)32 * i * K) = blk.codes16(v);
    }
  if (threadIdx.x == 0) scales[blockIdx.x] = blk.scale;
}

// ------------------------------------------------------------------- reader
// code * scale in fp32, rounded once to T.  BR: rows that share a scale.  Bound by
// HBM: 60 x 1408 x 2048 to fp16 in 78 us, 6.7 TB/s.
template <typename T, int BR>
__global__ void __launch_bounds__(256) fp8_dequant_kernel(const uint8_t* __restrict__ codes,
                                                          const float* __restrict__ scales, int E, int N, int K,
                                                          void* __restrict__ out) {
  pdl_wait();
  const uint32_t nb = (uint32_t)(K + 127) / 128, rb = (uint32_t)(N + BR - 1) / BR, rows = (uint32_t)E * N;
  for (RowWalk w(blockIdx.x * 256 + threadIdx.x, gridDim.x * 256, (uint32_t)K / 16); w.r < rows; w.next()) {
    const size_t i = (size_t)w.r * K + 16 * w.u;
    uint32_t sr = w.r;
    if constexpr (BR > 1) {
      const uint32_t e = w.r / N;
      sr = e * rb + (w.r - e * N) / BR;
    }
    const float s = scales[(size_t)sr * nb + w.u / 8];
    const uint4 c = *reinterpret_cast<const uint4*>(codes + i);
    float v[16];
    mx_from_e4m3x4(c.x, v);
    mx_from_e4m3x4(c.y, v + 4);
    mx_from_e4m3x4(c.z, v + 8);
    mx_from_e4m3x4(c.w, v + 12);
#pragma unroll
    for (int j = 0; j < 16; ++j) v[j] *= s;
    store16<T>(out, i, v);
  }
}

template <typename T>
static cudaError_t quantize_t(const void* x, int M, int K, const int32_t* pos, int k, uint8_t* codes, float* scales,
                              cudaStream_t st) {
  const dim3 g = fp8_grid((size_t)M * ((K + 127) / 128) * 8);
  return launch_kernel(pos ? fp8_rows_kernel<T, true> : fp8_rows_kernel<T, false>, g, dim3(256), 0, st, true, x, M, K, pos,
                       k, codes, scales);
}
template <typename T>
static cudaError_t swiglu_t(const void* h, int M, int I, uint8_t* codes, float* scales, cudaStream_t st) {
  return launch_kernel(fp8_swiglu_kernel<T>, fp8_grid((size_t)M * ((I + 127) / 128) * 8), dim3(256), 0, st, true, h, M, I,
                       codes, scales);
}
template <typename T>
static cudaError_t weights_t(const void* w, int E, int N, int K, uint8_t* codes, float* scales, cudaStream_t st) {
  const long long blocks = (long long)E * ((N + 127) / 128) * ((K + 127) / 128);
  if (blocks > 0x7fffffffLL) return cudaErrorInvalidValue;
  return launch_kernel(fp8_weights_kernel<T>, dim3((unsigned)blocks), dim3(256), 0, st, true, w, N, K, codes, scales);
}
template <typename T>
static cudaError_t dequant_t(const uint8_t* codes, const float* scales, int E, int N, int K, int block_rows, void* out,
                             cudaStream_t st) {
  const dim3 g = fp8_grid((size_t)E * N * (K / 16));
  return launch_kernel(block_rows == 1 ? fp8_dequant_kernel<T, 1> : fp8_dequant_kernel<T, 128>, g, dim3(256), 0, st, true,
                       codes, scales, E, N, K, out);
}
// fn(T{}) with the element type of a qmoe_dtype
template <typename F>
static cudaError_t by_type(int dtype, F fn) {
  if (dtype == QMOE_F32) return fn(float{});
  if (dtype == QMOE_BF16) return fn(__nv_bfloat16{});
  return fn(__half{});
}

cudaError_t launch_fp8_quantize(const void* x, int x_dtype, int T, int K, const int32_t* pos, int k, uint8_t* codes,
                                float* scales, cudaStream_t st) {
  return by_type(x_dtype, [&](auto t) { return quantize_t<decltype(t)>(x, T, K, pos, k, codes, scales, st); });
}
cudaError_t launch_fp8_swiglu(const void* h, int h_dtype, int M, int I, uint8_t* codes, float* scales, cudaStream_t st) {
  return by_type(h_dtype, [&](auto t) { return swiglu_t<decltype(t)>(h, M, I, codes, scales, st); });
}
cudaError_t launch_fp8_weights(const void* w, int w_dtype, int E, int N, int K, uint8_t* codes, float* scales,
                               cudaStream_t st) {
  return by_type(w_dtype, [&](auto t) { return weights_t<decltype(t)>(w, E, N, K, codes, scales, st); });
}
cudaError_t launch_fp8_dequant(const uint8_t* codes, const float* scales, int E, int N, int K, int block_rows, void* out,
                               int out_dtype, cudaStream_t st) {
  return by_type(out_dtype, [&](auto t) { return dequant_t<decltype(t)>(codes, scales, E, N, K, block_rows, out, st); });
}

}  // namespace qmoe
