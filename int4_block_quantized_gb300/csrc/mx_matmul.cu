// mx_matmul.cu -- product of a microscaled tensor with MXFP4 weights:
//   y[m, n] = sum over blocks b of X_x[m, b] X_w[n, b] sum_{k in b} x[m, k] w[n, k]
// with fp32 sums, rounded once to the output's type.
#include "launch.h"
#include "mx.cuh"

namespace qmoe {

// 32 x 32 outputs per CTA, one block (32 k) at a time: the block's codes of 32
// tokens and 32 weight rows are decoded into shared memory, scales applied.
template <typename TY, int FMT>
__global__ void __launch_bounds__(256) mx_matmul_kernel(const uint8_t* __restrict__ xc, const uint8_t* __restrict__ xs,
                                                        const uint8_t* __restrict__ wc, const uint8_t* __restrict__ ws,
                                                        int M, int N, int K, TY* __restrict__ y) {
  __shared__ float sx[32][33], sw[32][33];
  pdl_wait();
  const int kt = (K + 127) / 128, tid = threadIdx.x;
  const int nt = (N + 31) / 32, m0 = (int)(blockIdx.x / nt) * 32, n0 = (int)(blockIdx.x % nt) * 32;
  float acc[4] = {0.f, 0.f, 0.f, 0.f};
  for (int b = 0; b < K / 32; ++b) {
    const int r = tid >> 3, c = (tid & 7) * 4;  // 4 elements of row r
    {
      float v[8] = {0.f, 0.f, 0.f, 0.f, 0.f, 0.f, 0.f, 0.f};
      if (m0 + r < M) {
        const size_t e = (size_t)(m0 + r) * K + b * 32 + c;
        if (FMT == kMxfp8) mx_from_e4m3x4(*reinterpret_cast<const uint32_t*>(xc + e), v);
        else mx_from_e2m1x8(*reinterpret_cast<const uint16_t*>(xc + e / 2), v);
        const float X = mx_scale(xs[mx_scale_index(m0 + r, b, kt)]);
#pragma unroll
        for (int j = 0; j < 4; ++j) v[j] *= X;
      }
#pragma unroll
      for (int j = 0; j < 4; ++j) sx[r][c + j] = v[j];
    }
    {
      float v[8] = {0.f, 0.f, 0.f, 0.f, 0.f, 0.f, 0.f, 0.f};
      if (n0 + r < N) {
        mx_from_e2m1x8(*reinterpret_cast<const uint16_t*>(wc + ((size_t)(n0 + r) * K + b * 32 + c) / 2), v);
        const float X = mx_scale(ws[mx_scale_index(n0 + r, b, kt)]);
#pragma unroll
        for (int j = 0; j < 4; ++j) v[j] *= X;
      }
#pragma unroll
      for (int j = 0; j < 4; ++j) sw[r][c + j] = v[j];
    }
    __syncthreads();
    for (int k = 0; k < 32; ++k) {
      const float w = sw[tid & 31][k];
#pragma unroll
      for (int i = 0; i < 4; ++i) acc[i] = fmaf(sx[(tid >> 5) * 4 + i][k], w, acc[i]);
    }
    __syncthreads();
  }
  const int n = n0 + (tid & 31);
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    const int m = m0 + (tid >> 5) * 4 + i;
    if (m < M && n < N) {
      if constexpr (sizeof(TY) == 4) y[(size_t)m * N + n] = acc[i];
      else reinterpret_cast<uint16_t*>(y)[(size_t)m * N + n] = Half<TY>::from_float(acc[i]);
    }
  }
}

template <typename TY>
static cudaError_t launch_matmul_t(const uint8_t* xc, const uint8_t* xs, int x_format, const uint8_t* wc,
                                   const uint8_t* ws, int M, int N, int K, void* y, cudaStream_t st) {
  const long long tiles = (long long)((N + 31) / 32) * ((M + 31) / 32);
  if (tiles > 0x7fffffffLL) return cudaErrorInvalidValue;
  const dim3 g((unsigned)tiles);
  if (x_format == kMxfp8)
    return launch_kernel(mx_matmul_kernel<TY, kMxfp8>, g, dim3(256), 0, st, true, xc, xs, wc, ws, M, N, K,
                         static_cast<TY*>(y));
  return launch_kernel(mx_matmul_kernel<TY, kMxfp4>, g, dim3(256), 0, st, true, xc, xs, wc, ws, M, N, K,
                       static_cast<TY*>(y));
}

cudaError_t launch_mx_matmul(const uint8_t* xc, const uint8_t* xs, int x_format, const uint8_t* wc, const uint8_t* ws,
                             int M, int N, int K, void* y, int y_dtype, uint32_t* status, cudaStream_t st) {
  (void)status;
  if (y_dtype == QMOE_F32) return launch_matmul_t<float>(xc, xs, x_format, wc, ws, M, N, K, y, st);
  if (y_dtype == QMOE_BF16) return launch_matmul_t<__nv_bfloat16>(xc, xs, x_format, wc, ws, M, N, K, y, st);
  return launch_matmul_t<__half>(xc, xs, x_format, wc, ws, M, N, K, y, st);
}

}  // namespace qmoe
