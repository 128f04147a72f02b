// fp8_matmul.cu -- product of FP8 tensors with block scales, dense or grouped
// by expert:
//   y[m, n] = sum over blocks b of sx[m, b] sw[n / 128, b] sum_{k in b} x[m, k] w[n, k]
// with fp32 sums, rounded once to the output's type.  Grouped: row m meets the
// weights of the expert e with offsets[e] <= m < offsets[e + 1].
#include "fp8.cuh"
#include "launch.h"

namespace qmoe {

// The status word of the calls that bring none.
__device__ uint32_t g_fp8_status;

struct FmParams {
  const uint8_t *xc, *wc;
  const float *xs, *ws;
  const int32_t* offsets;
  void* y;
  uint32_t* status;
  int E, M, N, K, y_dtype;
};

__device__ __forceinline__ void fm_store(const FmParams& p, size_t i, float v) {
  if (p.y_dtype == QMOE_F32) static_cast<float*>(p.y)[i] = v;
  else static_cast<uint16_t*>(p.y)[i] = p.y_dtype == QMOE_BF16 ? Half<__nv_bfloat16>::from_float(v) : Half<__half>::from_float(v);
}

// A simple form: 64 x 64 outputs a CTA, 4 x 4 a thread, 32 k at a time.
__global__ void __launch_bounds__(256) fp8_matmul_kernel(const FmParams p) {
  pdl_wait();
  __shared__ float sx[32][68], sw[32][68];
  const int e = blockIdx.z, n0 = blockIdx.x * 64;
  int m0 = 0, m1 = p.M;
  if (p.offsets) {
    const int o0 = p.offsets[e], o1 = p.offsets[e + 1];
    m0 = min(max(o0, 0), p.M);
    m1 = min(max(o1, 0), p.M);
    if (m0 != o0 || m1 != o1 || m1 < m0) set_status(p.status ? p.status : &g_fp8_status, QMOE_ST_INDEX);
  }
  const int nb = (p.K + 127) / 128, rb = (p.N + 127) / 128;
  const int tx = threadIdx.x & 15, ty = threadIdx.x >> 4;
  const int lr = threadIdx.x >> 2, lk = (threadIdx.x & 3) * 8;
  for (int m = m0 + blockIdx.y * 64; m < m1; m += gridDim.y * 64) {
    float acc[4][4] = {};
    for (int k = 0; k < p.K; k += 32) {
      float v[8];
      auto fetch = [&](const uint8_t* base, size_t row, bool ok) {
        uint2 c = make_uint2(0, 0);
        if (ok && k + lk < p.K) c = *reinterpret_cast<const uint2*>(base + row * p.K + k + lk);
        mx_from_e4m3x4(c.x, v);
        mx_from_e4m3x4(c.y, v + 4);
      };
      fetch(p.xc, m + lr, m + lr < m1);
      const float s = m + lr < m1 ? p.xs[(size_t)(m + lr) * nb + k / 128] : 0.f;
      for (int j = 0; j < 8; ++j) sx[lk + j][lr] = v[j] * s;
      fetch(p.wc, (size_t)e * p.N + n0 + lr, n0 + lr < p.N);
      const float t = n0 + lr < p.N ? p.ws[((size_t)e * rb + (n0 + lr) / 128) * nb + k / 128] : 0.f;
      for (int j = 0; j < 8; ++j) sw[lk + j][lr] = v[j] * t;
      __syncthreads();
#pragma unroll 8
      for (int kk = 0; kk < 32; ++kk) {
        float a[4], b[4];
        for (int j = 0; j < 4; ++j) a[j] = sx[kk][ty * 4 + j], b[j] = sw[kk][tx * 4 + j];
        for (int i = 0; i < 4; ++i)
          for (int j = 0; j < 4; ++j) acc[i][j] = fmaf(a[i], b[j], acc[i][j]);
      }
      __syncthreads();
    }
    for (int i = 0; i < 4; ++i)
      for (int j = 0; j < 4; ++j)
        if (m + ty * 4 + i < m1 && n0 + tx * 4 + j < p.N) fm_store(p, (size_t)(m + ty * 4 + i) * p.N + n0 + tx * 4 + j, acc[i][j]);
  }
}

cudaError_t fp8_status_word(void** word) { return cudaGetSymbolAddress(word, g_fp8_status); }

cudaError_t launch_fp8_matmul(const uint8_t* xc, const float* xs, const uint8_t* wc, const float* ws,
                              const int32_t* offsets, int E, int M, int N, int K, void* y, int y_dtype, uint32_t* status,
                              cudaStream_t st) {
  FmParams p = {xc, wc, xs, ws, offsets, y, status, E, M, N, K, y_dtype};
  const int mt = (M + 63) / 64;
  return launch_kernel(fp8_matmul_kernel, dim3((N + 63) / 64, mt < 128 ? mt : 128, E), dim3(256), 0, st, true, p);
}

}  // namespace qmoe
