// mx.cu -- microscaled formats: quantisation (fp16 / bf16 / fp32 to MXFP8 or
// MXFP4), the reader, the layer stack's RMSNorm with the residual's addition
// and microscaled output, and the scale-layout adapters.
#include <math.h>

#include "launch.h"
#include "mx.cuh"

namespace qmoe {

// Grid of a grid-stride kernel over `work` threads of 256: at most 32 CTAs an
// SM (fp32 16384 x 8192 reads back in 102 us at 32, 108 at 16; without a cap
// 84480 x 2048 fp16 takes 80 us instead of 63).
static dim3 stride_grid(size_t work) {
  const size_t cap = (size_t)device_sm_count() * 32;
  const size_t b = (work + 255) / 256;
  return dim3((unsigned)(b < 1 ? 1 : b > cap ? cap : b));
}

// --------------------------------------------------------------- quantise
// s = floor(log2 max|v|) - emax, code = RN(v / 2^s): a thread takes half a
// block (16 elements), so a block's maximum needs one shuffle.  Bound by HBM:
// 84480 x 2048 fp16 to MXFP4 in 63 us, 6.9 TB/s.
template <typename T, int FMT>
__global__ void __launch_bounds__(256) mx_quantize_kernel(const void* __restrict__ x, int M, int K,
                                                          uint8_t* __restrict__ codes, uint8_t* __restrict__ scales) {
  pdl_wait();
  const uint32_t t0 = blockIdx.x * 256 + threadIdx.x, stride = gridDim.x * 256;
  const int kt = (K + 127) / 128;
  for (RowWalk w(t0, stride, (uint32_t)K / 16); w.r < (uint32_t)M; w.next()) {
    const size_t i = (size_t)w.r * K + 16 * w.u;
    float v[16];
    load16<T>(x, i, v);
    const uint32_t s = mx_encode16<FMT>(v, codes, i);
    if (!(w.u & 1)) scales[mx_scale_index((int)w.r, (int)w.u >> 1, kt)] = (uint8_t)s;
  }
  mx_zero_padding(scales, M, K, t0, stride);
}

template <typename T>
static cudaError_t launch_quantize_t(const void* x, int format, int M, int K, uint8_t* codes, uint8_t* scales,
                                     cudaStream_t st) {
  const dim3 g = stride_grid((size_t)M * (K / 16) + mx_padding_words(M, K));
  if (format == kMxfp8)
    return launch_kernel(mx_quantize_kernel<T, kMxfp8>, g, dim3(256), 0, st, true, x, M, K, codes, scales);
  return launch_kernel(mx_quantize_kernel<T, kMxfp4>, g, dim3(256), 0, st, true, x, M, K, codes, scales);
}

cudaError_t launch_mx_quantize(const void* x, int x_dtype, int format, int M, int K, uint8_t* codes, uint8_t* scales,
                               cudaStream_t st) {
  if (x_dtype == QMOE_F32) return launch_quantize_t<float>(x, format, M, K, codes, scales, st);
  if (x_dtype == QMOE_BF16) return launch_quantize_t<__nv_bfloat16>(x, format, M, K, codes, scales, st);
  return launch_quantize_t<__half>(x, format, M, K, codes, scales, st);
}

// ---------------------------------------------------------------- dequant
// code * X in fp32 (exact), rounded once to T.  Bound by HBM: 84480 x 2048
// MXFP4 to fp16 in 68 us, 6.4 TB/s.
template <typename T, int FMT>
__global__ void __launch_bounds__(256) mx_dequant_kernel(const uint8_t* __restrict__ codes,
                                                         const uint8_t* __restrict__ scales, int M, int K,
                                                         void* __restrict__ out) {
  pdl_wait();
  const int kt = (K + 127) / 128;
  for (RowWalk w(blockIdx.x * 256 + threadIdx.x, gridDim.x * 256, (uint32_t)K / 16); w.r < (uint32_t)M; w.next()) {
    const size_t i = (size_t)w.r * K + 16 * w.u;
    const float X = mx_scale(scales[mx_scale_index((int)w.r, (int)w.u >> 1, kt)]);
    float v[16];
    if constexpr (FMT == kMxfp8) {
      const uint4 c = *reinterpret_cast<const uint4*>(codes + i);
      mx_from_e4m3x4(c.x, v);
      mx_from_e4m3x4(c.y, v + 4);
      mx_from_e4m3x4(c.z, v + 8);
      mx_from_e4m3x4(c.w, v + 12);
    } else {
      const uint2 c = *reinterpret_cast<const uint2*>(codes + i / 2);
      mx_from_e2m1x8(c.x, v);
      mx_from_e2m1x8(c.y, v + 8);
    }
#pragma unroll
    for (int j = 0; j < 16; ++j) v[j] *= X;
    store16<T>(out, i, v);
  }
}

template <typename T>
static cudaError_t launch_dequant_t(const uint8_t* codes, const uint8_t* scales, int format, int M, int K, void* out,
                                    cudaStream_t st) {
  const dim3 g = stride_grid((size_t)M * (K / 16));
  if (format == kMxfp8)
    return launch_kernel(mx_dequant_kernel<T, kMxfp8>, g, dim3(256), 0, st, true, codes, scales, M, K, out);
  return launch_kernel(mx_dequant_kernel<T, kMxfp4>, g, dim3(256), 0, st, true, codes, scales, M, K, out);
}

cudaError_t launch_mx_dequant(const uint8_t* codes, const uint8_t* scales, int format, int M, int K, void* out,
                              int out_dtype, cudaStream_t st) {
  if (out_dtype == QMOE_F32) return launch_dequant_t<float>(codes, scales, format, M, K, out, st);
  if (out_dtype == QMOE_BF16) return launch_dequant_t<__nv_bfloat16>(codes, scales, format, M, K, out, st);
  return launch_dequant_t<__half>(codes, scales, format, M, K, out, st);
}

// ---------------------------------------------------------------- RMSNorm
// h = x + residual in fp32; residual_out = RN(h); y = h / sqrt(mean(h^2) +
// eps) * weight from the unrounded h, quantised like above.  One CTA per row,
// a thread to 16 elements, which it keeps in registers between the sum and the
// output (KEEP; rows beyond 16384 are read twice, and spill at this bound:
// 2048 x 20480 takes 92 us, 3.2 TB/s).  residual_out may be x or
// residual: each element is read and written by one thread, and nothing is
// written before the row's sum is complete.
// Bound by HBM.  32 registers a thread (the launch bound), so that 2048 threads
// fit an SM and one row's loads run during another's sum: 16384 x 4096 bf16
// with residual takes 70 us at 32 registers (6.76 TB/s) and 95 us at 55;
// reading the row twice instead of keeping it takes 76 us.  One thread per 16
// elements, and not 256 throughout: 16384 x 2048 takes 36 us instead of 45.
template <typename T>
__device__ __forceinline__ void norm_load(const void* x, const void* residual, size_t i, float (&v)[16]) {
  load16<T>(x, i, v);
  if (residual) {
    float r[16];
    load16<T>(residual, i, r);
#pragma unroll
    for (int j = 0; j < 16; ++j) v[j] += r[j];
  }
}

template <typename T, int FMT, bool KEEP>
__global__ void __launch_bounds__(1024, 2)
    mx_rmsnorm_kernel(const void* x, const void* residual, const void* weight, int M, int H, float eps,
                      void* residual_out, uint8_t* codes, uint8_t* scales) {
  pdl_wait();
  const int units = H / 16, kt = (H + 127) / 128, t = blockIdx.x, threads = blockDim.x;
  if (t >= M) {  // the last CTAs: the scale tiles' rows behind row M
    mx_zero_rows(scales, M, H, (t - M) * threads + threadIdx.x, (gridDim.x - M) * threads);
    return;
  }
  const size_t row = (size_t)t * H;
  float v[16];
  float ss = 0.f;
  for (int u = threadIdx.x; u < units; u += threads) {
    norm_load<T>(x, residual, row + u * 16, v);
#pragma unroll
    for (int j = 0; j < 16; ++j) ss = fmaf(v[j], v[j], ss);
    if (KEEP) break;
  }
  ss = warp_sum(ss);
  __shared__ float part[32];
  if ((threadIdx.x & 31) == 0) part[threadIdx.x >> 5] = ss;
  __syncthreads();
  // pairwise: the few large sums' roundings are all that the row's sum loses
  float tot = 0.f;
  for (int i = 0; i < threads / 32; i += 8) {
    float p[8];
#pragma unroll
    for (int j = 0; j < 8; ++j) p[j] = i + j < threads / 32 ? part[i + j] : 0.f;
    tot += ((p[0] + p[1]) + (p[2] + p[3])) + ((p[4] + p[5]) + (p[6] + p[7]));
  }
  // mean, + eps: each rounded to fp32.  (Against fp64 1030 of 2416 M codes fall
  // on the other side of a border, 1015 with 1 / sqrtf(tot / H + eps): chance.)
  const float inv = rsqrtf(__fadd_rn(__fmul_rn(tot, 1.0f / (float)H), eps));
  for (int u = threadIdx.x; u < units; u += threads) {
    if (!KEEP) norm_load<T>(x, residual, row + u * 16, v);
    if (residual_out) store16<T>(residual_out, row + u * 16, v);
#pragma unroll
    for (int j = 0; j < 16; ++j) v[j] *= inv;
    if (weight) {
      float w[16];
      load16<T>(weight, u * 16, w);
#pragma unroll
      for (int j = 0; j < 16; ++j) v[j] *= w[j];
    }
    const uint32_t s = mx_encode16<FMT>(v, codes, row + u * 16);
    if (!(u & 1)) scales[mx_scale_index(t, u >> 1, kt)] = (uint8_t)s;
    if (KEEP) break;
  }
  if (H / 32 + (int)threadIdx.x < 4 * kt) scales[mx_scale_index(t, H / 32 + threadIdx.x, kt)] = 0;
}

template <typename T, int FMT>
static cudaError_t launch_rmsnorm_t(const void* x, const void* residual, const void* weight, int M, int H, float eps,
                                    void* residual_out, uint8_t* codes, uint8_t* scales, cudaStream_t st) {
  const int threads = H > 16384 ? 1024 : (H / 16 + 31) / 32 * 32;
  const uint32_t pad = (mx_padding_words(M, H) + 4 * threads - 1) / (4 * threads);
  const long long grid = (long long)M + (pad < 64 ? pad : 64);
  if (grid > 0x7fffffffLL) return cudaErrorInvalidValue;
  return launch_kernel(H > 16384 ? mx_rmsnorm_kernel<T, FMT, false> : mx_rmsnorm_kernel<T, FMT, true>,
                       dim3((unsigned)grid), dim3(threads), 0, st, true, x, residual, weight, M, H, eps, residual_out,
                       codes, scales);
}

cudaError_t launch_mx_rmsnorm(const void* x, const void* residual, const void* weight, int act_dtype, int T, int H,
                              float eps, int format, void* residual_out, uint8_t* codes, uint8_t* scales,
                              cudaStream_t st) {
  auto go = [&](auto fn) { return fn(x, residual, weight, T, H, eps, residual_out, codes, scales, st); };
  if (act_dtype == QMOE_BF16)
    return format == kMxfp8 ? go(launch_rmsnorm_t<__nv_bfloat16, kMxfp8>) : go(launch_rmsnorm_t<__nv_bfloat16, kMxfp4>);
  return format == kMxfp8 ? go(launch_rmsnorm_t<__half, kMxfp8>) : go(launch_rmsnorm_t<__half, kMxfp4>);
}

// --------------------------------------------------------- scale adapters
// Row-major scales [R, K / 32] into tiles (padding zero), or back.
template <bool TO_TILES>
__global__ void __launch_bounds__(256) mx_retile_kernel(const uint8_t* __restrict__ in, uint8_t* __restrict__ out,
                                                        int R, int K) {
  pdl_wait();
  const uint32_t t0 = blockIdx.x * 256 + threadIdx.x, stride = gridDim.x * 256;
  const int nb = K / 32, kt = (K + 127) / 128;
  for (RowWalk w(t0, stride, (uint32_t)nb); w.r < (uint32_t)R; w.next()) {
    const size_t i = (size_t)w.r * nb + w.u, j = mx_scale_index((int)w.r, (int)w.u, kt);
    if (TO_TILES) out[j] = in[i];
    else out[i] = in[j];
  }
  if (TO_TILES) mx_zero_padding(out, R, K, t0, stride);
}

cudaError_t launch_mx_retile(const uint8_t* in, uint8_t* out, int R, int K, bool to_tiles, cudaStream_t st) {
  const dim3 g = stride_grid((size_t)R * (K / 32));
  if (to_tiles) return launch_kernel(mx_retile_kernel<true>, g, dim3(256), 0, st, true, in, out, R, K);
  return launch_kernel(mx_retile_kernel<false>, g, dim3(256), 0, st, true, in, out, R, K);
}

}  // namespace qmoe
