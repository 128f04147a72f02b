// dispatch.cu -- tokens in the order of their experts and back: a stable
// counting sort of the assignments, the tokens' rows written to their places,
// and the weighted sum of the experts' outputs with its gradient.
//
// An assignment a = t * k + j sends token t to expert ids[a]; its place pos[a]
// is its rank by (expert, a), or -1 where ids[a] is no expert.
#include "launch.h"
#include "mx.cuh"

namespace qmoe {

// --------------------------------------------------------------------- sort
// One cluster of C CTAs (one for few assignments).  Every warp takes a
// contiguous run of assignments and counts it by expert; the counts are summed
// over warps, CTAs (through distributed shared memory) and experts; then every
// warp walks its run again, 32 assignments at a time, and gives each its place:
// where its expert starts, plus the expert's assignments in earlier warps and
// rounds, plus those in lower lanes (match_any).  Bin E: no expert.
// Bound by latency: the chain of both walks and three barriers.
constexpr int kSortThreads = 1024, kSortWarps = kSortThreads / 32;
constexpr int kSortCluster = 8;

__global__ void __launch_bounds__(kSortThreads) sort_experts_kernel(const int32_t* __restrict__ ids, int A, int E,
                                                                    int32_t* __restrict__ offsets,
                                                                    int32_t* __restrict__ perm,
                                                                    int32_t* __restrict__ pos) {
  extern __shared__ uint32_t s_hist[];  // [kSortWarps][E + 1]
  __shared__ uint32_t s_total[kMaxExperts + 1], s_start[kMaxExperts + 1], s_sum[kSortWarps];
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5, bins = E + 1;
  const int C = (int)cluster_nctarank(), rank = (int)cluster_ctarank();
  const int per = (int)((((long long)A + C * kSortWarps - 1) / (C * kSortWarps) + 31) & ~31LL);
  const long long a0 = (long long)(rank * kSortWarps + warp) * per;
  const int n = (int)(a0 >= A ? 0 : min((long long)per, A - a0));
  uint32_t* hist = s_hist + warp * bins;
  for (int e = lane; e < bins; e += 32) hist[e] = 0;
  __syncwarp();
  pdl_wait();
  for (int i = lane; i < n; i += 32) atomicAdd(&hist[min((uint32_t)ids[a0 + i], (uint32_t)E)], 1u);
  __syncthreads();
  if (tid < bins) {
    uint32_t sum = 0;
    for (int w = 0; w < kSortWarps; ++w) {
      const uint32_t c = s_hist[w * bins + tid];
      s_hist[w * bins + tid] = sum;
      sum += c;
    }
    s_total[tid] = sum;
  }
  if (C > 1) cluster_sync_all();
  else __syncthreads();
  uint32_t all = 0, before = 0;
  if (tid < bins) {
    for (int r = 0; r < C; ++r) {
      const uint32_t c = C > 1 ? __float_as_uint(ld_dsmem_f32(reinterpret_cast<const float*>(&s_total[tid]), r)) : s_total[tid];
      before += r < rank ? c : 0;
      all += c;
    }
  }
  // exclusive sum over the bins (at most 257, threads of the first nine warps)
  uint32_t run = all;
#pragma unroll
  for (int o = 1; o < 32; o <<= 1) {
    const uint32_t up = __shfl_up_sync(0xffffffffu, run, o);
    if (lane >= o) run += up;
  }
  if (lane == 31) s_sum[warp] = run;
  __syncthreads();
  if (tid < bins) {
    uint32_t start = run - all;
    for (int w = 0; w < warp; ++w) start += s_sum[w];
    if (rank == 0 && offsets) offsets[tid] = (int32_t)start;
    s_start[tid] = start + before;
  }
  __syncthreads();
  for (int i = lane; i < ((n + 31) & ~31); i += 32) {
    const bool in = i < n;
    const uint32_t e = in ? min((uint32_t)ids[a0 + i], (uint32_t)E) : 0xffffffffu;
    const uint32_t peers = __match_any_sync(0xffffffffu, e);
    if (in) {
      const uint32_t p = s_start[e] + hist[e] + __popc(peers & ((1u << lane) - 1));
      const bool some = e < (uint32_t)E;
      if (perm) perm[p] = some ? (int32_t)(a0 + i) : -1;
      if (pos) pos[a0 + i] = some ? (int32_t)p : -1;
    }
    __syncwarp();
    if (in && (peers >> lane) == 1u) hist[e] += __popc(peers);  // the highest lane of its expert
    __syncwarp();
  }
  if (C > 1) cluster_sync_all();  // no CTA leaves while another may read its totals
}

cudaError_t launch_sort_experts(const int32_t* ids, int A, int E, int32_t* offsets, int32_t* perm, int32_t* pos,
                                cudaStream_t st) {
  const size_t smem = (size_t)kSortWarps * (E + 1) * 4;
  cudaLaunchConfig_t cfg = {};
  const int C = A > 4096 ? kSortCluster : 1;
  cfg.gridDim = dim3(C);
  cfg.blockDim = dim3(kSortThreads);
  cfg.dynamicSmemBytes = smem;
  cfg.stream = st;
  cudaLaunchAttribute attr[2];
  attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[0].val.programmaticStreamSerializationAllowed = 1;
  attr[1].id = cudaLaunchAttributeClusterDimension;
  attr[1].val.clusterDim.x = C;
  attr[1].val.clusterDim.y = attr[1].val.clusterDim.z = 1;
  cfg.attrs = attr;
  cfg.numAttrs = 2;
  return cudaLaunchKernelEx(&cfg, sort_experts_kernel, ids, A, E, offsets, perm, pos);
}

// ----------------------------------------------------------------- dispatch
static dim3 rows_grid(size_t threads) {
  const size_t cap = (size_t)device_sm_count() * 32;
  const size_t b = (threads + 255) / 256;
  return dim3((unsigned)(b < 1 ? 1 : b > cap ? cap : b));
}

// A token's row is read once and written to its k places, 16 bytes a thread.
// Bound by HBM.
__global__ void __launch_bounds__(256) dispatch_kernel(const uint4* __restrict__ x, int T, int units, int k,
                                                       const int32_t* __restrict__ pos, uint4* __restrict__ xs) {
  pdl_wait();
  const uint32_t rows = (uint32_t)T * k;
  for (RowWalk w(blockIdx.x * 256 + threadIdx.x, gridDim.x * 256, (uint32_t)units); w.r < (uint32_t)T; w.next()) {
    const uint4 v = x[(size_t)w.r * units + w.u];
    for (int j = 0; j < k; ++j) {
      const uint32_t p = (uint32_t)pos[(size_t)w.r * k + j];
      if (p < rows) xs[(size_t)p * units + w.u] = v;
    }
  }
}

cudaError_t launch_dispatch(const void* x, int row_bytes, int T, int k, const int32_t* pos, void* xs, cudaStream_t st) {
  const int units = row_bytes / 16;
  return launch_kernel(dispatch_kernel, rows_grid((size_t)T * units), dim3(256), 0, st, true,
                       static_cast<const uint4*>(x), T, units, k, pos, static_cast<uint4*>(xs));
}

// ------------------------------------------------------------------ combine
// eight elements of T at element i (a multiple of 8), 16-byte aligned
template <typename T>
__device__ __forceinline__ void load8(const void* base, size_t i, float (&v)[8]) {
  const uint4* p = reinterpret_cast<const uint4*>(static_cast<const uint8_t*>(base) + i * sizeof(T));
  if constexpr (sizeof(T) == 4) {
    const uint4 a = p[0], b = p[1];
    v[0] = __uint_as_float(a.x), v[1] = __uint_as_float(a.y), v[2] = __uint_as_float(a.z), v[3] = __uint_as_float(a.w);
    v[4] = __uint_as_float(b.x), v[5] = __uint_as_float(b.y), v[6] = __uint_as_float(b.z), v[7] = __uint_as_float(b.w);
  } else {
    const uint4 a = p[0];
    const uint32_t w[4] = {a.x, a.y, a.z, a.w};
#pragma unroll
    for (int j = 0; j < 4; ++j) {
      v[2 * j] = Half<T>::to_float((uint16_t)(w[j] & 0xffffu));
      v[2 * j + 1] = Half<T>::to_float((uint16_t)(w[j] >> 16));
    }
  }
}
template <typename T>
__device__ __forceinline__ void store8(void* base, size_t i, const float (&v)[8]) {
  uint4* p = reinterpret_cast<uint4*>(static_cast<uint8_t*>(base) + i * sizeof(T));
  if constexpr (sizeof(T) == 4) {
    p[0] = make_uint4(__float_as_uint(v[0]), __float_as_uint(v[1]), __float_as_uint(v[2]), __float_as_uint(v[3]));
    p[1] = make_uint4(__float_as_uint(v[4]), __float_as_uint(v[5]), __float_as_uint(v[6]), __float_as_uint(v[7]));
  } else {
    uint32_t w[4];
#pragma unroll
    for (int j = 0; j < 4; ++j)
      w[j] = (uint32_t)Half<T>::from_float(v[2 * j]) | (uint32_t)Half<T>::from_float(v[2 * j + 1]) << 16;
    p[0] = make_uint4(w[0], w[1], w[2], w[3]);
  }
}

// out[t] = residual[t] + sum_j w[t, j] ys[pos[t, j]], fp32 in this order, rounded
// once.  A thread takes 8 columns of a token.  Bound by HBM.
template <typename Y, typename O>
__global__ void __launch_bounds__(256) combine_kernel(const void* __restrict__ ys, const int32_t* __restrict__ pos,
                                                      const float* __restrict__ wt, const void* residual, int T, int H,
                                                      int k, void* out) {
  pdl_wait();
  const uint32_t rows = (uint32_t)T * k;
  for (RowWalk w(blockIdx.x * 256 + threadIdx.x, gridDim.x * 256, (uint32_t)H / 8); w.r < (uint32_t)T; w.next()) {
    const size_t i = (size_t)w.r * H + 8 * w.u;
    float s[8] = {};
    if (residual) load8<O>(residual, i, s);
    for (int j = 0; j < k; ++j) {
      const uint32_t p = (uint32_t)pos[(size_t)w.r * k + j];
      if (p >= rows) continue;
      const float f = wt ? wt[(size_t)w.r * k + j] : 1.f;
      float v[8];
      load8<Y>(ys, (size_t)p * H + 8 * w.u, v);
#pragma unroll
      for (int q = 0; q < 8; ++q) s[q] = fmaf(f, v[q], s[q]);
    }
    store8<O>(out, i, s);
  }
}

// dys[pos[t, j]] = w[t, j] dout[t], dw[t, j] = sum_h dout[t, h] ys[pos[t, j], h] (fp32).
// One warp per assignment; a token's warps are neighbours, so dout comes from
// L1 or L2 but once.  Bound by HBM.
template <typename Y, typename O>
__global__ void __launch_bounds__(256) combine_backward_kernel(const void* __restrict__ dout, const void* __restrict__ ys,
                                                               const int32_t* __restrict__ pos,
                                                               const float* __restrict__ wt, int T, int H, int k,
                                                               void* __restrict__ dys, float* __restrict__ dw) {
  pdl_wait();
  const uint32_t rows = (uint32_t)T * k, lane = threadIdx.x & 31;
  for (uint32_t a = blockIdx.x * 8 + threadIdx.x / 32; a < rows; a += gridDim.x * 8) {
    const uint32_t p = (uint32_t)pos[a];
    float dot = 0.f;
    if (p < rows) {
      const float f = wt ? wt[a] : 1.f;
      const size_t from = (size_t)(a / k) * H, to = (size_t)p * H;
      for (int h = lane * 8; h < H; h += 256) {
        float d[8], y[8];
        load8<O>(dout, from + h, d);
        if (dw) {
          load8<Y>(ys, to + h, y);
#pragma unroll
          for (int q = 0; q < 8; ++q) dot = fmaf(d[q], y[q], dot);
        }
        if (dys) {
#pragma unroll
          for (int q = 0; q < 8; ++q) y[q] = f * d[q];
          store8<Y>(dys, to + h, y);
        }
      }
    }
    if (dw) {
      dot = warp_sum(dot);
      if (lane == 0) dw[a] = dot;
    }
  }
}

template <typename F>
static cudaError_t by_type(int dtype, F fn) {
  if (dtype == QMOE_F32) return fn(float{});
  if (dtype == QMOE_BF16) return fn(__nv_bfloat16{});
  return fn(__half{});
}
template <typename F>
static cudaError_t by_types(int a, int b, F fn) {
  return by_type(a, [&](auto x) { return by_type(b, [&](auto y) { return fn(x, y); }); });
}

cudaError_t launch_combine(const void* ys, int ys_dtype, const int32_t* pos, const float* w, const void* residual, int T,
                           int H, int k, void* out, int out_dtype, cudaStream_t st) {
  return by_types(ys_dtype, out_dtype, [&](auto y, auto o) {
    return launch_kernel(combine_kernel<decltype(y), decltype(o)>, rows_grid((size_t)T * (H / 8)), dim3(256), 0, st, true, ys,
                         pos, w, residual, T, H, k, out);
  });
}
cudaError_t launch_combine_backward(const void* dout, int dout_dtype, const void* ys, int ys_dtype, const int32_t* pos,
                                    const float* w, int T, int H, int k, void* dys, float* dw, cudaStream_t st) {
  return by_types(ys_dtype, dout_dtype, [&](auto y, auto o) {
    return launch_kernel(combine_backward_kernel<decltype(y), decltype(o)>, rows_grid((size_t)T * k * 32), dim3(256), 0, st,
                         true, dout, ys, pos, w, T, H, k, dys, dw);
  });
}

}  // namespace qmoe
