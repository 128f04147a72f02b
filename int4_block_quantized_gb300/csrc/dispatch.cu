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
// rounds, plus those in lower lanes.  Lanes of one expert find each other by a
// vote on each bit of its number (match_any goes through the experts one by one).
// Bin E: no expert.  Bound by latency: the chain of both walks and the barriers, and
// for many assignments by the integer instructions of the votes, on few SMs: 131072
// to 256 experts take 12.1 us on 16 CTAs, 17.6 on 8 (with match_any 23).
constexpr int kSortCluster = 8, kSortWide = 16;  // CTAs; more than 8 are not promised, so they are asked for
constexpr int kSortAhead = 8;  // loads in flight a thread

// BITS: of a bin's number.
template <int BITS>
__global__ void __launch_bounds__(1024, 1) sort_experts_kernel(const int32_t* __restrict__ ids, int A, int E,
                                                            int32_t* __restrict__ offsets, int32_t* __restrict__ perm,
                                                            int32_t* __restrict__ pos) {
  extern __shared__ uint32_t s_hist[];  // [warps][E + 1]
  __shared__ uint32_t s_total[kMaxExperts + 1], s_start[kMaxExperts + 1], s_sum[32];
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5, warps = blockDim.x >> 5, bins = E + 1;
  const int C = (int)cluster_nctarank(), rank = (int)cluster_ctarank();
  const int per = (int)((((long long)A + C * warps - 1) / (C * warps) + 31) & ~31LL);
  const long long a0 = (long long)(rank * warps + warp) * per;
  const int n = (int)(a0 >= A ? 0 : min((long long)per, A - a0));
  const long long cta = A - (long long)rank * warps * per;  // assignments from this CTA's first on
  const int used = cta <= 0 ? 0 : (int)min((long long)warps, (cta + per - 1) / per);  // its warps with assignments
  uint32_t* hist = s_hist + warp * bins;
  if (n > 0)
    for (int e = lane; e < bins; e += 32) hist[e] = 0;
  __syncwarp();
  pdl_wait();
  // f(offset, bin) for 32 assignments of the run at a time, ~0 for the lanes behind its end
  auto walk = [&](auto f) {
    for (int i = 0; i < n; i += 32 * kSortAhead) {
      uint32_t e[kSortAhead];
#pragma unroll
      for (int j = 0; j < kSortAhead; ++j)
        e[j] = i + 32 * j + lane < n ? min((uint32_t)ids[a0 + i + 32 * j + lane], (uint32_t)E) : ~0u;
#pragma unroll
      for (int j = 0; j < kSortAhead; ++j) {
        if (i + 32 * j >= n) break;
        f(i + 32 * j + lane, e[j]);
      }
    }
  };
  walk([&](int, uint32_t e) {
    if (e != ~0u) atomicAdd(&hist[e], 1u);
  });
  __syncthreads();
  if (tid < bins) {
    uint32_t sum = 0;
    for (int w = 0; w < used; ++w) {
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
    if (C == 1) {
      all = s_total[tid];
    } else {
      for (int r0 = 0; r0 < C; r0 += kSortCluster)
#pragma unroll
        for (int r = r0; r < r0 + kSortCluster; ++r) {
          const uint32_t c = __float_as_uint(ld_dsmem_f32(reinterpret_cast<const float*>(&s_total[tid]), r));
          before += r < rank ? c : 0;
          all += c;
        }
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
  walk([&](int i, uint32_t e) {
    const bool in = e != ~0u;
    uint32_t peers = __ballot_sync(0xffffffffu, in);
#pragma unroll
    for (int b = 0; b < BITS; ++b) {
      const uint32_t one = __ballot_sync(0xffffffffu, e >> b & 1);
      peers &= e >> b & 1 ? one : ~one;
    }
    if (in) {
      const uint32_t p = s_start[e] + hist[e] + __popc(peers & ((1u << lane) - 1));
      const bool some = e < (uint32_t)E;
      if (perm) perm[p] = some ? (int32_t)(a0 + i) : -1;
      if (pos) pos[a0 + i] = some ? (int32_t)p : -1;
    }
    __syncwarp();
    if (in && (peers >> lane) == 1u) hist[e] += __popc(peers);  // the highest lane of its expert
    __syncwarp();
  });
  if (C > 1) cluster_sync_all();  // no CTA leaves while another may read its totals
}

cudaError_t launch_sort_experts(const int32_t* ids, int A, int E, int32_t* offsets, int32_t* perm, int32_t* pos,
                                cudaStream_t st) {
  const int threads = A > 1024 ? 1024 : 320;  // at least E + 1
  auto kernel = E < 64 ? sort_experts_kernel<6> : sort_experts_kernel<9>;
  cudaLaunchConfig_t cfg = {};
  cfg.blockDim = dim3(threads);
  cfg.dynamicSmemBytes = (size_t)(threads / 32) * (E + 1) * 4;
  cfg.stream = st;
  cudaLaunchAttribute attr[2];
  attr[0].id = cudaLaunchAttributeClusterDimension;
  attr[0].val.clusterDim.y = attr[0].val.clusterDim.z = 1;
  attr[1].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[1].val.programmaticStreamSerializationAllowed = 1;
  cfg.attrs = attr;
  auto clusters_of = [&](int C) {
    cfg.gridDim = dim3(C);
    attr[0].val.clusterDim.x = C;
  };
  int C = A > 4096 ? kSortCluster : 1;
  if (A > 32768) {
    static int wide[64][2] = {};  // 1: such clusters fit the device, 2: they do not
    int dev = 0;
    cudaError_t err = cudaGetDevice(&dev);
    if (err != cudaSuccess) return err;
    if (dev < 0 || dev >= 64) return cudaErrorInvalidDevice;
    int& known = wide[dev][E < 64];
    if (!known) {
      int n = 0;
      clusters_of(kSortWide);
      cfg.numAttrs = 1;
      cfg.dynamicSmemBytes = 32 * (kMaxExperts + 1) * 4;
      if ((err = cudaFuncSetAttribute(kernel, cudaFuncAttributeNonPortableClusterSizeAllowed, 1)) != cudaSuccess ||
          (err = cudaOccupancyMaxActiveClusters(&n, kernel, &cfg)) != cudaSuccess)
        return err;
      cfg.dynamicSmemBytes = (size_t)32 * (E + 1) * 4;
      known = n > 0 ? 1 : 2;
    }
    if (known == 1) C = kSortWide;
  }
  clusters_of(C);
  cfg.numAttrs = 2;
  return cudaLaunchKernelEx(&cfg, kernel, ids, A, E, offsets, perm, pos);
}

// ----------------------------------------------------------------- dispatch
static dim3 rows_grid(size_t threads) {
  const size_t cap = (size_t)device_sm_count() * 32;
  const size_t b = (threads + 255) / 256;
  return dim3((unsigned)(b < 1 ? 1 : b > cap ? cap : b));
}

// A token's row is read once and written to its k places, 16 bytes a thread.
// Bound by HBM: 16384 tokens of 2048 bf16 to 8 places each in 92 us, 6.4 TB/s.
__global__ void __launch_bounds__(256) dispatch_kernel(const uint4* __restrict__ x, int T, int units, int k,
                                                       const int32_t* __restrict__ pos, uint4* __restrict__ xs) {
  pdl_wait();
  const uint32_t rows = (uint32_t)T * k;
  for (RowWalk w(blockIdx.x * 256 + threadIdx.x, gridDim.x * 256, (uint32_t)units); w.r < (uint32_t)T; w.next()) {
    const uint4 v = x[(size_t)w.r * units + w.u];
    for (int j0 = 0; j0 < k; j0 += 4) {
      uint32_t p[4];
#pragma unroll
      for (int j = 0; j < 4; ++j) p[j] = j0 + j < k ? (uint32_t)pos[(size_t)w.r * k + j0 + j] : ~0u;
#pragma unroll
      for (int j = 0; j < 4; ++j)
        if (p[j] < rows) xs[(size_t)p[j] * units + w.u] = v;
    }
  }
}

cudaError_t launch_dispatch(const void* x, int row_bytes, int T, int k, const int32_t* pos, void* xs, cudaStream_t st) {
  const int units = row_bytes / 16;
  return launch_kernel(dispatch_kernel, rows_grid((size_t)T * units), dim3(256), 0, st, true,
                       static_cast<const uint4*>(x), T, units, k, pos, static_cast<uint4*>(xs));
}

// ------------------------------------------------------------------ combine
// eight elements of T, 16-byte aligned: loaded, and converted
template <typename T>
struct Eight {
  uint4 w[sizeof(T) / 2];
  __device__ __forceinline__ void load(const void* base, size_t i) {
    const uint4* p = reinterpret_cast<const uint4*>(static_cast<const uint8_t*>(base) + i * sizeof(T));
#pragma unroll
    for (uint32_t q = 0; q < sizeof(T) / 2; ++q) w[q] = p[q];
  }
  __device__ __forceinline__ void values(float (&v)[8]) const {
    if constexpr (sizeof(T) == 4) {
#pragma unroll
      for (int q = 0; q < 2; ++q) {
        v[4 * q] = __uint_as_float(w[q].x), v[4 * q + 1] = __uint_as_float(w[q].y);
        v[4 * q + 2] = __uint_as_float(w[q].z), v[4 * q + 3] = __uint_as_float(w[q].w);
      }
    } else {
      const uint32_t u[4] = {w[0].x, w[0].y, w[0].z, w[0].w};
#pragma unroll
      for (int j = 0; j < 4; ++j) {
        v[2 * j] = Half<T>::to_float((uint16_t)(u[j] & 0xffffu));
        v[2 * j + 1] = Half<T>::to_float((uint16_t)(u[j] >> 16));
      }
    }
  }
};
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
// once.  A thread takes 8 columns of a token, four assignments' loads in flight.
// Bound by HBM: 16384 tokens of 2048 bf16, 8 each, in 101 us, 6.6 TB/s (108 with one
// load in flight).
template <typename Y, typename O>
__global__ void __launch_bounds__(256) combine_kernel(const void* __restrict__ ys, const int32_t* __restrict__ pos,
                                                      const float* __restrict__ wt, const void* residual, int T, int H,
                                                      int k, void* out) {
  pdl_wait();
  const uint32_t rows = (uint32_t)T * k;
  for (RowWalk w(blockIdx.x * 256 + threadIdx.x, gridDim.x * 256, (uint32_t)H / 8); w.r < (uint32_t)T; w.next()) {
    const size_t i = (size_t)w.r * H + 8 * w.u, a = (size_t)w.r * k;
    float s[8] = {};
    if (residual) {
      Eight<O> r;
      r.load(residual, i);
      r.values(s);
    }
    for (int j0 = 0; j0 < k; j0 += 4) {
      uint32_t p[4];
      float f[4];
      Eight<Y> y[4];
#pragma unroll
      for (int j = 0; j < 4; ++j) {
        p[j] = j0 + j < k ? (uint32_t)pos[a + j0 + j] : ~0u;
        f[j] = wt && j0 + j < k ? wt[a + j0 + j] : 1.f;
      }
#pragma unroll
      for (int j = 0; j < 4; ++j)
        if (p[j] < rows) y[j].load(ys, (size_t)p[j] * H + 8 * w.u);
#pragma unroll
      for (int j = 0; j < 4; ++j)
        if (p[j] < rows) {
          float v[8];
          y[j].values(v);
#pragma unroll
          for (int q = 0; q < 8; ++q) s[q] = fmaf(f[j], v[q], s[q]);
        }
    }
    store8<O>(out, i, s);
  }
}

// dys[pos[t, j]] = w[t, j] dout[t], dw[t, j] = sum_h dout[t, h] ys[pos[t, j], h] (fp32).
// One warp per assignment, four steps of 256 columns in flight; a token's warps
// are neighbours, so dout comes from L1 or L2 but once.  dys may be ys: a thread
// has read what it writes.  Bound by HBM: 16384 x 8 rows of 2048 bf16 in 167 us,
// 6.7 TB/s.
template <typename Y, typename O>
__global__ void __launch_bounds__(256) combine_backward_kernel(const void* __restrict__ dout, const void* ys,
                                                               const int32_t* __restrict__ pos,
                                                               const float* __restrict__ wt, int T, int H, int k,
                                                               void* dys, float* __restrict__ dw) {
  pdl_wait();
  const uint32_t rows = (uint32_t)T * k, lane = threadIdx.x & 31;
  for (uint32_t a = blockIdx.x * 8 + threadIdx.x / 32; a < rows; a += gridDim.x * 8) {
    const uint32_t p = (uint32_t)pos[a];
    float dot = 0.f;
    if (p < rows) {
      const float f = wt ? wt[a] : 1.f;
      const size_t from = (size_t)(a / k) * H, to = (size_t)p * H;
      for (int h0 = lane * 8; h0 < H; h0 += 1024) {
        Eight<O> d[4];
        Eight<Y> y[4];
#pragma unroll
        for (int j = 0; j < 4; ++j)
          if (h0 + 256 * j < H) {
            d[j].load(dout, from + h0 + 256 * j);
            if (dw) y[j].load(ys, to + h0 + 256 * j);
          }
#pragma unroll
        for (int j = 0; j < 4; ++j)
          if (h0 + 256 * j < H) {
            float u[8], v[8];
            d[j].values(u);
            if (dw) {
              y[j].values(v);
#pragma unroll
              for (int q = 0; q < 8; ++q) dot = fmaf(u[q], v[q], dot);
            }
            if (dys) {
#pragma unroll
              for (int q = 0; q < 8; ++q) v[q] = f * u[q];
              store8<Y>(dys, to + h0 + 256 * j, v);
            }
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
