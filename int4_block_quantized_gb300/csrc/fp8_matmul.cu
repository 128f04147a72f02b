// fp8_matmul.cu -- product of FP8 tensors with block scales, dense or grouped
// by expert:
//   y[m, n] = sum over blocks b of sx[m, b] sw[n / 128, b] sum_{k in b} x[m, k] w[n, k]
// with fp32 sums, rounded once to the output's type.  Grouped: row m meets the
// weights of the expert e with offsets[e] <= m < offsets[e + 1].
//
// The scales are any fp32 numbers (for products of theirs that fp32 does not hold see
// fm_power), so the tensor cores (kind::f8f6f4) sum one
// block of 128 k at a time into a buffer of tensor memory of its own; eight warps
// read it from there, multiply with the block's scales and add to sums that they
// keep in registers, while the next block is multiplied into the next buffer.
// Two forms, by which operand the MMA has as its M = 128:
//   few tokens   128 weight rows (one scale block) by 16 to 128 tokens, so that a
//                few tokens cost a narrow MMA; K is split over the CTAs of a
//                cluster where there are few tiles.  Bound by the weights' bytes:
//                256 rows of 60 experts x 2816 x 2048 run at 6.8 TB/s; one token's
//                four experts take 8.8 us for 3.4 us of bytes (6.6 where these lie
//                in L2): their 88 tiles leave 64 of 152 SMs without one (K over two
//                CTAs each would be more than the SMs), and launch, first copies
//                and last block add to it.  16 x 8192 x 8192 runs on 128 SMs, 333 x
//                4099 x 1424, in the other form, on 99.
//   many tokens  128 tokens by 128 or 256 weight rows.  A block of 128 x 256 takes
//                860 cycles: a copy takes about 1700 to arrive and four stages of
//                48 KB fit, so that one is there every 780; reading, scaling and
//                adding takes 450 a warp, which two buffers leave in a chain with
//                the MMA's 515 and the hand-overs.  8192^3 in 400 to 415 us, 2.7
//                PFLOP/s, and 455 where it runs for seconds (the power limit,
//                1360 W, takes the clocks down to 1.67 GHz).
#include <cuda.h>

#include "fp8.cuh"
#include "launch.h"
#include "tmap.h"

namespace qmoe {

// Few tokens.  A block's scales are a vector over the tokens, which two warps put
// together in shared memory.  Tensor memory is read in the layout of 8 x 8
// fragments, in which a thread's neighbouring values are neighbouring tokens: one
// pair of scales serves eight values, and packed fp32 arithmetic does two at a
// time.  Warp 0 copies codes, 1 issues MMAs, 2 and 3 prepare scales, 4 to 11 scale
// and add the blocks' sums and write y.
constexpr int kFmThreads = 384;
constexpr uint32_t kFmSmem = 232448;  // 227 KB
constexpr uint32_t kFmBars = 1024;
constexpr uint32_t kFmTable = 3328;  // experts' first token tile, first and last row

struct FmParams {
  const uint8_t *xc, *wc;
  const float *xs, *ws;
  const int32_t* offsets;
  void* y;
  uint32_t* status;
  int E, M, N, K, y_dtype;
  int row_tiles;        // tiles of an expert's weight rows
  int wide_out;         // y: 16 bits, rows on 16-byte boundaries
  int wide_scales;      // four of a row's scales on 16 bytes
  int split, lsplit;    // CTAs of a cluster that share a tile's K, and the logarithm of that
  uint32_t stall;       // QMOE_DIAG_STALL_FP8_*: this role waits for what cannot arrive
  long long wait_limit; // SM cycles
};

template <int BN>
struct FmPlan {
  static constexpr uint32_t kA = 128 * 128, kB = BN * 128;  // a block's codes
  static constexpr int kBox = BN < 64 ? BN : 64;                 // tokens of a copy
  // buffers of tensor memory for the blocks' sums
  static constexpr int kBufs = BN >= 64 ? 512 / BN : 8;
  // tokens that a warp reads at once, and how often: two warps per lane quadrant take turns
  static constexpr int kW = BN >= 64 ? 32 : BN / 2, kQ = BN / 2 / kW, kG = kW / 8;
  static constexpr uint32_t kOut = 8 * kW * 64;                  // 32 outputs of kW tokens a warp, turned round there
  static constexpr int kQuads = 4;                               // scales: slots of four blocks
  static constexpr uint32_t kScales = kQuads * 4 * BN * 4;
  // a split tile's partial sums [split][tokens of a CTA / 2][128][2]: a place of
  // their own where they are small, else the ring once the cluster is done with it
  static constexpr uint32_t kPart = BN <= 64 ? BN * 512 : 0;
  static constexpr int kList = 64;                               // a CTA's first tiles, worked out at the start
  static constexpr uint32_t kFixed = kFmBars + kFmTable + kList * 16 + kOut + kScales + kPart;
  static constexpr uint32_t kAt = (kFixed + 1023) & ~1023u;      // the ring's place
  static constexpr uint32_t kStage = (kA + kB + 1023) & ~1023u;
  static constexpr int kStages0 = (int)((kFmSmem - 1024 - kAt) / kStage);
  static constexpr int kStages = kStages0 > 12 ? 12 : kStages0;
};

constexpr float kFmLargest = 3.40282347e38f;

// The status word of the calls that bring none.
__device__ uint32_t g_fp8_status;
__device__ __forceinline__ void fm_status(const FmParams& p, uint32_t bit) {
  set_status(p.status ? p.status : &g_fp8_status, bit);
}

// Bounded wait; gives up when another role has, or after the limit (about 2 s)
// with the status bit.  WARP: all lanes of the warp wait and agree on the answer
// by a vote (each may see the phase end at another poll).  The warp that issues
// MMAs has no votes: what its elected lane sees decides all that it does.
template <bool WARP = true>
__device__ __forceinline__ bool fm_wait(uint64_t* bar, uint32_t parity, const FmParams& p, volatile int* abort) {
  auto all = [](bool v) { return WARP ? __all_sync(0xffffffffu, v) != 0 : v; };
  if (all(mbar_try_wait(bar, parity))) return true;
  const long long t0 = clock64();
  while (!all(mbar_try_wait_sleep(bar, parity, 20000u))) {
    const bool late = clock64() - t0 > p.wait_limit;
    if (!all(!(late || *abort))) {
      if (late) fm_status(p, QMOE_ST_TIMEOUT);
      *abort = 1;
      return false;
    }
  }
  return true;
}

// The end of a warp that has issued `it` copies into a ring of S slots: it waits
// for the last use of each, time-out or not, so that no copy lands in shared
// memory that is another CTA's by then.  After a time-out slots may stay as they
// are; a copy lands within microseconds, so 10 ms for all of them do.
constexpr long long kFmSettleCycles = 20000000;
template <int S>
__device__ __forceinline__ void fm_settle(uint64_t* bars, int it, const FmParams& p, volatile int* abort) {
  const long long t0 = clock64();
  for (int n = max(it - S, 0); n < it; ++n)
    while (!mbar_try_wait_sleep(&bars[n % S], (n / S) & 1, 20000u)) {
      const long long t = clock64() - t0;
      if (*abort) {
        if (t > kFmSettleCycles) break;
      } else if (t > p.wait_limit) {
        fm_status(p, QMOE_ST_TIMEOUT);
        *abort = 1;
      }
    }
}

__device__ __forceinline__ void fm_store(const FmParams& p, size_t i, float v) {
  if (p.y_dtype == QMOE_F32) static_cast<float*>(p.y)[i] = v;
  else static_cast<uint16_t*>(p.y)[i] = p.y_dtype == QMOE_BF16 ? Half<__nv_bfloat16>::from_float(v) : Half<__half>::from_float(v);
}
// two results to the output's 16-bit type
__device__ __forceinline__ uint32_t fm_pack(const FmParams& p, f2 v) {
  if (p.y_dtype == QMOE_BF16) {
    const __nv_bfloat162 h = __floats2bfloat162_rn(v.x, v.y);
    return *reinterpret_cast<const uint32_t*>(&h);
  }
  const __half2 h = __floats2half2_rn(v.x, v.y);
  return *reinterpret_cast<const uint32_t*>(&h);
}

// A block's sum is multiplied with the product of its two scales.  Where that product
// is no normal number of fp32 although neither scale is 0, infinite or NaN, it has
// lost bits that the outcome has (2^-70 times 2^-70 with a sum of 2^20), or is
// infinite where the sum is 0 or small.  A token's outputs with such a product are
// worked out again at the end (fm_again).  What brings such a product back, or 1:
__device__ __forceinline__ float fm_power(float x, float w) {
  const float f = fabsf(x * w);
  if ((f >= 0x1p-126f && f <= kFmLargest) || x == 0.f || w == 0.f || !isfinite(x) || !isfinite(w)) return 1.f;
  return f < 1.f ? 0x1p64f : 0x1p-64f;
}
// The warps that prepare scales only keep the least and the largest of each kind, from
// which they tell whether some product could be out of range.  So the usual call takes
// 0 to 2 % longer than unasked, the smallest 5 (1 x 1408 x 2048: 3.36 -> 3.5 us); asked
// product by product, with the sums brought back in tensor memory, 8192^3 took 6 to 11.
struct FmRange {
  uint32_t least_x = ~0u, most_x = 0, least_w = ~0u, most_w = 0;  // bits
  __device__ __forceinline__ void token(float v) {
    least_x = min(least_x, __float_as_uint(v));
    most_x = max(most_x, __float_as_uint(v));
  }
  __device__ __forceinline__ void weight(float v) {
    least_w = min(least_w, __float_as_uint(v));
    most_w = max(most_w, __float_as_uint(v));
  }
  // exponents (biased by 127) of normal numbers below 2^-126 or above 2^127 together, or
  // numbers that are subnormal, 0 or negative
  __device__ __forceinline__ bool left() const {
    return (least_x >> 23) + (least_w >> 23) < 2 * 127 - 126 || (most_x >> 23) + (most_w >> 23) > 2 * 127 + 126 ||
           min(least_x, least_w) < 0x00800000u || max(most_x, most_w) >= 0x80000000u;
  }
};

// Outputs n .. n1 - 1 (in one block of 128) of token m again, if it has a product out of
// range.  The product is taken times a power of two that brings it back, rounded once;
// the block's sum, which is 0 or 2^-18 to 2^25 in magnitude, takes the inverse exactly.
// A warp calls it, a lane to an output, in plain fp32: 2048^3 with every token so 4.8 ms
// instead of 13 us, one token of 2048 0.15.
__device__ __forceinline__ void fm_again(const FmParams& p, int e, int n, int n1, int m) {
  const int lane = threadIdx.x & 31, nb = (p.K + 127) / 128;
  const float *xs = p.xs + (size_t)m * nb, *ws = p.ws + ((size_t)e * ((p.N + 127) / 128) + n / 128) * nb;
  bool out = false;
  for (int c = lane; c < nb; c += 32) out |= fm_power(xs[c], ws[c]) != 1.f;
  if (!__any_sync(0xffffffffu, out)) return;
  for (int i = n + lane; i < n1; i += 32) {
    const uint8_t *x = p.xc + (size_t)m * p.K, *w = p.wc + ((size_t)e * p.N + i) * p.K;
    float y = 0.f;
    for (int c = 0; c < nb; ++c) {
      float sum = 0.f;
#pragma unroll 1
      for (int k = c * 128; k < min(p.K, c * 128 + 128); k += 16) {
        const uint4 q = *reinterpret_cast<const uint4*>(x + k), r = *reinterpret_cast<const uint4*>(w + k);
        auto four = [&](uint32_t s, uint32_t t) {
          float a[4], b[4];
          mx_from_e4m3x4(s, a);
          mx_from_e4m3x4(t, b);
#pragma unroll
          for (int j = 0; j < 4; ++j) sum = fmaf(a[j], b[j], sum);
        };
        four(q.x, r.x), four(q.y, r.y), four(q.z, r.z), four(q.w, r.w);
      }
      const float u = xs[c], v = ws[c], power = fm_power(u, v);
      // (u times the power is exact: u is below 2^23 where the product is small, since v is
      // at least 2^-149, and above 1 where it is large)
      float s = u * power * v;
      if (power < 1.f) s = fminf(fmaxf(s, -kFmLargest), kFmLargest);  // a sum of 0 stays 0
      y = fmaf(sum * (1.f / power), s, y);
    }
    fm_store(p, (size_t)m * p.N + i, y);
  }
}

// 32 lanes x 8 G columns of tensor memory as fragments: r[i][j] holds columns
// 8 i + 2 (lane % 4) + {0, 1} of row lane / 4 + 8 j.
template <int G>
__device__ __forceinline__ void fm_load(uint32_t taddr, f2 (&r)[G][4]) {
  uint32_t lo[4 * G], hi[4 * G];
  if constexpr (G == 4) {
    tmem_ld_frag(taddr, lo, hi);
  } else if constexpr (G == 2) {
    asm volatile(
        "tcgen05.ld.sync.aligned.16x256b.x2.b32 {%0,%1,%2,%3,%4,%5,%6,%7}, [%16];\n"
        "tcgen05.ld.sync.aligned.16x256b.x2.b32 {%8,%9,%10,%11,%12,%13,%14,%15}, [%17];\n"
        "tcgen05.wait::ld.sync.aligned;"
        : "=r"(lo[0]), "=r"(lo[1]), "=r"(lo[2]), "=r"(lo[3]), "=r"(lo[4]), "=r"(lo[5]), "=r"(lo[6]), "=r"(lo[7]),
          "=r"(hi[0]), "=r"(hi[1]), "=r"(hi[2]), "=r"(hi[3]), "=r"(hi[4]), "=r"(hi[5]), "=r"(hi[6]), "=r"(hi[7])
        : "r"(taddr), "r"(taddr + (16u << 16))
        : "memory");
  } else {
    asm volatile(
        "tcgen05.ld.sync.aligned.16x256b.x1.b32 {%0,%1,%2,%3}, [%8];\n"
        "tcgen05.ld.sync.aligned.16x256b.x1.b32 {%4,%5,%6,%7}, [%9];\n"
        "tcgen05.wait::ld.sync.aligned;"
        : "=r"(lo[0]), "=r"(lo[1]), "=r"(lo[2]), "=r"(lo[3]), "=r"(hi[0]), "=r"(hi[1]), "=r"(hi[2]), "=r"(hi[3])
        : "r"(taddr), "r"(taddr + (16u << 16))
        : "memory");
  }
#pragma unroll
  for (int i = 0; i < G; ++i)
#pragma unroll
    for (int j = 0; j < 2; ++j) {
      r[i][j] = make_float2(__uint_as_float(lo[4 * i + 2 * j]), __uint_as_float(lo[4 * i + 2 * j + 1]));
      r[i][j + 2] = make_float2(__uint_as_float(hi[4 * i + 2 * j]), __uint_as_float(hi[4 * i + 2 * j + 1]));
    }
}

// D[tmem] (+)= A x B^T of e4m3 codes (shared-memory descriptors as sw128_desc,
// low words), 32 k, by the lane of a converged warp whose e is 1.
__device__ __forceinline__ void mma_f8(uint32_t e, uint32_t d, uint32_t a, uint32_t b, uint32_t idesc,
                                       uint32_t accumulate) {
  asm volatile(
      "{\n .reg .pred p, e;\n .reg .b64 a, b;\n mov.b64 a, {%1, %6};\n mov.b64 b, {%2, %6};\n"
      " setp.ne.b32 e, %5, 0;\n setp.ne.b32 p, %4, 0;\n"
      " @e tcgen05.mma.cta_group::1.kind::f8f6f4 [%0], a, b, %3, p;\n}" ::"r"(d),
      "r"(a), "r"(b), "r"(idesc), "r"(accumulate), "r"(e), "n"((1024u >> 4) | 1u << 14 | 2u << 29)
      : "memory");
}

__device__ __forceinline__ void fm_prefetch_map(const void* tmap) {
  asm volatile("prefetch.tensormap [%0];" ::"l"(reinterpret_cast<uint64_t>(tmap)) : "memory");
}

// A tile: the expert, which of its tiles of weight rows, tokens m0 .. m1 - 1.
struct alignas(16) FmTile {
  int e, rt, m0, m1;
};
struct FmTable {
  int first[kMaxExperts + 1];  // token tiles of the experts before
  int start[kMaxExperts], end[kMaxExperts];
};
static_assert(sizeof(FmTable) <= kFmTable, "table");

// The experts' rows and token tiles of BN; no tiles where the offsets are no
// offsets.  All threads of the CTA (at least as many as experts).
template <int BN>
__device__ __forceinline__ void fm_table(const FmParams& p, FmTable& tab, int* s_sum) {
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
  if (!p.offsets) {
    if (tid == 0) tab.first[0] = 0, tab.first[1] = (p.M + BN - 1) / BN, tab.start[0] = 0, tab.end[0] = p.M;
  } else {
    int sum = 0, bad = 0;
    if (tid < p.E) {
      const int a = p.offsets[tid], b = p.offsets[tid + 1];
      bad = a < 0 || b < a || b > p.M;
      tab.start[tid] = a;
      tab.end[tid] = b;
      sum = (int)(((long long)b - a + BN - 1) / BN);
    }
    bad = __syncthreads_or(bad);
    if (bad) sum = 0;
    if (bad && blockIdx.x == 0 && tid == 0) fm_status(p, QMOE_ST_INDEX);
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
      const int up = __shfl_up_sync(0xffffffffu, sum, o);
      if (lane >= o) sum += up;
    }
    if (warp < 8 && lane == 31) s_sum[warp] = sum;
    __syncthreads();
    if (tid < p.E) {
      for (int w = 0; w < warp; ++w) sum += s_sum[w];
      tab.first[tid + 1] = sum;
      if (tid == 0) tab.first[0] = 0;
    }
  }
  __syncthreads();
}

// Tile t: by expert, within it in groups of 8 row tiles, so that the tiles in
// flight share weights and tokens in L2.
template <int BN>
__device__ __forceinline__ FmTile fm_tile(const FmParams& p, const FmTable& tab, int t) {
  FmTile f;
  const int q = t / p.row_tiles;
  int lo = 0, hi = p.E;  // first[lo] <= q < first[hi]
  while (hi - lo > 1) {
    const int mid = (lo + hi) >> 1;
    if (tab.first[mid] <= q) lo = mid;
    else hi = mid;
  }
  const int tok = tab.first[lo + 1] - tab.first[lo];
  t -= tab.first[lo] * p.row_tiles;
  f.e = lo;
  f.rt = t;
  f.m0 = tab.start[lo];
  if (tok > 1) {
    const int per = 8 * tok, g = t / per, r = t - g * per, rows = min(8, p.row_tiles - g * 8);
    f.rt = g * 8 + r % rows;
    f.m0 += r / rows * BN;
  }
  f.m1 = min(f.m0 + BN, tab.end[lo]);
  return f;
}

template <int BN>
__global__ void __launch_bounds__(kFmThreads, 1)
    fp8_matmul_kernel(const __grid_constant__ CUtensorMap tm_w, const __grid_constant__ CUtensorMap tm_x,
                      const __grid_constant__ FmParams p) {
  using P = FmPlan<BN>;
  constexpr int S = P::kStages, NB = P::kBufs, SQ = P::kQuads;
  extern __shared__ __align__(1024) uint8_t smem_raw[];
  uint8_t* smem = smem_raw + ((1024u - (smem_u32(smem_raw) & 1023u)) & 1023u);
  uint64_t* full = reinterpret_cast<uint64_t*>(smem);
  uint64_t* empty = full + S;
  uint64_t* acc_full = empty + S;      // [NB]
  uint64_t* acc_free = acc_full + NB;  // [NB]
  uint64_t* sc_full = acc_free + NB;   // [SQ]
  uint64_t* sc_free = sc_full + SQ;    // [SQ]
  uint64_t* fin = sc_free + SQ;
  uint64_t* never = fin + 1;  // nothing arrives here (p.stall)
  uint32_t* s_tmem = reinterpret_cast<uint32_t*>(never + 1);
  volatile int* s_abort = reinterpret_cast<volatile int*>(s_tmem + 1);
  int* s_sum = reinterpret_cast<int*>(s_tmem + 2);  // [8]
  volatile int* s_left = s_sum + 8;  // a scale has left FmRange
  FmTable& tab = *reinterpret_cast<FmTable*>(smem + kFmBars);
  FmTile* list = reinterpret_cast<FmTile*>(smem + kFmBars + kFmTable);
  uint8_t* outbuf = smem + kFmBars + kFmTable + P::kList * sizeof(FmTile);
  float* scales = reinterpret_cast<float*>(outbuf + P::kOut);
  float* part_own = scales + P::kScales / 4;
  uint8_t* ring = smem + P::kAt;
  const int tid = threadIdx.x, lane = tid & 31;
  const int warp = __shfl_sync(0xffffffffu, tid >> 5, 0);  // known to be the same in all lanes

  // (by 32 threads: one takes 300 cycles for fifty barriers)
  if (warp == 2) {
    for (int i = lane; i < 2 * S + 2 * NB + 2 * SQ + 2; i += 32) {
      const int a = i - 2 * S, q = a - 2 * NB;
      mbar_init(&full[i], a >= NB && q < 0 ? 8 : q < 0 || q >= 2 * SQ ? 1 : q < SQ ? 2 : 8);
    }
    if (lane == 0) *s_abort = 0, *s_left = 0;
    fence_barrier_init();
  }
  if (warp == 1) {
    tmem_alloc(s_tmem, 512);
    tmem_relinquish();
  }
  if (warp == 0) fm_prefetch_map(&tm_w), fm_prefetch_map(&tm_x);
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  // all 512 columns are this CTA's, so they start at 0
  constexpr uint32_t tmem = 0;
  if (P::kPart && p.split > 1) cluster_arrive();  // this CTA runs: its shared memory may be written
  pdl_wait();
  pdl_trigger();

  fm_table<BN>(p, tab, s_sum);

  // this CTA's tiles and its share [c0, c1) of their blocks along K
  const int rank = p.split > 1 ? (int)cluster_ctarank() : 0;
  const int tiles = tab.first[p.E] * p.row_tiles;
  const int first = blockIdx.x >> p.lsplit, step = p.split > 1 ? max(tiles, (int)gridDim.x) : gridDim.x;
  const int nb = (p.K + 127) / 128;
  auto stalled = [&](uint32_t role) { return (p.stall & role) && !fm_wait(never, 0, p, s_abort); };
  const int c0 = nb * rank >> p.lsplit, c1 = nb * (rank + 1) >> p.lsplit;  // (nb is at most 2^24)
  // (a search and divisions of some 400 cycles, which every role would wait for
  // at each tile: 60 experts' 8192 rows 81 -> 77.5 us in the wide form, one token's
  // four experts 7.1 -> 6.5 with the barriers' setup by 32 threads)
  static_assert(sizeof(FmTile) == 16, "list");
  for (int i = tid; i < P::kList && first + (long long)i * step < tiles; i += kFmThreads)
    list[i] = fm_tile<BN>(p, tab, first + i * step);
  __syncthreads();
  auto nth = [&](int i, int t) { return i < P::kList ? list[i] : fm_tile<BN>(p, tab, t); };
  f2 acc[P::kQ][P::kG][4];
  bool left = false;  // the warps of the scales: FmRange

  if (warp == 0) {
    // ------------------------------------------------------------ codes
    int it = 0, s = 0;
    uint32_t ph = 0;
    bool ok = !stalled(QMOE_DIAG_STALL_FP8_CODES);
    const uint32_t el = elect_lane();
    for (int t = first, i = 0; t < tiles && ok; t += step, ++i) {
      const FmTile f = nth(i, t);
      const int row = f.e * p.N + f.rt * 128;
      const int boxes = (f.m1 - f.m0 + P::kBox - 1) / P::kBox;  // copies, as many as the tile has tokens
      for (int c = c0; c < c1; ++c, ++it) {
        if (it >= S) ok = fm_wait(&empty[s], ph ^ 1u, p, s_abort);
        if (!ok) break;
        if (el) {
          uint8_t* st = ring + s * P::kStage;
          mbar_arrive_expect_tx(&full[s], P::kA + boxes * P::kBox * 128);
          tma_load_2d(st, &tm_w, c * 128, row, &full[s]);
          for (int i = 0; i < boxes; ++i)
            tma_load_2d(st + P::kA + i * P::kBox * 128, &tm_x, c * 128, f.m0 + i * P::kBox, &full[s]);
        }
        __syncwarp();
        if (++s == S) {
          s = 0;
          ph ^= 1u;
        }
      }
    }
    if (lane == 0) fm_settle<S>(full, it, p, s_abort);
  } else if (warp == 1) {
    // ------------------------------------------------------------- MMAs
    int n = 0, s = 0;  // blocks so far
    uint32_t ph = 0;
    bool ok = !stalled(QMOE_DIAG_STALL_FP8_MMA), issued = false;
    const uint32_t el = elect_lane();
    for (int t = first, i = 0; t < tiles && ok; t += step, ++i) {
      const FmTile f = nth(i, t);
      const int cols = (f.m1 - f.m0 + 15) & ~15;
      // D fp32, A and B e4m3, both K-major
      const uint32_t idesc = 1u << 4 | (uint32_t)(cols >> 3) << 17 | (uint32_t)(128 >> 4) << 24;
      for (int c = c0; c < c1; ++c, ++n) {
        const int b = n % NB;
        if (n >= NB) ok = fm_wait<false>(&acc_free[b], (n / NB - 1) & 1, p, s_abort);
        if (ok) ok = fm_wait<false>(&full[s], ph, p, s_abort);
        if (!ok) break;
        tc_fence_after();
        const uint32_t st = (smem_u32(ring + s * P::kStage) >> 4) & 0x3FFFu;  // a descriptor's address field
        const uint32_t da = st | 1u << 16, db = (st + (P::kA >> 4)) | 1u << 16;
        const int left = p.K - c * 128;
#pragma unroll
        for (int j = 0; j < 4; ++j) {
          if (32 * j >= left) break;
          mma_f8(el, tmem + b * BN, da + 2 * j, db + 2 * j, idesc, j > 0);
        }
        mma_commit_mx<1>(el, &empty[s]);
        mma_commit_mx<1>(el, &acc_full[b]);
        issued = true;
        if (++s == S) {
          s = 0;
          ph ^= 1u;
        }
      }
    }
    if (issued) {  // all MMAs have finished before tensor memory is freed
      mma_commit_mx<1>(el, fin);
      if (el) mbar_wait(fin, 0, nullptr);
    }
  } else if (warp == 2 || warp == 3) {
    // ----------------------------------------- scales, four blocks at a time
    int it = 0;
    const int rb = (p.N + 127) / 128;
    FmRange range;
    bool ok = !stalled(QMOE_DIAG_STALL_FP8_SCALES);
    for (int t = first, i = 0; t < tiles && ok; t += step, ++i) {
      const FmTile f = nth(i, t);
      const int rt = f.rt;
      const float* ws = p.ws + ((size_t)f.e * rb + rt) * nb;
      for (int c = c0; c < c1; c += 4, ++it) {
        const int q = it % SQ;
        float w[4];
#pragma unroll
        for (int j = 0; j < 4; ++j) w[j] = rt < rb && c + j < c1 ? ws[c + j] : 1.f;  // (1: nobody reads it)
        if (it >= SQ) ok = fm_wait(&sc_free[q], (it / SQ - 1) & 1, p, s_abort);
        if (!ok) break;
        float* out = scales + q * 4 * BN;
#pragma unroll
        for (int i = (warp - 2) * 32 + lane; i < BN; i += 64) {
          float v[4] = {1.f, 1.f, 1.f, 1.f};
          if (f.m0 + i < f.m1) {
            const float* xs = p.xs + (size_t)(f.m0 + i) * nb + c;
            if (p.wide_scales) {
              const float4 u = *reinterpret_cast<const float4*>(xs);
              v[0] = u.x, v[1] = u.y, v[2] = u.z, v[3] = u.w;
            } else {
#pragma unroll
              for (int j = 0; j < 4; ++j) v[j] = c + j < c1 ? xs[j] : 1.f;
            }
          }
#pragma unroll
          for (int j = 0; j < 4; ++j) {
            out[j * BN + i] = v[j] * w[j];
            range.token(v[j]);
          }
        }
#pragma unroll
        for (int j = 0; j < 4; ++j) range.weight(w[j]);  // (not before the loads that follow w's)
        __syncwarp();
        if (lane == 0) mbar_arrive(&sc_full[q]);
      }
    }
    left = range.left();
  } else if (warp >= 4) {
    // ------------------------------------- the blocks' sums, scaled and added
    const int qd = warp & 3, set = (warp - 4) >> 2;
    uint8_t* buf = outbuf + (warp - 4) * (P::kW * 64);
    int n = 0, it = 0;
    bool ok = !stalled(QMOE_DIAG_STALL_FP8_OUTPUT);
    for (int t = first, i = 0; t < tiles && ok; t += step, ++i) {
      const FmTile f = nth(i, t);
      const int cols = f.m1 - f.m0;
#pragma unroll
      for (int q = 0; q < P::kQ; ++q)
#pragma unroll
        for (int i = 0; i < P::kG; ++i)
#pragma unroll
          for (int j = 0; j < 4; ++j) acc[q][i][j] = make_float2(0.f, 0.f);
      for (int c = c0; c < c1; ++c, ++n) {
        const int b = n % NB, sub = (c - c0) & 3, slot = it % SQ;
        if (sub == 0) ok = fm_wait(&sc_full[slot], (it / SQ) & 1, p, s_abort);
        if (ok) ok = fm_wait(&acc_full[b], (n / NB) & 1, p, s_abort);
        if (!ok) break;
        tc_fence_after();
        const float* sc = scales + (slot * 4 + sub) * BN + 2 * (lane & 3);
        const uint32_t d = tmem + ((uint32_t)(qd * 32) << 16) + b * BN;
#pragma unroll
        for (int q = 0; q < P::kQ; ++q) {
          const int col = (2 * q + set) * P::kW;
          if (col < cols) {
            f2 v[P::kG][4];
            fm_load<P::kG>(d + col, v);
#pragma unroll
            for (int i = 0; i < P::kG; ++i) {
              const f2 s = *reinterpret_cast<const f2*>(sc + col + 8 * i);
#pragma unroll
              for (int j = 0; j < 4; ++j) acc[q][i][j] = ffma2(v[i][j], s, acc[q][i][j]);
            }
          }
        }
        tc_fence_before();
        __syncwarp();
        if (lane == 0) {
          mbar_arrive(&acc_free[b]);
          if (sub == 3 || c + 1 == c1) mbar_arrive(&sc_free[slot]);
        }
        if (sub == 3 || c + 1 == c1) ++it;
      }
      if (!ok || p.split > 1) break;
      const int n0 = f.rt * 128 + qd * 32;
#pragma unroll
      for (int q = 0; q < P::kQ; ++q) {
        const int col = (2 * q + set) * P::kW, m = f.m0 + col;
        if (m >= f.m1 || n0 >= p.N) continue;
        if (p.wide_out) {
          // token 8 i + lane % 8 is a row of 64 bytes; its four 16-byte pieces
          // (8 outputs each) are permuted against bank conflicts
          const uint32_t a = smem_u32(buf) + (lane & 7) * 64 + (((lane >> 3) ^ ((lane >> 1) & 3)) << 4);
#pragma unroll
          for (int i = 0; i < P::kG; ++i)
            stmatrix_t4(a + i * 512, fm_pack(p, acc[q][i][0]), fm_pack(p, acc[q][i][1]), fm_pack(p, acc[q][i][2]),
                        fm_pack(p, acc[q][i][3]));
          __syncwarp();
          const int tok = lane >> 2, piece = lane & 3;
          uint16_t* y = static_cast<uint16_t*>(p.y) + (size_t)(m + tok) * p.N + n0 + piece * 8;
#pragma unroll
          for (int i = 0; i < P::kG; ++i, y += (size_t)8 * p.N)
            if (m + 8 * i + tok < f.m1 && n0 + piece * 8 < p.N)
              *reinterpret_cast<uint4*>(y) =
                  *reinterpret_cast<const uint4*>(buf + i * 512 + tok * 64 + ((piece ^ ((tok >> 1) & 3)) << 4));
          __syncwarp();
        } else {
#pragma unroll
          for (int i = 0; i < P::kG; ++i)
#pragma unroll
            for (int j = 0; j < 4; ++j) {
              const int nn = n0 + (lane >> 2) + 8 * j, mm = m + 8 * i + 2 * (lane & 3);
              if (nn < p.N) {
                if (mm < f.m1) fm_store(p, (size_t)mm * p.N + nn, acc[q][i][j].x);
                if (mm + 1 < f.m1) fm_store(p, (size_t)(mm + 1) * p.N + nn, acc[q][i][j].y);
              }
            }
        }
      }
    }
  }
  __syncwarp();
  if (p.split > 1) {
    // Each CTA sends its partial sums of tokens j to CTA j / per, which adds
    // them in rank order and writes y.  (A cluster without a tile only keeps
    // the barriers.)
    float* part = P::kPart ? part_own : reinterpret_cast<float*>(ring);
    const bool some = first < tiles;
    FmTile f = {0, 0, 0, 0};
    if (some) f = list[0];
    const int rows = f.m1 - f.m0, per = max(2, BN / p.split), lper = 31 - __clz(per);
    if (!P::kPart) cluster_arrive();
    cluster_wait();
    if (warp >= 4) {
      const int qd = warp & 3, set = (warp - 4) >> 2;
#pragma unroll
      for (int q = 0; q < P::kQ; ++q)
#pragma unroll
        for (int i = 0; i < P::kG; ++i) {
          const int tok = (2 * q + set) * P::kW + 8 * i + 2 * (lane & 3);
          if (tok < rows) {
            const uint32_t to = peer_u32(part + (((size_t)rank * per + (tok & (per - 1))) * 64 + qd * 32 + (lane >> 2)) * 2, tok >> lper);
#pragma unroll
            for (int j = 0; j < 4; ++j)
              asm volatile("st.shared::cluster.v2.f32 [%0], {%1, %2};" ::"r"(to + 64 * j), "f"(acc[q][i][j].x), "f"(acc[q][i][j].y)
                           : "memory");
          }
        }
    }
    if (left)
      for (int r = 0; r < p.split; ++r)
        asm volatile("st.shared::cluster.u32 [%0], %1;" ::"r"(peer_u32(const_cast<int*>(s_left), r)), "r"(1) : "memory");
    __syncwarp();
    cluster_sync_all();
    const int mine = min(per, rows - rank * per);
    const f2* p2 = reinterpret_cast<const f2*>(part);
    for (int i = tid; i < (mine + 1) / 2 * 128; i += blockDim.x) {
      const int nn = f.rt * 128 + (i & 127), j = rank * per + (i >> 7) * 2;
      if (nn < p.N) {
        f2 v = p2[i];
        for (int r = 1; r < p.split; ++r) v = fadd2(v, p2[r * per * 64 + i]);
        const size_t o = (size_t)(f.m0 + j) * p.N + nn;
        fm_store(p, o, v.x);
        if (j + 1 < rows) fm_store(p, o + p.N, v.y);
      }
    }
  } else if (left) {
    *s_left = 1;
  }
  tc_fence_before();
  __syncthreads();
  if (warp == 1) {
    tc_fence_after();
    tmem_dealloc(tmem, 512);
  }
  if (*s_left) {
    const int per = max(2, BN / p.split);  // a CTA's tokens of a split tile
    for (int t = first, i = 0; t < tiles; t += step, ++i) {
      const FmTile f = nth(i, t);
      const int a = f.m0 + rank * per, n0 = f.rt * 128, many = (p.split > 1 ? min(a + per, f.m1) : f.m1) - a;
      for (int j = warp; j < 4 * many; j += kFmThreads / 32)
        fm_again(p, f.e, n0 + (j & 3) * 32, min(p.N, n0 + (j & 3) * 32 + 32), a + j / 4);
    }
  }
}

// ------------------------------------------------------------- many tokens
// Here 128 tokens are the MMA's M operand and BN weight rows its N: a thread of
// the warps that add has a token to itself, so that a block's scale is one number
// to it, and reads tensor memory in whole rows (32x32b, measured at 18 cycles for
// 32 columns of a warp; fragments take 32), 16 columns ahead of its sums.  Warp 0
// copies codes, 1 issues MMAs, 2 prepares scales, 4 to 11 add and write y, two to
// each lane quadrant with a half of the columns each.  Measured at 8192^3 and not
// kept (400 to 415 us, for seconds 455): pairs of CTAs (cta_group::2) 415, for
// seconds 437; a buffer handed back by halves 423 to 450; sixteen adding warps 497;
// three stages 432; blocks issued by two warps in turn 403.
constexpr int kFwThreads = 384;
// 256 outputs: the adding warps hold 128 sums a thread and take registers of the
// others: 256 x 208 + 128 x 88 = 384 x 168, which the launch has (checked there).
constexpr int kFwRegs = 168, kFwManyRegs = 208, kFwFewRegs = 88;
static_assert(256 * kFwManyRegs + 128 * kFwFewRegs <= kFwThreads * kFwRegs, "registers");

template <int BN>
struct FwPlan {
  static constexpr uint32_t kA = 128 * 128, kB = BN * 128, kStage = kA + kB;  // a block's codes
  static constexpr int kBufs = 512 / BN;
  static constexpr int kHalves = BN / 128;                        // scale blocks of a tile's weight rows
  static constexpr int kC = BN / 2 / 16;                          // a warp's columns, 16 at a time
  static constexpr int kQuads = 2;                                // scales: slots of four blocks
  static constexpr uint32_t kScales = kQuads * 4 * kHalves * 512;
  static constexpr uint32_t kOut = 8 * 32 * 17 * 4;               // rows of y that are not written in wide words
  static constexpr int kList = 64;                                // a CTA's first tiles, worked out at the start
  static constexpr uint32_t kAt = (kFmBars + kFmTable + kList * 32 + kScales + kOut + 1023) & ~1023u;
  static constexpr int kStages = (int)((kFmSmem - 1024 - kAt) / kStage);
};

__device__ __forceinline__ void fw_load(uint32_t taddr, uint32_t (&r)[16]) {
  asm volatile(
      "tcgen05.ld.sync.aligned.32x32b.x16.b32 {%0,%1,%2,%3,%4,%5,%6,%7,%8,%9,%10,%11,%12,%13,%14,%15}, [%16];"
      : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3]), "=r"(r[4]), "=r"(r[5]), "=r"(r[6]), "=r"(r[7]), "=r"(r[8]),
        "=r"(r[9]), "=r"(r[10]), "=r"(r[11]), "=r"(r[12]), "=r"(r[13]), "=r"(r[14]), "=r"(r[15])
      : "r"(taddr)
      : "memory");
}
// waits for the loads so far; the registers pass through, so that no use of
// theirs is scheduled before
__device__ __forceinline__ void fw_wait(uint32_t (&r)[16]) {
  asm volatile("tcgen05.wait::ld.sync.aligned;"
               : "+r"(r[0]), "+r"(r[1]), "+r"(r[2]), "+r"(r[3]), "+r"(r[4]), "+r"(r[5]), "+r"(r[6]), "+r"(r[7]),
                 "+r"(r[8]), "+r"(r[9]), "+r"(r[10]), "+r"(r[11]), "+r"(r[12]), "+r"(r[13]), "+r"(r[14]), "+r"(r[15])
               :
               : "memory");
}

struct alignas(16) FwTile : FmTile {
  int n0, n1;  // outputs
};

template <int BN>
__global__ void __launch_bounds__(kFwThreads, 1)
    fp8_wide_kernel(const __grid_constant__ CUtensorMap tm_w, const __grid_constant__ CUtensorMap tm_x,
                    const __grid_constant__ FmParams p) {
  using P = FwPlan<BN>;
  constexpr int BT = 128;  // tokens of a tile
  constexpr int S = P::kStages, NB = P::kBufs, SQ = P::kQuads;
  extern __shared__ __align__(1024) uint8_t smem_raw[];
  uint8_t* smem = smem_raw + ((1024u - (smem_u32(smem_raw) & 1023u)) & 1023u);
  uint64_t* full = reinterpret_cast<uint64_t*>(smem);
  uint64_t* empty = full + S;
  uint64_t* acc_full = empty + S;      // [NB]
  uint64_t* acc_free = acc_full + NB;  // [NB]
  uint64_t* sc_full = acc_free + NB;   // [SQ]
  uint64_t* sc_free = sc_full + SQ;    // [SQ]
  uint64_t* fin = sc_free + SQ;
  uint64_t* never = fin + 1;  // nothing arrives here (p.stall)
  uint32_t* s_tmem = reinterpret_cast<uint32_t*>(never + 1);
  volatile int* s_abort = reinterpret_cast<volatile int*>(s_tmem + 1);
  int* s_sum = reinterpret_cast<int*>(s_tmem + 2);  // [8]
  volatile int* s_left = s_sum + 8;  // a scale has left FmRange
  FmTable& tab = *reinterpret_cast<FmTable*>(smem + kFmBars);
  FwTile* list = reinterpret_cast<FwTile*>(smem + kFmBars + kFmTable);
  float* scales = reinterpret_cast<float*>(smem + kFmBars + kFmTable + P::kList * sizeof(FwTile));
  uint8_t* outbuf = reinterpret_cast<uint8_t*>(scales) + P::kScales;
  uint8_t* ring = smem + P::kAt;
  const int tid = threadIdx.x, lane = tid & 31;
  const int warp = __shfl_sync(0xffffffffu, tid >> 5, 0);  // known to be the same in all lanes

  if (warp == 2) {
    for (int i = lane; i < 2 * S + 2 * NB + 2 * SQ + 2; i += 32) {
      const int a = i - 2 * S, q = a - 2 * NB;
      mbar_init(&full[i], (a >= NB && q < 0) || (q >= SQ && q < 2 * SQ) ? 8 : 1);
    }
    if (lane == 0) *s_abort = 0, *s_left = 0;
    fence_barrier_init();
  }
  if (warp == 1) {
    tmem_alloc(s_tmem, 512);
    tmem_relinquish();
  }
  if (warp == 0) fm_prefetch_map(&tm_w), fm_prefetch_map(&tm_x);
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  constexpr uint32_t tmem = 0;  // all 512 columns are this CTA's
  pdl_wait();
  pdl_trigger();
  fm_table<BT>(p, tab, s_sum);

  // The tiles of a last round that fewer than half of the CTAs would have are
  // dealt in halves of their outputs (8192^3: 14 rounds of which the last is half as long).
  const int tiles = tab.first[p.E] * p.row_tiles, nb = (p.K + 127) / 128, rest = tiles % (int)gridDim.x;
  const int whole = BN == 256 && 2 * rest <= (int)gridDim.x ? tiles - rest : tiles, parts = 2 * tiles - whole;
  auto part = [&](int v) {
    const int h = v - whole;
    FwTile f = {fm_tile<BT>(p, tab, h < 0 ? v : whole + h / 2)};
    f.n0 = f.rt * BN + (h > 0 && h % 2 ? BN / 2 : 0);
    f.n1 = min(p.N, f.n0 + (h < 0 ? BN : BN / 2));
    return f;  // (an empty half where the outputs end before it)
  };
  // (as in the form for few tokens)
  static_assert(sizeof(FwTile) == 32, "list");
  for (int i = tid; i < P::kList && blockIdx.x + (long long)i * gridDim.x < parts; i += kFwThreads)
    list[i] = part(blockIdx.x + i * gridDim.x);
  __syncthreads();
  auto nth = [&](int i, int t) { return i < P::kList ? list[i] : part(t); };
  auto stalled = [&](uint32_t role) { return (p.stall & role) && !fm_wait(never, 0, p, s_abort); };
  if (warp >= 4) {
    if (BN == 256) asm volatile("setmaxnreg.inc.sync.aligned.u32 %0;" ::"n"(kFwManyRegs));
    // ------------------------------------- the blocks' sums, scaled and added
    const int qd = warp & 3, set = warp >= 8;
    float* buf = reinterpret_cast<float*>(outbuf) + (warp - 4) * 32 * 17;
    int n = 0, it = 0;
    bool ok = !stalled(QMOE_DIAG_STALL_FP8_OUTPUT);
    for (int t = blockIdx.x, i = 0; t < parts && ok; t += gridDim.x, ++i) {
      const FwTile f = nth(i, t);
      if (f.n1 <= f.n0) continue;
      const int n0 = f.n0 + set * (BN / 2), cols = f.n1 - n0;      // this warp's columns
      const int m0 = f.m0 + qd * 32;                               // and tokens
      const bool live = cols > 0 && m0 < f.m1;
      float acc[P::kC][16];
#pragma unroll
      for (int q = 0; q < P::kC; ++q)
#pragma unroll
        for (int j = 0; j < 16; ++j) acc[q][j] = 0.f;
      // `ready`: what is waited for next had come when this was last looked at,
      // which is under the last sums of the block before, so that the answer's
      // latency costs nothing
      bool ready = false;
      for (int c = 0; c < nb; ++c, ++n) {
        const int b = n % NB, sub = c & 3, slot = it % SQ;
        if (!__all_sync(0xffffffffu, ready)) {
          if (sub == 0) ok = fm_wait(&sc_full[slot], (it / SQ) & 1, p, s_abort);
          if (ok) ok = fm_wait(&acc_full[b], (n / NB) & 1, p, s_abort);
          if (!ok) break;
        }
        tc_fence_after();
        const uint32_t d = tmem + ((uint32_t)(qd * 32) << 16) + b * BN + set * (BN / 2);
        uint32_t v[2][16];
        if (live) fw_load(d, v[0]);
        const float s = scales[((slot * 4 + sub) * P::kHalves + (P::kHalves > 1 ? set : 0)) * 128 + qd * 32 + lane];
        auto freed = [&]() {
          tc_fence_before();
          __syncwarp();
          if (lane == 0) mbar_arrive(&acc_free[b]);
          if (sub == 3) ++it;
          ready = c + 1 < nb && mbar_try_wait(&acc_full[(n + 1) % NB], ((n + 1) / NB) & 1) &&
                  (sub != 3 || mbar_try_wait(&sc_full[it % SQ], (it / SQ) & 1));
        };
        if (live) {
#pragma unroll
          for (int q = 0; q < P::kC; ++q) {
            fw_wait(v[q & 1]);
            if (q + 1 < P::kC) fw_load(d + 16 * (q + 1), v[(q + 1) & 1]);
            else freed();  // the last sums are still to come, but the buffer has been read
#pragma unroll
            for (int j = 0; j < 16; ++j) acc[q][j] = fmaf(__uint_as_float(v[q & 1][j]), s, acc[q][j]);
          }
        } else {
          freed();
        }
        if ((sub == 3 || c + 1 == nb) && lane == 0) mbar_arrive(&sc_free[slot]);
      }
      if (nb & 3) ++it;
      if (!ok) break;
      if (!live) continue;
      if (p.wide_out) {
        // 32 tokens x 64 bytes at a time through shared memory (the four 16-byte
        // pieces of a row permuted against bank conflicts), so that four lanes
        // write 64 bytes of a row: a row to each lane takes 32 cycles a store
        uint8_t* row = reinterpret_cast<uint8_t*>(buf) + lane * 64;
        const int w32 = p.y_dtype == QMOE_F32, x = lane >> 1 & 3;
        auto out = [&](int col, int per) {  // columns col .. + 64 bytes, `per` of them to 16 bytes
          __syncwarp();
          const int piece = lane & 3;
#pragma unroll
          for (int i = 0; i < 4; ++i) {
            const int r = 8 * i + (lane >> 2);
            const uint4 v = *reinterpret_cast<const uint4*>(reinterpret_cast<uint8_t*>(buf) + r * 64 + ((piece ^ (r >> 1 & 3)) << 4));
            if (m0 + r < f.m1 && col + piece * per < cols)
              *reinterpret_cast<uint4*>(static_cast<uint8_t*>(p.y) + ((size_t)(m0 + r) * p.N + n0 + col + piece * per) * (w32 ? 4 : 2)) = v;
          }
          __syncwarp();
        };
        if (w32) {
#pragma unroll
          for (int q = 0; q < P::kC; ++q)
            if (16 * q < cols) {
#pragma unroll
              for (int j = 0; j < 4; ++j)
                *reinterpret_cast<float4*>(row + ((j ^ x) << 4)) = make_float4(acc[q][4 * j], acc[q][4 * j + 1], acc[q][4 * j + 2], acc[q][4 * j + 3]);
              out(16 * q, 4);
            }
        } else {
#pragma unroll
          for (int q = 0; q < P::kC; q += 2)
            if (16 * q < cols) {
#pragma unroll
              for (int j = 0; j < 4; ++j) {
                const float* a = acc[q + j / 2] + 8 * (j & 1);
                *reinterpret_cast<uint4*>(row + ((j ^ x) << 4)) =
                    make_uint4(fm_pack(p, make_float2(a[0], a[1])), fm_pack(p, make_float2(a[2], a[3])),
                               fm_pack(p, make_float2(a[4], a[5])), fm_pack(p, make_float2(a[6], a[7])));
              }
              out(16 * q, 8);
            }
        }
      } else {
        // 32 tokens x 16 columns at a time through shared memory, so that
        // neighbouring lanes write neighbouring columns; the type and the address are
        // settled outside the loop (4096 x 8195 x 2048 bf16: 96 -> 80 us; a loop
        // unrolled in full, 81, takes registers that rows on 16 bytes miss: 6 %)
#pragma unroll
        for (int q = 0; q < P::kC; ++q) {
          if (16 * q < cols) {
#pragma unroll
            for (int j = 0; j < 16; ++j) buf[lane * 17 + j] = acc[q][j];
            __syncwarp();
            const int col = lane & 15, rows = 16 * q + col < cols ? f.m1 - m0 : 0;
            const float* from = buf + (lane >> 4) * 17 + col;
            const size_t to = (size_t)(m0 + (lane >> 4)) * p.N + n0 + 16 * q + col, step = 2 * (size_t)p.N;
            if (p.y_dtype == QMOE_F32) {
              float* y = static_cast<float*>(p.y) + to;
#pragma unroll 4
              for (int r = 0; r < 32; r += 2, y += step)
                if (r + (lane >> 4) < rows) *y = from[r * 17];
            } else {
              uint16_t* y = static_cast<uint16_t*>(p.y) + to;
#pragma unroll 4
              for (int r = 0; r < 32; r += 2, y += step)
                if (r + (lane >> 4) < rows) *y = (uint16_t)fm_pack(p, make_float2(from[r * 17], 0.f));
            }
            __syncwarp();
          }
        }
      }
    }
    __syncwarp();
    if (ok && *s_left)
      for (int t = blockIdx.x, i = 0; t < parts; t += gridDim.x, ++i) {
        const FwTile f = nth(i, t);
        const int n0 = f.n0 + set * (BN / 2), n1 = min(f.n1, n0 + BN / 2);
        for (int m = f.m0 + qd * 32; m < min(f.m1, f.m0 + qd * 32 + 32); ++m)
          if (n0 < n1) fm_again(p, f.e, n0, n1, m);
      }
  } else {
    if (BN == 256) asm volatile("setmaxnreg.dec.sync.aligned.u32 %0;" ::"n"(kFwFewRegs));
    if (warp == 0) {
      // ------------------------------------------------------------ codes
      int it = 0, s = 0;
      uint32_t ph = 0;
      bool ok = !stalled(QMOE_DIAG_STALL_FP8_CODES);
      const uint32_t el = elect_lane();
      for (int t = blockIdx.x, i = 0; t < parts && ok; t += gridDim.x, ++i) {
        const FwTile f = nth(i, t);
        if (f.n1 <= f.n0) continue;
        const int xb = (f.m1 - f.m0 + 63) / 64, wb = (f.n1 - f.n0 + 63) / 64;  // copies of 64 rows
        for (int c = 0; c < nb; ++c, ++it) {
          if (it >= S) ok = fm_wait(&empty[s], ph ^ 1u, p, s_abort);
          if (!ok) break;
          if (el) {
            uint8_t* st = ring + s * P::kStage;
            mbar_arrive_expect_tx(&full[s], (xb + wb) * 64 * 128);
            for (int i = 0; i < xb; ++i) tma_load_2d(st + i * 8192, &tm_x, c * 128, f.m0 + 64 * i, &full[s]);
            for (int i = 0; i < wb; ++i)
              tma_load_2d(st + P::kA + i * 8192, &tm_w, c * 128, f.e * p.N + f.n0 + 64 * i, &full[s]);
          }
          __syncwarp();
          if (++s == S) {
            s = 0;
            ph ^= 1u;
          }
        }
      }
      if (lane == 0) fm_settle<S>(full, it, p, s_abort);
    } else if (warp == 1) {
      // ------------------------------------------------------------- MMAs
      int n = 0, s = 0;  // blocks so far
      uint32_t ph = 0;
      bool ok = !stalled(QMOE_DIAG_STALL_FP8_MMA), issued = false;
      const uint32_t el = elect_lane();
      for (int t = blockIdx.x, i = 0; t < parts && ok; t += gridDim.x, ++i) {
        const FwTile f = nth(i, t);
        if (f.n1 <= f.n0) continue;
        const int cols = (f.n1 - f.n0 + 15) & ~15;
        const uint32_t idesc = 1u << 4 | (uint32_t)(cols >> 3) << 17 | (uint32_t)(BT >> 4) << 24;
        for (int c = 0; c < nb; ++c, ++n) {
          const int b = n % NB;
          ok = fm_wait<false>(&full[s], ph, p, s_abort);
          if (ok && n >= NB) ok = fm_wait<false>(&acc_free[b], (n / NB - 1) & 1, p, s_abort);
          if (!ok) break;
          tc_fence_after();
          const uint32_t st = (smem_u32(ring + s * P::kStage) >> 4) & 0x3FFFu;  // a descriptor's address field
          const uint32_t da = st | 1u << 16, db = (st + (P::kA >> 4)) | 1u << 16;
          const int left = p.K - c * 128;
#pragma unroll
          for (int j = 0; j < 4; ++j) {
            if (32 * j >= left) break;
            mma_f8(el, tmem + b * BN, da + 2 * j, db + 2 * j, idesc, j > 0);
          }
          mma_commit_mx<1>(el, &empty[s]);
          mma_commit_mx<1>(el, &acc_full[b]);
          issued = true;
          if (++s == S) {
            s = 0;
            ph ^= 1u;
          }
        }
      }
      if (issued) {  // all MMAs have finished before tensor memory is freed
        mma_commit_mx<1>(el, fin);
        if (el) mbar_wait(fin, 0, nullptr);
      }
    } else if (warp == 2) {
      // ------------ scales of 128 tokens by kHalves weight blocks, four k blocks at a time
      int it = 0;
      const int rb = (p.N + 127) / 128;
      FmRange range;
      bool ok = !stalled(QMOE_DIAG_STALL_FP8_SCALES);
      for (int t = blockIdx.x, i = 0; t < parts && ok; t += gridDim.x, ++i) {
        const FwTile f = nth(i, t);
        if (f.n1 <= f.n0) continue;
        const float* ws = p.ws + ((size_t)f.e * rb + f.n0 / 128) * nb;
        for (int c = 0; c < nb; c += 4, ++it) {
          const int q = it % SQ;
          float v[4][4], w[P::kHalves][4];
#pragma unroll
          for (int h = 0; h < P::kHalves; ++h)
#pragma unroll
            for (int j = 0; j < 4; ++j) w[h][j] = f.n0 / 128 + h < rb && c + j < nb ? ws[h * nb + c + j] : 1.f;  // (1: nobody reads it)
#pragma unroll
          for (int i = 0; i < 4; ++i) {
#pragma unroll
            for (int j = 0; j < 4; ++j) v[i][j] = 1.f;
            if (f.m0 + 32 * i + lane < f.m1) {
              const float* xs = p.xs + (size_t)(f.m0 + 32 * i + lane) * nb + c;
              if (p.wide_scales) {
                const float4 u = *reinterpret_cast<const float4*>(xs);
                v[i][0] = u.x, v[i][1] = u.y, v[i][2] = u.z, v[i][3] = u.w;
              } else {
#pragma unroll
                for (int j = 0; j < 4; ++j) v[i][j] = c + j < nb ? xs[j] : 1.f;
              }
            }
          }
          if (it >= SQ) ok = fm_wait(&sc_free[q], (it / SQ - 1) & 1, p, s_abort);
          if (!ok) break;
          float* out = scales + q * 4 * P::kHalves * 128;
#pragma unroll
          for (int j = 0; j < 4; ++j)
#pragma unroll
            for (int h = 0; h < P::kHalves; ++h)
#pragma unroll
              for (int i = 0; i < 4; ++i) out[(j * P::kHalves + h) * 128 + 32 * i + lane] = v[i][j] * w[h][j];
#pragma unroll
          for (int j = 0; j < 4; ++j) {
#pragma unroll
            for (int h = 0; h < P::kHalves; ++h) range.weight(w[h][j]);
#pragma unroll
            for (int i = 0; i < 4; ++i) range.token(v[i][j]);
          }
          if (range.left()) *s_left = 1;
          __syncwarp();
          if (lane == 0) mbar_arrive(&sc_full[q]);
        }
      }
    }
  }
  __syncwarp();
  tc_fence_before();
  __syncthreads();
  if (warp == 1) {
    tc_fence_after();
    tmem_dealloc(tmem, 512);
  }
}

// Most token tiles that rows of E experts can make.
static long long fm_token_tiles(const FmParams& p, int bn) {
  if (!p.offsets) return (p.M + bn - 1) / bn;
  const long long most = p.M / bn + (p.E < p.M ? p.E : p.M);
  return most < p.M ? most : p.M;
}

template <int BN>
static cudaError_t launch_fm(FmParams p, int split, const uint8_t* xc, const uint8_t* wc, cudaStream_t st) {
  using P = FmPlan<BN>;
  static_assert(P::kStages >= 3 && P::kBufs * BN <= 512, "plan");
  static_assert((2 * P::kStages + 2 * P::kBufs + 2 * P::kQuads + 2) * 8 + 44 <= kFmBars, "barriers");
  p.split = split;
  p.lsplit = split == 8 ? 3 : split / 2;
  p.row_tiles = (p.N + 127) / 128;
  const long long tiles = fm_token_tiles(p, BN) * p.row_tiles;
  if (tiles > (1LL << 27)) return cudaErrorInvalidValue;
  CUtensorMap tw, tx;
  if (!make_map(&tw, wc, CU_TENSOR_MAP_DATA_TYPE_UINT8, 1, p.K, (uint64_t)p.E * p.N, 128, 128, CU_TENSOR_MAP_SWIZZLE_128B,
                CU_TENSOR_MAP_L2_PROMOTION_L2_256B) ||
      !make_map(&tx, xc, CU_TENSOR_MAP_DATA_TYPE_UINT8, 1, p.K, p.M, 128, P::kBox, CU_TENSOR_MAP_SWIZZLE_128B,
                CU_TENSOR_MAP_L2_PROMOTION_L2_256B))
    return cudaErrorNotSupported;
  p.wide_out = p.y_dtype != QMOE_F32 && p.N % 8 == 0 && !(reinterpret_cast<uintptr_t>(p.y) & 15);
  p.wide_scales = split == 1 && p.K % 512 == 0 && !(reinterpret_cast<uintptr_t>(p.xs) & 15);
  const int sms = device_sm_count();
  auto kernel = fp8_matmul_kernel<BN>;
  // All of the SM's shared memory, used or not: the CTA takes all of its tensor
  // memory, and a CTA of another kernel that waits for some (or has some) must
  // not share the SM: two clusters could then wait for one another.
  cudaError_t err = ensure_smem(kernel, kFmSmem);
  if (err != cudaSuccess) return err;
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3((unsigned)(p.split > 1 ? tiles * p.split : tiles < sms ? tiles : sms));
  cfg.blockDim = dim3(kFmThreads);
  cfg.dynamicSmemBytes = kFmSmem;
  cfg.stream = st;
  cudaLaunchAttribute attr[2];
  attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[0].val.programmaticStreamSerializationAllowed = 1;
  attr[1].id = cudaLaunchAttributeClusterDimension;
  attr[1].val.clusterDim.x = p.split;
  attr[1].val.clusterDim.y = attr[1].val.clusterDim.z = 1;
  cfg.attrs = attr;
  cfg.numAttrs = 2;
  return cudaLaunchKernelEx(&cfg, kernel, tw, tx, p);
}

template <int BN>
static cudaError_t launch_fw(FmParams p, const uint8_t* xc, const uint8_t* wc, cudaStream_t st) {
  using P = FwPlan<BN>;
  static_assert(P::kStages >= 3, "plan");
  static_assert((2 * P::kStages + 2 * P::kBufs + 2 * P::kQuads + 2) * 8 + 44 <= kFmBars, "barriers");
  p.split = 1;
  p.row_tiles = (p.N + BN - 1) / BN;
  const long long tiles = fm_token_tiles(p, 128) * p.row_tiles;
  if (tiles > (1LL << 27)) return cudaErrorInvalidValue;
  CUtensorMap tw, tx;
  if (!make_map(&tw, wc, CU_TENSOR_MAP_DATA_TYPE_UINT8, 1, p.K, (uint64_t)p.E * p.N, 128, 64, CU_TENSOR_MAP_SWIZZLE_128B,
                CU_TENSOR_MAP_L2_PROMOTION_L2_256B) ||
      !make_map(&tx, xc, CU_TENSOR_MAP_DATA_TYPE_UINT8, 1, p.K, p.M, 128, 64, CU_TENSOR_MAP_SWIZZLE_128B,
                CU_TENSOR_MAP_L2_PROMOTION_L2_256B))
    return cudaErrorNotSupported;
  p.wide_out = p.N % (p.y_dtype == QMOE_F32 ? 4 : 8) == 0 && !(reinterpret_cast<uintptr_t>(p.y) & 15);
  p.wide_scales = p.K % 512 == 0 && !(reinterpret_cast<uintptr_t>(p.xs) & 15);
  const int sms = device_sm_count();
  auto kernel = fp8_wide_kernel<BN>;
  const cudaError_t err = ensure_smem(kernel, kFmSmem);  // all of it, as above
  if (err != cudaSuccess) return err;
  if (BN == 256) {  // the warps' shares of the registers wait for what the launch does not have
    static int regs = 0;
    if (!regs) {
      cudaFuncAttributes a;
      const cudaError_t e = cudaFuncGetAttributes(&a, kernel);
      if (e != cudaSuccess) return e;
      regs = a.numRegs;
    }
    if (regs < kFwRegs) return cudaErrorInvalidDeviceFunction;
  }
  return launch_kernel(kernel, dim3((unsigned)(tiles < sms ? tiles : sms)), dim3(kFwThreads), kFmSmem, st, true, tw, tx, p);
}

// CTAs of clusters of `split` (2, 4, 8) that the device holds at once, one CTA
// to an SM.  A query that fails fails the call: with a guess in its place, the
// same call would sum in another order another time.
static cudaError_t fm_capacity(int split, int* ctas) {
  static int cached[64][4] = {};  // CTAs + 1
  const int l = split == 8 ? 3 : split == 4 ? 2 : 1;
  int dev = 0;
  cudaError_t err = cudaGetDevice(&dev);
  if (err != cudaSuccess) return err;
  if (dev < 0 || dev >= 64) return cudaErrorInvalidDevice;
  if (!cached[dev][l]) {
    auto kernel = fp8_matmul_kernel<16>;
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = dim3(split);
    cfg.blockDim = dim3(kFmThreads);
    cfg.dynamicSmemBytes = kFmSmem;
    cudaLaunchAttribute attr;
    attr.id = cudaLaunchAttributeClusterDimension;
    attr.val.clusterDim.x = split;
    attr.val.clusterDim.y = attr.val.clusterDim.z = 1;
    cfg.attrs = &attr;
    cfg.numAttrs = 1;
    int n = 0;
    if ((err = ensure_smem(kernel, kFmSmem)) != cudaSuccess ||
        (err = cudaOccupancyMaxActiveClusters(&n, kernel, &cfg)) != cudaSuccess)
      return err;
    cached[dev][l] = n * split + 1;
  }
  *ctas = cached[dev][l] - 1;
  return cudaSuccess;
}

// wide 0: bn tokens a tile, 128 weight rows; 1: 128 tokens, bn weight rows.
struct FmChoice {
  int bn, wide, split;
};

// The form by an estimate of its time in ns: a start, the blocks of the CTA with
// the most tiles (a narrower MMA is not proportionally faster), what each further
// tile adds (rows of y off 16 bytes leave the wide forms slowly), the exchange of a
// split tile's sums; at least what the operands' bytes take.  Where experts share
// the rows, each is taken to have as many, and a last tile half full.
// The constants are fits to 410 measured sizes, dense and grouped, of which 15 are
// then more than 5 % off the best form, the worst 29 % (71 tokens x 8, 8 experts).
// Some of them on GB300 (us, the forms of a row side by side, before FmRange's 0 to 0.2;
// tokens x outputs a tile / CTAs along K):
//      1 x 1408 x 2048      16x128/8 3.4  /4 3.6  /2 4.2  /1 5.2
//     16 x 8192 x 8192      64x128/2 14.2  16x128/2 14.6  /1 16.6
//     64 x 2048 x 5632      32x128/4 6.9  64x128/4 7.5  /1 12.7
//    512 x 1408 x 2048      64x128 7.0  128x128 8.1  128x256 11.2
//   2048 x 1408 x 2048      128x256 11.6  128x128 13.9  64x128 15.5
//   8192 x 8192 x 8192      128x256 400 to 415  128x128 490  64x128 810
//    4 rows of 4 experts    x 2816 x 2048: 16x128/1 6.5  /2 11
//   8192 rows of 60 experts x 2816 x 2048: 128x256 77  128x128 83  64x128 100
static cudaError_t fm_choose(const FmParams& p, FmChoice* choice) {
  static const struct {
    int bn, wide, start, block, tile, exchange, odd;  // odd: a tile more where rows of y are off 16 bytes
  } kinds[] = {{16, 0, 2422, 246, 709, 361, 0},   {32, 0, 3172, 223, 977, 223, 0}, {64, 0, 3725, 230, 1097, 1045, 0},
               {128, 0, 4089, 462, 1631, 679, 0}, {128, 1, 3990, 269, 1413, 0, 664}, {256, 1, 6800, 348, 3068, 0, 1940}};
  int capacity[9] = {};
  for (int split = 2; split <= 8; split *= 2) {
    const cudaError_t err = fm_capacity(split, &capacity[split]);
    if (err != cudaSuccess) return err;
  }
  const long long nb = (p.K + 127) / 128, active = p.offsets ? (p.E < p.M ? p.E : p.M) : 1, each = (p.M + active - 1) / active;
  const double bytes = (double)active * p.N * p.K + (double)p.M * p.K + 2.0 * p.M * p.N, least_time = 3523 + bytes / 7000;
  double least = -1;
  for (const auto& k : kinds) {
    if (!k.wide && k.bn < 64 && each > 4 * k.bn) continue;
    const int bt = k.wide ? 128 : k.bn, br = k.wide ? k.bn : 128;
    const long long rows = (p.N + br - 1) / br, some = p.offsets ? p.M / bt + active / 2 : (p.M + bt - 1) / bt;
    const long long tiles = rows * (some > active ? some : active), of = k.wide ? p.N : each;
    const double block = k.block * (0.52 + 0.48 * (of < k.bn ? (int)of : k.bn) / k.bn);
    const int tile = k.tile + (p.N % 8 ? k.odd : 0);
    for (int split = 1; split <= 8; split *= 2) {
      if (split > 1 && (!k.exchange || split > nb || rows * fm_token_tiles(p, k.bn) * split > capacity[split])) break;
      const long long slots = split > 1 ? tiles : device_sm_count(), rounds = (tiles + slots - 1) / slots;
      const double one = (double)((nb + split - 1) / split) * block;
      const double t = k.start + one + (double)(rounds - 1) * (one + tile) + (split > 1 ? k.exchange : 0);
      const double total = (t > least_time ? t : least_time) + 0.05 * t;
      if (least < 0 || total < least) {
        least = total;
        *choice = {k.bn, k.wide, split};
      }
    }
  }
  return cudaSuccess;
}

cudaError_t fp8_status_word(void** word) { return cudaGetSymbolAddress(word, g_fp8_status); }

static FmParams fm_params(const float* xs, const float* ws, const int32_t* offsets, int E, int M, int N, int K) {
  FmParams p = {};
  p.xs = xs;
  p.ws = ws;
  p.offsets = offsets;
  p.E = E;
  p.M = M;
  p.N = N;
  p.K = K;
  return p;
}

cudaError_t fp8_matmul_variant(bool grouped, int E, int M, int N, int K, int* tile, int* wide, int* split) {
  static const int32_t some = 0;  // looked at for being given alone
  const FmParams p = fm_params(nullptr, nullptr, grouped ? &some : nullptr, E, M, N, K);
  FmChoice c = {};
  const cudaError_t err = fm_choose(p, &c);
  *tile = c.bn;
  *wide = c.wide;
  *split = c.split;
  return err;
}

cudaError_t launch_fp8_matmul(const uint8_t* xc, const float* xs, const uint8_t* wc, const float* ws,
                              const int32_t* offsets, int E, int M, int N, int K, void* y, int y_dtype, uint32_t* status,
                              uint32_t wait_limit_kilocycles, uint32_t stall, cudaStream_t st) {
  FmParams p = fm_params(xs, ws, offsets, E, M, N, K);
  p.xc = xc;
  p.wc = wc;
  p.y = y;
  p.y_dtype = y_dtype;
  p.status = status;
  p.stall = stall;
  p.wait_limit = wait_limit_kilocycles ? (long long)wait_limit_kilocycles << 10 : kWaitLimitCycles;
  FmChoice c = {};
  const cudaError_t err = fm_choose(p, &c);
  if (err != cudaSuccess) return err;
  if (c.wide) return c.bn == 256 ? launch_fw<256>(p, xc, wc, st) : launch_fw<128>(p, xc, wc, st);
  if (c.bn == 16) return launch_fm<16>(p, c.split, xc, wc, st);
  if (c.bn == 32) return launch_fm<32>(p, c.split, xc, wc, st);
  if (c.bn == 64) return launch_fm<64>(p, c.split, xc, wc, st);
  return launch_fm<128>(p, c.split, xc, wc, st);
}

}  // namespace qmoe
