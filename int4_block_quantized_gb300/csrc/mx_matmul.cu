// mx_matmul.cu -- product of a microscaled tensor with MXFP4 weights:
//   y[m, n] = sum over blocks b of X_x[m, b] X_w[n, b] sum_{k in b} x[m, k] w[n, k]
// with fp32 sums, rounded once to the output's type.
//
// The tensor cores multiply block-scaled operands directly
// (tcgen05.mma.block_scale): codes go from HBM to shared memory and scales on
// to tensor memory as they are, no thread touches either.  Weight rows are
// the MMA's M = 128 operand and tokens its N, so that one token costs a
// narrow MMA and not a 128-row one.  A pipeline stage is 128 bytes per row:
//   MXFP4 x: 256 k (kind::mxf4, four MMAs of 64 k, two scale words);
//   MXFP8 x: 128 k (kind::mxf8f6f4, four MMAs of 32 k, one scale word), the
//            e2m1 codes widened on the way in to 16 codes per 16 bytes, the
//            first 8 of them used.
#include <cuda.h>

#include "launch.h"
#include "mx.cuh"
#include "tmap.h"

namespace qmoe {

constexpr int kMmThreads = 352;       // warps 0 and 6 copy, warp 1 issues MMAs, warps 2-5 and 7-10 write y
constexpr int kMmFillThreads = 640;   // + warps 11-18: codes widened by loads and stores, 19: their copies (see FILL)
constexpr uint32_t kMmSmem = 232448;  // 227 KB
constexpr uint32_t kMmBars = 1024;

struct MmParams {
  const uint8_t *xs, *ws, *wc;
  void* y;
  uint32_t* status;
  int M, N, K, y_dtype;
  int row_tiles, tok_tiles, kt;  // tiles of 128 weight rows, of BN tokens; scale tiles along K
  int wide_out;                  // y: 16 bits, rows on 16-byte boundaries
  int split;                     // CTAs of a cluster that share a tile's K
  uint32_t stall;                // QMOE_DIAG_STALL_MX_*: this role waits for what cannot arrive
  long long wait_limit;          // SM cycles
};

template <int XF, int BN, int CG, bool FILL = false>
struct MmPlan {
  static constexpr int kStageK = XF == kMxfp4 ? 256 : 128;  // elements
  static constexpr int kWords = kStageK / 128;              // scale tiles of a stage along K
  static constexpr int kTokSf = (BN + 127) / 128;           // scale tiles of a stage along the tokens
  static constexpr uint32_t kA = 128 * 128, kB = BN / CG * 128;  // one CTA's share
  // bytes that a weight copy reports: those read, also where the codes are widened
  static constexpr uint32_t kTxA = XF == kMxfp4 ? kA : kA / 2;
  static constexpr uint32_t kSf = 512 * kWords * (1 + kTokSf);
  static constexpr uint32_t kAb = (kA + kB + 1023) & ~1023u;
  // a split tile's partial sums [split][tokens of a CTA / 4][128][4]: a place of
  // their own where they are small, else the ring once the cluster is done with it
  static constexpr uint32_t kPart = BN <= 64 ? (BN < 32 ? 32 : BN) * 512 : 0;
  // 2 KB per output warp: 32 tokens x 32 outputs of 16 bits, turned round there
  static constexpr uint32_t kOut = BN >= 32 ? 8 * 2048 : 0;
  // FILL: packed weight codes on their way, 128 rows x 64 bytes a stage
  static constexpr int kRawSlots = !FILL ? 0 : BN <= 64 ? 6 : 4;
  static constexpr uint32_t kRaw = kRawSlots * 128 * 64;
  static constexpr int kStages0 = (int)((kMmSmem - kMmBars - 1024 - kPart - kOut - kRaw) / (kAb + kSf));
  static constexpr int kStages = kStages0 > 12 ? 12 : kStages0;
  static constexpr uint32_t kTotal = kMmBars + kOut + kRaw + kStages * (kAb + kSf) + kPart + 1024;
  // tensor memory: two accumulators, then the stage's scales.  At 256 tokens
  // the two overlap by 32 columns, since the scales need 24 of the 512.
  static constexpr bool kOverlap = BN == 256;
  static constexpr uint32_t kAcc1 = kOverlap ? 224 : BN;
  static constexpr uint32_t kSfa = kAcc1 + BN;
  static constexpr uint32_t kSfb = kSfa + 4 * kWords;
  static constexpr uint32_t kCols0 = kSfb + 4 * kWords * kTokSf;
};

// The status word of the calls that bring none.
__device__ uint32_t g_mx_status;
__device__ __forceinline__ void mm_timed_out(const MmParams& p) {
  set_status(p.status ? p.status : &g_mx_status, QMOE_ST_TIMEOUT);
}

// Bounded wait; gives up when another role has, or after the limit (about 2 s)
// with the status bit.  WARP: all lanes of the warp wait, and they agree on the
// answer (each may see the phase end at another poll, and aligned instructions
// or warp barriers follow).  The warp that issues MMAs has neither: what its
// elected lane sees decides all that it does, and the other lanes only follow.
// (With votes there, 16 x 8192 x 8192 takes 0.1 us more.)
template <bool WARP = true>
__device__ __forceinline__ bool mm_wait(uint64_t* bar, uint32_t parity, const MmParams& p, volatile int* abort) {
  auto all = [](bool v) { return WARP ? __all_sync(0xffffffffu, v) != 0 : v; };
  if (all(mbar_try_wait(bar, parity))) return true;
  const long long t0 = clock64();
  while (!all(mbar_try_wait_sleep(bar, parity, 20000u))) {
    const bool late = clock64() - t0 > p.wait_limit;
    if (!all(!(late || *abort))) {
      if (late) mm_timed_out(p);
      *abort = 1;
      return false;
    }
  }
  return true;
}

// The end of a warp that has issued `it` copies into a ring of S slots: it
// waits for the last use of each, time-out or not (a role that gives up does so
// at any time, also after this warp's last step), so that no copy lands in
// shared memory that is another CTA's by then.  After a time-out slots may stay
// as they are; a copy lands within microseconds, so 10 ms for all of them do.
constexpr long long kMmSettleCycles = 20000000;
template <int S>
__device__ __forceinline__ void mm_settle(uint64_t* bars, int it, const MmParams& p, volatile int* abort) {
  const long long t0 = clock64();
  for (int n = max(it - S, 0); n < it; ++n)  // the oldest first: no poll is left when the last has come
    while (!mbar_try_wait_sleep(&bars[n % S], (n / S) & 1, 20000u)) {
      const long long t = clock64() - t0;
      if (*abort) {
        if (t > kMmSettleCycles) break;
      } else if (t > p.wait_limit) {
        mm_timed_out(p);
        *abort = 1;
      }
    }
}

__device__ __forceinline__ void mm_store(const MmParams& p, size_t i, float v) {
  if (p.y_dtype == QMOE_F32) static_cast<float*>(p.y)[i] = v;
  else static_cast<uint16_t*>(p.y)[i] = p.y_dtype == QMOE_BF16 ? Half<__nv_bfloat16>::from_float(v) : Half<__half>::from_float(v);
}

// two results to the output's 16-bit type
__device__ __forceinline__ uint32_t mm_pack(const MmParams& p, uint32_t a, uint32_t b) {
  if (p.y_dtype == QMOE_BF16) {
    const __nv_bfloat162 h = __floats2bfloat162_rn(__uint_as_float(a), __uint_as_float(b));
    return *reinterpret_cast<const uint32_t*>(&h);
  }
  const __half2 h = __floats2half2_rn(__uint_as_float(a), __uint_as_float(b));
  return *reinterpret_cast<const uint32_t*>(&h);
}

// W tokens' results of one output column: y[i], y[i + N], ... , the first `rows` of them.
template <int W>
__device__ __forceinline__ void mm_store_cols(const MmParams& p, size_t i, int rows, const uint32_t (&v)[W]) {
  const size_t N = p.N;
  if (p.y_dtype == QMOE_F32) {
    uint32_t* y = static_cast<uint32_t*>(p.y) + i;
#pragma unroll
    for (int j = 0; j < W; ++j, y += N)
      if (j < rows) *y = v[j];
    return;
  }
  uint16_t* y = static_cast<uint16_t*>(p.y) + i;
#pragma unroll
  for (int j = 0; j < W; j += 2) {
    const uint32_t u = mm_pack(p, v[j], v[j + 1]);
    if (j < rows) *y = (uint16_t)(u & 0xffffu);
    y += N;
    if (j + 1 < rows) *y = (uint16_t)(u >> 16);
    y += N;
  }
}

// Tile t of the grid: groups of 8 row tiles, so that the tiles in flight share
// weights and tokens in L2.
__device__ __forceinline__ void mm_tile(const MmParams& p, int t, int& rt, int& tt) {
  const int per = 8 * p.tok_tiles, g = t / per, r = t - g * per;
  const int rows = min(8, p.row_tiles - g * 8);
  rt = g * 8 + r % rows;
  tt = r / rows;
}

// FILL (MXFP8 x only): the TMA copy that widens e2m1 codes wants rows of a
// multiple of 128 codes on 32-byte boundaries; other weights come packed and
// eight warps spread them in shared memory.
template <int XF, int BN, int CG, bool FILL>
__global__ void __launch_bounds__(FILL ? kMmFillThreads : kMmThreads, 1)
    mx_matmul_kernel(const __grid_constant__ CUtensorMap tm_w, const __grid_constant__ CUtensorMap tm_x,
                     const __grid_constant__ CUtensorMap tm_ws, const __grid_constant__ CUtensorMap tm_xs,
                     const MmParams p) {
  using P = MmPlan<XF, BN, CG, FILL>;
  constexpr int S = P::kStages;
  extern __shared__ __align__(1024) uint8_t smem_raw[];
  uint8_t* smem = smem_raw + ((1024u - (smem_u32(smem_raw) & 1023u)) & 1023u);
  uint64_t* full = reinterpret_cast<uint64_t*>(smem);
  uint64_t* empty = full + S;
  uint64_t* acc_full = empty + S;       // [2]
  uint64_t* acc_free = acc_full + 2;    // [2]
  uint64_t* fin = acc_free + 2;
  uint64_t* raw_full = fin + 1;  // [kRawSlots]
  uint64_t* raw_empty = raw_full + P::kRawSlots;
  uint64_t* never = raw_empty + P::kRawSlots;  // nothing arrives here (p.stall)
  uint32_t* s_tmem = reinterpret_cast<uint32_t*>(never + 1);
  volatile int* s_abort = reinterpret_cast<volatile int*>(s_tmem + 1);
  uint8_t* outbuf = smem + kMmBars;  // 1024-byte aligned, as the ring behind it
  uint8_t* raw = outbuf + P::kOut;
  uint8_t* ring = raw + P::kRaw;
  uint8_t* sfring = ring + S * P::kAb;
  const int tid = threadIdx.x, lane = tid & 31;
  const int warp = __shfl_sync(0xffffffffu, tid >> 5, 0);  // known to be the same in all lanes

  if (tid == 0) {
    for (int s = 0; s < S; ++s) {
      mbar_init(&full[s], FILL ? 6 : 2);
      mbar_init(&empty[s], 1);
    }
    for (int b = 0; b < 2; ++b) {
      mbar_init(&acc_full[b], 1);
      mbar_init(&acc_free[b], 8 * CG);
    }
    mbar_init(fin, 1);
    mbar_init(never, 1);
    for (int s = 0; s < P::kRawSlots; ++s) {
      mbar_init(&raw_full[s], 1);
      mbar_init(&raw_empty[s], 4);
    }
    *s_abort = 0;
    fence_barrier_init();
  }
  if (warp == 1) {
    if (CG == 1) {
      tmem_alloc(s_tmem, 512);
      tmem_relinquish();
    } else {
      tmem_alloc2(s_tmem, 512);
      tmem_relinquish2();
    }
  }
  tc_fence_before();
  __syncthreads();
  if (CG == 2) cluster_sync_all();  // the pair's barriers are set up
  tc_fence_after();
  // all 512 columns are this CTA's, so they start at 0
  constexpr uint32_t tmem = 0;
  if (P::kPart && p.split > 1) cluster_arrive();  // this CTA runs: its shared memory may be written
  pdl_wait();
  pdl_trigger();

  // this CTA's tiles and its share [c0, c1) of their stages along K
  const int rank = p.split > 1 ? (int)cluster_ctarank() : 0;
  const int half = CG == 2 ? (int)cluster_ctarank() : 0;  // of the pair's rows and tokens
  const int tiles = p.row_tiles * p.tok_tiles;
  const int first = blockIdx.x / (CG * p.split), step = p.split > 1 ? tiles : gridDim.x / CG;
  const int chunks = (p.K + P::kStageK - 1) / P::kStageK;
  auto stalled = [&](uint32_t role) { return (p.stall & role) && !mm_wait(never, 0, p, s_abort); };
  const int c0 = (int)((long long)chunks * rank / p.split), c1 = (int)((long long)chunks * (rank + 1) / p.split);

  if (warp == 0 || warp == 6) {
    // ------------------------------ copies: warp 0 the codes, warp 6 the scales
    int it = 0, s = 0;
    uint32_t ph = 0;
    bool ok = !stalled(warp == 0 ? QMOE_DIAG_STALL_MX_CODES : QMOE_DIAG_STALL_MX_SCALES);
    const uint32_t el = elect_lane();
    for (int t = first; t < tiles && ok; t += step) {
      int rt, tt;
      mm_tile(p, t, rt, tt);
      const int m0 = tt * BN, r = rt * CG + half;
      // scale tiles of the tokens: those that exist (128-row tiles m0 / 128 ..)
      const int t0 = m0 >> 7, nt = min(P::kTokSf, ((p.M + 127) >> 7) - t0);
      for (int c = c0; c < c1; ++c, ++it) {
        if (it >= S) ok = mm_wait(&empty[s], ph ^ 1u, p, s_abort);
        if (!ok) break;
        if (el) {
          const int q0 = c * P::kWords, nq = min(P::kWords, p.kt - q0);
          uint8_t* st = ring + s * P::kAb;
          uint8_t* sf = sfring + s * P::kSf;
          if constexpr (CG == 2) {
            // both CTAs report to the leader; scale tiles that do not exist read as zeros
            const uint32_t bar = peer_u32(&full[s], 0);
            if (warp == 0) {
              if (half == 0) mbar_arrive_expect_tx(&full[s], 2 * (P::kTxA + P::kB));
              tma_load_2d_pair(st, &tm_w, c * 128, r * 128, bar);
              tma_load_2d_pair(st + P::kA, &tm_x, c * 128, m0 + half * (BN / 2), bar);
            } else {
              if (half == 0) mbar_arrive_expect_tx(&full[s], 2 * P::kSf);
              tma_load_2d_pair(sf, &tm_ws, 0, r * p.kt + q0, bar);
              for (int i = 0; i < P::kTokSf; ++i)
                tma_load_2d_pair(sf + 512 * P::kWords * (1 + i), &tm_xs, 0, (t0 + i) * p.kt + q0, bar);
            }
          } else if (warp == 0) {
            mbar_arrive_expect_tx(&full[s], (FILL ? 0u : P::kTxA) + P::kB);
            if (!FILL) tma_load_2d(st, &tm_w, c * 128, rt * 128, &full[s]);
            tma_load_2d(st + P::kA, &tm_x, c * 128, m0, &full[s]);
          } else {
            mbar_arrive_expect_tx(&full[s], 512u * nq * (1 + nt));
            bulk_g2s(sf, p.ws + ((size_t)rt * p.kt + q0) * 512, 512u * nq, &full[s]);
            for (int i = 0; i < nt; ++i)
              bulk_g2s(sf + 512 * P::kWords * (1 + i), p.xs + ((size_t)(t0 + i) * p.kt + q0) * 512, 512u * nq, &full[s]);
          }
        }
        __syncwarp();
        if (++s == S) {
          s = 0;
          ph ^= 1u;
        }
      }
    }
    // A pair's stages are counted in the leader alone, but both CTAs see the
    // commits that give slots back (and stay until these have arrived).
    if (lane == 0) mm_settle<S>(CG == 1 ? full : empty, it, p, s_abort);
  } else if (warp == 1 && half == 0) {
    // --------------------------------------------------------------- MMAs
    int n = 0, s = 0;
    uint32_t ph = 0;
    bool ok = !stalled(QMOE_DIAG_STALL_MX_MMA), issued = false;
    const uint32_t el = elect_lane();
    for (int t = first; t < tiles && ok; t += step, ++n) {
      const int b = n & 1;
      int rt, tt;
      mm_tile(p, t, rt, tt);
      if (P::kOverlap) {
        if (n >= 1) ok = mm_wait<false>(&acc_free[0], (n - 1) & 1, p, s_abort);
      } else {
        if (n >= 2) ok = mm_wait<false>(&acc_free[b], ((n >> 1) - 1) & 1, p, s_abort);
      }
      if (!ok) break;
      tc_fence_after();
      const uint32_t d = tmem + (b ? P::kAcc1 : 0);
      // 64 or 192 tokens: an odd token tile starts in the middle of a scale tile
      const uint32_t sfb = tmem + P::kSfb + (BN % 128 == 64 ? 2 * (tt & 1) : 0);
      // one stage: its scales, then its MMAs (the first `words` scale words and
      // `mmas` instructions: fewer only where K ends)
      auto issue = [&](int slot, bool first_stage, int words, int mmas) {
        const uint32_t st = (smem_u32(ring + slot * P::kAb) >> 4) & 0x3FFFu;  // a descriptor's address field
        const uint32_t sf = (smem_u32(sfring + slot * P::kSf) >> 4) & 0x3FFFu;
#pragma unroll
        for (int q = 0; q < P::kWords; ++q) {
          if (q >= words) break;
          tmem_cp_scales<CG>(el, tmem + P::kSfa + 4 * q, sf + 32 * q);
#pragma unroll
          for (int i = 0; i < P::kTokSf; ++i)
            tmem_cp_scales<CG>(el, tmem + P::kSfb + 4 * (q * P::kTokSf + i), sf + 32 * (P::kWords * (1 + i) + q));
        }
        const uint32_t da = st | 1u << 16, db = (st + (P::kA >> 4)) | 1u << 16;
#pragma unroll
        for (int j = 0; j < 4; ++j) {
          if (j >= mmas) break;
          const uint32_t acc = (j > 0 || !first_stage) ? 1u : 0u;
          if (XF == kMxfp4)
            mma_mxf4<CG>(el, d, da + 2 * j, db + 2 * j, idesc_mx(128 * CG, BN, 1, 1, 2 * (j & 1), 2 * (j & 1)),
                         tmem + P::kSfa + 4 * (j >> 1), sfb + 4 * P::kTokSf * (j >> 1), acc);
          else
            mma_mxf8f6f4<CG>(el, d, da + 2 * j, db + 2 * j, idesc_mx(128 * CG, BN, 5, 0, j, j), tmem + P::kSfa, sfb, acc);
        }
        mma_commit_mx<CG>(el, &empty[slot]);
      };
      bool ready = mbar_try_wait(&full[s], ph);
      for (int c = c0; c < c1; ++c) {
        if (!ready) ok = mm_wait<false>(&full[s], ph, p, s_abort);
        if (!ok) break;
        const int slot = s;
        if (++s == S) {
          s = 0;
          ph ^= 1u;
        }
        ready = c + 1 < c1 && mbar_try_wait(&full[s], ph);  // the next stage's answer arrives meanwhile
        tc_fence_after();
        const int left = p.K - c * P::kStageK;  // elements from here on
        if (left >= P::kStageK) issue(slot, c == c0, P::kWords, 4);
        else issue(slot, c == c0, (left + 127) / 128, (left + P::kStageK / 4 - 1) / (P::kStageK / 4));
        issued = true;
      }
      if (ok) mma_commit_mx<CG>(el, &acc_full[b]);
    }
    if (issued) {  // all MMAs have finished before tensor memory is freed
      if (CG == 1) mma_commit_mx<1>(el, fin);
      else mma_commit_mx2_own(el, fin);  // a commit to the peer's barrier too could arrive there when it has left
      if (el) mbar_wait(fin, 0, nullptr);
    }
  } else if (warp >= 2 && warp < 11) {
    // ------------------------------------------------------------- outputs
    // Two warps per lane quadrant take the accumulator's chunks in turn (one
    // warp needed longer for 256 tokens than the MMAs of 2048 k).
    const int qd = warp & 3, row = qd * 32 + lane, set = warp > 6;
    uint8_t* buf = outbuf + (warp - 2 - set) * 2048;
    int n = 0;
    const bool ok = !stalled(QMOE_DIAG_STALL_MX_OUTPUT);
    for (int t = first; t < tiles && ok; t += step, ++n) {
      const int b = n & 1;
      int rt, tt;
      mm_tile(p, t, rt, tt);
      if (!mm_wait(&acc_full[b], (n >> 1) & 1, p, s_abort)) break;
      tc_fence_after();
      const uint32_t d = tmem + ((uint32_t)(qd * 32) << 16) + (b ? P::kAcc1 : 0);
      const int m0 = tt * BN, nn = (rt * CG + half) * 128 + row;
      constexpr int W = BN < 32 ? BN : 32, C = BN / W;
      auto freed = [&](uint64_t* bar) {
        tc_fence_before();
        __syncwarp();
        if (lane == 0) {
          if (CG == 1) mbar_arrive(bar);
          else mbar_arrive_cluster(peer_u32(bar, 0));
        }
      };
      if (P::kOverlap && set) freed(&acc_free[0]);  // done with the tile before, and not the first chunk's
      if (p.split == 1) {
        for (int i = set; i < C; i += 2) {
          // the columns that the other accumulator shares come first
          const int c = P::kOverlap && b == 0 ? (i + C - 1) % C : i;
          const int m = m0 + c * W;
          if constexpr (W == 32) {
            if (p.wide_out) {
              uint32_t lo[16], hi[16];
              tmem_ld_frag(d + c * W, lo, hi);
              if (P::kOverlap && i == 0) freed(&acc_free[0]);
              const int n0 = nn - lane;
              if (m >= p.M || n0 >= p.N) continue;
              // token 8 g + lane % 8 is a row of 64 bytes; its four 16-byte
              // pieces (8 outputs each) are permuted against bank conflicts
              const uint32_t a = smem_u32(buf) + (lane & 7) * 64 + (((lane >> 3) ^ ((lane >> 1) & 3)) << 4);
#pragma unroll
              for (int g = 0; g < 4; ++g)
                stmatrix_t4(a + g * 512, mm_pack(p, lo[4 * g], lo[4 * g + 1]), mm_pack(p, lo[4 * g + 2], lo[4 * g + 3]),
                            mm_pack(p, hi[4 * g], hi[4 * g + 1]), mm_pack(p, hi[4 * g + 2], hi[4 * g + 3]));
              __syncwarp();
              const int tok = lane >> 2, piece = lane & 3;
              uint16_t* y = static_cast<uint16_t*>(p.y) + (size_t)(m + tok) * p.N + n0 + piece * 8;
#pragma unroll
              for (int g = 0; g < 4; ++g, y += (size_t)8 * p.N)
                if (m + 8 * g + tok < p.M && n0 + piece * 8 < p.N)
                  *reinterpret_cast<uint4*>(y) =
                      *reinterpret_cast<const uint4*>(buf + g * 512 + tok * 64 + ((piece ^ ((tok >> 1) & 3)) << 4));
              __syncwarp();
              continue;
            }
          }
          uint32_t v[W];
          if constexpr (W == 32) tmem_ld32(d + c * W, v);
          else tmem_ld16(d + c * W, v);
          if (P::kOverlap && i == 0) freed(&acc_free[0]);
          if (nn < p.N && m < p.M) mm_store_cols<W>(p, (size_t)m * p.N + nn, p.M - m, v);
        }
        if (!P::kOverlap) freed(&acc_free[b]);
      }
    }
  } else if (FILL && warp == kMmFillThreads / 32 - 1) {
    // ------------------------- packed weight codes, as far ahead as slots allow
    constexpr int R = P::kRawSlots ? P::kRawSlots : 1;
    int it = 0, s = 0;
    uint32_t ph = 0;
    bool ok = true;
    const uint32_t el = elect_lane();
    for (int t = first; t < tiles && ok; t += step) {
      int rt, tt;
      mm_tile(p, t, rt, tt);
      for (int c = c0; c < c1; ++c, ++it) {
        if (it >= R) ok = mm_wait(&raw_empty[s], ph ^ 1u, p, s_abort);
        if (!ok) break;
        if (el) {
          mbar_arrive_expect_tx(&raw_full[s], 128 * 64);
          tma_load_2d(raw + s * 128 * 64, &tm_w, c * 64, rt * 128, &raw_full[s]);
        }
        __syncwarp();
        if (++s == R) {
          s = 0;
          ph ^= 1u;
        }
      }
    }
    if (lane == 0) mm_settle<R>(raw_full, it, p, s_abort);
  } else if (FILL && warp >= kMmThreads / 32) {
    // ---------------------- codes of ragged rows spread to 16 bytes per 8 (MXFP8 x)
    // Two groups of four warps take turns at the stages; a warp takes 32 rows,
    // four lanes the 64 bytes of a row.  (The codes come by TMA and not by
    // loads of these warps, whose fence between stores and MMAs waits for loads
    // in flight too: 16 x 8192 x 8160 takes 11.8 us so, and 512 x 8192 x 8160
    // 41.6; with loads 16.9 and 49.  Widened by TMA, K = 8192 takes 9.3 and 24.)
    const int group = warp >= kMmThreads / 32 + 4;
    const int r0 = ((warp - kMmThreads / 32) & 3) * 32 + (lane >> 2), piece = lane & 3;
    constexpr int R = P::kRawSlots ? P::kRawSlots : 1;
    const int mine = first < tiles ? (tiles - 1 - first) / step + 1 : 0;
    const long long total = (long long)mine * (c1 - c0);
    int s = group, rs = group;
    uint32_t ph = 0, rph = 0;
    const bool ok = !stalled(QMOE_DIAG_STALL_MX_SPREAD);
    for (long long n = group; n < total && ok; n += 2) {
      if (!mm_wait(&raw_full[rs], rph, p, s_abort)) break;
      const uint4* src = reinterpret_cast<const uint4*>(raw + rs * 128 * 64 + r0 * 64 + piece * 16);
      uint4 v[4];
#pragma unroll
      for (int i = 0; i < 4; ++i) v[i] = src[32 * i];
      if (n >= S && !mm_wait(&empty[s], ph ^ 1u, p, s_abort)) break;
      // 16-byte pieces 2 piece and 2 piece + 1 of the row, swizzled by row % 8 = r0 % 8
      uint8_t* st = ring + s * P::kAb + r0 * 128;
      uint4* lo = reinterpret_cast<uint4*>(st + (((2 * piece) ^ (r0 & 7)) << 4));
      uint4* hi = reinterpret_cast<uint4*>(st + (((2 * piece + 1) ^ (r0 & 7)) << 4));
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        lo[64 * i] = make_uint4(v[i].x, v[i].y, 0, 0);
        hi[64 * i] = make_uint4(v[i].z, v[i].w, 0, 0);
      }
      asm volatile("fence.proxy.async.shared::cta;" ::: "memory");
      __syncwarp();
      if (lane == 0) {
        mbar_arrive(&full[s]);
        mbar_arrive(&raw_empty[rs]);  // only now: what was read has been stored
      }
      s += 2;
      if (s >= S) {
        s -= S;
        ph ^= 1u;
      }
      rs += 2;
      if (rs >= R) {
        rs -= R;
        rph ^= 1u;
      }
    }
  }
  __syncwarp();
  if (p.split > 1) {
    // Each CTA sends its partial sums of tokens j to CTA j / per, which adds
    // them in rank order and writes y.
    float* part = reinterpret_cast<float*>(P::kPart ? sfring + S * P::kSf : ring);
    int rt, tt;
    mm_tile(p, first, rt, tt);
    const int rows = min(BN, p.M - tt * BN), per = max(4, BN / p.split), lper = 31 - __clz(per);
    if (!P::kPart) cluster_arrive();
    cluster_wait();
    if (warp >= 2 && warp < 11 && warp != 6) {
      const int qd = warp & 3, row = qd * 32 + lane;
      constexpr int W = BN < 32 ? BN : 32;
#pragma unroll 1
      for (int c = warp > 6 ? W : 0; c < rows; c += 2 * W) {
        uint32_t v[W];
        if constexpr (W == 32) tmem_ld32(tmem + ((uint32_t)(qd * 32) << 16) + c, v);
        else tmem_ld16(tmem + ((uint32_t)(qd * 32) << 16) + c, v);
#pragma unroll
        for (int j = 0; j < W; j += 4)
          if (c + j < rows)
            st_dsmem_v4(part + ((rank * per + ((c + j) & (per - 1))) * 128 + 4 * row), (c + j) >> lper, v[j], v[j + 1],
                        v[j + 2], v[j + 3]);
      }
    }
    __syncwarp();
    cluster_sync_all();
    const int mine = min(per, rows - rank * per);
    const float4* p4 = reinterpret_cast<const float4*>(part);
    for (int i = tid; i < (mine + 3) / 4 * 128; i += blockDim.x) {
      const int nn = rt * 128 + (i & 127), j = rank * per + (i >> 7) * 4;
      if (nn < p.N) {
        float4 v = p4[i];
        for (int r = 1; r < p.split; ++r) {
          const float4 u = p4[r * per * 32 + i];
          v.x += u.x, v.y += u.y, v.z += u.z, v.w += u.w;
        }
        const size_t o = (size_t)(tt * BN + j) * p.N + nn;
        mm_store(p, o, v.x);
        if (j + 1 < rows) mm_store(p, o + p.N, v.y);
        if (j + 2 < rows) mm_store(p, o + 2 * (size_t)p.N, v.z);
        if (j + 3 < rows) mm_store(p, o + 3 * (size_t)p.N, v.w);
      }
    }
  }
  tc_fence_before();
  __syncthreads();
  if (CG == 2) cluster_sync_all();  // neither CTA leaves while the other may use its memory
  if (warp == 1) {
    tc_fence_after();
    if (CG == 1) tmem_dealloc(tmem, 512);
    else tmem_dealloc2(tmem, 512);
  }
}

template <int XF, int BN, int CG, bool FILL>
static cudaError_t launch_mm(MmParams p, int split, const uint8_t* xc, cudaStream_t st) {
  using P = MmPlan<XF, BN, CG, FILL>;
  static_assert(P::kTotal <= kMmSmem && P::kCols0 <= 512, "plan");
  p.split = split;
  p.row_tiles = (p.N + 128 * CG - 1) / (128 * CG);
  p.tok_tiles = (p.M + BN - 1) / BN;
  const long long tiles = (long long)p.row_tiles * p.tok_tiles;
  if (tiles > (1LL << 27)) return cudaErrorInvalidValue;
  CUtensorMap tw, tx;
  EncodeTiledFn fn = encode_fn();
  if (!fn) return cudaErrorNotSupported;
  const cuuint32_t es[2] = {1, 1};
  auto map = [&](CUtensorMap* m, const void* base, CUtensorMapDataType dt, uint64_t inner, uint64_t rows,
                 uint64_t stride, uint32_t box_rows) {
    const cuuint64_t dims[2] = {inner, rows}, strides[1] = {stride};
    const cuuint32_t box[2] = {128, box_rows};
    return fn(m, dt, 2, const_cast<void*>(base), dims, strides, box, es, CU_TENSOR_MAP_INTERLEAVE_NONE,
              CU_TENSOR_MAP_SWIZZLE_128B, CU_TENSOR_MAP_L2_PROMOTION_L2_256B,
              CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) == CUDA_SUCCESS;
  };
  const uint64_t half = p.K / 2;
  if (!map(&tx, xc, CU_TENSOR_MAP_DATA_TYPE_UINT8, XF == kMxfp4 ? half : p.K, p.M, XF == kMxfp4 ? half : p.K, BN / CG))
    return cudaErrorNotSupported;
  if (FILL) {  // packed, 64 bytes a row
    const cuuint64_t dims[2] = {half, (cuuint64_t)p.N}, strides[1] = {half};
    const cuuint32_t box[2] = {64, 128};
    if (fn(&tw, CU_TENSOR_MAP_DATA_TYPE_UINT8, 2, const_cast<uint8_t*>(p.wc), dims, strides, box, es,
           CU_TENSOR_MAP_INTERLEAVE_NONE, CU_TENSOR_MAP_SWIZZLE_NONE, CU_TENSOR_MAP_L2_PROMOTION_L2_256B,
           CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) != CUDA_SUCCESS)
      return cudaErrorNotSupported;
  } else if (XF == kMxfp4) {
    if (!map(&tw, p.wc, CU_TENSOR_MAP_DATA_TYPE_UINT8, half, p.N, half, 128)) return cudaErrorNotSupported;
  } else {
    if (!map(&tw, p.wc, CU_TENSOR_MAP_DATA_TYPE_16U4_ALIGN16B, p.K, p.N, half, 128)) return cudaErrorNotSupported;
  }
  CUtensorMap tws = tw, txs = tx;
  if (CG == 2) {  // scale tiles as rows of 128 words
    const cuuint32_t box[2] = {128, (cuuint32_t)P::kWords};
    const cuuint64_t stride[1] = {512};
    const cuuint64_t dw[2] = {128, (cuuint64_t)((p.N + 127) / 128) * p.kt}, dx[2] = {128, (cuuint64_t)((p.M + 127) / 128) * p.kt};
    auto smap = [&](CUtensorMap* m, const void* base, const cuuint64_t* dims) {
      return fn(m, CU_TENSOR_MAP_DATA_TYPE_UINT32, 2, const_cast<void*>(base), dims, stride, box, es,
                CU_TENSOR_MAP_INTERLEAVE_NONE, CU_TENSOR_MAP_SWIZZLE_NONE, CU_TENSOR_MAP_L2_PROMOTION_L2_256B,
                CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) == CUDA_SUCCESS;
    };
    if (!smap(&tws, p.ws, dw) || !smap(&txs, p.xs, dx)) return cudaErrorNotSupported;
  }
  p.wide_out = p.y_dtype != QMOE_F32 && p.N % 8 == 0 && !(reinterpret_cast<uintptr_t>(p.y) & 15);
  const int sms = device_sm_count();
  auto kernel = mx_matmul_kernel<XF, BN, CG, FILL>;
  // All of the SM's shared memory, used or not: the CTA takes all of its tensor
  // memory, and a CTA of another kernel that waits for some (or has some) must
  // not share the SM: two clusters could then wait for one another.
  cudaError_t err = ensure_smem(kernel, kMmSmem);
  if (err != cudaSuccess) return err;
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3((unsigned)(p.split > 1 ? tiles * p.split : CG * (tiles < sms / CG ? tiles : sms / CG)));
  cfg.blockDim = dim3(FILL ? kMmFillThreads : kMmThreads);
  cfg.dynamicSmemBytes = kMmSmem;
  cfg.stream = st;
  cudaLaunchAttribute attr[2];
  attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[0].val.programmaticStreamSerializationAllowed = 1;
  attr[1].id = cudaLaunchAttributeClusterDimension;
  attr[1].val.clusterDim.x = p.split * CG;
  attr[1].val.clusterDim.y = attr[1].val.clusterDim.z = 1;
  cfg.attrs = attr;
  cfg.numAttrs = 2;
  return cudaLaunchKernelEx(&cfg, kernel, tw, tx, tws, txs, p);
}

// CTAs of clusters of `split` (2, 4, 8) that the device holds at once, one CTA
// to an SM.  A query that fails fails the call: with a guess in its place, the
// same call would sum in another order another time.
static cudaError_t mm_capacity(int split, int* ctas) {
  static int cached[64][4] = {};  // CTAs + 1
  const int l = split == 8 ? 3 : split == 4 ? 2 : 1;
  int dev = 0;
  cudaError_t err = cudaGetDevice(&dev);
  if (err != cudaSuccess) return err;
  if (dev < 0 || dev >= 64) return cudaErrorInvalidDevice;
  if (!cached[dev][l]) {
    auto kernel = mx_matmul_kernel<kMxfp4, 16, 1, false>;
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = dim3(split);
    cfg.blockDim = dim3(kMmThreads);
    cfg.dynamicSmemBytes = kMmSmem;
    cudaLaunchAttribute attr;
    attr.id = cudaLaunchAttributeClusterDimension;
    attr.val.clusterDim.x = split;
    attr.val.clusterDim.y = attr.val.clusterDim.z = 1;
    cfg.attrs = &attr;
    cfg.numAttrs = 1;
    int n = 0;
    if ((err = ensure_smem(kernel, kMmSmem)) != cudaSuccess ||
        (err = cudaOccupancyMaxActiveClusters(&n, kernel, &cfg)) != cudaSuccess)
      return err;
    cached[dev][l] = n * split + 1;
  }
  *ctas = cached[dev][l] - 1;
  return cudaSuccess;
}

// Tokens per tile (and a pair of CTAs or one) and CTAs per tile along K, by an
// estimate of the time in ns: a start, the stages of the CTA with the most
// tiles, what each further tile adds beyond its MMAs (at least its epilogue's
// time in all, which short K leave bare), and the exchange of a split tile's
// sums.  The constants are fits to measured kernel times on GB300
// (us; x in MXFP8; tokens a tile / CTAs along K, 2 x for a pair):
//     16 x 1408 x 2048    16/8 3.9   16/4 4.0   16/2 4.4   16/1 4.7
//     64 x 2048 x 5632    64/4 6.0   64/2 7.6   64/1 9.6   128/4 7.1  128/1 9.9
//    512 x 1408 x 2048    64/1 5.3   128/1 6.0  192/1 7.3  2x192/1 7.8  2x256/1 9.1
//   2048 x 1408 x 2048    192/1 8.0  2x192/1 8.6  128/1 9.7  2x256/1 9.9  64/1 11.4
//    512 x 8192 x 8192    2x256/1 24  128/1 28  2x192/1 33  192/1 35  64/1 46
//   2048 x 8192 x 8192    2x192/1 82  192/1 85  2x256/1 87  128/1 89  64/1 154
//   2048 x 11264 x 2048   2x192/1 33  2x256/1 34  192/1 37  128/1 39  64/1 59
//   4096 x 8192 x 2048 (x in MXFP4)  2x256/1 30  2x192/1 35
//   4085 x 3895 x 512 (x in MXFP4)  128/1 13.1  192/1 13.4  64/1 13.9  2x256/1 15.4  2x192/1 16.9
//   8192 x 8192 x 8192 (x in MXFP4)  2x256/1 156 to 166  2x192/1 155 to 169 (the power limit's doing)
// (192 tokens: two whole accumulators fit tensor memory; at 256 the next tile's
// first MMA waits until the epilogue has taken the shared columns.)
struct MmChoice {
  int bn, cg, split;
};
static cudaError_t mm_choose(int M, int N, int chunks, bool fill, MmChoice* choice) {
  static const struct {
    int bn, cg, start, stage, tile, epilogue, exchange;
  } kinds[] = {{16, 1, 1900, 170, 300, 200, 1200},   {32, 1, 2000, 170, 350, 300, 1300},
               {64, 1, 2900, 165, 500, 850, 1400},   {128, 1, 3600, 185, 1200, 1350, 2900},
               {192, 1, 3900, 250, 800, 1900, 0},    {192, 2, 4200, 240, 300, 3000, 0},
               {256, 2, 4600, 300, 1250, 2700, 0}};
  int capacity[9] = {};
  for (int split = 2; split <= 8; split *= 2) {
    const cudaError_t err = mm_capacity(split, &capacity[split]);
    if (err != cudaSuccess) return err;
  }
  long long least = -1;
  for (const auto& k : kinds) {
    if (k.bn < 64 && M > k.bn) continue;  // 16 and 32 tokens: a single tile, at the head of its scale tile
    if (k.cg == 2 && fill) continue;
    const int stage = fill ? 230 + k.bn / 2 : k.stage;  // codes widened by warps: 240 ns at 16 tokens, 340 at 192
    const long long tiles = (long long)((N + 128 * k.cg - 1) / (128 * k.cg)) * ((M + k.bn - 1) / k.bn);
    for (int split = 1; split <= 8; split *= 2) {
      if (split > 1 && (!k.exchange || split > chunks || tiles * split > capacity[split])) break;
      const long long slots = split > 1 ? tiles : device_sm_count() / k.cg;
      const long long rounds = (tiles + slots - 1) / slots;
      const long long one = (long long)((chunks + split - 1) / split) * stage, more = one + k.tile;
      const long long t = k.start + one + (rounds - 1) * (more > k.epilogue ? more : k.epilogue) +
                          (split > 1 ? k.exchange : 0);
      if (least < 0 || t < least) {
        least = t;
        *choice = {k.bn, k.cg, split};
      }
    }
  }
  return cudaSuccess;
}

// MXFP8 x: codes that TMA cannot widen (mx_matmul_kernel)
static bool mm_fill(int x_format, int K, const uint8_t* wc) {
  return x_format == kMxfp8 && (K % 128 || (reinterpret_cast<uintptr_t>(wc) & 31));
}
static cudaError_t mm_choose(int x_format, int M, int N, int K, bool fill, MmChoice* choice) {
  const int stage = x_format == kMxfp4 ? MmPlan<kMxfp4, 128, 1>::kStageK : MmPlan<kMxfp8, 128, 1>::kStageK;
  return mm_choose(M, N, (K + stage - 1) / stage, fill, choice);
}

cudaError_t mx_matmul_variant(int x_format, const uint8_t* wc, int M, int N, int K, int* tokens, int* pair, int* split,
                              int* spread) {
  MmChoice c = {};
  const bool fill = mm_fill(x_format, K, wc);
  const cudaError_t err = mm_choose(x_format, M, N, K, fill, &c);
  *tokens = c.bn;
  *pair = c.cg == 2;
  *split = c.split;
  *spread = fill;
  return err;
}

template <int XF, bool FILL>
static cudaError_t launch_mm_bn(const MmParams& p, const uint8_t* xc, cudaStream_t st) {
  MmChoice c = {};
  const cudaError_t err = mm_choose(XF, p.M, p.N, p.K, FILL, &c);
  if (err != cudaSuccess) return err;
  switch (c.bn) {
    case 16: return launch_mm<XF, 16, 1, FILL>(p, c.split, xc, st);
    case 32: return launch_mm<XF, 32, 1, FILL>(p, c.split, xc, st);
    case 64: return launch_mm<XF, 64, 1, FILL>(p, c.split, xc, st);
    case 128: return launch_mm<XF, 128, 1, FILL>(p, c.split, xc, st);
  }
  if constexpr (!FILL) {
    if (c.bn == 256) return launch_mm<XF, 256, 2, false>(p, 1, xc, st);
    if (c.cg == 2) return launch_mm<XF, 192, 2, false>(p, 1, xc, st);
  }
  return launch_mm<XF, 192, 1, FILL>(p, 1, xc, st);
}

cudaError_t mx_status_word(void** word) { return cudaGetSymbolAddress(word, g_mx_status); }

cudaError_t launch_mx_matmul(const uint8_t* xc, const uint8_t* xs, int x_format, const uint8_t* wc, const uint8_t* ws,
                             int M, int N, int K, void* y, int y_dtype, uint32_t* status,
                             uint32_t wait_limit_kilocycles, uint32_t stall, cudaStream_t st) {
  MmParams p = {};
  p.stall = stall;
  p.wait_limit = wait_limit_kilocycles ? (long long)wait_limit_kilocycles << 10 : kWaitLimitCycles;
  p.xs = xs;
  p.ws = ws;
  p.wc = wc;
  p.y = y;
  p.status = status;
  p.M = M;
  p.N = N;
  p.K = K;
  p.y_dtype = y_dtype;
  p.kt = (K + 127) / 128;
  if (x_format == kMxfp4) return launch_mm_bn<kMxfp4, false>(p, xc, st);
  if (mm_fill(x_format, K, wc)) return launch_mm_bn<kMxfp8, true>(p, xc, st);
  return launch_mm_bn<kMxfp8, false>(p, xc, st);
}

}  // namespace qmoe
