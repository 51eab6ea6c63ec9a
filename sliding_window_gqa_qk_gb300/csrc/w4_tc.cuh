// Products of more than a few rows with 4-bit weights, on the tensor cores'
// tcgen05 form (bf16 library).
//
// Few rows are bound by the weights' bytes, many by the products; between the
// two lies turning numbers into operands, which every CTA does for the weights of
// its own tile only. A tile is 128 weight rows (the products' M: the lanes of
// tensor memory, so that a thread owns a row) by MB rows of x (their N, 64 to
// 256), K in stages of 128:
//   warps 0-15  in four groups that take every fourth stage. A thread turns one
//               row's 128 numbers of the stage to bf16, times their step, and
//               puts them into tensor memory, from where the products take them;
//               afterwards the epilogue. The rows of x too where they are e4m3
//               (widened to bf16, exact, into shared memory).
//   warp 16     TMA producer of the rows of x in bf16 (or, in e4m3, as they are);
//   warp 17     MMA issuer: eight M = 128, N = MB, K = 16 products a stage;
//   warp 18     TMA producer of the weights as they lie in memory.
// Why so: weights as operands in shared memory are 256 bytes a row and stage
// written and read again, 512 clocks of shared memory where a stage's bytes take
// the memory 378; in tensor memory they cost none. The packed numbers come as
// 128-byte rows with the 128-byte swizzle, in which the 16-byte pieces of a
// thread's row (64 bytes apart for neighbouring rows) meet no bank twice. Loaded
// ahead into registers they made every 64 columns wait for memory at the fence.
// Measured (GB300): 8192 x 8192, 64 rows 23 us, 256 rows 29 us; 2048 rows through
// 2048 x 2048 21 us, of which about 6 are the way in and out of the kernel. Up to
// 128 rows the issue of the products bounds it, 45 to 64 clocks each (eight a
// stage) however narrow they are; with 256 rows the products themselves, 128 each.
// Rounding: a weight enters as bf16(s (n - 8)): its 11 bits lose up to three,
// less than 2^-8 of the weight (3.9e-3 for s = 148 / 128, n - 8 = 7). The error is
// relative to the sum of sizes |x w|: as y's own bf16 rounding where that sum does
// not cancel, above it where it does. (The form for few rows keeps s out of the
// products; here that would take the sums out of tensor memory every 64 columns.)
// Few tiles: K is split over a cluster of up to 8 CTAs, which add their sums up
// through distributed shared memory, in rank order.
#pragma once

#include "tc_gemm.cuh"
#include "w4.cuh"

namespace swa {
namespace w4 {

constexpr int kTcGroup = 4, kTcGroups = 4;       // warps of a group, groups
constexpr int kTcDequant = kTcGroup * kTcGroups, kTcTma = kTcDequant, kTcMma = kTcTma + 1, kTcRaw = kTcMma + 1;
constexpr int kTcThreads = 32 * (kTcRaw + 1);
constexpr int kTcRows = 128, kTcPanels = kTcRows / kRows;
constexpr int kSub = 2;                          // 64-column steps of a stage
constexpr int kTcStages = 4;                     // stages of weights in tensor memory, 64 columns each
constexpr uint32_t kTcAcol = 256;                // their first column, behind the sums

template <int MB, bool X8>
struct TcShape {
  static constexpr int kB = MB * kCols * 2;      // x as operand, of a step
  // Stages of x. Up to 128 rows they go with those of the weights: the issuer then has one wait and one commit a
  // stage beside its eight products, which take 45 to 64 clocks each to issue however narrow they are (a wait and a
  // commit of their own for every 64 columns of x: 27 us for 22). The warps that turn the stage's weights wait for its
  // x too, and arrive for both: a copy that the issuer's barrier counted itself could not be waited for on the way out,
  // once warps that give up arrive there no more.
  static constexpr bool kJoint = MB <= 128;
  static constexpr int kXs = kJoint ? kTcStages : 3;
  // A stage's place in either ring is always the same group's: a wait for a
  // phase then never comes before the one in front of it is over.
  static constexpr int kRaws = MB == 256 || (X8 && MB == 128) ? 4 : 8;
  static constexpr int kRawW = kTcPanels * kSub * 512, kRawS = kTcPanels * kSub * 32, kRawX = X8 ? kSub * MB * kCols : 0;
  static constexpr int oRawW = kXs * kSub * kB, oRawX = oRawW + kRaws * kRawW, oRawS = oRawX + kRaws * kRawX,
                       oBar = oRawS + kRaws * kRawS;
  static constexpr int kBytes = oBar + 512;
  static constexpr int FULL = 0, EMPTY = kTcStages, XFULL = 2 * kTcStages, XEMPTY = XFULL + kXs, RAW = XEMPTY + kXs,
                       RAWFREE = RAW + kRaws, ACC = RAWFREE + kRaws, COUNT = ACC + 1;
  static_assert(kBytes <= 232448 && COUNT * 8 + 8 <= 512 && oRawW % 1024 == 0 && oRawX % 128 == 0 && oRawS % 128 == 0, "");
  static_assert(kRaws % kTcGroups == 0 && kTcStages % kTcGroups == 0 && (!kJoint || kXs == kTcStages), "");
  static_assert(MB * kTcRows * 4 <= oRawS && MB <= static_cast<int>(kTcAcol), "the sums fit shared memory and their columns");
};

// Where a call without a workspace leaves what its waits report.
__device__ uint32_t g_unreported;

struct TcArgs {
  LinArgs l;
  int mt;                     // tiles along the rows of x
  int splits, per;            // CTAs of a tile (the cluster), stages of each
  uint32_t* status;
  uint64_t wait_limit_ns;
};

__device__ __forceinline__ uint32_t mul_bf16x2(uint32_t a, __nv_bfloat162 s) {
  const __nv_bfloat162 r = __hmul2(*reinterpret_cast<const __nv_bfloat162*>(&a), s);
  return *reinterpret_cast<const uint32_t*>(&r);
}
// 128 + n of two numbers, to (n - 8) s
__device__ __forceinline__ uint32_t weight2(uint32_t v, __nv_bfloat162 s) {
  const __nv_bfloat162 r = __hadd2(*reinterpret_cast<const __nv_bfloat162*>(&v), __floats2bfloat162_rn(-136.f, -136.f));
  return mul_bf16x2(*reinterpret_cast<const uint32_t*>(&r), s);
}
// Two e4m3 numbers as bf16 (exact).
__device__ __forceinline__ uint32_t e4m3_bf16x2(uint32_t two) {
  const __half2_raw h = __nv_cvt_fp8x2_to_halfraw2(static_cast<__nv_fp8x2_storage_t>(two), __NV_E4M3);
  const float2 f = __half22float2(__half2(h));
  return pack_bf16x2(f.x, f.y);
}

template <int MB, bool X8, bool kPolled>
__global__ void __launch_bounds__(kTcThreads, 1)
    linear_tc_kernel(const __grid_constant__ CUtensorMap tmX, const __grid_constant__ CUtensorMap tmW,
                     const __grid_constant__ CUtensorMap tmS, const __grid_constant__ TcArgs a) {
  using S = TcShape<MB, X8>;
  constexpr int ST = kTcStages, RS = S::kRaws, XS = S::kXs;
  extern __shared__ __align__(1024) uint8_t smem[];
  const uint32_t sbase = smem_u32(smem);
  if (sbase & 1023u) {   // swizzle atoms need 1024-byte aligned tiles (uniform over the grid)
    if (threadIdx.x == 0) atomicOr(a.status != nullptr ? a.status : &g_unreported, DEV_ERR_BOUNDS);
    return;
  }
  uint32_t* tmem_sh = reinterpret_cast<uint32_t*>(smem + S::oBar + S::COUNT * 8);
  uint32_t* abort_flag = tmem_sh + 1;
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
  uint32_t* status = a.status != nullptr ? a.status : &g_unreported;
  const WaitCtl<kPolled> ctl{abort_flag, status, a.wait_limit_ns};
  auto bar = [&](int i) { return sbase + S::oBar + 8u * static_cast<uint32_t>(i); };
  const int rank = static_cast<int>(blockIdx.x) % a.splits, tile = static_cast<int>(blockIdx.x) / a.splits;
  const int m0 = tile % a.mt * MB, n0 = tile / a.mt * kTcRows;
  const int Q = (a.l.K + kCols - 1) / kCols;
  const int q0 = rank * a.per * kSub, stages = max(0, (min(Q, q0 + a.per * kSub) - q0 + kSub - 1) / kSub);

  if (tid == 0) {
    *abort_flag = 0;
    for (int s = 0; s < ST; ++s) {
      mbar_init(bar(S::FULL + s), kTcGroup);
      mbar_init(bar(S::EMPTY + s), 1);
    }
    for (int s = 0; s < XS; ++s) {
      mbar_init(bar(S::XFULL + s), 1);
      mbar_init(bar(S::XEMPTY + s), 1);
    }
    for (int s = 0; s < RS; ++s) {
      mbar_init(bar(S::RAW + s), 1);
      mbar_init(bar(S::RAWFREE + s), kTcGroup);
    }
    mbar_init(bar(S::ACC), 1);
    fence_mbar_init();
  }
  if (warp == kTcMma) {
    tmem_alloc(smem_u32(tmem_sh), 512);
    tmem_relinquish();
  }
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  const uint32_t tmem = *tmem_sh;
  const uint32_t quarter = static_cast<uint32_t>(warp & 3) * 32;      // lanes of tensor memory that this warp reaches

  bool ok = true;
  if (warp < kTcDequant) {
    // row quarter + lane: panel, row r + 8 hi of it; its numbers are every second nibble of lanes 4 r .. 4 r + 3's words
    const int r = lane & 7, hi = lane >> 3 & 1, panel = (warp & 3) * 2 + (lane >> 4);
    const int gt = tid % (32 * kTcGroup);
    for (int k = warp / kTcGroup; k < stages; k += kTcGroups) {
      const int st = k % ST, raw = k % RS;
      if (!(ok = mbar_wait_warp(bar(S::RAW + raw), (k / RS) & 1, ctl))) break;
      uint4 v[kSub][4];
      uint32_t sc[kSub];
#pragma unroll
      for (int u = 0; u < kSub; ++u) {
        const uint32_t at = sbase + S::oRawW + raw * S::kRawW + (panel * kSub + u) * 512 + (r >> 1) * 128;
#pragma unroll
        for (int j = 0; j < 4; ++j) v[u][j] = ld_shared_v4u(at + static_cast<uint32_t>((4 * (r & 1) + j) ^ ((r >> 1) + 4 * u)) * 16);
        asm volatile("ld.shared.u16 %0, [%1];" : "=r"(sc[u]) : "r"(sbase + S::oRawS + raw * S::kRawS + (panel * kSub + u) * 32 + 4 * r + 2 * hi) : "memory");
      }
      if (!X8) {
        __syncwarp();
        if (lane == 0) mbar_arrive(bar(S::RAWFREE + raw));
      }
      if (k >= ST && !(ok = mbar_wait_warp(bar(S::EMPTY + st), (k / ST - 1) & 1, ctl))) break;
      tc_fence_after();
#pragma unroll
      for (int u = 0; u < kSub; ++u) {
        const __nv_bfloat16 s1 = __ushort_as_bfloat16(static_cast<unsigned short>(sc[u]));
        const __nv_bfloat162 s2 = __halves2bfloat162(s1, s1);
        uint32_t x[32];
#pragma unroll
        for (int j = 0; j < 4; ++j) {
          const uint32_t word[4] = {v[u][j].x, v[u][j].y, v[u][j].z, v[u][j].w};
#pragma unroll
          for (int w = 0; w < 4; ++w) {
            const uint32_t y = word[w] >> (4 * hi);
            x[8 * j + 2 * w] = weight2(kv4::and_or(y, 0x000F000Fu, 0x43004300u), s2);
            x[8 * j + 2 * w + 1] = weight2(kv4::and_or(y >> 8, 0x000F000Fu, 0x43004300u), s2);
          }
        }
        tmem_st32(tmem + (quarter << 16) + kTcAcol + static_cast<uint32_t>(st * kSub + u) * 32, x);
      }
      if constexpr (X8) {
        constexpr int XP = kSub * MB * 4 / (32 * kTcGroup);     // pieces of 16 columns of x
#pragma unroll
        for (int u = 0; u < XP; ++u) {
          const int unit = gt + 32 * kTcGroup * u, m = unit % (MB * 4) >> 2, c = (unit & 3) * 2;
          const uint4 v = ld_shared_v4u(sbase + S::oRawX + raw * S::kRawX + unit * 16);
          const uint32_t b = sbase + static_cast<uint32_t>(st * kSub + unit / (MB * 4)) * S::kB + (m >> 3) * 1024 + (m & 7) * 128;
          const uint32_t e[4] = {v.x, v.y, v.z, v.w};
#pragma unroll
          for (int h = 0; h < 2; ++h)
            st_shared_v4(b + static_cast<uint32_t>((c + h) ^ (m & 7)) * 16, e4m3_bf16x2(e[2 * h] & 0xFFFFu), e4m3_bf16x2(e[2 * h] >> 16),
                         e4m3_bf16x2(e[2 * h + 1] & 0xFFFFu), e4m3_bf16x2(e[2 * h + 1] >> 16));
        }
        fence_async_smem();
      }
      tmem_wait_st();
      if (!X8 && S::kJoint && !(ok = mbar_wait_warp(bar(S::XFULL + st), (k / ST) & 1, ctl))) break;
      tc_fence_before();
      __syncwarp();
      if (lane == 0) {
        mbar_arrive(bar(S::FULL + st));
        if (X8) mbar_arrive(bar(S::RAWFREE + raw));
      }
    }
  } else if (warp == kTcTma) {
    if (!X8 && lane == 0) {
      tma_prefetch_desc(&tmX);
      constexpr int full = S::XFULL, empty = S::kJoint ? S::EMPTY : S::XEMPTY;
      int k = 0;
      for (; k < stages; ++k) {
        const int st = k % XS;
        if (k >= XS && !mbar_wait(bar(empty + st), (k / XS - 1) & 1, ctl)) break;
        mbar_arrive_expect_tx(bar(full + st), kSub * S::kB);
        for (int u = 0; u < kSub; ++u)
          tma_load_2d(sbase + static_cast<uint32_t>(st * kSub + u) * S::kB, &tmX, bar(full + st), (q0 + k * kSub + u) * kCols, m0);
      }
      // what was issued lands before the memory is given back (those who wait for it may have given up)
      for (int i = max(0, k - XS); i < k; ++i) mbar_wait_drain(bar(full + i % XS), (i / XS) & 1, kDrainLimitNs);
    }
  } else if (warp == kTcRaw) {
    if (lane == 0) {
      tma_prefetch_desc(&tmW);
      tma_prefetch_desc(&tmS);
      if (X8) tma_prefetch_desc(&tmX);
      int i = 0;
      for (; i < stages; ++i) {
        const int st = i % RS, k = q0 + i * kSub;
        if (i >= RS && !mbar_wait(bar(S::RAWFREE + st), (i / RS - 1) & 1, ctl)) break;
        mbar_arrive_expect_tx(bar(S::RAW + st), S::kRawW + S::kRawS + S::kRawX);
        tma_load_4d(sbase + S::oRawW + st * S::kRawW, &tmW, bar(S::RAW + st), 0, 0, k, n0 / kRows);
        tma_load_4d(sbase + S::oRawS + st * S::kRawS, &tmS, bar(S::RAW + st), 0, k, n0 / kRows, 0);
        if (X8)
          for (int e = 0; e < kSub; ++e)
            tma_load_2d(sbase + S::oRawX + st * S::kRawX + e * (MB * kCols), &tmX, bar(S::RAW + st), (k + e) * kCols, m0);
      }
      for (int e = max(0, i - RS); e < i; ++e) mbar_wait_drain(bar(S::RAW + e % RS), (e / RS) & 1, kDrainLimitNs);   // as above
    }
  } else if (lane == 0) {
    constexpr uint32_t id = idesc_bf16_f32(kTcRows, MB, 0, 0);
    const uint64_t dB = sdesc_sw128(sbase, 16, 1024);
    for (int k = 0; k < stages; ++k) {
      const int st = k % ST, xs = k % XS;
      if (!(ok = mbar_wait(bar(S::FULL + st), (k / ST) & 1, ctl))) break;
      if (!S::kJoint && !(ok = mbar_wait(bar(S::XFULL + xs), (k / XS) & 1, ctl))) break;
      tc_fence_after();
      const uint32_t ta = tmem + kTcAcol + static_cast<uint32_t>(st) * (kSub * 32);
      const uint64_t db = sdesc_add(dB, xs * kSub * S::kB);
      static_for<0, kSub * kCols / 16>([&](auto kc) {
        constexpr int kk = decltype(kc)::value, u = kk / (kCols / 16), e = kk % (kCols / 16);
        umma_ts_imm<id, kk * 8, u * (S::kB >> 4) + e * 2>(tmem, ta, db, (k > 0 || kk > 0) ? 1u : 0u, 1u);
      });
      umma_commit(bar(S::EMPTY + st));
      if (!S::kJoint) umma_commit(bar(S::XEMPTY + xs));
    }
    umma_commit(bar(S::ACC));         // every product issued has completed, after a wait that ran out too
    mbar_wait_drain(bar(S::ACC), 0, kDrainLimitNs);
  }

  __syncwarp();
  // ---------------- epilogue: the sums to shared memory, [MB][128] over the operands; thread = weight row ----------------
  float* part = reinterpret_cast<float*>(smem);
  if (warp < kTcDequant && ok) ok = mbar_wait_warp(bar(S::ACC), 0, ctl);
  tc_fence_after();
  if (warp < kTcDequant && ok) {
    for (int c = (warp >> 2) * 32; c < MB; c += kTcDequant * 8) {
      uint32_t d[32];
      tmem_ld32(tmem + (quarter << 16) + c, d);
      tmem_wait_ld(d);
#pragma unroll
      for (int i = 0; i < 32; ++i) part[(c + i) * kTcRows + quarter + lane] = stages > 0 ? __uint_as_float(d[i]) : 0.f;
    }
  }
  __syncwarp();
  tc_fence_before();
  if (a.splits > 1)
    asm volatile("barrier.cluster.arrive.release.aligned;\n\tbarrier.cluster.wait.acquire.aligned;" ::: "memory");
  else
    __syncthreads();
  // this CTA's share of the rows of x, eight weight rows a thread
  if (warp < kTcDequant && ok) {
    const int per = MB / a.splits;
    const bool wide = a.l.N % 8 == 0;
    for (int i = tid; i < per * (kTcRows / 8); i += kTcDequant * 32) {
      const int c = rank * per + i / (kTcRows / 8), f = i % (kTcRows / 8) * 8, m = m0 + c, n = n0 + f;
      if (m >= a.l.M || n >= a.l.N) continue;
      float v[8] = {};
      const uint32_t mine = sbase + static_cast<uint32_t>(c * kTcRows + f) * 4;
      for (int s = 0; s < a.splits; ++s) {
        uint32_t there;
        float4 x, y;
        asm volatile("mapa.shared::cluster.u32 %0, %1, %2;" : "=r"(there) : "r"(mine), "r"(s));
        asm volatile("ld.shared::cluster.v4.f32 {%0, %1, %2, %3}, [%4];" : "=f"(x.x), "=f"(x.y), "=f"(x.z), "=f"(x.w) : "r"(there) : "memory");
        asm volatile("ld.shared::cluster.v4.f32 {%0, %1, %2, %3}, [%4];" : "=f"(y.x), "=f"(y.y), "=f"(y.z), "=f"(y.w) : "r"(there + 16) : "memory");
        v[0] += x.x; v[1] += x.y; v[2] += x.z; v[3] += x.w;
        v[4] += y.x; v[5] += y.y; v[6] += y.z; v[7] += y.w;
      }
      finish8<X8 ? kX8 : kXElem>(a.l, m, n, wide, v);
    }
  }
  __syncwarp();
  if (a.splits > 1) asm volatile("barrier.cluster.arrive.release.aligned;\n\tbarrier.cluster.wait.acquire.aligned;" ::: "memory");
  if (warp == kTcMma) tmem_dealloc(tmem, 512);
}

// Tensor map of e4m3 rows [M][K], boxes of 64 columns x `rows`, not swizzled.
// Strides count in 16 bytes: K has to be a multiple of 16.
inline bool map_bytes(CUtensorMap* m, const void* base, long long K, long long M, int rows) {
  auto fn = tc::encode_fn();
  if (fn == nullptr) return false;
  cuuint64_t dims[2] = {static_cast<cuuint64_t>(K), static_cast<cuuint64_t>(M)}, strides[1] = {static_cast<cuuint64_t>(K)};
  cuuint32_t box[2] = {kCols, static_cast<cuuint32_t>(rows)}, es[2] = {1, 1};
  return fn(m, CU_TENSOR_MAP_DATA_TYPE_UINT8, 2, const_cast<void*>(base), dims, strides, box, es, CU_TENSOR_MAP_INTERLEAVE_NONE,
            CU_TENSOR_MAP_SWIZZLE_NONE, CU_TENSOR_MAP_L2_PROMOTION_L2_256B, CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) == CUDA_SUCCESS;
}

// Tensor maps of packed weights in 8-byte elements, boxes of a stage's tiles of
// the panels of a tile of y: the numbers as 128-byte rows [panel][tile][4], swizzled,
// and the steps [panel][tile], 32 bytes each. Beyond the last tile and panel: zeros.
inline bool map_w4(CUtensorMap* w, CUtensorMap* s, const void* base, long long panels, long long tiles) {
  auto fn = tc::encode_fn();
  if (fn == nullptr) return false;
  const cuuint64_t t = static_cast<cuuint64_t>(tiles), p = static_cast<cuuint64_t>(panels);
  cuuint64_t dw[4] = {16, 4, t, p}, sw[3] = {128, kTileBytes, t * kTileBytes};
  cuuint32_t bw[4] = {16, 4, kSub, kTcPanels}, es[4] = {1, 1, 1, 1};
  cuuint64_t ds[4] = {4, t, p, 1}, ss[3] = {kTileBytes, t * kTileBytes, t * kTileBytes};
  cuuint32_t bs[4] = {4, kSub, kTcPanels, 1};
  return fn(w, CU_TENSOR_MAP_DATA_TYPE_INT64, 4, const_cast<void*>(base), dw, sw, bw, es, CU_TENSOR_MAP_INTERLEAVE_NONE,
            CU_TENSOR_MAP_SWIZZLE_128B, CU_TENSOR_MAP_L2_PROMOTION_L2_256B, CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) == CUDA_SUCCESS &&
         fn(s, CU_TENSOR_MAP_DATA_TYPE_INT64, 4, static_cast<uint8_t*>(const_cast<void*>(base)) + 512, ds, ss, bs, es,
            CU_TENSOR_MAP_INTERLEAVE_NONE, CU_TENSOR_MAP_SWIZZLE_NONE, CU_TENSOR_MAP_L2_PROMOTION_NONE,
            CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) == CUDA_SUCCESS;
}

// CTAs of a tile: as many as fill the GPU, with two stages each at least.
inline int tc_splits(long long tiles, int stages) {
  int s = 1;
  while (s < 8 && tiles * s * 2 <= 152 && stages / (s * 2) >= 2) s *= 2;
  return s;
}

template <int MB, bool X8>
swa_status launch_linear_tc(const LinArgs& l, uint32_t* status, uint64_t wait_ns, cudaStream_t st) {
  using S = TcShape<MB, X8>;
  CUtensorMap map{}, wmap{}, smap{};
  if (!map_w4(&wmap, &smap, l.w4, (l.N + kRows - 1) / kRows, (l.K + kCols - 1) / kCols)) return SWA_ERR_CUDA;
  if (X8 ? !map_bytes(&map, l.x, l.K, l.M, MB) : !tc::map_2d(&map, l.x, l.K, l.M, l.K, MB)) return SWA_ERR_CUDA;
  TcArgs a{};
  a.l = l;
  a.mt = (l.M + MB - 1) / MB;
  const long long tiles = static_cast<long long>(a.mt) * ((l.N + kTcRows - 1) / kTcRows);
  const int stages = (l.K + kSub * kCols - 1) / (kSub * kCols);
  a.splits = tc_splits(tiles, stages);
  a.per = (stages + a.splits - 1) / a.splits;
  a.status = status;
  a.wait_limit_ns = wait_ns;
  auto launch = [&](auto kern) {
    if (cudaFuncSetAttribute(kern, cudaFuncAttributeMaxDynamicSharedMemorySize, S::kBytes) != cudaSuccess) {
      cudaGetLastError();
      return SWA_ERR_CUDA;
    }
    return launch_cluster(kern, tiles * a.splits, kTcThreads, S::kBytes, a.splits, st, map, wmap, smap, a);
  };
  return wait_ns < kPollBelowNs ? launch(linear_tc_kernel<MB, X8, true>) : launch(linear_tc_kernel<MB, X8, false>);
}

}  // namespace w4
}  // namespace swa
