// Weights held in 4 bits, and products of a few rows with them.
//
//   y[m, n] = xs[m] sum_k x[m, k] W[n, k] + add[m, n],   W[n, k] = s[n, k / 64] (c[n, k] - 8)
//
// c in 0..15, one bf16 step s per weight row and 64 columns:
//   s = bf16(max|w| / 7) over the group, c = clamp(floor(w / s + 8.5), 0, 15), 8 where s = 0.
//
// Layout: [N / 16][K / 64] tiles (both rounded up; what is beyond N or K has c =
// 8, s = 0) of 544 bytes: 512 bytes of numbers, 16 per lane of a warp, then the
// 16 rows' steps. Lane 4 r + j holds rows r and r + 8, columns 16 j .. 16 j + 15,
// as the operand registers of four m16n8k16 products: word w, low nibble first,
// the numbers of row r + 8 hi and column 16 j + 4 w + 2 q + e for e = 0, 1, q =
// 0, 1, hi = 0, 1. (The order of a product's columns is free as long as both
// operands have the same one; this one makes a lane's part of a row of x 16
// neighbours.) Step 2 r + hi is that of row r + 8 hi.
#pragma once

#include <cuda_fp16.h>
#include <cuda_fp8.h>

#include "kv4_attn.cuh"

namespace swa {
namespace w4 {

constexpr int kRows = 16, kCols = 64;
constexpr int kTileBytes = 544;
constexpr int kMaxN = 1 << 24, kMaxK = 1 << 24, kMaxM = INT32_MAX - 255;

// ---------------------------------------------------------------------------
// Packing. A warp a tile: lane 4 r + j reads its two rows' 16 columns.
// ---------------------------------------------------------------------------
struct PackArgs {
  int N, K;
  const elem_t* w;      // [N, K]
  uint8_t* w4;
};

// The number of w at step s > 0: floor(w / s + 8.5) within 0..15. The candidate
// of the approximate quotient is settled by comparing with its borders, which
// are products of a few bits with a bf16 step: exact in fp32.
__device__ __forceinline__ uint32_t number(float w, float s) {
  float n = floorf(w / s + 8.5f);
  n = fminf(fmaxf(n, 0.f), 15.f);
  if (n > 0.f && w < (n - 8.5f) * s) n -= 1.f;
  if (n < 15.f && w >= (n - 7.5f) * s) n += 1.f;
  return static_cast<uint32_t>(n);
}

__global__ void __launch_bounds__(256) pack_kernel(const __grid_constant__ PackArgs a) {
  const int lane = threadIdx.x & 31, r = lane >> 2, j = lane & 3;
  const int Q = (a.K + kCols - 1) / kCols;
  const long long tiles = static_cast<long long>((a.N + kRows - 1) / kRows) * Q;
  for (long long t = grid_warp(); t < tiles; t += grid_warps()) {
    const int n0 = static_cast<int>(t / Q) * kRows, k0 = static_cast<int>(t % Q) * kCols + 16 * j;
    float x[2][16], s[2];
#pragma unroll
    for (int hi = 0; hi < 2; ++hi) {
      const int n = n0 + r + 8 * hi;
      const elem_t* p = a.w + static_cast<long long>(n) * a.K + k0;
      float top = 0.f;
#pragma unroll
      for (int i = 0; i < 16; ++i) {
        x[hi][i] = n < a.N && k0 + i < a.K ? to_f32(p[i]) : 0.f;
        top = kv4::max_nan(top, fabsf(x[hi][i]));
      }
      top = kv4::max_nan(top, __shfl_xor_sync(0xffffffffu, top, 1));
      top = kv4::max_nan(top, __shfl_xor_sync(0xffffffffu, top, 2));
      s[hi] = kv4::to_bf16(__fdiv_rn(top, 7.0f));
      if (s[hi] < kv4::kFlatStep) s[hi] = 0.f;
      if (!isfinite(s[hi])) s[hi] = __int_as_float(0x7fffffff);    // the group reads back as NaN
    }
    uint32_t word[4];
#pragma unroll
    for (int w = 0; w < 4; ++w) {
      word[w] = 0;
#pragma unroll
      for (int e = 0; e < 2; ++e)
#pragma unroll
        for (int q = 0; q < 2; ++q)
#pragma unroll
          for (int hi = 0; hi < 2; ++hi) {
            const uint32_t n = s[hi] > 0.f ? number(x[hi][4 * w + 2 * q + e], s[hi]) : 8u;
            word[w] |= n << (4 * (4 * e + 2 * q + hi));
          }
    }
    uint8_t* tile = a.w4 + t * kTileBytes;
    *reinterpret_cast<uint4*>(tile + 16 * lane) = make_uint4(word[0], word[1], word[2], word[3]);
    if (j == 0) *reinterpret_cast<uint32_t*>(tile + 512 + 4 * r) = pack_bf16x2(s[0], s[1]);
  }
}

// The weights that the numbers stand for, rounded to elem (exact in fp32).
__global__ void __launch_bounds__(256) unpack_kernel(int N, int K, const uint8_t* __restrict__ w4, elem_t* __restrict__ w) {
  const int lane = threadIdx.x & 31, r = lane >> 2, j = lane & 3;
  const int Q = (K + kCols - 1) / kCols;
  const long long tiles = static_cast<long long>((N + kRows - 1) / kRows) * Q;
  for (long long t = grid_warp(); t < tiles; t += grid_warps()) {
    const int n0 = static_cast<int>(t / Q) * kRows, k0 = static_cast<int>(t % Q) * kCols + 16 * j;
    const uint8_t* tile = w4 + t * kTileBytes;
    const uint4 v = *reinterpret_cast<const uint4*>(tile + 16 * lane);
    const uint32_t word[4] = {v.x, v.y, v.z, v.w};
    const uint32_t sc = *reinterpret_cast<const uint32_t*>(tile + 512 + 4 * r);
#pragma unroll
    for (int hi = 0; hi < 2; ++hi) {
      const int n = n0 + r + 8 * hi;
      const float s = __uint_as_float(hi ? sc & 0xFFFF0000u : sc << 16);
      if (n >= N) continue;
      elem_t* p = w + static_cast<long long>(n) * K + k0;
#pragma unroll
      for (int i = 0; i < 16; ++i) {
        const int nib = 4 * (i & 1) + 2 * (i >> 1 & 1) + hi;
        const float c = static_cast<float>(static_cast<int>(word[i / 4] >> (4 * nib) & 15u) - 8);
        if (k0 + i < K) p[i] = from_f32<elem_t>(c * s);
      }
    }
  }
}

// ---------------------------------------------------------------------------
// Products of few rows, on m16n8k16: a tile is the 16-row operand, made from
// the numbers' bits as in the cache's attention, eight rows of x are the other.
// n - 8 is exact in bf16 and fp16 and so are its products with an entry of x, so
// a tile's sums (64 columns) round only as fp32 adds do; the step multiplies
// them once a tile, in fp32.
//   x bf16: as it is.   x e4m3: widened to fp16 (exact), with fp16 numbers.
//   x fp32: three bf16 terms of 8 bits each, cut off, which hold it exactly.
// Small layers (linear_kernel, and all of the fp32 library): the warps of a CTA
// take every fourth (eighth) tile of the same 16 weight rows, x straight from
// memory, and add their sums up in shared memory, in their order. This is
// latency: one token through 1536 x 768 weights takes 2.2 us.
// ---------------------------------------------------------------------------
enum XKind { kXElem, kX8 };

struct LinArgs {
  int M, N, K;
  const void* x;              // [M, K] elem or e4m3
  const float* xs;            // [M], e4m3 only
  const uint8_t* w4;
  const elem_t* add;          // [M, N] or NULL (may be y)
  elem_t* y;                  // [M, N]
};

constexpr int kTerms = sizeof(elem_t) == 4 ? 3 : 1;

// 16 entries of a row of x as operand registers: b[term][word][2].
template <XKind X>
struct XFrag {
  static constexpr int T = X == kX8 ? 1 : kTerms;
  uint32_t b[T][4][2];
};

template <XKind X>
__device__ __forceinline__ void load_x(const LinArgs& a, int m, int k, XFrag<X>& f) {
  const bool on0 = m < a.M && k < a.K, on1 = m < a.M && k + 8 < a.K;      // K is a multiple of 8
  const long long at = static_cast<long long>(m) * a.K + k;
  if constexpr (X == kX8) {
    const uint8_t* p = static_cast<const uint8_t*>(a.x) + at;
    uint2 u = make_uint2(0u, 0u), v = make_uint2(0u, 0u);
    if (on0) u = *reinterpret_cast<const uint2*>(p);
    if (on1) v = *reinterpret_cast<const uint2*>(p + 8);
    const uint32_t w[4] = {u.x, u.y, v.x, v.y};
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      const __half2_raw lo = __nv_cvt_fp8x2_to_halfraw2(static_cast<__nv_fp8x2_storage_t>(w[i] & 0xFFFFu), __NV_E4M3);
      const __half2_raw hi = __nv_cvt_fp8x2_to_halfraw2(static_cast<__nv_fp8x2_storage_t>(w[i] >> 16), __NV_E4M3);
      f.b[0][i][0] = static_cast<uint32_t>(lo.x) | static_cast<uint32_t>(lo.y) << 16;
      f.b[0][i][1] = static_cast<uint32_t>(hi.x) | static_cast<uint32_t>(hi.y) << 16;
    }
  } else if constexpr (kTerms == 1) {
    const elem_t* p = static_cast<const elem_t*>(a.x) + at;
    uint4 u = make_uint4(0u, 0u, 0u, 0u), v = u;
    if (on0) u = ld16(p);
    if (on1) v = ld16(p + 8);
    f.b[0][0][0] = u.x; f.b[0][0][1] = u.y; f.b[0][1][0] = u.z; f.b[0][1][1] = u.w;
    f.b[0][2][0] = v.x; f.b[0][2][1] = v.y; f.b[0][3][0] = v.z; f.b[0][3][1] = v.w;
  } else {
    const float* p = reinterpret_cast<const float*>(a.x) + at;
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      float4 u = make_float4(0.f, 0.f, 0.f, 0.f);
      if (i < 2 ? on0 : on1) u = *reinterpret_cast<const float4*>(p + 4 * i);
      const float e[4] = {u.x, u.y, u.z, u.w};
      uint32_t t[3][4];
#pragma unroll
      for (int c = 0; c < 4; ++c) {
        float rest = e[c];
        const bool odd = (__float_as_uint(rest) & 0x7F800000u) == 0x7F800000u;   // an infinity or a NaN is its own first term
#pragma unroll
        for (int s = 0; s < 3; ++s) {
          const uint32_t bits = odd ? (s == 0 ? __float_as_uint(rest) | (rest != rest ? 0x400000u : 0u) : 0u) : __float_as_uint(rest);
          t[s][c] = bits & 0xFFFF0000u;
          if (!odd) rest -= __uint_as_float(t[s][c]);
        }
      }
#pragma unroll
      for (int s = 0; s < 3; ++s) {
        f.b[s % XFrag<X>::T][i][0] = t[s][0] >> 16 | t[s][1];
        f.b[s % XFrag<X>::T][i][1] = t[s][2] >> 16 | t[s][3];
      }
    }
  }
}

// 16 bytes that no one else reads.
__device__ __forceinline__ uint4 ld_once(const void* p) {
  uint4 v;
  asm volatile("ld.global.nc.L1::no_allocate.v4.u32 {%0, %1, %2, %3}, [%4];" : "=r"(v.x), "=r"(v.y), "=r"(v.z), "=r"(v.w) : "l"(p));
  return v;
}

template <XKind X>
__device__ __forceinline__ void widen(uint32_t w, uint32_t (&h)[4]) {
  if constexpr (X == kX8) kv4::widen_f16(w, h); else kv4::widen_bf16(w, h);
}
template <XKind X>
__device__ __forceinline__ void mma(float (&c)[4], const uint32_t (&h)[4], const uint32_t (&b)[2]) {
  if constexpr (X == kX8) kv4::mma_f16(c, h[0], h[1], h[2], h[3], b[0], b[1]);
  else kv4::mma_bf16(c, h[0], h[1], h[2], h[3], b[0], b[1]);
}

// Eight sums of row m of x and weight rows n .. n + 7 into y.
template <XKind X>
__device__ __forceinline__ void finish8(const LinArgs& a, int m, int n, bool wide, float (&y)[8]) {
  const float xs = X == kX8 ? a.xs[m] : 1.0f;
  const long long at = static_cast<long long>(m) * a.N + n;
#if !defined(SWA_ELEM_FP32)
  if (wide) {
    float b[8] = {};
    if (a.add != nullptr) unpack16(ld16(a.add + at), b);
#pragma unroll
    for (int e = 0; e < 8; ++e) y[e] = fmaf(y[e], xs, b[e]);
    st16(a.y + at, pack16(y));
    return;
  }
#endif
#pragma unroll
  for (int e = 0; e < 8; ++e)
    if (n + e < a.N) a.y[at + e] = from_f32<elem_t>(fmaf(y[e], xs, a.add != nullptr ? to_f32(a.add[at + e]) : 0.f));
}

// NT operands of eight rows of x, NW warps.
template <XKind X, int NT, int NW>
__global__ void __launch_bounds__(NW * 32) linear_kernel(const __grid_constant__ LinArgs a) {
  constexpr int MB = 8 * NT, kAhead = 2;
  __shared__ float part[NW][MB][kRows + 1];
  const int tid = threadIdx.x, lane = tid & 31, wid = tid >> 5, r = lane >> 2, j = lane & 3;
  const int P = (a.N + kRows - 1) / kRows, Q = (a.K + kCols - 1) / kCols;
  const int panel = static_cast<int>(blockIdx.x % P), m0 = static_cast<int>(blockIdx.x / P) * MB;
  const uint8_t* w = a.w4 + static_cast<long long>(panel) * Q * kTileBytes;
  uint4 v[kAhead];
  uint32_t sc[kAhead];
  auto load = [&](int i, int q) {
    if (q < Q) {
      const uint8_t* tile = w + static_cast<long long>(q) * kTileBytes;
      v[i] = ld_once(tile + 16 * lane);
      sc[i] = *reinterpret_cast<const uint32_t*>(tile + 512 + 4 * r);
    }
  };
  float acc[NT][4] = {};
#pragma unroll
  for (int i = 0; i < kAhead; ++i) load(i, wid + i * NW);
  for (int q0 = wid; q0 < Q; q0 += NW * kAhead) {
#pragma unroll
    for (int i = 0; i < kAhead; ++i) {
      const int q = q0 + i * NW;
      if (q >= Q) break;
      XFrag<X> f[NT];
#pragma unroll
      for (int t = 0; t < NT; ++t) load_x<X>(a, m0 + 8 * t + r, q * kCols + 16 * j, f[t]);
      const uint32_t word[4] = {v[i].x, v[i].y, v[i].z, v[i].w};
      uint32_t h[4][4];
#pragma unroll
      for (int k = 0; k < 4; ++k) widen<X>(word[k], h[k]);
      const float s0 = __uint_as_float(sc[i] << 16), s1 = __uint_as_float(sc[i] & 0xFFFF0000u);
      load(i, q + NW * kAhead);
#pragma unroll
      for (int t = 0; t < NT; ++t) {
        float d[4] = {};
#pragma unroll
        for (int s = XFrag<X>::T - 1; s >= 0; --s)
#pragma unroll
          for (int k = 0; k < 4; ++k) mma<X>(d, h[k], f[t].b[s][k]);
        acc[t][0] = fmaf(s0, d[0], acc[t][0]);
        acc[t][1] = fmaf(s0, d[1], acc[t][1]);
        acc[t][2] = fmaf(s1, d[2], acc[t][2]);
        acc[t][3] = fmaf(s1, d[3], acc[t][3]);
      }
    }
  }
#pragma unroll
  for (int t = 0; t < NT; ++t)
#pragma unroll
    for (int e = 0; e < 4; ++e) part[wid][8 * t + 2 * j + (e & 1)][r + 8 * (e >> 1)] = acc[t][e];
  __syncthreads();
  for (int i = tid; i < MB * kRows; i += NW * 32) {
    const int m = m0 + i / kRows, n = panel * kRows + i % kRows;
    if (m >= a.M || n >= a.N) continue;
    float y = part[0][i / kRows][i % kRows];
#pragma unroll
    for (int k = 1; k < NW; ++k) y += part[k][i / kRows][i % kRows];
    if (a.xs != nullptr) y *= a.xs[m];
    const long long at = static_cast<long long>(m) * a.N + n;
    if (a.add != nullptr) y += to_f32(a.add[at]);
    a.y[at] = from_f32<elem_t>(y);
  }
}

#if !defined(SWA_ELEM_FP32)
// ---------------------------------------------------------------------------
// Large layers: the same products, bound by the weights' bytes up to the rows
// whose products take longer (a product takes 2.5 clocks of an SM, a tile four of
// them for every eight rows of x, and its bytes 24 clocks).
//   - The eight warps of a CTA hold different panels (PN each) and go through the
//     same columns, of which x is in shared memory, 512 at a time, two buffers:
//     straight from memory every tile waited for L2 (15.6 us at 8192 x 8192 and one
//     row, 27 us from nine on, for 12.4 and 16 here).
//   - kAhead tiles a panel are in flight in registers, straight from memory.
//   - K is split over a cluster of up to 8 CTAs, which add their sums up through
//     distributed shared memory, in rank order.
// ---------------------------------------------------------------------------
constexpr int kWideWarps = 8, kChunk = 512, kAhead = 4;

template <XKind X, int NT, int PN>
struct WideShape {
  static constexpr int row = kChunk * 2 + 16;          // bytes of a row of x: lanes 4 r + j meet no bank twice
  static constexpr int buf = 8 * NT * row;
  static constexpr int RN = kWideWarps * PN * kRows;
  static constexpr int sums = 8 * NT * RN * 4;
  static constexpr int bytes = 2 * buf > sums ? 2 * buf : sums;
};
struct WideArgs {
  LinArgs l;
  int splits, per;      // CTAs of a group of panels (the cluster), chunks of each
};

template <XKind X, int NT, int PN>
__global__ void __launch_bounds__(kWideWarps * 32, 2) linear_wide_kernel(const __grid_constant__ WideArgs a) {
  using S = WideShape<X, NT, PN>;
  constexpr int MB = 8 * NT, RN = S::RN, kTiles = kChunk / kCols;
  extern __shared__ __align__(128) uint8_t smem[];
  const uint32_t sbase = smem_u32(smem);
  const int tid = threadIdx.x, lane = tid & 31, wid = tid >> 5, r = lane >> 2, j = lane & 3;
  const int P = (a.l.N + kRows - 1) / kRows, Q = (a.l.K + kCols - 1) / kCols;
  const int rank = static_cast<int>(blockIdx.x) % a.splits, group = static_cast<int>(blockIdx.x) / a.splits;
  const int q0 = rank * a.per * kTiles, q1 = min(Q, q0 + a.per * kTiles);
  const uint8_t* w[PN];
#pragma unroll
  for (int p = 0; p < PN; ++p)      // (a panel behind the last: the last again, not stored)
    w[p] = a.l.w4 + static_cast<long long>(min((group * kWideWarps + wid) * PN + p, P - 1)) * Q * kTileBytes;
  uint4 v[kAhead][PN];
  uint32_t sc[kAhead][PN];
  auto load = [&](int i, int q) {
    if (q < q1) {
#pragma unroll
      for (int p = 0; p < PN; ++p) {
        const uint8_t* tile = w[p] + static_cast<long long>(q) * kTileBytes;
        v[i][p] = ld_once(tile + 16 * lane);
        sc[i][p] = *reinterpret_cast<const uint32_t*>(tile + 512 + 4 * r);
      }
    }
  };
#pragma unroll
  for (int i = 0; i < kAhead; ++i) load(i, q0 + i);
  // x of chunk c into its buffer, in pieces of 8 columns (K is a multiple of 8); zeros beyond M and K. e4m3 is
  // widened to fp16 on the way, through registers: get() before the chunk in front of it is worked on, put() after.
  constexpr int kPieces = kChunk / 8, kMine = X == kX8 ? MB * kPieces / (kWideWarps * 32) : 1;
  uint2 x8[kMine];
  auto get = [&](int c) {
    if constexpr (X == kX8) {
#pragma unroll
      for (int u = 0; u < kMine; ++u) {
        const int i = tid + u * kWideWarps * 32, m = i / kPieces, k = (q0 + c * kTiles) * kCols + i % kPieces * 8;
        x8[u] = make_uint2(0u, 0u);
        if (m < a.l.M && k < a.l.K) x8[u] = *reinterpret_cast<const uint2*>(static_cast<const uint8_t*>(a.l.x) + static_cast<long long>(m) * a.l.K + k);
      }
    } else {
      for (int i = tid; i < MB * kPieces; i += kWideWarps * 32) {
        const int m = i / kPieces, k = (q0 + c * kTiles) * kCols + i % kPieces * 8;
        const bool on = m < a.l.M && k < a.l.K;
        const elem_t* src = static_cast<const elem_t*>(a.l.x) + (on ? static_cast<long long>(m) * a.l.K + k : 0);
        asm volatile("cp.async.cg.shared.global [%0], [%1], 16, %2;" ::"r"(sbase + (c & 1) * S::buf + m * S::row + i % kPieces * 16), "l"(src),
                     "r"(on ? 16 : 0)
                     : "memory");
      }
      asm volatile("cp.async.commit_group;" ::: "memory");
    }
  };
  auto put = [&](int c) {
    if constexpr (X == kX8) {
#pragma unroll
      for (int u = 0; u < kMine; ++u) {
        const int i = tid + u * kWideWarps * 32;
        const uint32_t e[4] = {x8[u].x & 0xFFFFu, x8[u].x >> 16, x8[u].y & 0xFFFFu, x8[u].y >> 16};
        uint32_t h[4];
#pragma unroll
        for (int k = 0; k < 4; ++k) {
          const __half2_raw t = __nv_cvt_fp8x2_to_halfraw2(static_cast<__nv_fp8x2_storage_t>(e[k]), __NV_E4M3);
          h[k] = static_cast<uint32_t>(t.x) | static_cast<uint32_t>(t.y) << 16;
        }
        st_shared_v4(sbase + (c & 1) * S::buf + i / kPieces * S::row + i % kPieces * 16, h[0], h[1], h[2], h[3]);
      }
    }
  };
  float acc[PN][NT][4] = {};
  const int chunks = (q1 - q0 + kTiles - 1) / kTiles;      // (below 1: this rank has no columns)
  if (chunks > 0) get(0);
  for (int c = 0; c < chunks; ++c) {
    put(c);
    if (c + 1 < chunks) {
      get(c + 1);
      asm volatile("cp.async.wait_group 1;" ::: "memory");
    } else {
      asm volatile("cp.async.wait_group 0;" ::: "memory");
    }
    __syncthreads();
    const uint8_t* xb = smem + (c & 1) * S::buf;
#pragma unroll
    for (int tq = 0; tq < kTiles; ++tq) {
      const int q = q0 + c * kTiles + tq, i = tq % kAhead;
      if (q >= q1) break;
      uint32_t h[PN][4][4];
      float s0[PN], s1[PN];
#pragma unroll
      for (int p = 0; p < PN; ++p) {
        const uint32_t word[4] = {v[i][p].x, v[i][p].y, v[i][p].z, v[i][p].w};
#pragma unroll
        for (int k = 0; k < 4; ++k) widen<X>(word[k], h[p][k]);
        s0[p] = __uint_as_float(sc[i][p] << 16);
        s1[p] = __uint_as_float(sc[i][p] & 0xFFFF0000u);
      }
      load(i, q + kAhead);
#pragma unroll
      for (int t = 0; t < NT; ++t) {
        uint32_t b[4][2];
        const uint8_t* at = xb + (8 * t + r) * S::row + (tq * kCols + 16 * j) * 2;
        const uint4 u = *reinterpret_cast<const uint4*>(at), z = *reinterpret_cast<const uint4*>(at + 16);
        b[0][0] = u.x; b[0][1] = u.y; b[1][0] = u.z; b[1][1] = u.w;
        b[2][0] = z.x; b[2][1] = z.y; b[3][0] = z.z; b[3][1] = z.w;
#pragma unroll
        for (int p = 0; p < PN; ++p) {
          float d[4] = {};
#pragma unroll
          for (int k = 0; k < 4; ++k) mma<X>(d, h[p][k], b[k]);
          acc[p][t][0] = fmaf(s0[p], d[0], acc[p][t][0]);
          acc[p][t][1] = fmaf(s0[p], d[1], acc[p][t][1]);
          acc[p][t][2] = fmaf(s1[p], d[2], acc[p][t][2]);
          acc[p][t][3] = fmaf(s1[p], d[3], acc[p][t][3]);
        }
      }
    }
    __syncthreads();       // the buffer is free
  }
  // the sums, [MB][RN]
  float* part = reinterpret_cast<float*>(smem);
#pragma unroll
  for (int p = 0; p < PN; ++p)
#pragma unroll
    for (int t = 0; t < NT; ++t)
#pragma unroll
      for (int e = 0; e < 4; ++e)
        part[(8 * t + 2 * j + (e & 1)) * RN + (wid * PN + p) * kRows + r + 8 * (e >> 1)] = acc[p][t][e];
  if (a.splits > 1)
    asm volatile("barrier.cluster.arrive.release.aligned;\n\tbarrier.cluster.wait.acquire.aligned;" ::: "memory");
  else
    __syncthreads();
  // this CTA's share of them, eight weight rows a thread
  const int share = (MB * RN / 8 + a.splits - 1) / a.splits;
  const bool wide = a.l.N % 8 == 0;
  for (int i = rank * share + tid; i < min((rank + 1) * share, MB * RN / 8); i += kWideWarps * 32) {
    const int m = i / (RN / 8), f = i % (RN / 8) * 8, n = group * RN + f;
    if (m >= a.l.M || n >= a.l.N) continue;
    float y[8] = {};
    const uint32_t mine = sbase + static_cast<uint32_t>(m * RN + f) * 4;
    for (int s = 0; s < a.splits; ++s) {
      uint32_t there;
      float4 u, z;
      asm volatile("mapa.shared::cluster.u32 %0, %1, %2;" : "=r"(there) : "r"(mine), "r"(s));
      asm volatile("ld.shared::cluster.v4.f32 {%0, %1, %2, %3}, [%4];" : "=f"(u.x), "=f"(u.y), "=f"(u.z), "=f"(u.w) : "r"(there) : "memory");
      asm volatile("ld.shared::cluster.v4.f32 {%0, %1, %2, %3}, [%4];" : "=f"(z.x), "=f"(z.y), "=f"(z.z), "=f"(z.w) : "r"(there + 16) : "memory");
      y[0] += u.x; y[1] += u.y; y[2] += u.z; y[3] += u.w;
      y[4] += z.x; y[5] += z.y; y[6] += z.z; y[7] += z.w;
    }
    finish8<X>(a.l, m, n, wide, y);
  }
  if (a.splits > 1) asm volatile("barrier.cluster.arrive.release.aligned;\n\tbarrier.cluster.wait.acquire.aligned;" ::: "memory");
}
#endif

// A launch in clusters of `size` CTAs.
template <typename K, typename... A>
swa_status launch_cluster(K kern, long long grid, int threads, int smem, int size, cudaStream_t st, const A&... args) {
  if (grid > INT32_MAX) return SWA_ERR_UNSUPPORTED;
  cudaLaunchConfig_t cfg{};
  cfg.gridDim = dim3(static_cast<unsigned>(grid));
  cfg.blockDim = dim3(static_cast<unsigned>(threads));
  cfg.dynamicSmemBytes = static_cast<size_t>(smem);
  cfg.stream = st;
  cudaLaunchAttribute at{};
  at.id = cudaLaunchAttributeClusterDimension;
  at.val.clusterDim.x = static_cast<unsigned>(size);
  at.val.clusterDim.y = at.val.clusterDim.z = 1;
  cfg.attrs = &at;
  cfg.numAttrs = 1;
  const bool ok = cudaLaunchKernelEx(&cfg, kern, args...) == cudaSuccess;
  return cudaGetLastError() == cudaSuccess && ok ? SWA_OK : SWA_ERR_CUDA;      // (told here, and not again by the next launch)
}

}  // namespace w4
}  // namespace swa
