// The norm in front of a layer as an operator of its own, and its backward.
//
//   h = x + a (rounded to elem),  y = g h rstd,  rstd = 1 / sqrt(mean(h^2) + eps)
//
// y as elem, or in 8 bits with one scale a row:
//   u = g h,  n = e4m3(448 u / max|u|),  scale = max|u| rstd / 448,  y ~ n scale
// (the row's rstd cancels in n, so a number does not depend on its rounding).
//
// Bound by the bytes of x, a, h and y: each is touched once, so a row stays in
// registers between the sums and the stores. One warp holds a row of up to 128
// 16-byte vectors, 128 threads one of up to 512, 512 threads one of up to 2048;
// longer rows are read again for every pass. Sums are fp32.
//
// Borders of e4m3: an entry whose quotient fp32 cannot tell from a border
// between two numbers is settled exactly. Products g h are held as a pair of
// floats (fma gives what the product's rounding left), the largest of the row
// likewise, and the comparison with the border in between, (mid) max|u| against
// 448 |u|, is exact in fp64: 48 bits times at most 5. Ties go to even.
#pragma once

#include <cuda_fp8.h>

#include "rowwise.cuh"

namespace swa {
namespace norm {

constexpr int kEpl = 16 / static_cast<int>(sizeof(elem_t));   // elements of a 16-byte vector
constexpr int kMaxC = 65536;
constexpr int kLoopThreads = 512;

struct FwdArgs {
  long long rows;
  int C;
  float eps;
  const elem_t* x; const elem_t* add;   // [rows, C]; add or NULL
  const float* gain;                    // [C] or NULL
  elem_t* h;                            // [rows, C], or NULL where there is no add
  elem_t* y; uint8_t* y8;               // one of them
  float* scale; float* rstd;            // [rows]; rstd or NULL
};

__device__ __forceinline__ float max_nan(float a, float b) {
  float r;
  asm("max.NaN.f32 %0, %1, %2;" : "=f"(r) : "f"(a), "f"(b));
  return r;
}

// Sum or maximum over the threads of a row. buf: 2 x (warps of the row) floats of
// shared memory, used in turn, so that one barrier a reduction suffices.
template <int TPR, bool kMax>
__device__ __forceinline__ float row_reduce(float v, float* buf, int& turn) {
#pragma unroll
  for (int o = 16; o > 0; o >>= 1) {
    const float w = __shfl_xor_sync(0xffffffffu, v, o);
    v = kMax ? max_nan(v, w) : v + w;
  }
  if constexpr (TPR > 32) {
    constexpr int NW = TPR / 32;
    float* b = buf + turn * NW;
    turn ^= 1;
    if ((threadIdx.x & 31) == 0) b[threadIdx.x >> 5] = v;
    __syncthreads();
    v = b[0];
#pragma unroll
    for (int i = 1; i < NW; ++i) v = kMax ? max_nan(v, b[i]) : v + b[i];
  }
  return v;
}

// The e4m3 number of |u| 448 / top, as t = |u| inv in fp32 found it, where that
// is too close to a border to tell: u and top as pairs of floats.
__device__ __noinline__ uint8_t settle8(float p, float e, float top, float etop, float t) {
  const float a = fabsf(t);
  // the border next to t, and the numbers on either side
  const float unit = a < 0.015625f ? 0.001953125f : __uint_as_float((__float_as_uint(a) & 0x7F800000u)) * 0.125f;
  const float below = floorf(a / unit) * unit, mid = below + 0.5f * unit;      // powers of two: exact
  const double u = fabs(static_cast<double>(p) + static_cast<double>(e)) * 448.0;
  const double m = (static_cast<double>(top) + static_cast<double>(etop)) * static_cast<double>(mid);
  const bool odd = static_cast<int>(below / unit) & 1;
  const bool up = u > m || (u == m && odd);
  return __nv_cvt_float_to_fp8(copysignf(up ? below + unit : below, t), __NV_SATFINITE, __NV_E4M3);
}
// Whether t lies within 2^-20 of itself of a border between two e4m3 numbers
// (the quotient's error is below 2^-21.9: four roundings).
__device__ __forceinline__ bool near8(float t) {
  const float a = fabsf(t);
  if (a >= 0.015625f) {
    const int low = static_cast<int>(__float_as_uint(a) & 0xFFFFFu) - 0x80000;    // three fraction bits stay
    return low >= -8 && low <= 8;
  }
  const float v = a * 512.0f, f = v - floorf(v) - 0.5f;
  return fabsf(f) <= v * 9.6e-7f;
}

__device__ __forceinline__ void gains(const float* gain, int c, float (&g)[kEpl]) {
  if (gain != nullptr) {
    ldf<kEpl>(gain + c, g);
  } else {
#pragma unroll
    for (int i = 0; i < kEpl; ++i) g[i] = 1.0f;
  }
}

// A vector of h from x and add, stored where h is kept.
__device__ __forceinline__ uint4 take(const FwdArgs& a, long long at) {
  uint4 v = ld16(a.x + at);
  if (a.add != nullptr) {
    float f[kEpl], g[kEpl];
    unpack16(v, f);
    unpack16(ld16(a.add + at), g);
#pragma unroll
    for (int i = 0; i < kEpl; ++i) f[i] += g[i];
    v = pack16(f);
  }
  return v;
}

// One vector of y. c: its first channel.
template <bool kFp8>
__device__ __forceinline__ void put(const FwdArgs& a, long long at, int c, float (&f)[kEpl], float mul, float inv, float top,
                                    float etop) {
  float g[kEpl];
  gains(a.gain, c, g);
  if constexpr (!kFp8) {
#pragma unroll
    for (int i = 0; i < kEpl; ++i) f[i] = f[i] * mul * g[i];
    st16(a.y + at, pack16(f));
  } else {
    uint32_t w[kEpl / 4];
    bool close = false;
    float t[kEpl];
#pragma unroll
    for (int i = 0; i < kEpl; ++i) {
      t[i] = f[i] * g[i] * inv;
      close |= near8(t[i]);
    }
#pragma unroll
    for (int i = 0; i < kEpl / 4; ++i) {
      const uint32_t lo = __nv_cvt_float2_to_fp8x2(make_float2(t[4 * i], t[4 * i + 1]), __NV_SATFINITE, __NV_E4M3);
      const uint32_t hi = __nv_cvt_float2_to_fp8x2(make_float2(t[4 * i + 2], t[4 * i + 3]), __NV_SATFINITE, __NV_E4M3);
      w[i] = lo | hi << 16;
    }
    if (close) {
#pragma unroll
      for (int i = 0; i < kEpl; ++i) {
        if (!near8(t[i])) continue;
        const float p = f[i] * g[i];
        const uint32_t n = settle8(p, fmaf(f[i], g[i], -p), top, etop, t[i]);
        w[i / 4] = (w[i / 4] & ~(255u << (8 * (i & 3)))) | n << (8 * (i & 3));
      }
    }
    if constexpr (kEpl == 8) {
      *reinterpret_cast<uint2*>(a.y8 + at) = make_uint2(w[0], w[1]);
    } else {
      *reinterpret_cast<uint32_t*>(a.y8 + at) = w[0];
    }
  }
}

// What a row's entries are multiplied by before anything else: 1, or a power of
// two where the sum ss of their squares leaves fp32's range or its normal numbers.
__device__ __forceinline__ float rescue(float ss) { return ss > 0x1p100f ? 0x1p-80f : (ss < 0x1p-80f ? 0x1p80f : 1.0f); }
// Rows whose largest |g h| is below this are zero in 8 bits: 448 over it would
// near fp32's end.
constexpr float kLeast8 = 0x1p-100f;

// TPR threads hold a row, VPT vectors each; VPT 0: rows of any length, read
// again for every pass (from h, which this thread has just written, where there
// is an add).
template <int TPR, int VPT, bool kFp8>
__global__ void __launch_bounds__(TPR == 32 ? 256 : TPR) fwd_kernel(const __grid_constant__ FwdArgs a) {
  constexpr int RPB = TPR == 32 ? 8 : 1;
  constexpr bool kLoop = VPT == 0;
  constexpr int V = kLoop ? 1 : VPT;
  __shared__ float buf[TPR == 32 ? 1 : 2 * TPR / 32];
  int turn = 0;
  const int t = TPR == 32 ? threadIdx.x & 31 : threadIdx.x;
  const int nv = a.C / kEpl;
  for (long long r = static_cast<long long>(blockIdx.x) * RPB + (TPR == 32 ? threadIdx.x >> 5 : 0); r < a.rows;
       r += static_cast<long long>(gridDim.x) * RPB) {
    const long long base = r * a.C;
    uint4 v[V];
    const elem_t* src = a.add != nullptr ? a.h : a.x;      // of a row that is read again
    auto each = [&](auto f) {          // f(channel, the entries) over this thread's vectors
      if constexpr (kLoop) {
        for (int i = t; i < nv; i += TPR) {
          float e[kEpl];
          unpack16(ld16(src + base + static_cast<long long>(i) * kEpl), e);
          f(i * kEpl, e);
        }
      } else {
#pragma unroll
        for (int k = 0; k < V; ++k) {
          if (t + k * TPR < nv) {
            float e[kEpl];
            unpack16(v[k], e);
            f((t + k * TPR) * kEpl, e);
          }
        }
      }
    };
    if constexpr (kLoop) {
      if (a.h != nullptr)
        for (int i = t; i < nv; i += TPR) st16(a.h + base + static_cast<long long>(i) * kEpl, take(a, base + static_cast<long long>(i) * kEpl));
    } else {
#pragma unroll
      for (int k = 0; k < V; ++k)
        if (t + k * TPR < nv) v[k] = take(a, base + (t + k * TPR) * kEpl);
      if (a.h != nullptr) {
#pragma unroll
        for (int k = 0; k < V; ++k)
          if (t + k * TPR < nv) st16(a.h + base + (t + k * TPR) * kEpl, v[k]);
      }
    }
    auto squares = [&](float down) {
      float ss = 0.f;
      each([&](int, float (&e)[kEpl]) {
#pragma unroll
        for (int i = 0; i < kEpl; ++i) ss = fmaf(e[i] * down, e[i] * down, ss);
      });
      return row_reduce<TPR, false>(ss, buf, turn);
    };
    const float plain = squares(1.0f), down = rescue(plain);
    float mul = rsqrtf(plain / a.C + a.eps);              // of entries times down
    if (down < 1.0f || (down > 1.0f && a.eps < 0x1p-40f)) mul = rsqrtf(squares(down) / a.C + a.eps * down * down);
    else if (down > 1.0f) mul *= 1.0f / down;             // eps is all that counts
    float top = 0.f, etop = 0.f, inv = 0.f;
    if constexpr (kFp8) {
      each([&](int c, float (&e)[kEpl]) {
        float g[kEpl];
        gains(a.gain, c, g);
#pragma unroll
        for (int i = 0; i < kEpl; ++i) top = max_nan(top, fabsf(e[i] * down * g[i]));
      });
      top = row_reduce<TPR, true>(top, buf, turn);
      if (a.gain != nullptr) {           // what the rounding of the largest product left
        etop = -INFINITY;
        each([&](int c, float (&e)[kEpl]) {
          float g[kEpl];
          gains(a.gain, c, g);
#pragma unroll
          for (int i = 0; i < kEpl; ++i) {
            const float p = e[i] * down * g[i];
            if (fabsf(p) == top) etop = fmaxf(etop, copysignf(1.0f, p) * fmaf(e[i] * down, g[i], -p));
          }
        });
        etop = row_reduce<TPR, true>(etop, buf, turn);
      }
      const bool fine = top < INFINITY;      // a NaN or an infinity: the whole row reads back as NaN
      const bool some = top >= kLeast8;
      inv = !fine ? __int_as_float(0x7fffffff) : (some ? 448.0f / top : 0.f);
      if (t == 0) a.scale[r] = !fine ? __int_as_float(0x7fffffff) : (some ? top * mul * (1.0f / 448.0f) : 0.f);
    }
    if (t == 0 && a.rstd != nullptr) a.rstd[r] = mul * down;
    each([&](int c, float (&e)[kEpl]) {
#pragma unroll
      for (int i = 0; i < kEpl; ++i) e[i] *= down;
      put<kFp8>(a, base + c, c, e, mul, inv, top, etop);
    });
  }
}

// ---------------------------------------------------------------------------
// Backward: with xh = h rstd and d = g dy,
//   dx = rstd (d - xh mean(d xh)) + dh,   dg = sum over rows of dy xh.
// A thread has the same channels in every row of its block, so the gain's
// gradient is summed in registers over the block's rows (in its row of the
// workspace where a row does not fit them), written once a block, and the
// blocks' rows are added in their order: results repeat bit by bit.
// ---------------------------------------------------------------------------
struct BwdArgs {
  long long rows;
  int C;
  const elem_t* h; const float* rstd; const float* gain;
  const elem_t* dy; const elem_t* dh;   // dh or NULL
  elem_t* dx;
  float* part;                          // [blocks][C], or NULL: no gradient of the gain
};

// A row's three tensors are loaded together and its products with the gain are
// kept, so that the gain is read once a row (32768 x 768 in bf16: 66 us with dh loaded
// behind the sum and the gain read twice, 42 so; its bytes take 30). Rows of many
// threads meet at a barrier, with nothing in flight but what was asked for before
// it: the next row is, where registers hold it (5001 x 8192 in fp32: 106 us without,
// 86 so, its bytes 73; 8192 x 4096 in bf16 51, its bytes 40). The blocks are as many
// as run at once with 128 registers a thread.
template <int TPR, int VPT>
__global__ void __launch_bounds__(TPR == 32 ? 256 : TPR, TPR == 32 ? 2 : 512 / TPR) bwd_kernel(const __grid_constant__ BwdArgs a) {
  constexpr int RPB = TPR == 32 ? 8 : 1;
  constexpr bool kLoop = VPT == 0, kNext = !kLoop && TPR > 32 && (kEpl == 4 || VPT < 3);
  constexpr int V = kLoop ? 1 : VPT;
  __shared__ float buf[TPR == 32 ? 1 : 2 * TPR / 32];
  extern __shared__ float sums[];        // TPR == 32: [C] of the block
  int turn = 0;
  const int t = TPR == 32 ? threadIdx.x & 31 : threadIdx.x;
  const int nv = a.C / kEpl;
  float acc[V][kEpl] = {};
  float* mine = a.part != nullptr ? a.part + static_cast<long long>(blockIdx.x) * a.C : nullptr;
  bool first = true;
  uint4 hv[V], dv[V], ev[V];
  float rs = 0.f;
  auto load = [&](long long r) {
    const long long base = r * a.C;
    rs = a.rstd[r];
#pragma unroll
    for (int k = 0; k < V; ++k) {
      if (t + k * TPR >= nv) continue;
      const long long at = base + static_cast<long long>(t + k * TPR) * kEpl;
      hv[k] = ld16(a.h + at);
      dv[k] = ld16(a.dy + at);
      if (a.dh != nullptr) ev[k] = ld16(a.dh + at);
    }
  };
  // (dy xh) into the gain's sums; d = g dy and its product with xh
  auto products = [&](const uint4& hr, const uint4& dr, int c, float rstd, float (&d)[kEpl], float (&w)[kEpl], float& dot) {
    float x[kEpl], g[kEpl];
    unpack16(hr, x);
    unpack16(dr, d);
    gains(a.gain, c, g);
#pragma unroll
    for (int e = 0; e < kEpl; ++e) {
      const float n = x[e] * rstd;
      w[e] = d[e] * n;
      d[e] *= g[e];
      dot = fmaf(d[e], n, dot);
    }
  };
  auto write = [&](const uint4& hr, const uint4& er, long long at, float rstd, float mean, float (&d)[kEpl]) {
    float x[kEpl];
    unpack16(hr, x);
#pragma unroll
    for (int e = 0; e < kEpl; ++e) d[e] = rstd * fmaf(-x[e] * rstd, mean, d[e]);
    if (a.dh != nullptr) {
      unpack16(er, x);
#pragma unroll
      for (int e = 0; e < kEpl; ++e) d[e] += x[e];
    }
    st16(a.dx + at, pack16(d));
  };
  const long long stride = static_cast<long long>(gridDim.x) * RPB;
  long long r = static_cast<long long>(blockIdx.x) * RPB + (TPR == 32 ? threadIdx.x >> 5 : 0);
  if (kNext && r < a.rows) load(r);
  for (; r < a.rows; r += stride) {
    const long long base = r * a.C;
    float dot = 0.f;
    if constexpr (kLoop) {
      const float rstd = a.rstd[r];
      for (int i = t; i < nv; i += TPR) {
        const long long at = base + static_cast<long long>(i) * kEpl;
        float d[kEpl], w[kEpl];
        products(ld16(a.h + at), ld16(a.dy + at), i * kEpl, rstd, d, w, dot);
        if (mine != nullptr) {
          float sum[kEpl] = {};
          if (!first) ldf<kEpl>(mine + i * kEpl, sum);
#pragma unroll
          for (int e = 0; e < kEpl; ++e) sum[e] += w[e];
          stf<kEpl>(mine + i * kEpl, sum);
        }
      }
      const float mean = row_reduce<TPR, false>(dot, buf, turn) / a.C;
      for (int i = t; i < nv; i += TPR) {
        const long long at = base + static_cast<long long>(i) * kEpl;
        const uint4 x = ld16(a.h + at);
        float d[kEpl], w[kEpl], none = 0.f;
        products(x, ld16(a.dy + at), i * kEpl, rstd, d, w, none);
        write(x, a.dh != nullptr ? ld16(a.dh + at) : x, at, rstd, mean, d);
      }
      first = false;
    } else {
      if (!kNext) load(r);
      float d[V][kEpl];
#pragma unroll
      for (int k = 0; k < V; ++k) {
        if (t + k * TPR >= nv) continue;
        float w[kEpl];
        products(hv[k], dv[k], (t + k * TPR) * kEpl, rs, d[k], w, dot);
#pragma unroll
        for (int e = 0; e < kEpl; ++e) acc[k][e] += w[e];
      }
      uint4 h0[V], e0[V];
      const float rs0 = rs;
#pragma unroll
      for (int k = 0; k < V; ++k) {
        h0[k] = hv[k];
        e0[k] = ev[k];
      }
      if (kNext && r + stride < a.rows) load(r + stride);
      const float mean = row_reduce<TPR, false>(dot, buf, turn) / a.C;
#pragma unroll
      for (int k = 0; k < V; ++k)
        if (t + k * TPR < nv) write(h0[k], e0[k], base + static_cast<long long>(t + k * TPR) * kEpl, rs0, mean, d[k]);
    }
  }
  if (mine == nullptr || kLoop) return;
  if constexpr (TPR == 32) {             // the block's eight rows of sums, warp after warp
    for (int w = 0; w < 8; ++w) {
      if ((threadIdx.x >> 5) == w) {
#pragma unroll
        for (int k = 0; k < V; ++k) {
          if (t + k * 32 >= nv) continue;
          float s[kEpl];
          if (w > 0) {
            ldf<kEpl>(sums + (t + k * 32) * kEpl, s);
#pragma unroll
            for (int e = 0; e < kEpl; ++e) acc[k][e] += s[e];
          }
          stf<kEpl>((w == 7 ? mine : sums) + (t + k * 32) * kEpl, acc[k]);
        }
      }
      __syncthreads();
    }
  } else {
#pragma unroll
    for (int k = 0; k < V; ++k)
      if (t + k * TPR < nv) stf<kEpl>(mine + (t + k * TPR) * kEpl, acc[k]);
  }
}

// dgain[c] = sum over n rows of part. A block: 32 channels, 8 warps that take
// every eighth row.
__global__ void __launch_bounds__(256) gain_kernel(const float* __restrict__ part, int n, int C, float* __restrict__ dgain) {
  __shared__ float s[8][32];
  const int lane = threadIdx.x & 31, w = threadIdx.x >> 5, c = blockIdx.x * 32 + lane;
  float v = 0.f;
  if (c < C) {
#pragma unroll 8
    for (int i = w; i < n; i += 8) v += part[static_cast<long long>(i) * C + c];
  }
  s[w][lane] = v;
  __syncthreads();
  if (w == 0 && c < C) {
#pragma unroll
    for (int i = 1; i < 8; ++i) v += s[i][lane];
    dgain[c] = v;
  }
}

// Threads of a row and vectors of a thread: f(integral constants TPR, VPT). The
// backward pass, which holds a row three times, takes more threads for long ones.
template <int N>
struct Int { static constexpr int value = N; };
template <bool kBwd, typename F>
void by_width(int C, F f) {
  const int nv = C / kEpl;
  if (nv <= 32) f(Int<32>{}, Int<1>{});
  else if (nv <= 64) f(Int<32>{}, Int<2>{});
  else if (nv <= 96) f(Int<32>{}, Int<3>{});
  else if (nv <= 128) f(Int<32>{}, Int<4>{});
  else if (nv <= 256) f(Int<128>{}, Int<2>{});
  else if (nv <= 512) {
    if constexpr (kBwd) f(Int<256>{}, Int<2>{});
    else if (nv <= 384) f(Int<128>{}, Int<3>{});
    else f(Int<128>{}, Int<4>{});
  }
  else if (nv <= 1024) f(Int<512>{}, Int<2>{});
  else if (nv <= 1536) f(Int<512>{}, Int<3>{});
  else if (nv <= 2048) f(Int<512>{}, Int<4>{});
  else f(Int<kLoopThreads>{}, Int<0>{});
}
// Blocks of a call: a wave of the GPU's, by threads an SM holds.
template <bool kBwd>
int row_blocks(long long rows, int C) {
  int tpr = 0;
  by_width<kBwd>(C, [&](auto t, auto) { tpr = decltype(t)::value; });
  const int threads_per_sm = kBwd ? 512 : 2048;
  const long long want = tpr == 32 ? (rows + 7) / 8 : rows;
  const long long cap = 152LL * (threads_per_sm / (tpr == 32 ? 256 : tpr));
  return static_cast<int>(want < 1 ? 1 : (want < cap ? want : cap));
}

}  // namespace norm
}  // namespace swa
