// Rotary positions as operators of their own: the cosine / sine tables
// (scaled for long contexts) and the rotation of q and k by such tables, in
// the split-half or the interleaved layout, of the whole head or its first
// channels. The attention's prologue (rowwise.cuh rotate_row) keeps its fused
// form of the split-half rotation of whole heads; these cover the rest, and
// build the tables both read.
#pragma once

#include "common.cuh"
#include "rowwise.cuh"

namespace swa {

constexpr int kMaxRot = 128;        // channels turned at most (the largest head)
constexpr int kTableThreads = 256;
constexpr int kRopeThreads = 128;

// ---------------------------------------------------------------------------
// Tables: cos[t][c], sin[t][c] of t * theta_c.
//
// A position far out makes the angle thousands of turns, and fp32 (or an
// fp32 reduction) would lose the fraction that matters. The angle is kept in
// turns as a 64-bit fixed-point fraction instead: phi_c = theta_c / (2 pi)
// scaled by 2^64 and multiplied by the integer t modulo 2^64 leaves the
// fraction of a turn exactly, with no floating-point reduction and no fp64
// arithmetic (this GPU has little of it). Its top 32 bits are the angle; the
// nearest quarter turn comes off as an integer, and what is left, at most an
// eighth of a turn either way, goes through the Taylor polynomials of sine
// (to x^9) and cosine (to x^8), which are good to 2 10^-9 and 3 10^-8 there.
// ---------------------------------------------------------------------------
struct RopeTableArgs {
  unsigned long long turn[kMaxRot / 2];  // theta_c / (2 pi) * 2^64
  float* cos;
  float* sin;
  long long n;       // vectors of four columns: rows * half / 4
  int half;          // columns (a multiple of 8)
  unsigned first;    // position of the first row
  float amplitude;
};

// Sine and cosine of frac / 2^32 turns.
__device__ __forceinline__ void sincos_turn(uint32_t frac, float& sn, float& cs) {
  const uint32_t q = (frac + 0x20000000u) >> 30;                       // nearest quarter
  const float x = static_cast<float>(static_cast<int>(frac - (q << 30))) * 1.4629180792671596e-9f;   // 2 pi / 2^32
  const float y = x * x;
  const float s = fmaf(x * y, fmaf(y, fmaf(y, fmaf(y, 1.0f / 362880.0f, -1.0f / 5040.0f), 1.0f / 120.0f), -1.0f / 6.0f), x);
  const float c = fmaf(y, fmaf(y, fmaf(y, fmaf(y, 1.0f / 40320.0f, -1.0f / 720.0f), 1.0f / 24.0f), -0.5f), 1.0f);
  const float a = q & 1u ? c : s, b = q & 1u ? s : c;
  sn = __uint_as_float(__float_as_uint(a) ^ ((q & 2u) << 30));
  cs = __uint_as_float(__float_as_uint(b) ^ (((q + 1u) & 2u) << 30));
}

__global__ void __launch_bounds__(kTableThreads) rope_table_kernel(const __grid_constant__ RopeTableArgs a) {
  __shared__ unsigned long long turn[kMaxRot / 2];
  if (threadIdx.x < kMaxRot / 2) turn[threadIdx.x] = a.turn[threadIdx.x];
  __syncthreads();
  const int q = a.half / 4;
  for (long long i = static_cast<long long>(blockIdx.x) * kTableThreads + threadIdx.x; i < a.n;
       i += static_cast<long long>(gridDim.x) * kTableThreads) {
    // rows < 2^31 and q <= 16: the quotient by a 64-bit division only where i is that large
    const unsigned row = i < UINT32_MAX ? static_cast<unsigned>(i) / q : static_cast<unsigned>(i / q);
    const int c = static_cast<int>(i - static_cast<long long>(row) * q) * 4;
    const unsigned long long t = a.first + row;
    float cs[4], sn[4];
#pragma unroll
    for (int j = 0; j < 4; ++j) {
      sincos_turn(static_cast<uint32_t>((turn[c + j] * t) >> 32), sn[j], cs[j]);
      cs[j] *= a.amplitude;
      sn[j] *= a.amplitude;
    }
    reinterpret_cast<float4*>(a.cos)[i] = make_float4(cs[0], cs[1], cs[2], cs[3]);
    reinterpret_cast<float4*>(a.sin)[i] = make_float4(sn[0], sn[1], sn[2], sn[3]);
  }
}

// ---------------------------------------------------------------------------
// Rotation of q and k.
//
// A thread owns one unit of channels of one position: the 16 bytes of
// channels c.. and their partners (split-half), 16 bytes that hold whole
// pairs (interleaved), or 16 bytes past the turned part (copied when the
// output is another tensor). It reads the unit's cosines and sines once and
// walks over some of the position's heads with them, a batch of heads' loads
// in flight at a time (six 16-byte loads where a unit is two pieces, four where
// it is one: 24 more registers for eight cost 9 % on a layer of 16 x 2048
// positions). Every element is read and written by the same thread,
// reads first, so the rotation also runs in place. Bound by memory: 16 x 2048
// positions, 6 + 3 heads of 128, bf16: 25.0 us, 6.1 TB/s, 90 % of the measured
// copy rate; 2 x 16384, 16 + 4 heads, fp32: 101 us, 98 %.
// ---------------------------------------------------------------------------
constexpr int kRopeBatch[2] = {3, 4};    // split-half, interleaved

struct RopeArgs {
  const elem_t* q; const elem_t* k;   // [N, Hq, d], [N, Hkv, d] or NULL
  elem_t* qo; elem_t* ko;
  const float* cos; const float* sin; // [rows][rot / 2]
  const int32_t* pos;                 // [N] or NULL: position n % T
  long long N;                        // B * T
  int T, rows, d, rot;
  int Hq, Hkv;                        // 0 for a tensor that is not given
  int turned, units;                  // units of a position: turned, and all
  int heads;                          // heads of one thread
  float sgn;                          // 1, or -1 for the transposed rotation
  bool fresh;                         // rows that are not turned become zero
  uint32_t* status;                   // or NULL
};

template <bool INTER>
__global__ void __launch_bounds__(kRopeThreads) rope_kernel(const __grid_constant__ RopeArgs a) {
  constexpr int EPL = 16 / static_cast<int>(sizeof(elem_t)), kBatch = kRopeBatch[INTER];
  const long long id = static_cast<long long>(blockIdx.x) * kRopeThreads + threadIdx.x;
  const long long n = id / a.units;
  if (n >= a.N) return;
  const int u = static_cast<int>(id - n * a.units);
  const int p = a.pos ? a.pos[n] : static_cast<int>(n % a.T);
  const int half = a.rot / 2;
  const bool turn = u < a.turned;
  const int c = turn ? u * EPL : a.rot + (u - a.turned) * EPL;
  const int H = a.Hq + a.Hkv;
  const int h0 = blockIdx.y * a.heads, h1 = h0 + a.heads < H ? h0 + a.heads : H;
  if (p < 0 || p >= a.rows) {   // left as it was, or zero, and reported
    if (u == 0 && blockIdx.y == 0 && a.status) atomicOr(a.status, DEV_ERR_BOUNDS);
    if (a.fresh) {
#pragma unroll 1
      for (int h = h0; h < h1; ++h) {
        elem_t* out = (h < a.Hq ? a.qo + (n * a.Hq + h) * a.d : a.ko + (n * a.Hkv + (h - a.Hq)) * a.d) + c;
        st16(out, make_uint4(0u, 0u, 0u, 0u));
        if (!INTER && turn) st16(out + half, make_uint4(0u, 0u, 0u, 0u));
      }
    }
    return;
  }
  constexpr int NP = INTER ? EPL / 2 : EPL;   // pairs of the unit
  float cs[NP], sn[NP];
  if (turn) {
    const long long at = static_cast<long long>(p) * half + (INTER ? c / 2 : c);
    if constexpr (NP == 2) {
      const float2 x = *reinterpret_cast<const float2*>(a.cos + at), y = *reinterpret_cast<const float2*>(a.sin + at);
      cs[0] = x.x; cs[1] = x.y; sn[0] = y.x; sn[1] = y.y;
    } else {
      ldf<NP>(a.cos + at, cs);
      ldf<NP>(a.sin + at, sn);
    }
#pragma unroll
    for (int i = 0; i < NP; ++i) sn[i] *= a.sgn;
  }
  for (int h = h0; h < h1; h += kBatch) {
    uint4 x[kBatch], y[kBatch];
    elem_t* out[kBatch];
#pragma unroll
    for (int i = 0; i < kBatch; ++i) {
      if (h + i >= h1) continue;
      const bool is_q = h + i < a.Hq;
      const long long off = is_q ? (n * a.Hq + h + i) * a.d + c : (n * a.Hkv + (h + i - a.Hq)) * a.d + c;
      const elem_t* src = (is_q ? a.q : a.k) + off;
      out[i] = (is_q ? a.qo : a.ko) + off;
      x[i] = ld16(src);
      if (!INTER && turn) y[i] = ld16(src + half);
    }
#pragma unroll
    for (int i = 0; i < kBatch; ++i) {
      if (h + i >= h1) continue;
      if (!turn) {
        st16(out[i], x[i]);
        continue;
      }
      float f[EPL], g[EPL];
      unpack16(x[i], f);
      if constexpr (INTER) {
#pragma unroll
        for (int j = 0; j < NP; ++j) {
          g[2 * j] = fmaf(f[2 * j], cs[j], f[2 * j + 1] * sn[j]);
          g[2 * j + 1] = fmaf(f[2 * j + 1], cs[j], -f[2 * j] * sn[j]);
        }
        st16(out[i], pack16(g));
      } else {
        unpack16(y[i], g);
        float lo[EPL], hi[EPL];
#pragma unroll
        for (int j = 0; j < EPL; ++j) {
          lo[j] = fmaf(f[j], cs[j], g[j] * sn[j]);
          hi[j] = fmaf(g[j], cs[j], -f[j] * sn[j]);
        }
        st16(out[i], pack16(lo));
        st16(out[i] + half, pack16(hi));
      }
    }
  }
}

// Rotation of one row held by the LPR lanes of a RowMap<D> (EPL channels
// each), in either layout, of the first rot channels; cos, sin point at the
// position's row of the tables. Every lane of the warp calls it (shuffles).
template <int D>
__device__ __forceinline__ void rotate_lanes(float (&x)[RowMap<D>::EPL], const float* cos, const float* sin, int rot,
                                             int interleaved, bool valid) {
  using M = RowMap<D>;
  constexpr int EPL = M::EPL;
  const int lane = threadIdx.x & 31, cl = lane % M::LPR, c0 = cl * EPL, half = rot / 2;
  if (interleaved) {
    if (valid && c0 < rot) {
#pragma unroll
      for (int j = 0; j < EPL / 2; ++j) {
        const float c = cos[c0 / 2 + j], s = sin[c0 / 2 + j], a = x[2 * j], b = x[2 * j + 1];
        x[2 * j] = fmaf(a, c, b * s);
        x[2 * j + 1] = fmaf(b, c, -a * s);
      }
    }
    return;
  }
  // rot / 2 is a multiple of 8 channels, so partners sit whole lanes apart
  const int shift = half / EPL;
  const int from = c0 < half ? lane + shift : (c0 < rot ? lane - shift : lane);
  float p[EPL];
#pragma unroll
  for (int i = 0; i < EPL; ++i) p[i] = __shfl_sync(0xffffffffu, x[i], from);
  if (valid && c0 < rot) {
    float cs[EPL], sn[EPL];
    const int c = c0 < half ? c0 : c0 - half;
    ldf<EPL>(cos + c, cs);
    ldf<EPL>(sin + c, sn);
    const float sg = c0 < half ? 1.f : -1.f;
#pragma unroll
    for (int i = 0; i < EPL; ++i) x[i] = fmaf(x[i], cs[i], sg * p[i] * sn[i]);
  }
}

}  // namespace swa
