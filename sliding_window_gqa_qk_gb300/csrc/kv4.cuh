// The paged cache of keys and values held in 4 bits: its layout, the plan of
// a serving step (pages, slots, positions), the append that rotates, norms
// and quantises new rows into it, and the read that turns rows back.
//
// Layout: [n_pages][Hkv][page / 16] tiles of 18 d bytes; a tile holds 16
// consecutive tokens of one kv head:
//   8 d   keys, token by token, d / 2 bytes each
//   8 d   values, token pair by token pair, d bytes each
//   d     16 x d / 64 pairs (s, z) of the keys, bf16
//   d     16 x d / 64 pairs (s, z) of the values, bf16
// A stored number n = 0..15 of a 64-channel group stands for s (n - 8) + z.
// The order of the numbers inside a row is the one in which the attention's
// matrix instructions take them, so that a lane's 16 bytes of a row are
// exactly its operand registers (kv4_attn.cuh):
//   keys    position (j, g, i) of a token's row: channel 64 g + 16 j + i,
//           j = 0..3, i = 0..15;
//   values  position (r, g, u, token of the pair, i) of a pair's row: channel
//           64 g + 8 r + 4 u + i, r = 0..7, u = 0..1, i = 0..3. One token
//           owns 16-bit pieces, so appends of neighbours never share a store.
// Low nibble first throughout.
#pragma once

#include "common.cuh"
#include "rope.cuh"
#include "rowwise.cuh"

namespace swa {
namespace kv4 {

constexpr int kTile = 16;    // tokens of a tile

__host__ __device__ constexpr int tile_bytes(int d) { return 18 * d; }

// n / d for n < 2^31 by a multiplication: with l = ceil(log2 d) and
// m = ceil(2^(31 + l) / d), n m 2^-(31 + l) exceeds n / d by less than 1 / d.
struct FastDiv {
  uint32_t d, mul;
  int shift;
  __device__ __forceinline__ uint32_t div(uint32_t n) const { return d == 1 ? n : __umulhi(n, mul) >> shift; }
};
inline FastDiv fast_div(uint32_t d) {
  FastDiv f{d, 0, 0};
  int l = 0;
  while ((1ull << l) < d) ++l;
  if (l > 0) {
    f.mul = static_cast<uint32_t>(((1ull << (31 + l)) + d - 1) / d);
    f.shift = l - 1;
  }
  return f;
}

struct Cache {
  uint8_t* data;
  int n_pages, page, Hkv;
  FastDiv per_page;      // tiles of a page and kv head; there are fewer than 2^31 such tiles
};

// The tile of `slot` (page * page size + offset) of kv head h.
template <int D>
__device__ __forceinline__ uint8_t* tile_of(const Cache& c, long long slot, int h) {
  const uint32_t t = static_cast<uint32_t>(slot / kTile);
  const uint32_t pg = c.per_page.div(t);
  const long long at = (static_cast<long long>(pg) * c.Hkv + h) * c.per_page.d + (t - pg * c.per_page.d);
  return c.data + at * tile_bytes(D);
}

// max / min that keep a NaN (fmaxf and fminf drop it).
__device__ __forceinline__ float max_nan(float a, float b) {
  float r;
  asm("max.NaN.f32 %0, %1, %2;" : "=f"(r) : "f"(a), "f"(b));
  return r;
}
__device__ __forceinline__ float max_nan(float a, float b, float c) {
  float r;
  asm("max.NaN.f32 %0, %1, %2, %3;" : "=f"(r) : "f"(a), "f"(b), "f"(c));
  return r;
}
__device__ __forceinline__ float min_nan(float a, float b, float c) {
  float r;
  asm("min.NaN.f32 %0, %1, %2, %3;" : "=f"(r) : "f"(a), "f"(b), "f"(c));
  return r;
}
__device__ __forceinline__ float min_nan(float a, float b) {
  float r;
  asm("min.NaN.f32 %0, %1, %2;" : "=f"(r) : "f"(a), "f"(b));
  return r;
}

// ---------------------------------------------------------------------------
// Quantisation of a row held by RowMap<D> lanes. Per group of 64 channels:
//   s = bf16((max - min) / 15),  z = bf16(min + 8 s),
//   n = clamp(floor((x - z) / s + 8 + 1/2), 0, 15),   n = 8 where s = 0.
// s and z are bf16 (not fp16): values are unnormalised and may pass fp16's
// range; z is the group's centre rather than its minimum, which makes it
// small and its rounding finer. A group that holds an infinity or a NaN, or
// whose span overflows, gets s = z = NaN, so that it reads back as NaN.
//
// A border between two numbers, or between two bf16 steps, splits values that
// fp32 arithmetic cannot always tell apart. Two cases:
//   - Values of plain layers enter exactly (bf16), and many sit on a border (one
//     Gaussian value in 450): x, z and s are short numbers. The number found with an approximate
//     reciprocal is settled by the remainder x - z - n s, which fma gives
//     exactly (kExact). (x - z itself rounds where x is far smaller than z; that
//     decides only for a border at 0 and an x within 2^-25 z of it, which goes
//     up from either side, both numbers being as near.)
//   - Keys, and values with an embedding, are results of fp32 arithmetic. A
//     row with an entry or a step closer to a border than that arithmetic is
//     good for is done again in fp64: the numbers a row is held as then
//     follow the formula, not the rounding of a kernel. A centre close to a
//     border of its own counts only where the other rounding would change a
//     number (most centres lie near 0, where bf16's steps are fine); else it
//     may stay one rounding off, by less than 2^-8 of itself. About one row
//     in 500 takes that way.
// ---------------------------------------------------------------------------
// Steps below 1e-36 (whose reciprocal nears fp32's end) count as 0.
constexpr float kFlatStep = 1e-36f;
struct Group {
  float s, z;
};
__device__ __forceinline__ float to_bf16(float x) { return __bfloat162float(__float2bfloat16_rn(x)); }
__device__ __forceinline__ float rcp_approx(float x) {
  float r;
  asm("rcp.approx.ftz.f32 %0, %1;" : "=f"(r) : "f"(x));
  return r;
}

// Distance of x from the nearest border between two bf16 roundings, given
// its rounding y.
__device__ __forceinline__ float bf16_margin(float x, float y) {
  return __uint_as_float(__float_as_uint(x) & 0x7F800000u) * 0.00390625f - fabsf(x - y);   // half a step: 2^(e - 8)
}

// x / 15, correctly rounded where the quotient is a normal number (compared with
// the division over every fraction, which a power of two does not change): the
// product with 1 / 15 and one correction by its remainder.
__device__ __forceinline__ float over_15(float x) {
  const float q = x * (1.0f / 15.0f);
  return fmaf(fmaf(-15.0f, q, x), 1.0f / 15.0f, q);
}

// step and centre. Unless kExact, err is what the entries may be off by, as a
// multiple of the row's largest: slack becomes that, plus a step of the
// centre's where it may round either way, and near is set where the step may.
template <int D, bool kExact>
__device__ __forceinline__ Group group_scale(const float (&x)[RowMap<D>::EPL], float err, float& slack, bool& near) {
  constexpr int EPL = RowMap<D>::EPL;
  constexpr int GL = 64 / EPL;   // lanes of a group
  float lo = min_nan(x[0], x[1]), hi = max_nan(x[0], x[1]);
#pragma unroll
  for (int i = 2; i < EPL; i += 2) {
    lo = min_nan(lo, x[i], x[i + 1]);
    hi = max_nan(hi, x[i], x[i + 1]);
  }
#pragma unroll
  for (int o = GL / 2; o > 0; o >>= 1) {
    lo = min_nan(lo, __shfl_xor_sync(0xffffffffu, lo, o));
    hi = max_nan(hi, __shfl_xor_sync(0xffffffffu, hi, o));
  }
  Group g;
  const float s = over_15(hi - lo);
  g.s = to_bf16(s);
  if (g.s < kFlatStep) g.s = 0.0f;
  const float z = fmaf(8.0f, g.s, lo);
  g.z = to_bf16(z);
  if (!isfinite(g.s) || !isfinite(g.z)) g.s = g.z = __int_as_float(0x7fffffff);
  if (!kExact) {
    float top = fmaxf(fabsf(lo), fabsf(hi));
    if (D == 128) top = fmaxf(top, __shfl_xor_sync(0xffffffffu, top, GL));   // a rotated pair may span the groups
    slack = err * top;
    near = bf16_margin(s, g.s) <= 0.2f * slack;      // both ends over 15, and a rounding
    if (bf16_margin(z, g.z) <= 1.25f * slack) slack += __uint_as_float(__float_as_uint(z) & 0x7F800000u) * 0.0078125f;
  }
  return g;
}

// The lane's EPL numbers, four bits each, lowest channel lowest. A saturating
// multiply-add keeps (x - z) / (15 s) + 8 / 15 within [0, 1]; 15 times that
// plus 1.5 * 2^23 is rounded to an integer, which sits in the low bits, and the
// words add up as whole numbers. kExact: rounded a little low, so that only
// a remainder of half a step or more is left to settle, upwards. Otherwise gap
// becomes the least distance of an entry from a border.
template <int D, bool kExact>
__device__ __forceinline__ uint32_t quantise_lane(const float (&x)[RowMap<D>::EPL], const Group& g, float& gap) {
  constexpr int EPL = RowMap<D>::EPL;
  constexpr float kRound = 12582912.0f, kLow = kExact ? 1.0f / 4096.0f : 0.0f;
  const bool flat = !(g.s > 0.0f);       // step 0, or NaN
  const float inv = rcp_approx(g.s) * (1.0f / 15.0f), half = 0.5f * g.s;
  const float off = fmaf(-g.z, inv, (8.0f - kLow) / 15.0f);
  uint32_t w = 0, ones = 0;
  float far = 0.0f;                      // largest distance from a number, in steps
#pragma unroll
  for (int i = 0; i < EPL; ++i) {
    float n = kExact ? __saturatef(fmaf(x[i] - g.z, inv, (8.0f - kLow) / 15.0f)) : __saturatef(fmaf(x[i], inv, off));
    float b = fmaf(n, 15.0f, kRound);
    if (kExact) {
      const float r = fmaf((kRound + 8.0f) - b, g.s, x[i] - g.z);      // x - z - (n - 8) s
      b = fminf(b + (r >= half ? 1.0f : 0.0f), kRound + 15.0f);
    } else {
      far = fmaxf(far, fabsf(fmaf(n, 15.0f, kRound - b)));
    }
    w += __float_as_uint(b) << (4 * i);
    ones += __float_as_uint(kRound) << (4 * i);
  }
  if (!kExact) gap = flat ? INFINITY : (0.5f - far) * g.s;
  return flat ? 0x88888888u >> (32 - 4 * EPL) : w - ones;
}

// The same in fp64, of a group that is finite: its comparisons would drop a NaN
// (see settled()). Every lane of the warp calls it.
template <int D>
__device__ __forceinline__ uint32_t quantise_f64(const double (&x)[RowMap<D>::EPL], Group& g) {
  constexpr int EPL = RowMap<D>::EPL;
  constexpr int GL = 64 / EPL;
  double lo = x[0], hi = x[0];
#pragma unroll
  for (int i = 1; i < EPL; ++i) {
    lo = x[i] < lo ? x[i] : lo;
    hi = x[i] > hi ? x[i] : hi;
  }
#pragma unroll
  for (int o = GL / 2; o > 0; o >>= 1) {
    const double a = __shfl_xor_sync(0xffffffffu, lo, o), b = __shfl_xor_sync(0xffffffffu, hi, o);
    lo = a < lo ? a : lo;
    hi = b > hi ? b : hi;
  }
  g.s = to_bf16(static_cast<float>((hi - lo) * (1.0 / 15.0)));
  if (g.s < kFlatStep) g.s = 0.0f;
  g.z = to_bf16(static_cast<float>(fma(8.0, static_cast<double>(g.s), lo)));
  const bool flat = !(g.s > 0.0f);
  const float inv = flat ? 0.0f : rcp_approx(g.s);
  const double half = 0.5 * static_cast<double>(g.s);
  uint32_t w = 0;
#pragma unroll
  for (int i = 0; i < EPL; ++i) {
    const double v = x[i] - static_cast<double>(g.z);
    float n = rintf(static_cast<float>(v) * inv);
    const double r = fma(-static_cast<double>(n), static_cast<double>(g.s), v);
    n += r >= half ? 1.0f : 0.0f;
    n -= r < -half ? 1.0f : 0.0f;
    n = fminf(fmaxf(n, -8.0f), 7.0f);
    w |= (flat ? 8u : static_cast<uint32_t>(static_cast<int>(n) + 8)) << (4 * i);
  }
  return w;
}

// ---------------------------------------------------------------------------
// Append
// ---------------------------------------------------------------------------
struct AppendArgs {
  Cache c;
  uint32_t N;                          // tokens of this launch: N * Hkv < 2^31
  FastDiv heads, seq;                  // by Hkv, by T
  uint32_t t0;                         // position of the launch's first token where pos is NULL
  float eps, ve_scale;
  int vocab;
  const elem_t* k; const elem_t* v;    // [N, Hkv, D]
  const float* gk;
  const elem_t* ve; const int32_t* tok; const float* gate;
  const elem_t* gx; long long gx_stride; const float* gw; int gch;   // learned gate, gw NULL: none
  const float* rcos; const float* rsin; int rows, rot, interleaved;  // rcos NULL: none
  const int32_t* pos; const int64_t* slot;
  uint32_t* status;                    // or NULL
};

// Whether a lane takes the fp64 result of its row: where the row has a close
// entry, unless fp32 found the lane's group not finite. The row's other group
// may be what was close.
__device__ __forceinline__ bool settled(unsigned close, const Group& fp32) { return close != 0 && !isnan(fp32.s); }

// What fp32 arithmetic may leave an entry off by, in units of 2^-24 of the
// row's largest entry. Rotation, norm and gain, in fp32 and fp64 on 200,000
// Gaussian rows: 0.41 rms; more than 3 in one row of 54, more than 4 in one of
// 2400, 4.7 at most. At 4, one row in 550 goes the slow way.
constexpr float kKeyErr = 4.0f * 5.9604645e-8f;
constexpr float kMixErr = 4.0f * 5.9604645e-8f;
constexpr int kAppendWarps = 4;      // a small block: one slow row holds up few others

// 1 / sqrt(x), x >= 0 of any size: an even power of two is taken out, and one
// Newton step from the fp32 root of the rest squares its 2^-22, which is enough
// here. Infinity gives 2^-512, which keeps an infinity one and leaves nothing of
// a number.
__device__ __forceinline__ double rsqrt_f64(double x) {
  const int hi = __double2hiint(x), k = ((hi >> 20) - 1023) & ~1;
  const double m = __hiloint2double(hi - k * (1 << 20), __double2loint(x));   // within [1, 4)
  const double r0 = rsqrtf(static_cast<float>(m));
  const double r = r0 * fma(-0.5 * m * r0, r0, 1.5) * __hiloint2double((1023 - k / 2) * (1 << 20), 0);
  return x > 0.0 ? r : static_cast<double>(rsqrtf(static_cast<float>(x)));     // 0 and NaN
}

// The rotated and normed key row in fp64 (row: its index, p its position),
// quantised; every lane of the warp calls it.
template <int D>
__device__ __noinline__ uint32_t key_f64(const AppendArgs& a, uint32_t row, int p, bool on, Group* out) {
  using M = RowMap<D>;
  constexpr int EPL = M::EPL;
  const int cl = (threadIdx.x & 31) % M::LPR, c0 = cl * EPL, half = a.rot / 2;
  const elem_t* k = a.k + static_cast<long long>(on ? row : 0) * D;
  double x[EPL], ss = 0.0;
#pragma unroll
  for (int i = 0; i < EPL; ++i) {
    const int c = c0 + i;
    x[i] = on ? to_f32(k[c]) : 0.0;
    if (a.rcos != nullptr && c < a.rot && on) {
      const int col = a.interleaved ? c / 2 : (c < half ? c : c - half);
      const int to = a.interleaved ? c ^ 1 : (c < half ? c + half : c - half);
      const bool first = a.interleaved ? (c & 1) == 0 : c < half;
      const long long at = static_cast<long long>(p) * half + col;
      const double o = static_cast<double>(to_f32(k[to])) * a.rsin[at];
      x[i] = fma(x[i], static_cast<double>(a.rcos[at]), first ? o : -o);
    }
    ss = fma(x[i], x[i], ss);
  }
#pragma unroll
  for (int o = M::LPR / 2; o > 0; o >>= 1) ss += __shfl_xor_sync(0xffffffffu, ss, o);
  const double rstd = rsqrt_f64(fma(ss, 1.0 / D, static_cast<double>(a.eps)));
#pragma unroll
  for (int i = 0; i < EPL; ++i) x[i] = x[i] * rstd * (a.gk ? a.gk[c0 + i] : 1.0f);
  Group g;
  const uint32_t w = quantise_f64<D>(x, g);
  *out = g;
  return w;
}
// A value row with its embedding in fp64, from its fp32 parts.
template <int D>
__device__ __noinline__ uint32_t mix_f64(const AppendArgs& a, uint32_t row, const elem_t* ve, float gate, bool on, Group* out) {
  constexpr int EPL = RowMap<D>::EPL;
  const int c0 = ((threadIdx.x & 31) % RowMap<D>::LPR) * EPL;
  double x[EPL];
  const double f = static_cast<double>(a.ve_scale) * gate;
#pragma unroll
  for (int i = 0; i < EPL; ++i) {
    x[i] = on ? to_f32(a.v[static_cast<long long>(row) * D + c0 + i]) : 0.0;
    if (on && ve != nullptr) x[i] = fma(f, static_cast<double>(to_f32(ve[c0 + i])), x[i]);
  }
  Group g;
  const uint32_t w = quantise_f64<D>(x, g);
  *out = g;
  return w;
}

// Lanes as in the other row-wise kernels: LPR lanes hold one row of D
// channels, 16 bytes each, and a warp works on RPI rows (token, head) at a
// time, key and value together. MIX: a value embedding.
// It should be bound by memory (4 D bytes in, 18 D / 16 out per row) and is
// bound by instructions, about 35 per channel and lane: 16384 tokens of 3 heads of
// 128 take 24.8 us, 1.3 TB/s, of which the steps and centres (computed by all
// lanes of a group) are 5.5 us, rotation 2.5, the keys' numbers 2.3, stores 2.1,
// fp64 rows 0.7. 64 single tokens take 3.0 us, a chain of dependent loads.
// Blocks of four warps, not persistent, against eight, eight per SM: 32 us.
template <int D, bool MIX>
__global__ void __launch_bounds__(kAppendWarps * 32) append_kernel(const __grid_constant__ AppendArgs a) {
  using M = RowMap<D>;
  constexpr int EPL = M::EPL, NG = D / 64;
  constexpr bool kPlainExact = !MIX && sizeof(elem_t) == 2;    // fp32 values: x - z may round
  const int lane = threadIdx.x & 31, cl = lane % M::LPR, c0 = cl * EPL;
  const uint32_t Hkv = a.heads.d, rows = a.N * Hkv;
  const long long cap = static_cast<long long>(a.c.n_pages) * a.c.page;
  const unsigned rows_mask = M::LPR == 32 ? 0xffffffffu : ((1u << M::LPR) - 1u) << (lane / M::LPR * M::LPR);
  float gk[EPL];
#pragma unroll
  for (int i = 0; i < EPL; ++i) gk[i] = a.gk ? a.gk[c0 + i] : 1.0f;
  for (uint32_t r0 = static_cast<uint32_t>(grid_warp()) * M::RPI; r0 < rows;
       r0 += static_cast<uint32_t>(grid_warps()) * M::RPI) {
    const uint32_t row = r0 + lane / M::LPR;
    bool on = row < rows;
    const uint32_t n = on ? a.heads.div(row) : 0;
    const int h = static_cast<int>(on ? row - n * Hkv : 0);
    const long long slot = on ? a.slot[n] : -1;
    uint4 kr = make_uint4(0u, 0u, 0u, 0u), vr = kr, er = kr;
    if (on) {
      kr = ld16(a.k + static_cast<long long>(row) * D + c0);
      vr = ld16(a.v + static_cast<long long>(row) * D + c0);
    }
    int p = 0;
    uint32_t bad = 0;
    if (on && a.rcos != nullptr) {
      const uint32_t t = a.t0 + n;
      p = a.pos ? a.pos[n] : static_cast<int>(t - a.seq.div(t) * a.seq.d);
      if (slot >= 0 && (p < 0 || p >= a.rows)) bad = DEV_ERR_BOUNDS;
    }
    if (on && slot != -1 && (slot < 0 || slot >= cap)) bad = DEV_ERR_BOUNDS;
    on = on && slot >= 0 && !bad;
    const elem_t* ve = nullptr;
    float gate = 1.0f;
    if (MIX) {
      const int tok = on ? a.tok[n] : 0;
      if (on && tok >= 0 && tok < a.vocab) {
        ve = a.ve + (static_cast<long long>(tok) * Hkv + h) * D;
        er = ld16(ve + c0);
      } else if (on) {
        bad |= DEV_ERR_TOKEN;
      }
      if (a.gw != nullptr) {
        float z = 0.f;
        if (on) {
          const elem_t* xr = a.gx + n * a.gx_stride;
          for (int c = cl; c < a.gch; c += M::LPR) z = fmaf(a.gw[h * a.gch + c], to_f32(xr[c]), z);
        }
        gate = 2.0f / (1.0f + expf(-row_sum<M::LPR>(z)));
      } else if (on && a.gate != nullptr) {
        gate = a.gate[static_cast<long long>(n) * Hkv + h];
      }
    }
    // key: rotation, RMSNorm
    float x[EPL];
    unpack16(kr, x);
    if (a.rcos != nullptr) {
      const long long at = on ? static_cast<long long>(p) * (a.rot / 2) : 0;
      rotate_lanes<D>(x, a.rcos + at, a.rsin + at, a.rot, a.interleaved, on);
    }
    float ss = 0.f;
#pragma unroll
    for (int i = 0; i < EPL; ++i) ss = fmaf(x[i], x[i], ss);
    ss = row_sum<M::LPR>(ss);
    // A mean square past fp32 makes every entry 0 (or NaN), whose step of 0 lies
    // on a border: such a row is done in fp64.
    const float rstd = rsqrtf(ss / D + a.eps);
#pragma unroll
    for (int i = 0; i < EPL; ++i) x[i] = x[i] * rstd * gk[i];
    float slack = 0.f, gap = 0.f;
    bool near = false;
    Group sk = group_scale<D, false>(x, kKeyErr, slack, near);
    uint32_t wk = quantise_lane<D, false>(x, sk, gap);
    unsigned close = __ballot_sync(0xffffffffu, on && (near || gap <= slack));
    if (close) {
      Group s2;
      const uint32_t w2 = key_f64<D>(a, row, p, on, &s2);
      if (settled(close & rows_mask, sk)) {
        wk = w2;
        sk = s2;
      }
    }
    // value, with its embedding
    unpack16(vr, x);
    if (MIX) {
      float e[EPL];
      unpack16(er, e);
      const float f = a.ve_scale * gate;
#pragma unroll
      for (int i = 0; i < EPL; ++i) x[i] = fmaf(f, e[i], x[i]);
    }
    Group sv = group_scale<D, kPlainExact>(x, kMixErr, slack, near);
    uint32_t wv = quantise_lane<D, kPlainExact>(x, sv, gap);
    if (!kPlainExact) {
      close = __ballot_sync(0xffffffffu, on && (near || gap <= slack));
      if (close) {
        Group s2;
        const uint32_t w2 = mix_f64<D>(a, row, ve, gate, on, &s2);
        if (settled(close & rows_mask, sv)) {
          wv = w2;
          sv = s2;
        }
      }
    }
    if (bad && cl == 0 && a.status) atomicOr(a.status, bad);
    if (!on) continue;
    uint8_t* tile = tile_of<D>(a.c, slot, h);
    const int t = static_cast<int>(slot) & (kTile - 1);
    const int g = c0 / 64, x0 = c0 % 64;
    // keys: nibble ((x / 16) NG + g) 16 + x % 16 of the row
    const int nk = ((x0 / 16) * NG + g) * 16 + x0 % 16;
    uint8_t* krow = tile + t * (D / 2);
    // values: 16-bit piece (((x / 8) NG + g) 2 + (x / 4) % 2) 2 + token
    uint16_t* vrow = reinterpret_cast<uint16_t*>(tile + 8 * D + (t / 2) * D);
    const int pv = (((x0 / 8) * NG + g) * 2 + (x0 / 4) % 2) * 2 + (t & 1);
    if constexpr (EPL == 8) {
      reinterpret_cast<uint32_t*>(krow)[nk / 8] = wk;
      vrow[pv] = static_cast<uint16_t>(wv);
      vrow[pv + 2] = static_cast<uint16_t>(wv >> 16);
    } else {
      reinterpret_cast<uint16_t*>(krow)[nk / 4] = static_cast<uint16_t>(wk);
      vrow[pv] = static_cast<uint16_t>(wv);
    }
    if (x0 == 0) {
      uint32_t* sc = reinterpret_cast<uint32_t*>(tile + 16 * D);
      sc[t * NG + g] = pack_bf16x2(sk.s, sk.z);
      sc[(kTile + t) * NG + g] = pack_bf16x2(sv.s, sv.z);
    }
  }
}

// ---------------------------------------------------------------------------
// Read: the rows of slots as the values they stand for.
// ---------------------------------------------------------------------------
struct ReadArgs {
  Cache c;
  uint32_t N;                // tokens of this launch: N * Hkv < 2^31
  FastDiv heads;             // by Hkv
  const int64_t* slot;
  elem_t* k; elem_t* v;      // [N, Hkv, D]
  uint32_t* status;          // or NULL
};

// Bound by the rows written: 16384 tokens of 3 heads of 128 take 6.3 us, 5.1
// TB/s read and written, 75 % of the measured copy rate.
template <int D>
__global__ void __launch_bounds__(kRowWarps * 32) read_kernel(const __grid_constant__ ReadArgs a) {
  using M = RowMap<D>;
  constexpr int EPL = M::EPL, NG = D / 64;
  const int lane = threadIdx.x & 31, cl = lane % M::LPR, c0 = cl * EPL;
  const uint32_t Hkv = a.heads.d, rows = a.N * Hkv;
  const long long cap = static_cast<long long>(a.c.n_pages) * a.c.page;
  const int g = c0 / 64, x0 = c0 % 64;
  const int nk = ((x0 / 16) * NG + g) * 16 + x0 % 16;
  for (uint32_t row = static_cast<uint32_t>(grid_warp()) * M::RPI + lane / M::LPR; row < rows;
       row += static_cast<uint32_t>(grid_warps()) * M::RPI) {
    const uint32_t n = a.heads.div(row);
    const int h = static_cast<int>(row - n * Hkv);
    const long long slot = a.slot[n];
    float x[EPL] = {}, y[EPL] = {};
    if (slot >= 0 && slot < cap) {
      const uint8_t* tile = tile_of<D>(a.c, slot, h);
      const int t = static_cast<int>(slot) & (kTile - 1);
      const uint8_t* krow = tile + t * (D / 2);
      const uint16_t* vrow = reinterpret_cast<const uint16_t*>(tile + 8 * D + (t / 2) * D);
      const int pv = (((x0 / 8) * NG + g) * 2 + (x0 / 4) % 2) * 2 + (t & 1);
      uint32_t wk, wv;
      if constexpr (EPL == 8) {
        wk = reinterpret_cast<const uint32_t*>(krow)[nk / 8];
        wv = vrow[pv] | static_cast<uint32_t>(vrow[pv + 2]) << 16;
      } else {
        wk = reinterpret_cast<const uint16_t*>(krow)[nk / 4];
        wv = vrow[pv];
      }
      const uint32_t* sc = reinterpret_cast<const uint32_t*>(tile + 16 * D);
      const uint32_t a0 = sc[t * NG + g], b0 = sc[(kTile + t) * NG + g];
      const float ks = __uint_as_float(a0 << 16), kz = __uint_as_float(a0 & 0xFFFF0000u);
      const float vs = __uint_as_float(b0 << 16), vz = __uint_as_float(b0 & 0xFFFF0000u);
#pragma unroll
      for (int i = 0; i < EPL; ++i) {
        x[i] = fmaf(ks, static_cast<float>(static_cast<int>((wk >> (4 * i)) & 15u) - 8), kz);
        y[i] = fmaf(vs, static_cast<float>(static_cast<int>((wv >> (4 * i)) & 15u) - 8), vz);
      }
    } else if (slot != -1 && cl == 0 && a.status) {
      atomicOr(a.status, DEV_ERR_BOUNDS);
    }
    st16(a.k + static_cast<long long>(row) * D + c0, pack16(x));
    st16(a.v + static_cast<long long>(row) * D + c0, pack16(y));
  }
}

// ---------------------------------------------------------------------------
// Plan of a step: request b holds lens[b] tokens and gets new_lens[b] more.
//   held_b = ceil(lens_b / P), want_b = ceil((lens_b + new_b) / P) - held_b,
//   off_b = sum of the wants before b; its new pages are
//   free[head + off_b ..], its tokens' slots follow.
// Every block does the whole scan itself (a few thousand requests at most,
// two integers each, from L2) and keeps it in shared memory, so one launch
// serves every token and no block waits on another. Latency bounds it: 64
// requests of one token 5.3 us, 1000 requests of 104,000 tokens 7.1 us (their
// bytes would take 0.3), 633 requests of one token 7.3 us on 20 blocks and 21.4
// on the one that their tokens fill.
// ---------------------------------------------------------------------------
constexpr int kPlanThreads = 512;
constexpr int kPlanMaxB = 8192;      // 12 bytes of shared memory per request
constexpr int kPlanTokens = 4;       // consecutive tokens of a thread

struct PlanArgs {
  int B, page, n_pages, max_pages, n_free, n_tokens;
  const int32_t* lens; const int32_t* new_lens;    // new_lens NULL: one each
  int32_t* table;                                  // [B][max_pages]
  const int32_t* free_pages; const int32_t* head;
  int64_t* slot; int32_t* pos; int32_t* row;       // [n_tokens]
  int32_t* cu; int32_t* lens_out; int32_t* head_out;
  uint32_t* status;
};

// Pages of len tokens, len >= 0: the sum may pass 2^31, but not 2^32.
__device__ __forceinline__ int plan_pages(const PlanArgs& a, int len) {
  return static_cast<int>((static_cast<uint32_t>(len) + static_cast<uint32_t>(a.page) - 1u) / static_cast<uint32_t>(a.page));
}

struct PlanReq {
  int len, fresh, held, want;
  bool ok;      // plausible, and fits its table row
};
__device__ __forceinline__ PlanReq plan_req(const PlanArgs& a, int b) {
  PlanReq r;
  r.len = a.lens[b];
  r.fresh = a.new_lens ? a.new_lens[b] : 1;
  const long long end = static_cast<long long>(r.len) + r.fresh;
  r.ok = r.len >= 0 && r.fresh >= 0 && end <= static_cast<long long>(a.max_pages) * a.page;
  r.fresh = r.fresh < 0 ? 0 : r.fresh;
  r.held = r.ok ? plan_pages(a, r.len) : 0;
  r.want = r.ok ? plan_pages(a, static_cast<int>(end)) - r.held : 0;
  return r;
}

__global__ void __launch_bounds__(kPlanThreads) plan_kernel(const __grid_constant__ PlanArgs a) {
  extern __shared__ int plan_smem[];
  int* s_cu = plan_smem;              // [B + 1], clamped to INT_MAX
  int* s_off = plan_smem + a.B + 1;   // [B]: off_b, or -1 for a refused request
  int* s_len = s_off + a.B;           // [B]
  __shared__ long long s_wn[kPlanThreads / 32], s_ww[kPlanThreads / 32];
  __shared__ unsigned long long s_head;
  const int tid = threadIdx.x, lane = tid & 31, wid = tid >> 5;
  const int per = (a.B + kPlanThreads - 1) / kPlanThreads;
  const int b0 = tid * per < a.B ? tid * per : a.B, b1 = b0 + per < a.B ? b0 + per : a.B;
  const int head = *a.head;
  const long long avail = head >= 0 && head <= a.n_free ? a.n_free - head : 0;
  long long sn = 0, sw = 0;
  for (int b = b0; b < b1; ++b) {
    const PlanReq r = plan_req(a, b);
    sn += r.fresh;
    sw += r.want;
  }
  long long en = sn, ew = sw;   // inclusive over the warp
#pragma unroll
  for (int o = 1; o < 32; o <<= 1) {
    const long long x = __shfl_up_sync(0xffffffffu, en, o), y = __shfl_up_sync(0xffffffffu, ew, o);
    if (lane >= o) { en += x; ew += y; }
  }
  if (lane == 31) { s_wn[wid] = en; s_ww[wid] = ew; }
  if (tid == 0) s_head = 0;
  __syncthreads();
  for (int w = 0; w < wid; ++w) { en += s_wn[w]; ew += s_ww[w]; }
  en -= sn;
  ew -= sw;
  uint32_t bad = head < 0 || head > a.n_free ? DEV_ERR_BOUNDS : 0u;
  unsigned long long last = 0;   // pages given out
  for (int b = b0; b < b1; ++b) {
    const PlanReq r = plan_req(a, b);
    const bool fits = r.ok && (r.want == 0 || ew + r.want <= avail) && en + r.fresh <= a.n_tokens;
    if (!fits) bad |= DEV_ERR_BOUNDS;
    s_cu[b] = static_cast<int>(en < INT32_MAX ? en : INT32_MAX);
    s_off[b] = fits ? static_cast<int>(r.want ? ew : 0) : -1;
    s_len[b] = r.len;
    if (fits && r.want && static_cast<unsigned long long>(ew + r.want) > last) last = ew + r.want;
    if (blockIdx.x == 0) {
      a.cu[b] = s_cu[b];
      a.lens_out[b] = fits ? r.len + r.fresh : r.len;
    }
    en += r.fresh;
    ew += r.want;
  }
  if (last) atomicMax(&s_head, last);
  if (b1 == a.B && b0 < a.B) s_cu[a.B] = static_cast<int>(en < INT32_MAX ? en : INT32_MAX);
  if (a.B == 0 && tid == 0) s_cu[0] = 0;
  __syncthreads();
  if (blockIdx.x == 0 && tid == 0) {
    a.cu[a.B] = s_cu[a.B];
    *a.head_out = head + static_cast<int>(s_head);
  }
  // the new pages into the table: a warp a request
  const int nw = gridDim.x * (kPlanThreads / 32);
  for (int b = blockIdx.x * (kPlanThreads / 32) + wid; b < a.B; b += nw) {
    if (s_off[b] < 0) continue;
    const PlanReq r = plan_req(a, b);
    for (int i = lane; i < r.want; i += 32) {
      const int pg = a.free_pages[head + s_off[b] + i];
      if (pg < 0 || pg >= a.n_pages) bad |= DEV_ERR_BOUNDS;
      a.table[static_cast<long long>(b) * a.max_pages + r.held + i] = pg;
    }
  }
  // tokens
  const int total = s_cu[a.B];
  const long long nt = (a.n_tokens + kPlanTokens - 1) / kPlanTokens;
  for (long long u = static_cast<long long>(blockIdx.x) * kPlanThreads + tid; u < nt;
       u += static_cast<long long>(gridDim.x) * kPlanThreads) {
    const int i0 = static_cast<int>(u * kPlanTokens);
    int b = -1;
    long long slot[kPlanTokens];
    int pos[kPlanTokens], row[kPlanTokens];
#pragma unroll
    for (int j = 0; j < kPlanTokens; ++j) {
      const int i = i0 + j;
      slot[j] = -1; pos[j] = 0; row[j] = -1;
      if (i >= total || i >= a.n_tokens) continue;
      if (b < 0) {   // the last request that begins at or before i
        int lo = 0, hi = a.B - 1;
        while (lo < hi) {
          const int m = (lo + hi + 1) >> 1;
          if (s_cu[m] <= i) lo = m; else hi = m - 1;
        }
        b = lo;
      }
      while (s_cu[b + 1] <= i) ++b;
      const int len = s_len[b];
      const long long t64 = static_cast<long long>(len) + (i - s_cu[b]);
      const int t = len >= 0 && t64 < static_cast<long long>(a.max_pages) * a.page ? static_cast<int>(t64) : 0;
      row[j] = b;
      pos[j] = t;
      if (s_off[b] < 0) continue;   // (a request that goes lies inside its row)
      const int held = plan_pages(a, len), pj = t / a.page;
      const int pg = pj < held ? a.table[static_cast<long long>(b) * a.max_pages + pj]
                               : a.free_pages[head + s_off[b] + (pj - held)];
      if (pg >= 0 && pg < a.n_pages) slot[j] = static_cast<long long>(pg) * a.page + (t - pj * a.page);
      else bad |= DEV_ERR_BOUNDS;
    }
    if (i0 + kPlanTokens <= a.n_tokens) {
      longlong2* sp = reinterpret_cast<longlong2*>(a.slot + i0);
      sp[0] = make_longlong2(slot[0], slot[1]);
      sp[1] = make_longlong2(slot[2], slot[3]);
      *reinterpret_cast<int4*>(a.pos + i0) = make_int4(pos[0], pos[1], pos[2], pos[3]);
      *reinterpret_cast<int4*>(a.row + i0) = make_int4(row[0], row[1], row[2], row[3]);
    } else {
      for (int j = 0; j < kPlanTokens && i0 + j < a.n_tokens; ++j) {
        a.slot[i0 + j] = slot[j];
        a.pos[i0 + j] = pos[j];
        a.row[i0 + j] = row[j];
      }
    }
  }
  if (bad && a.status) atomicOr(a.status, bad);
}

}  // namespace kv4
}  // namespace swa
