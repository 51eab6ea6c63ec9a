// Attention of one new token per request over the 4-bit paged cache.
//
// o = sum_j p_j v_j / sum_j p_j, p_j = exp(scale <q, k_j>): each key and value
// is read once, so the bytes of the cache bound it, and everything else has
// to stay below what a tile's 18 D bytes cost the memory (about 100 clocks of
// an SM at D = 128).
//
// What that asks for, and what is done:
//   - Loads. A tile (16 tokens of one kv head, keys, values and scales) is
//     one contiguous block, fetched by one bulk copy into the warp's own ring
//     of kStages buffers: no registers and no address arithmetic are spent on
//     bytes in flight. A warp walks its tiles alone; the warps of a CTA meet
//     only at the end.
//   - Products. Per 4-bit number one multiply-add for every query head of the
//     group is more than the fp32 units have time for, so both products run
//     on matrix instructions with the cache as the 16-row operand: S^T = K Q^T
//     (16 keys x 8 columns) and O^T += V^T P^T (16 channels x 8 columns). The
//     operand registers are made straight from the numbers' bits: (x & 15) |
//     0x6400 is the fp16 number 1024 + n (0x4300: bf16, 128 + n), and one
//     exact subtraction leaves n - 8 (numbers as the low bits of a float of a
//     known power of two: Kim, Henry, Fahim and Awadalla 2022, "Who Says
//     Elephants Can't Run"). The cache's order of numbers makes a
//     lane's 16 bytes of a row exactly its operand registers, so there is no
//     exchange between lanes. (tcgen05 takes its operands from shared or
//     tensor memory: the converted tiles, four times the bytes, would have to
//     be written there first, and its 128-row tiles would hold 8 useful
//     columns as well.)
//   - Precision. A group has few query heads, so the eight columns hold four
//     heads as two terms each: q as fp16 hi + lo (scaled by a power of two
//     into fp16's range), P as bf16 hi + lo (bf16, because P times a step has
//     any size). Products of n - 8 with them are exact in the accumulators;
//     the second terms cost nothing where a group has at most four heads. That
//     is 22 bits of q, whose 2^-22 of a logit is below what the norm's and
//     the sum's fp32 roundings leave (a third term would be a product more),
//     and 16 bits of P, far below a bf16 o's 8; an fp32 o's 24 get a third term
//     of P.
//   - Scales. s and z of a (token, 64 channels) leave the products:
//     <q, k> = sum_g s_g <q, n - 8>_g + z_g sum(q)_g, and sum_j p_j v_j =
//     sum_j (p_j s_j) (n_j - 8) + sum_j p_j z_j, the last one number per group.
//   - Softmax. The running maximum is raised only when a logit passes it by
//     2^8 (in base 2), which a vote of the warp finds out: the reduction over
//     lanes and the rescaling are left out of nearly every tile.
//   - Few requests. A request's tiles are split into chunks of one CTA each;
//     with more than one, each writes its partial result, and the CTA that
//     finishes last joins them in the order of the chunks.
//
// Measured (GB300, graph of calls, bf16): 32 requests of 57k to 65k tokens, 16 / 4
// heads of 128: 212 us, 5.33 TB/s, 78 % of the measured copy rate. The same
// kernel with the arithmetic taken out streams the cache in 166 us (the copy
// rate), with the copies taken out it computes in 184 us; the two overlap but
// not wholly. About 300 instructions a warp and tile, 160 of them turning
// numbers into operands; 57 % of the ALU pipe, 24 % of the tensor pipe. At d =
// 64 a token has half the bytes and the same softmax: 48 % of the copy rate.
// Short requests pay a CTA's set-up and end, about 3 us.
#pragma once

#include <cuda_fp16.h>

#include "kv4.cuh"

namespace swa {
namespace kv4 {

constexpr int kAttnWarps = 4;
constexpr int kStages = 2;               // steps of two tiles in flight per warp
// P in fp32 calls: a third term, or the second's rounding would show in o
constexpr bool kThreeTerms = sizeof(elem_t) == 4;
constexpr int kColQ = 4;                 // query heads of one 8-column operand
constexpr int kMaxSplits = 512;          // CTAs of one request and kv head
// CTAs an SM holds, by head dim and 8-column operands; it bounds the registers
// of a thread (128, or 255 for two). Measured on 16 requests of 32768 tokens, 4 kv
// heads: d = 128, eight query heads a kv head: two 92.6 us, three (spills) 97; d =
// 64, eight: two 67.2, three 56.9, four 55.3; d = 64, four: four 43.2, five 43.2,
// six 46.1.
constexpr int attn_ctas_per_sm(int d, int operands) { return operands == 1 || d == 64 ? 4 : 2; }

struct AttnArgs {
  Cache c;
  int B, Hq, max_pages, window;          // window < 0: none
  float scale, eps;
  const elem_t* q;                       // [B, Hq, D]
  const float* gq;
  const float* rcos; const float* rsin; int rows, rot, interleaved;   // rcos NULL: none
  const int32_t* table; const int32_t* lens;
  elem_t* o; float* lse;                 // [B, Hq, D], [B, Hq]
  int chunk, splits;                     // tiles of a CTA, CTAs of a request
  int groups;                            // CTAs that share a kv head's query heads
  unsigned* count;                       // [B * Hkv * groups] finished chunks, 0 between calls
  float* part;                           // [B * Hkv * groups][splits][heads][D]: partial O
  float2* part_ml;                       // [B * Hkv * groups][splits][heads]: their M, L
  uint32_t* status;
  uint64_t wait_limit_ns;
};

template <int D>
struct AttnShape {
  static constexpr int TB = tile_bytes(D);
  static constexpr int NG = D / 64;
  static constexpr int W = D / 32;       // 32-bit words of a lane's piece of a row
};

// Shared memory of a CTA: rings (re-used for the join), queries, barriers.
template <int D, int NT>
struct AttnSmem {
  static constexpr int ring = kAttnWarps * kStages * 2 * AttnShape<D>::TB;
  static constexpr int join = kAttnWarps * NT * kColQ * (D + 2) * 4;
  static constexpr int bars = (ring > join ? ring : join + 127) / 128 * 128;
  static constexpr int qs = bars + (kAttnWarps * kStages * 8 + 15) / 16 * 16;    // read 16 bytes at a time
  static constexpr int qf = qs + NT * kColQ * 2 * D * 2;        // fp16 hi, lo rows
  static constexpr int flags = qf + NT * kColQ * 4 * 4;         // factor, sums per group
  static constexpr int bytes = flags + 16;
  static_assert(bars % 128 == 0 && qs % 16 == 0 && qf % 16 == 0 && flags % 16 == 0, "");
};

__device__ __forceinline__ void mma_f16(float (&c)[4], uint32_t a0, uint32_t a1, uint32_t a2, uint32_t a3, uint32_t b0,
                                        uint32_t b1) {
  asm("mma.sync.aligned.m16n8k16.row.col.f32.f16.f16.f32 {%0,%1,%2,%3}, {%4,%5,%6,%7}, {%8,%9}, {%0,%1,%2,%3};"
      : "+f"(c[0]), "+f"(c[1]), "+f"(c[2]), "+f"(c[3])
      : "r"(a0), "r"(a1), "r"(a2), "r"(a3), "r"(b0), "r"(b1));
}
// the same onto zeros
__device__ __forceinline__ void mma_f16_first(float (&c)[4], uint32_t a0, uint32_t a1, uint32_t a2, uint32_t a3, uint32_t b0,
                                              uint32_t b1) {
  asm("mma.sync.aligned.m16n8k16.row.col.f32.f16.f16.f32 {%0,%1,%2,%3}, {%4,%5,%6,%7}, {%8,%9}, {%10,%10,%10,%10};"
      : "=f"(c[0]), "=f"(c[1]), "=f"(c[2]), "=f"(c[3])
      : "r"(a0), "r"(a1), "r"(a2), "r"(a3), "r"(b0), "r"(b1), "f"(0.f));
}
__device__ __forceinline__ void mma_bf16(float (&c)[4], uint32_t a0, uint32_t a1, uint32_t a2, uint32_t a3, uint32_t b0,
                                         uint32_t b1) {
  asm("mma.sync.aligned.m16n8k16.row.col.f32.bf16.bf16.f32 {%0,%1,%2,%3}, {%4,%5,%6,%7}, {%8,%9}, {%0,%1,%2,%3};"
      : "+f"(c[0]), "+f"(c[1]), "+f"(c[2]), "+f"(c[3])
      : "r"(a0), "r"(a1), "r"(a2), "r"(a3), "r"(b0), "r"(b1));
}
// 8x8 transpose of 16-bit elements across the warp.
__device__ __forceinline__ uint32_t transpose8(uint32_t x) {
  uint32_t r;
  asm("movmatrix.sync.aligned.m8n8.trans.b16 %0, %1;" : "=r"(r) : "r"(x));
  return r;
}
// (x & mask) | bits as the one instruction it is
__device__ __forceinline__ uint32_t and_or(uint32_t x, uint32_t mask, uint32_t bits) {
  uint32_t r;
  asm("lop3.b32 %0, %1, %2, %3, 0xEA;" : "=r"(r) : "r"(x), "r"(mask), "r"(bits));
  return r;
}
// Eight numbers of a word as four fp16 pairs (number i, number i + 4) - 8.
__device__ __forceinline__ void widen_f16(uint32_t x, uint32_t (&h)[4]) {
  const __half2 low = __floats2half2_rn(-1032.f, -1032.f), sixteenth = __floats2half2_rn(0.0625f, 0.0625f),
                high = __floats2half2_rn(-72.f, -72.f);
  auto h2 = [](uint32_t v) { return *reinterpret_cast<__half2*>(&v); };
  auto u = [](__half2 v) { return *reinterpret_cast<uint32_t*>(&v); };
  const uint32_t y = x >> 8;
  h[0] = u(__hadd2(h2(and_or(x, 0x000F000Fu, 0x64006400u)), low));                  // 1024 + n
  h[1] = u(__hfma2(h2(and_or(x, 0x00F000F0u, 0x64006400u)), sixteenth, high));     // 1024 + 16 n
  h[2] = u(__hadd2(h2(and_or(y, 0x000F000Fu, 0x64006400u)), low));
  h[3] = u(__hfma2(h2(and_or(y, 0x00F000F0u, 0x64006400u)), sixteenth, high));
}
// The same as bf16 (whose 7 fraction bits leave no place for the second form).
__device__ __forceinline__ void widen_bf16(uint32_t x, uint32_t (&h)[4]) {
  const __nv_bfloat162 off = __floats2bfloat162_rn(-136.f, -136.f);
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    uint32_t v = and_or(x >> (4 * i), 0x000F000Fu, 0x43004300u);                    // 128 + n
    const __nv_bfloat162 r = __hadd2(*reinterpret_cast<__nv_bfloat162*>(&v), off);
    h[i] = *reinterpret_cast<const uint32_t*>(&r);
  }
}

template <int W>
__device__ __forceinline__ void ld_words(const uint8_t* p, uint32_t (&w)[W]) {
  if constexpr (W == 4) {
    const uint4 t = *reinterpret_cast<const uint4*>(p);
    w[0] = t.x; w[1] = t.y; w[2] = t.z; w[3] = t.w;
  } else {
    const uint2 t = *reinterpret_cast<const uint2*>(p);
    w[0] = t.x; w[1] = t.y;
  }
}
// The (s, z) pairs of one token, NG groups.
template <int NG>
__device__ __forceinline__ void ld_scales(const uint8_t* p, float (&s)[NG], float (&z)[NG]) {
  uint32_t w[NG];
  if constexpr (NG == 2) {
    const uint2 t = *reinterpret_cast<const uint2*>(p);
    w[0] = t.x; w[1] = t.y;
  } else {
    w[0] = *reinterpret_cast<const uint32_t*>(p);
  }
#pragma unroll
  for (int g = 0; g < NG; ++g) {
    s[g] = __uint_as_float(w[g] << 16);
    z[g] = __uint_as_float(w[g] & 0xFFFF0000u);
  }
}

// A query row by one warp: rotation, norm, gain, softmax scale and log2 e, a
// power of two that brings the largest entry into [2^13, 2^14), and the two
// fp16 terms, into shared memory; f[0] = the inverse power, f[1 + g] = the
// sum over group g. x == NULL: a row of zeros.
template <int D>
__device__ __forceinline__ void query_row(const AttnArgs& a, const elem_t* q, int pos, __half* dst, float* f) {
  constexpr int E = D / 32;
  const int lane = threadIdx.x & 31, c0 = lane * E;
  float x[E] = {}, g[E], ss = 0.f;
#pragma unroll
  for (int i = 0; i < E; ++i) g[i] = 1.0f;
  if (q != nullptr) {
    // all loads before any use: this is latency in front of every CTA
    load_vec<E>(q + c0, x);
    if (a.gq != nullptr) load_vec<E>(a.gq + c0, g);
    if (a.rcos != nullptr && c0 < a.rot) {
      const int half = a.rot / 2;
      const long long row = static_cast<long long>(pos) * half;
      if (a.interleaved) {
        float c[E / 2], s[E / 2];
#pragma unroll
        for (int i = 0; i < E / 2; ++i) {
          c[i] = a.rcos[row + c0 / 2 + i];
          s[i] = a.rsin[row + c0 / 2 + i];
        }
#pragma unroll
        for (int i = 0; i < E / 2; ++i) {
          const float u = x[2 * i], v = x[2 * i + 1];
          x[2 * i] = fmaf(u, c[i], v * s[i]);
          x[2 * i + 1] = fmaf(v, c[i], -u * s[i]);
        }
      } else {      // half is a multiple of 8: the lane's channels lie on one side of it
        const bool first = c0 < half;
        float y[E], c[E], s[E];
        load_vec<E>(q + (first ? c0 + half : c0 - half), y);
        load_vec<E>(a.rcos + row + (first ? c0 : c0 - half), c);
        load_vec<E>(a.rsin + row + (first ? c0 : c0 - half), s);
#pragma unroll
        for (int i = 0; i < E; ++i) x[i] = fmaf(x[i], c[i], (first ? y[i] : -y[i]) * s[i]);
      }
    }
#pragma unroll
    for (int i = 0; i < E; ++i) ss = fmaf(x[i], x[i], ss);
  }
  ss = warp_sum(ss);
  float eps = a.eps;
  if (ss == INFINITY) {      // the squares pass fp32: the same of 2^-80 of the row
    constexpr float kDown = 0x1p-80f;
    ss = 0.f;
#pragma unroll
    for (int i = 0; i < E; ++i) {
      x[i] *= kDown;
      ss = fmaf(x[i], x[i], ss);
    }
    ss = warp_sum(ss);
    eps = eps * kDown * kDown;
  }
  const float mul = rsqrtf(ss / D + eps) * (a.scale * 1.4426950408889634f);
  float top = 0.f;
#pragma unroll
  for (int i = 0; i < E; ++i) {
    x[i] *= mul * g[i];
    if (q == nullptr) x[i] = 0.f;
    top = fmaxf(top, fabsf(x[i]));
  }
#pragma unroll
  for (int o = 16; o > 0; o >>= 1) top = fmaxf(top, __shfl_xor_sync(0xffffffffu, top, o));
  // exponent of top, kept where both the power and its inverse are normal
  int e = static_cast<int>((__float_as_uint(top) >> 23) & 255u) - 127;
  e = e < -100 ? -100 : (e > 100 ? 100 : e);
  const float up = __uint_as_float(static_cast<uint32_t>(127 + 13 - e) << 23);
  float sum = 0.f;
#pragma unroll
  for (int i = 0; i < E; ++i) {
    const float v = x[i] * up;
    const __half hi = __float2half_rn(v);
    const __half lo = __float2half_rn(v - __half2float(hi));
    const int at = ((c0 + i) & ~7) + ((c0 + i) & 3) * 2 + (((c0 + i) >> 2) & 1);   // pairs (i, i + 4) side by side
    dst[at] = hi;
    dst[D + at] = lo;
    sum += v;
  }
  // lanes of one group: 64 / E
#pragma unroll
  for (int o = 32 / E; o > 0; o >>= 1) sum += __shfl_xor_sync(0xffffffffu, sum, o);
  if (lane == 0) {
    f[0] = __uint_as_float(static_cast<uint32_t>(127 - 13 + e) << 23);
    f[1] = sum;
  }
  if (D == 128 && lane == 16) f[2] = sum;
}

// o and lse of one head from its sums, by one warp. No key: 0 and -infinity;
// a NaN stays one.
template <int D>
__device__ __forceinline__ void finish_head(const AttnArgs& a, long long head, float (&o)[D / 32], float top, float sum) {
  constexpr int E = D / 32;
  const int lane = threadIdx.x & 31;
  const float inv = sum == 0.f ? 0.f : 1.0f / sum;
#pragma unroll
  for (int e = 0; e < E; ++e) o[e] *= inv;
  store_vec<E>(a.o + head * D + lane * E, o);
  if (lane == 0) a.lse[head] = sum == 0.f ? -INFINITY : (top + log2f(sum)) * 0.6931471805599453f;
}

template <int D, int NT, bool kPolled>
__global__ void __launch_bounds__(kAttnWarps * 32, attn_ctas_per_sm(D, NT)) attn_kernel(const __grid_constant__ AttnArgs a) {
  using S = AttnShape<D>;
  using M = AttnSmem<D, NT>;
  constexpr int NG = S::NG, W = S::W, NQ = NT * kColQ;
  extern __shared__ __align__(128) uint8_t smem[];
  const int tid = threadIdx.x, lane = tid & 31, wid = tid >> 5;
  const int r = lane >> 2, j = lane & 3;
  const int b = blockIdx.z, h = blockIdx.y / a.groups, qg = blockIdx.y - h * a.groups;
  const int G = a.Hq / a.c.Hkv;
  const int nq = min(NQ, G - qg * NQ);                     // query heads of this CTA
  const long long hq0 = static_cast<long long>(b) * a.Hq + h * G + qg * NQ;

  // what of the request this chunk holds
  uint32_t bad = 0;
  int len = a.lens[b];
  const long long cap = static_cast<long long>(a.max_pages) * a.c.page;
  if (len < 0 || len > cap) {
    bad = DEV_ERR_BOUNDS;
    len = len < 0 ? 0 : static_cast<int>(cap);
  }
  if (a.rcos != nullptr && len > a.rows) {
    bad = DEV_ERR_BOUNDS;
    len = 0;
  }
  const int lo = a.window >= 0 && len - 1 - a.window > 0 ? len - 1 - a.window : 0;
  const int t_lo = lo / kTile, t_hi = (len + kTile - 1) / kTile;     // tiles [t_lo, t_hi)
  const int chunks = max(1, (t_hi - t_lo + a.chunk - 1) / a.chunk);
  if (blockIdx.x >= chunks) return;
  const int t0 = t_lo + blockIdx.x * a.chunk, t1 = min(t_hi, t0 + a.chunk);

  const uint32_t bars = smem_u32(smem + M::bars) + wid * kStages * 8;
  uint32_t* flags = reinterpret_cast<uint32_t*>(smem + M::flags);    // [0] abort, [1] last
  if (lane == 0) {
    for (int s = 0; s < kStages; ++s) mbar_init(bars + 8 * s, 1);
    fence_mbar_init();
  }
  if (tid == 0) flags[0] = 0;
  __syncwarp();

  // Step n of this warp is the tiles t0 + 2 (wid + n * kAttnWarps) and the one
  // behind it, which share a stage. Pages are looked up 32 tiles (16 steps)
  // at a time, a lane a tile.
  const int n_mine = (t1 - t0 + 1) / 2 > wid ? ((t1 - t0 + 1) / 2 - wid + kAttnWarps - 1) / kAttnWarps : 0;
  uint8_t* ring = smem + wid * kStages * 2 * S::TB;
  const uint32_t ring_u = smem_u32(ring);
  const int per_page = a.c.page / kTile;
  const long long head_off = static_cast<long long>(h) * per_page;
  long long tile_at = -1;  // of the lane's tile in the cache; -1: none
  uint32_t gone = 0;       // two bits per stage: tiles that are not there
  auto issue = [&](int n) {
    if ((n & 15) == 0) {
      const int t = t0 + 2 * (wid + (n + (lane >> 1)) * kAttnWarps) + (lane & 1);
      tile_at = -1;
      if (t < t1) {
        const int pi = t / per_page;
        const int pg = a.table[static_cast<long long>(b) * a.max_pages + pi];
        if (pg >= 0 && pg < a.c.n_pages)
          tile_at = static_cast<long long>(pg) * a.c.Hkv * per_page + head_off + (t - pi * per_page);
        else
          bad = DEV_ERR_BOUNDS;
      }
    }
    const int st = n % kStages;
    const long long at = __shfl_sync(0xffffffffu, tile_at, ((2 * n) & 31) + (lane & 1));
    const uint32_t there = __ballot_sync(0xffffffffu, at >= 0) & 3u;
    gone = (gone & ~(3u << (2 * st))) | ((there ^ 3u) << (2 * st));
    if (lane == 0) mbar_arrive_expect_tx(bars + 8 * st, __popc(there) * S::TB);
    __syncwarp();
    if (lane < 2 && at >= 0) bulk_load(ring_u + (st * 2 + lane) * S::TB, a.c.data + at * S::TB, S::TB, bars + 8 * st);
  };
  for (int n = 0; n < kStages && n < n_mine; ++n) issue(n);

  // the queries
  __half* qs = reinterpret_cast<__half*>(smem + M::qs);
  float* qf = reinterpret_cast<float*>(smem + M::qf);
  for (int i = wid; i < NQ; i += kAttnWarps)
    query_row<D>(a, i < nq && len > 0 ? a.q + (hq0 + i) * D : nullptr, len - 1, qs + i * 2 * D, qf + i * 4);
  __syncthreads();
  uint32_t qb[NT][2 * W][2];       // operand registers: column lane / 4 = 2 head + term
  float qfac[NT], qsum[NT][NG];
#pragma unroll
  for (int nt = 0; nt < NT; ++nt) {
    const __half* row = qs + (nt * kColQ + (r >> 1)) * 2 * D + (r & 1) * D;
#pragma unroll
    for (int w = 0; w < W; ++w) {
      const uint4 c = *reinterpret_cast<const uint4*>(row + (w / 2) * 64 + j * 16 + (w & 1) * 8);
      qb[nt][2 * w][0] = c.x; qb[nt][2 * w][1] = c.y;
      qb[nt][2 * w + 1][0] = c.z; qb[nt][2 * w + 1][1] = c.w;
    }
    qfac[nt] = qf[(nt * kColQ + j) * 4];
#pragma unroll
    for (int g = 0; g < NG; ++g) qsum[nt][g] = qf[(nt * kColQ + j) * 4 + 1 + g];
  }

  const WaitCtl<kPolled> ctl{flags, a.status, a.wait_limit_ns};
  float acc[NT][2 * W][4] = {};
  float m[NT], l[NT] = {}, zs[NT][NG] = {};
#pragma unroll
  for (int nt = 0; nt < NT; ++nt) m[nt] = -1e30f;
  int n = 0;
  for (; n < n_mine; ++n) {
    const int st = n % kStages;
    if (!mbar_wait_warp(bars + 8 * st, (n / kStages) & 1, ctl)) break;
    const uint8_t* tile = ring + st * 2 * S::TB;
    const int key0 = (t0 + 2 * (wid + n * kAttnWarps)) * kTile;
    float s[2][NT][2];       // logits (base 2): tile, column, key r or r + 8
#pragma unroll
    for (int q = 0; q < 2; ++q) {
      uint32_t ka[W], kb[W];
      ld_words<W>(tile + q * S::TB + r * (D / 2) + j * (D / 8), ka);
      ld_words<W>(tile + q * S::TB + (r + 8) * (D / 2) + j * (D / 8), kb);
      float sa[NG], za[NG], sb[NG], zb[NG];
      ld_scales<NG>(tile + q * S::TB + 16 * D + r * (4 * NG), sa, za);
      ld_scales<NG>(tile + q * S::TB + 16 * D + (r + 8) * (4 * NG), sb, zb);
      float d[NT][NG][4];
#pragma unroll
      for (int w = 0; w < W; ++w) {
        uint32_t x[4], y[4];
        widen_f16(ka[w], x);
        widen_f16(kb[w], y);
#pragma unroll
        for (int nt = 0; nt < NT; ++nt) {
          if (w & 1)
            mma_f16(d[nt][w / 2], x[0], y[0], x[1], y[1], qb[nt][2 * w][0], qb[nt][2 * w][1]);
          else
            mma_f16_first(d[nt][w / 2], x[0], y[0], x[1], y[1], qb[nt][2 * w][0], qb[nt][2 * w][1]);
          mma_f16(d[nt][w / 2], x[2], y[2], x[3], y[3], qb[nt][2 * w + 1][0], qb[nt][2 * w + 1][1]);
        }
      }
#pragma unroll
      for (int nt = 0; nt < NT; ++nt) {
        float u = 0.f, v = 0.f;
#pragma unroll
        for (int g = 0; g < NG; ++g) {
          u = fmaf(sa[g], d[nt][g][0] + d[nt][g][1], fmaf(za[g], qsum[nt][g], u));
          v = fmaf(sb[g], d[nt][g][2] + d[nt][g][3], fmaf(zb[g], qsum[nt][g], v));
        }
        s[q][nt][0] = u * qfac[nt];
        s[q][nt][1] = v * qfac[nt];
      }
    }
    float sv[2][2][NG], zv[2][2][NG];
#pragma unroll
    for (int q = 0; q < 2; ++q) {
      ld_scales<NG>(tile + q * S::TB + 17 * D + r * (4 * NG), sv[q][0], zv[q][0]);
      ld_scales<NG>(tile + q * S::TB + 17 * D + (r + 8) * (4 * NG), sv[q][1], zv[q][1]);
    }
    const uint32_t miss = gone >> (2 * st) & 3u;
    if (key0 < lo || key0 + 2 * kTile > len || miss) {       // keys outside, or not there, count nothing
#pragma unroll
      for (int q = 0; q < 2; ++q) {
#pragma unroll
        for (int i = 0; i < 2; ++i) {
          const int key = key0 + q * kTile + r + 8 * i;
          if (key < lo || key >= len || (miss >> q & 1u)) {
#pragma unroll
            for (int nt = 0; nt < NT; ++nt) s[q][nt][i] = -INFINITY;
#pragma unroll
            for (int g = 0; g < NG; ++g) sv[q][i][g] = zv[q][i][g] = 0.f;
          }
        }
      }
    }
    float top[NT];
    bool raise = false;
#pragma unroll
    for (int nt = 0; nt < NT; ++nt) {
      top[nt] = fmaxf(fmax3(s[0][nt][0], s[0][nt][1], s[1][nt][0]), s[1][nt][1]);
      raise |= top[nt] > m[nt] + 8.f;
    }
    if (__any_sync(0xffffffffu, raise)) {
#pragma unroll
      for (int nt = 0; nt < NT; ++nt) {
        float x = top[nt];
#pragma unroll
        for (int o = 4; o < 32; o <<= 1) x = fmaxf(x, __shfl_xor_sync(0xffffffffu, x, o));
        const float mn = fmaxf(m[nt], x), al = ex2_approx(m[nt] - mn);
        m[nt] = mn;
        l[nt] *= al;
#pragma unroll
        for (int g = 0; g < NG; ++g) zs[nt][g] *= al;
#pragma unroll
        for (int i = 0; i < 2 * W; ++i)
#pragma unroll
          for (int k = 0; k < 4; ++k) acc[nt][i][k] *= al;
      }
    }
    uint32_t va[2][W], vb[2][W];
#pragma unroll
    for (int q = 0; q < 2; ++q) {
      ld_words<W>(tile + q * S::TB + 8 * D + j * D + r * (D / 8), va[q]);
      ld_words<W>(tile + q * S::TB + 8 * D + (j + 4) * D + r * (D / 8), vb[q]);
    }
    __syncwarp();
    if (n + kStages < n_mine) issue(n + kStages);   // every lane has its words
#pragma unroll
    for (int q = 0; q < 2; ++q) {
      uint32_t pb[NT][NG][2], pc[NT][NG][2];
#pragma unroll
      for (int nt = 0; nt < NT; ++nt) {
#pragma unroll
        for (int i = 0; i < 2; ++i) {
          const float p = ex2_approx(s[q][nt][i] - m[nt]);
          l[nt] += p;
#pragma unroll
          for (int g = 0; g < NG; ++g) {
            zs[nt][g] = fmaf(p, zv[q][i][g], zs[nt][g]);
            const float w = p * sv[q][i][g];
            const float hi = __uint_as_float(pack_bf16x2(0.f, w));       // rounded, in the high half
            const uint32_t both = pack_bf16x2(hi, w - hi);
            pb[nt][g][i] = transpose8(both);
            if (kThreeTerms) pc[nt][g][i] = transpose8(pack_bf16x2(w - hi - __uint_as_float(both & 0xFFFF0000u), 0.f));
          }
        }
      }
#pragma unroll
      for (int w = 0; w < W; ++w) {
        uint32_t x[4], y[4];
        widen_bf16(va[q][w], x);
        widen_bf16(vb[q][w], y);
#pragma unroll
        for (int nt = 0; nt < NT; ++nt) {
          mma_bf16(acc[nt][2 * w], x[0], x[1], y[0], y[1], pb[nt][w / 2][0], pb[nt][w / 2][1]);
          mma_bf16(acc[nt][2 * w + 1], x[2], x[3], y[2], y[3], pb[nt][w / 2][0], pb[nt][w / 2][1]);
          if (kThreeTerms) {
            mma_bf16(acc[nt][2 * w], x[0], x[1], y[0], y[1], pc[nt][w / 2][0], pc[nt][w / 2][1]);
            mma_bf16(acc[nt][2 * w + 1], x[2], x[3], y[2], y[3], pc[nt][w / 2][0], pc[nt][w / 2][1]);
          }
        }
      }
    }
  }
  // a wait that ran out: the copies still on their way land before the memory is used again
  for (int k = n; k < n_mine && k < n + kStages; ++k) mbar_wait_drain(bars + 8 * (k % kStages), (k / kStages) & 1, kDrainLimitNs);
  if (bad) atomicOr(a.status, bad);

  // join the warps: O, M, L of each query head into shared memory
  __syncthreads();
  float* jo = reinterpret_cast<float*>(smem);                    // [warp][NQ][D]
  float* jm = jo + kAttnWarps * NQ * D;                          // [warp][NQ][2]: M, L
#pragma unroll
  for (int nt = 0; nt < NT; ++nt) {
#pragma unroll
    for (int o = 4; o < 32; o <<= 1) {
      l[nt] += __shfl_xor_sync(0xffffffffu, l[nt], o);
#pragma unroll
      for (int g = 0; g < NG; ++g) zs[nt][g] += __shfl_xor_sync(0xffffffffu, zs[nt][g], o);
    }
    const int i = wid * NQ + nt * kColQ + j;
#pragma unroll
    for (int w = 0; w < W; ++w) {
      const float(&x)[4] = acc[nt][2 * w], (&y)[4] = acc[nt][2 * w + 1];
      const float z = zs[nt][w / 2];
      *reinterpret_cast<float4*>(jo + i * D + (w / 2) * 64 + r * 8 + (w & 1) * 4) =
          make_float4(x[0] + x[1] + z, x[2] + x[3] + z, y[0] + y[1] + z, y[2] + y[3] + z);
    }
    if (r == 0) {
      jm[2 * i] = m[nt];
      jm[2 * i + 1] = l[nt];
    }
  }
  __syncthreads();
  constexpr int E = D / 32;
  const int item = (b * a.c.Hkv + h) * a.groups + qg;
  const long long part0 = static_cast<long long>(item) * a.splits * NQ;
  for (int i = wid; i < nq; i += kAttnWarps) {      // a warp a head, E channels a lane
    float top = -1e30f, sum = 0.f, o[E] = {};
#pragma unroll
    for (int k = 0; k < kAttnWarps; ++k) top = fmaxf(top, jm[2 * (k * NQ + i)]);
#pragma unroll
    for (int k = 0; k < kAttnWarps; ++k) {
      const float f = ex2_approx(jm[2 * (k * NQ + i)] - top);
      sum = fmaf(f, jm[2 * (k * NQ + i) + 1], sum);
      float x[E];
      load_vec<E>(jo + (k * NQ + i) * D + lane * E, x);
#pragma unroll
      for (int e = 0; e < E; ++e) o[e] = fmaf(f, x[e], o[e]);
    }
    if (chunks == 1) {
      finish_head<D>(a, hq0 + i, o, top, sum);
    } else {
      const long long at = part0 + static_cast<long long>(blockIdx.x) * NQ + i;
      store_vec<E>(a.part + at * D + lane * E, o);
      if (lane == 0) a.part_ml[at] = make_float2(top, sum);
    }
  }
  if (chunks == 1) return;
  __syncthreads();
  if (tid == 0) {
    __threadfence();      // after the barrier it covers what the CTA wrote
    flags[1] = atomicAdd(a.count + item, 1u) == static_cast<unsigned>(chunks - 1);
  }
  __syncthreads();
  if (!flags[1]) return;
  __threadfence();
  if (tid == 0) a.count[item] = 0;        // for the next call

  // join the chunks: a warp every fourth one, all heads of it at once (their
  // loads wait together), then the warps as above, with M common to all
  float top[NQ], sum[NQ] = {}, o[NQ][E] = {};
#pragma unroll
  for (int i = 0; i < NQ; ++i) top[i] = -1e30f;
  for (int k = lane; k < chunks; k += 32) {
#pragma unroll
    for (int i = 0; i < NQ; ++i)
      if (i < nq) top[i] = fmaxf(top[i], __ldcg(a.part_ml + part0 + k * NQ + i).x);
  }
#pragma unroll
  for (int i = 0; i < NQ; ++i)
#pragma unroll
    for (int x = 16; x > 0; x >>= 1) top[i] = fmaxf(top[i], __shfl_xor_sync(0xffffffffu, top[i], x));
#pragma unroll 4
  for (int k = wid; k < chunks; k += kAttnWarps) {
#pragma unroll
    for (int i = 0; i < NQ; ++i) {
      if (i >= nq) continue;
      const long long at = part0 + static_cast<long long>(k) * NQ + i;
      const float2 ml = __ldcg(a.part_ml + at);
      float x[E];
      if constexpr (E == 4) {
        const float4 v = __ldcg(reinterpret_cast<const float4*>(a.part + at * D + lane * E));
        x[0] = v.x; x[1] = v.y; x[2] = v.z; x[3] = v.w;
      } else {
        const float2 v = __ldcg(reinterpret_cast<const float2*>(a.part + at * D + lane * E));
        x[0] = v.x; x[1] = v.y;
      }
      const float f = ex2_approx(ml.x - top[i]);
      sum[i] = fmaf(f, ml.y, sum[i]);
#pragma unroll
      for (int e = 0; e < E; ++e) o[i][e] = fmaf(f, x[e], o[i][e]);
    }
  }
#pragma unroll
  for (int i = 0; i < NQ; ++i) {
    store_vec<E>(jo + (wid * NQ + i) * D + lane * E, o[i]);
    if (lane == 0) {
      jm[2 * (wid * NQ + i)] = top[i];
      jm[2 * (wid * NQ + i) + 1] = sum[i];
    }
  }
  __syncthreads();
  for (int i = wid; i < nq; i += kAttnWarps) {
    float total = 0.f, y[E] = {};
#pragma unroll
    for (int k = 0; k < kAttnWarps; ++k) {
      total += jm[2 * (k * NQ + i) + 1];
      float x[E];
      load_vec<E>(jo + (k * NQ + i) * D + lane * E, x);
#pragma unroll
      for (int e = 0; e < E; ++e) y[e] += x[e];
    }
    finish_head<D>(a, hq0 + i, y, jm[2 * i], total);
  }
}

// Chunks: a CTA's tiles and the CTAs of the longest request, from what the
// host knows (the table's width and the window, not the lengths). The number
// of splits is the one with the least estimated time, in tiles of one CTA: a
// chunk and the set-up of a CTA, as often as the CTAs fill the GPU, and for
// more than one split the join, a tail of the last CTA; the mean of a batch
// of full-length requests (whole rounds of CTAs) and of one that is ragged
// (half the CTAs have work). Measured on 32 requests x 4096 tiles, 4 kv
// heads: chunks of 64, 96, 216, 256 and 432 tiles take 243, 226, 212, 216 and
// 214 us; 16 ragged requests of at most 313 tiles, 6 kv heads: chunks of 32 and
// 56 tiles 14.9 and 18.4 us; one request of 10 tiles 3.9 us in one CTA, 5.4 us
// in two.
// Partial results are kept for at most kPartRounds rounds of CTAs, so that a
// workspace has one size whatever the batch, the lengths and the window.
constexpr long long kPartRounds = 8;
constexpr long long attn_slots(int d, int operands) { return 152LL * attn_ctas_per_sm(d, operands); }   // of a GB300
constexpr long long attn_part_floats(int d, int operands) {
  return kPartRounds * attn_slots(d, operands) * operands * kColQ * (d + 2);
}
struct AttnSplit {
  int heads, groups;     // query heads of a CTA, CTAs per kv head
  int chunk, splits;
  long long items;
};
inline AttnSplit attn_split(int B, int Hq, int Hkv, int d, int page, int max_pages, int window) {
  constexpr long long kSetup = 12, kJoin = 6, kStep = 2 * kAttnWarps;
  AttnSplit s;
  const int G = Hq / Hkv;
  s.heads = G <= kColQ ? kColQ : 2 * kColQ;
  s.groups = (G + s.heads - 1) / s.heads;
  s.items = static_cast<long long>(B) * Hkv * s.groups;
  const long long cap = static_cast<long long>(max_pages) * page;
  long long keys = cap;
  if (window >= 0 && window + 1LL + kTile < cap) keys = window + 1LL + kTile;    // the window may begin inside a tile
  const long long tiles = (keys + kTile - 1) / kTile;
  const long long slots = attn_slots(d, s.heads / kColQ);
  long long best = 0, chunk = 0;
  for (long long n = 1; n <= kMaxSplits; ++n) {
    const long long c = ((tiles + n - 1) / n + kStep - 1) / kStep * kStep, real = (tiles + c - 1) / c;
    if (real > 1 && s.items * real > kPartRounds * slots) break;
    const long long own = (c < tiles ? c : tiles) + kSetup, half = s.items * real / 2;
    const long long t = (half > slots ? half * own / slots : own) + (s.items * real + slots - 1) / slots * own +
                        (real > 1 ? kJoin + real / 2 : 0);
    if (n == 1 || t < best) {
      best = t;
      chunk = c;
    }
    if (c == kStep) break;
  }
  s.chunk = static_cast<int>(chunk);
  s.splits = static_cast<int>((tiles + chunk - 1) / chunk);
  return s;
}

}  // namespace kv4
}  // namespace swa
