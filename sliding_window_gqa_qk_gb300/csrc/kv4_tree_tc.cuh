// Attention of a request's drafted tokens on the tensor cores' tcgen05 form (bf16
// library, head dim 128): more than 16 (token, head) rows of a kv head.
//
// With many rows the m16n8k16 form (kv4_tree.cuh) is held by its products and by
// the softmax beside them: 16 requests of 32768 tokens, 64 rows for each of 4 kv
// heads, took it 548 us where the cache's bytes take the memory 43 and the products
// 34. This form takes 173, and is held by the softmax warps' round of a block, 2600
// clocks: their exponentials, P's stores, and the waits for S around them. (With 32
// rows a CTA 201; with a thread's 16 rows instead of 32 its registers spill, 335.)
// Here a block is 128 keys (eight tiles), the lanes of tensor memory:
//   S^T[keys x rows]     = K Q^T    K from tensor memory (a lane a key), Q from
//                                   shared memory, rows twice: q's two fp16 terms
//   O^T[channels x rows] += V^T P^T V^T from tensor memory (a lane a channel), P
//                                   from shared memory
// so that the numbers go from their bits to operands without passing shared
// memory again, and S comes out with a thread a key: its scales and masks are the
// thread's own, and both terms of a row's q lie in its own lane.
//   soft    NR / 8 warps  a thread a key, 32 rows: S, mask, exponentials, P, sums
//   keys    8 warps       numbers of a block's keys to fp16, times their steps: exact
//                         (11 bits), since each key's steps and centres are first
//                         brought to size by a power of two, which the softmax takes
//                         out again. Centres are a ninth product of 16: <q, k> =
//                         sum_g s_g <q, n - 8>_g + z_g sum(q)_g. Also the values'
//                         scales, cleaned: keys that are not there, or not finite, 0.
//   values  4 warps       numbers to fp16, times step plus centre: 11 bits, as P has
//                         (with 8 of each, in bf16, o was up to 2.5e-3 off where its own
//                         rounding makes 1.7e-3). A key whose values are not about 1
//                         has them brought there by a power of two that P takes on and
//                         its sum takes off: see value_shift
//   mma     2 threads      products of 16: nine of S a block, eight of O. One after the
//                         other by one thread they were 17 times 90 to 100 clocks of issue
//                         a block, beside the other warps' work; S and O have one each
//   load    1 warp        bulk copies of tiles, kTtRing blocks in flight
// Maximum: a row's is that of the first block in which it sees a key, where P is 2^4,
// and is raised only when P would pass 2^15, which the four warps of its 32 rows find
// out together; then they rescale O in tensor memory themselves. So P leaves fp16 2^29
// below that first maximum (what a million keys there would count is below o's own
// rounding), and has 2^11 above it: logits of a standard deviation of 0.9 and 2.3 take
// 173 us, of 3.7 181, of 4.6 193, of 9.2 254 (from 2^8: 173 and 178, 210, 231, 279; from 2^2: 173, 175,
// 184, 239). 183 where every key's values are shifted.
// A key whose scales are not finite counts as 0 in the products, for a product would
// bring a NaN to rows that do not see it: the rows that see it are made NaN at the
// end (keys' scales: through S, per row).
#pragma once

#include "kv4_tree.cuh"
#include "tc_fwd.cuh"

namespace swa {
namespace kv4 {

constexpr int kTtD = 128, kTtKeys = 128, kTtTiles = kTtKeys / kTile;
constexpr int kTtRing = 6;                       // blocks of packed tiles in flight
constexpr int kTtScales = 8;                      // blocks whose scales are kept: see the keys' warps
constexpr float kTtBase = 4.f, kTtRaise = 15.f;

template <int NR>
struct TtShape {
  static constexpr int soft = NR / 8, keys0 = soft, values0 = soft + 8, mma = soft + 12, mma_o = mma + 1, load = mma + 2;
  static constexpr int warps = soft + 16;        // whole groups of four, for the registers; the last does nothing
  // registers of a thread: at launch, then softmax, keys and values, the rest (soft 128 threads for each 32 rows)
  static constexpr int regs0 = 80, regs_soft = 112, regs_convert = 72, regs_rest = 40;
  static_assert(128 * (NR / 32 * regs_soft + 3 * regs_convert + regs_rest) <= warps * 32 * regs0, "");
  static constexpr int N = 2 * NR;               // columns of S: both terms
  // tensor memory
  static constexpr uint32_t cS = 0, cO = 128, cK = 192, cV = 336, kstep = 72, vstep = 64;
  // shared memory
  static constexpr int q_block = N * 128;        // 64 K elements of every row, 128-byte swizzle
  static constexpr int oQ = 0, oP = 3 * q_block, p_buf = kTtKeys * 128, oRing = oP + 2 * p_buf, block = kTtTiles * tile_bytes(kTtD);
  static constexpr int oFk = oRing + kTtRing * block;          // [kTtScales][128] {factor, flags}
  static constexpr int oVs = oFk + kTtScales * kTtKeys * 8;    // [kTtScales][2 groups][128] steps, then centres, fp16
  static constexpr int oRow = oVs + kTtScales * 2 * 2 * kTtKeys * 2;   // TreeRow [NR]
  static constexpr int oM = oRow + NR * 16;                    // maxima, negated, and their rises [NR] each
  static constexpr int oRed = oM + 2 * NR * 4;                 // [4][NR]
  static constexpr int oNan = oRed + 4 * NR * 4;               // [NR]
  static constexpr int oFresh = oNan + NR * 4;                 // [NR], then one for each 32 rows
  static constexpr int oPos = oFresh + NR * 4 + 16;            // [kTreeTokens]
  static constexpr int oMiss = oPos + kTreeTokens * 4;         // [kTtRing]
  static constexpr int oBar = (oMiss + kTtRing * 4 + 15) / 16 * 16;
  static constexpr int RAW = 0, RAWFREE = kTtRing, KFULL = 2 * kTtRing, KFREE = KFULL + 2, SFULL = KFREE + 2, SFREE = SFULL + 1,
                       PFULL = SFREE + 1, VFULL = PFULL + 2, PVDONE = VFULL + 2, SCALES = PVDONE + 2, FINAL = SCALES + kTtScales,
                       COUNT = FINAL + 1;
  static constexpr int bytes = oBar + COUNT * 8 + 32;
  static constexpr int oJoin = oRing;                          // [NR][128] fp32, over the ring
  static_assert(bytes <= 232448 && NR * kTtD * 4 <= kTtRing * block && oRing % 128 == 0 && block % 128 == 0, "");
};

__device__ __forceinline__ void tmem_st_16x128_x2(uint32_t taddr, uint32_t a, uint32_t b, uint32_t c, uint32_t d) {
  asm volatile("tcgen05.st.sync.aligned.16x128b.x2.b32 [%0], {%1, %2, %3, %4};" ::"r"(taddr), "r"(a), "r"(b), "r"(c), "r"(d) : "memory");
}
__device__ __forceinline__ void tmem_st_16x128_x16(uint32_t taddr, const uint32_t (&r)[32]) {
  asm volatile(
      "tcgen05.st.sync.aligned.16x128b.x16.b32 [%0], {%1, %2, %3, %4, %5, %6, %7, %8, %9, %10, "
      "%11, %12, %13, %14, %15, %16, %17, %18, %19, %20, %21, %22, %23, %24, %25, %26, %27, "
      "%28, %29, %30, %31, %32};" ::"r"(taddr),
      SWA_I32(r)
      : "memory");
}
__device__ __forceinline__ void tmem_st_16x128_x8(uint32_t taddr, const uint32_t (&r)[16]) {
  asm volatile(
      "tcgen05.st.sync.aligned.16x128b.x8.b32 [%0], {%1, %2, %3, %4, %5, %6, %7, %8, %9, %10, "
      "%11, %12, %13, %14, %15, %16};" ::"r"(taddr),
      "r"(r[0]), "r"(r[1]), "r"(r[2]), "r"(r[3]), "r"(r[4]), "r"(r[5]), "r"(r[6]), "r"(r[7]), "r"(r[8]), "r"(r[9]), "r"(r[10]),
      "r"(r[11]), "r"(r[12]), "r"(r[13]), "r"(r[14]), "r"(r[15])
      : "memory");
}
// Order of floats as whole numbers.
__device__ __forceinline__ int ordered(float x) {
  const int i = __float_as_int(x);
  return i ^ ((i >> 31) & 0x7fffffff);
}
__device__ __forceinline__ float unordered(int i) { return __int_as_float(i ^ ((i >> 31) & 0x7fffffff)); }
__device__ __forceinline__ uint32_t hmul2_u(uint32_t a, __half2 b) {
  const __half2 r = __hmul2(*reinterpret_cast<const __half2*>(&a), b);
  return *reinterpret_cast<const uint32_t*>(&r);
}
__device__ __forceinline__ uint32_t hfma2_u(uint32_t a, uint32_t s, uint32_t z) {
  const __half2 r = __hfma2(*reinterpret_cast<const __half2*>(&a), *reinterpret_cast<const __half2*>(&s), *reinterpret_cast<const __half2*>(&z));
  return *reinterpret_cast<const uint32_t*>(&r);
}
__device__ __forceinline__ uint32_t pack_f16x2(float lo, float hi) {
  const __half2 r = __floats2half2_rn(lo, hi);
  return *reinterpret_cast<const uint32_t*>(&r);
}
constexpr uint32_t kKeyOff = 4u;                 // flags of a key: no such key; 1, 2: values of group 0, 1 not finite
// Size of a group's values, whose step and centre are w (bf16), as an exponent of fp32; 0: nothing, -1: not finite. The
// values are below four times it.
__device__ __forceinline__ int value_size(uint32_t w) {
  const int es = w >> 7 & 255u, ez = w >> 23 & 255u;
  return max(es, ez) == 255 ? -1 : max(es > 0 ? es + 3 : 0, ez);
}
// Power of two e by which a key's values of size `top` are taken down (up below 0). 0 for those of 2^-4 to 2^5, which
// need none of it: with P beside them as little as 2^-29 of a row's largest, what is cut off P (2^-25) is below 2^-19 of
// the row's sum there; values of all that fp16 holds, 2^-12 to 2^13, would make it 2^-3. Never below -85, so that P's sum,
// whose terms are P 2^-e, stays in fp32. (Keys whose values lie 2^120 apart leave it.)
__device__ __forceinline__ int value_shift(int top) {
  const int e = top - 127;
  return top <= 0 ? 0 : (e > 4 ? e - 4 : (e < -4 ? max(e + 4, -85) : 0));
}
__device__ __forceinline__ float exp2i(int e) { return __uint_as_float(static_cast<uint32_t>(127 + e) << 23); }

template <int NR, bool kPolled>
__global__ void __launch_bounds__(TtShape<NR>::warps * 32, 1) tree_tc_kernel(const __grid_constant__ TreeAttnArgs a) {
  using S = TtShape<NR>;
  constexpr int D = kTtD, E = D / 32, TB = tile_bytes(D);
  extern __shared__ __align__(1024) uint8_t smem[];
  const uint32_t sbase = smem_u32(smem);
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
  const TreeShare share = tree_share<NR, S::warps * 32>(a);
  if (share.none) return;
  const int b = share.b, h = share.h, qg = share.qg;
  const int G = a.Hq / a.c.Hkv;
  uint32_t bad = 0;
  const TreeReq req = tree_req(a.cu, a.lens, b, a.N, a.max_new, static_cast<long long>(a.max_pages) * a.c.page);
  if (req.bad || (sbase & 1023u)) bad = DEV_ERR_BOUNDS;      // (swizzle atoms need 1024-byte aligned tiles)
  if (share.ci == 0 && qg == 0) tree_zero<D, S::warps>(a, req, b, h, G);
  if (bad && tid == 0) atomicOr(a.status, bad);
  const int row_q0 = qg * NR, nq = min(NR, req.n * G - row_q0);
  if (nq <= 0 || (sbase & 1023u)) return;
  const int len = req.ctx + req.n;
  const int lo = a.window >= 0 && req.ctx - a.window > 0 ? req.ctx - a.window : 0;
  const int t_lo = lo / kTile, t_hi = (len + kTile - 1) / kTile;     // tiles [t_lo, t_hi)
  const int chunks = max(1, (t_hi - t_lo + share.chunk - 1) / share.chunk);
  if (share.ci >= chunks) return;
  const int t0 = t_lo + share.ci * share.chunk, t1 = min(t_hi, t0 + share.chunk);
  const int blocks = (t1 - t0 + kTtTiles - 1) / kTtTiles;

  auto bar = [&](int i) { return sbase + S::oBar + 8u * static_cast<uint32_t>(i); };
  uint32_t* flags = reinterpret_cast<uint32_t*>(smem + S::oBar + S::COUNT * 8);    // abort, last, tensor memory, lowest key seen by all
  TreeRow* rows = reinterpret_cast<TreeRow*>(smem + S::oRow);
  int* tpos = reinterpret_cast<int*>(smem + S::oPos);
  float* rowm = reinterpret_cast<float*>(smem + S::oM);          // maxima, negated, then their last rises
  uint32_t* rownan = reinterpret_cast<uint32_t*>(smem + S::oNan);
  volatile int* fresh = reinterpret_cast<volatile int*>(smem + S::oFresh);
  const WaitCtl<kPolled> ctl{flags, a.status, a.wait_limit_ns};
  if (tid == 0) {
    for (int i = 0; i < kTtRing; ++i) {
      mbar_init(bar(S::RAW + i), 1);
      mbar_init(bar(S::RAWFREE + i), 12);
    }
    for (int i = 0; i < 2; ++i) {
      mbar_init(bar(S::KFULL + i), 8);
      mbar_init(bar(S::KFREE + i), 1);
      mbar_init(bar(S::PFULL + i), S::soft);
      mbar_init(bar(S::VFULL + i), 4);
      mbar_init(bar(S::PVDONE + i), 1);
    }
    for (int i = 0; i < kTtScales; ++i) mbar_init(bar(S::SCALES + i), 8);
    mbar_init(bar(S::SFULL), 1);
    mbar_init(bar(S::SFREE), S::soft);
    mbar_init(bar(S::FINAL), 2);
    fence_mbar_init();
    flags[0] = 0;
    flags[3] = 0;
  }
  if (warp == S::mma) {
    tmem_alloc(smem_u32(flags + 2), 512);
    tmem_relinquish();
  }
  tree_rows<NR, S::warps * 32>(a, req, row_q0, nq, G, rows, tpos, bad);       // (row i by thread i)
  static_assert(NR <= S::warps * 32, "");
  for (int i = tid; i < NR; i += S::warps * 32) {
    rowm[i] = 0.f;
    rownan[i] = 0;
    fresh[i] = rows[i].lo != INT32_MAX;       // no key seen yet
    if (i < NR / 32) fresh[NR + i] = 1;       // some of these 32 rows: its blocks take the way of a raise
  }
  // the centres' K block: zeros beside the two sums
  for (int i = tid; warp < S::mma && i < S::N * 2; i += S::mma * 32)
    st_shared_v4(sbase + S::oQ + 2 * S::q_block + (i >> 1) * 128 + ((i & 1) ^ (i >> 1 & 7)) * 16, 0u, 0u, 0u, 0u);
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  const uint32_t tmem = flags[2];

  bool ok = true;
  const int q4 = warp & 3;                                       // quarter of tensor memory
  const uint32_t lanes = static_cast<uint32_t>(q4 * 32) << 16;
  // Every entry of a normed query is below sqrt(D) max|gain|: one power of two for all rows.
  float up;
  {
    float top = 1.f;
    if (a.gq != nullptr) {
      float g[E];
      load_vec<E>(a.gq + lane * E, g);
      top = fmaxf(fmaxf(fabsf(g[0]), fabsf(g[1])), fmaxf(fabsf(g[2]), fabsf(g[3])));
#pragma unroll
      for (int o = 16; o > 0; o >>= 1) top = fmaxf(top, __shfl_xor_sync(0xffffffffu, top, o));
    }
    top *= 11.3137085f * 1.4426950408889634f * a.scale;
    int e = static_cast<int>((__float_as_uint(top) >> 23) & 255u) - 127;
    e = e < -100 ? -100 : (e > 100 ? 100 : e);
    up = __uint_as_float(static_cast<uint32_t>(127 + 13 - e) << 23);
  }
  const float down = 1.0f / up;                                  // a power of two
  auto at = [&](int n, int k) {                                  // K element k of row n of Q
    return reinterpret_cast<__half*>(smem + S::oQ + (k >> 6) * S::q_block + n * 128 + (((k & 63) >> 3) ^ (n & 7)) * 16 + (k & 7) * 2);
  };
  if (warp < S::mma) {
    tree_sight<NR, S::mma>(a, req, rows, tpos, warp);
    query_rows<D>(a, warp, NR, S::mma, up,
        [&](int i, int& pos) -> const elem_t* {
          const int row = row_q0 + i;
          pos = rows[i].pos;
          return rows[i].lo != INT32_MAX ? a.q + (static_cast<long long>(req.row0 + row / G) * a.Hq + h * G + row % G) * D : nullptr;
        },
        [&](int i, int c, __half hi, __half lo2) {
          // the order in which a lane's numbers of a key make its operand: pair k of lane j in column 4 k + j
          const int k = 4 * (2 * (c >> 6) + ((c & 15) >> 3)) + (c & 3), j = (c & 63) >> 4, e = 2 * (4 * k + j) + ((c & 7) >> 2);
          *at(i, e) = hi;
          *at(NR + i, e) = lo2;
        },
        [&](int i, int g, float, float sum) {
          const float v = sum * 0.015625f;                       // below 2^14 again
          const __half hi = __float2half_rn(v);
          *at(i, 128 + g) = hi;
          *at(NR + i, 128 + g) = __float2half_rn(v - __half2float(hi));
        });
  }
  // Q is written: the warps up to the issuer meet here (the loader has work of its own till the end)
  if (warp <= S::mma_o) {
    if (warp < S::mma && lane == 0) {
      int low = 0;
      for (int i = warp; i < NR; i += S::mma) low = max(low, rows[i].lo == INT32_MAX ? 0 : rows[i].lo);
      atomicMax(reinterpret_cast<int*>(flags + 3), low);
    }
    fence_async_smem();
    named_bar_sync(1, (S::mma_o + 1) * 32);
  }
  const int all_lo = static_cast<int>(*reinterpret_cast<volatile uint32_t*>(flags + 3));

  if (warp < S::soft) setmaxnreg_inc<S::regs_soft>();
  else if (warp < S::mma) setmaxnreg_dec<S::regs_convert>();
  else setmaxnreg_dec<S::regs_rest>();
  if (warp < S::soft) {
    // ---------------- softmax: thread = key q4 * 32 + lane, rows r0 .. r0 + 31 ----------------
    const int key_in = q4 * 32 + lane, half = warp >> 2, r0 = half * 32;
    const int my_bar = 2 + half;
    // (A wait that ran out ends no warp's loop here: the four warps of these rows meet at barriers in it that have no
    // time limit. Those that go on do so without waiting, on whatever lies there.)
    float l[32];
#pragma unroll
    for (int i = 0; i < 32; ++i) l[i] = 0.f;
    for (int n = 0; n < blocks; ++n) {
      const int key0 = (t0 + n * kTtTiles) * kTile, key = key0 + key_in;
      ok = ok && mbar_wait_warp(bar(S::SFULL), n & 1, ctl);
      tc_fence_after();
      const float2 fk = *reinterpret_cast<const float2*>(smem + S::oFk + (n % kTtScales * kTtKeys + key_in) * 8);
      const uint32_t kflag = __float_as_uint(fk.y);
      float x[32];
      {
        uint32_t hi[32], lw[32];
        tmem_ld32(tmem + lanes + S::cS + r0, hi);
        tmem_ld32(tmem + lanes + S::cS + NR + r0, lw);
        tmem_wait_ld(hi);
        reg_fence(lw);
#pragma unroll
        for (int i = 0; i < 32; i += 2)
          fadd2(x[i], x[i + 1], __uint_as_float(hi[i]), __uint_as_float(hi[i + 1]), __uint_as_float(lw[i]), __uint_as_float(lw[i + 1]));
      }
      tc_fence_before();
      __syncwarp();
      if (lane == 0) mbar_arrive(bar(S::SFREE));
      const float f = fk.x * down;
#pragma unroll
      for (int i = 0; i < 32; i += 4) {       // relative to the rows' maxima from here on
        const float4 m = *reinterpret_cast<const float4*>(rowm + r0 + i);
        ffma2(x[i], x[i + 1], x[i], x[i + 1], f, f, m.x, m.y);
        ffma2(x[i + 2], x[i + 3], x[i + 2], x[i + 3], f, f, m.z, m.w);
      }
      const bool edge = key0 < all_lo || key0 + kTtKeys > req.ctx;        // of the block
      // (one branch for both that are seldom: with one of their own for the shifts 178 us for 173)
      if (edge || (kflag & ~3u)) {
        if (kflag >> 8) {
          const float shift = static_cast<float>(static_cast<int>(kflag) >> 8);
#pragma unroll
          for (int i = 0; i < 32; i += 2) fadd2_acc(x[i], x[i + 1], shift, shift);
        }
        if (edge || (kflag & kKeyOff)) {
          const int d = key - req.ctx;
#pragma unroll
          for (int i = 0; i < 32; ++i) {
            const int4 w = *reinterpret_cast<const int4*>(rows + r0 + i);    // lo, pos, seen
            const uint32_t word = static_cast<uint32_t>(d & 32 ? w.w : w.z);
            const bool on = (d < 0 ? key >= w.x : (d < kTreeTokens) & static_cast<bool>(word >> (d & 31) & 1u)) & !(kflag & kKeyOff);
            if (!on) x[i] = -INFINITY;
          }
        }
      }
      if (kflag & 3u) {                 // values that are not finite: the rows that see them say so at the end
#pragma unroll
        for (int i = 0; i < 32; ++i)
          if (x[i] != -INFINITY) atomicOr(rownan + r0 + i, kflag & 3u);
      }
      // does a logit pass its row's maximum by too much?
      float over = fmax3(x[0], x[1], x[2]);
#pragma unroll
      for (int i = 3; i < 31; i += 2) over = fmax3(over, x[i], x[i + 1]);
      over = fmaxf(over, x[31]);
      if (fresh[NR + half] || !named_bar_and(my_bar, 128, !(over > kTtRaise))) {
        int* red = reinterpret_cast<int*>(smem + S::oRed) + q4 * NR + r0;
#pragma unroll
        for (int i = 0; i < 32; ++i) {
          const int t = __reduce_max_sync(0xffffffffu, ordered(x[i] == x[i] ? x[i] : -INFINITY));
          if (lane == i) red[i] = t;
        }
        named_bar_sync(my_bar, 128);
        if (q4 == 0) {
          int t = red[lane];
#pragma unroll
          for (int w = 1; w < 4; ++w) t = max(t, red[w * NR + lane]);
          // by how much the row's maximum rises; a first one may be below 0, where it starts
          const float top = unordered(t);
          const bool first = fresh[r0 + lane], none = first && top == -INFINITY;
          const float rise = none ? 0.f : (first ? top - kTtBase : fmaxf(top - kTtBase, 0.f));
          rowm[r0 + lane] -= rise;
          rowm[NR + r0 + lane] = rise;
          fresh[r0 + lane] = none;
          const bool some = __any_sync(0xffffffffu, none);
          if (lane == 0) fresh[NR + half] = some;
        }
        named_bar_sync(my_bar, 128);
#pragma unroll
        for (int i = 0; i < 32; ++i) x[i] -= rowm[NR + r0 + i];
        if (n > 0) {
          // O of the blocks in front of this one, in tensor memory: these rows' columns of this quarter's channels
          ok = ok && mbar_wait_warp(bar(S::PVDONE + ((n - 1) & 1)), ((n - 1) >> 1) & 1, ctl);
          tc_fence_after();
          uint32_t o[32];
          tmem_ld32(tmem + lanes + S::cO + r0, o);
          tmem_wait_ld(o);
#pragma unroll
          for (int i = 0; i < 32; ++i) {
            const float rise = rowm[NR + r0 + i], al = rise > 0.f ? ex2_approx(-rise) : 1.f;     // (below 0: nothing summed yet)
            o[i] = __float_as_uint(__uint_as_float(o[i]) * al);
            l[i] *= al;
          }
          tmem_st32(tmem + lanes + S::cO + r0, o);
          tmem_wait_st();
        }
      }
      if (n >= 2) ok = ok && mbar_wait_warp(bar(S::PVDONE + (n & 1)), ((n >> 1) - 1) & 1, ctl);
      const uint32_t p = sbase + S::oP + (n & 1) * S::p_buf + key_in * 128;
      // (read again: a register that is kept till here is one that spills)
      const float back = exp2i(-(*reinterpret_cast<volatile int*>(smem + S::oFk + (n % kTtScales * kTtKeys + key_in) * 8 + 4) >> 8));
#pragma unroll
      for (int i = 0; i < 32; i += 8) {
        uint32_t w[4];
#pragma unroll
        for (int e = 0; e < 8; e += 2) {
          const float p0 = ex2_approx(x[i + e]), p1 = ex2_approx(x[i + e + 1]);
          ffma2(l[i + e], l[i + e + 1], p0, p1, back, back, l[i + e], l[i + e + 1]);
          w[e / 2] = pack_f16x2(p0, p1);
        }
        st_shared_v4(p + static_cast<uint32_t>(((r0 + i) >> 3) ^ (key_in & 7)) * 16, w[0], w[1], w[2], w[3]);
      }
      fence_async_smem();
      tc_fence_before();
      __syncwarp();
      if (lane == 0) mbar_arrive(bar(S::PFULL + (n & 1)));
    }
    // sums over the warp's keys: lane i keeps row i's
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) {
      const bool up_half = lane & o;
#pragma unroll
      for (int i = 0; i < o; ++i) {
        const float send = up_half ? l[i] : l[i + o], keep = up_half ? l[i + o] : l[i];
        l[i] = keep + __shfl_xor_sync(0xffffffffu, send, o);
      }
    }
    reinterpret_cast<float*>(smem + S::oRed)[q4 * NR + r0 + lane] = l[0];
  } else if (warp < S::values0) {
    // ---------------- keys: a tile a warp, as operands of lanes 32 q4 + 16 u .. ----------------
    const int r = lane >> 2, j = lane & 3, u = (warp - S::keys0) >> 2, tile = 2 * q4 + u;
    for (int n = 0; n < blocks; ++n) {
      const int st = n % kTtRing, ks = n & 1;
      if (!(ok = mbar_wait_warp(bar(S::RAW + st), (n / kTtRing) & 1, ctl))) break;
      const uint32_t miss = *reinterpret_cast<volatile uint32_t*>(smem + S::oMiss + 4 * st);
      const uint8_t* at = smem + S::oRing + st * S::block + tile * TB;
      uint32_t kw[2][4];
      float s[2][2], z[2][2];
#pragma unroll
      for (int i = 0; i < 2; ++i) {
        ld_words<4>(at + (r + 8 * i) * (D / 2) + j * 16, kw[i]);
        ld_scales<2>(at + 16 * D + (r + 8 * i) * 8, s[i], z[i]);
      }
      const int key_tile = (t0 + n * kTtTiles + tile) * kTile;
      // lane = (token, group): steps and centres of the values, in fp16, 0 where they are not to be used, and the token's flags
      uint32_t value = *reinterpret_cast<const uint32_t*>(at + 17 * D + lane * 4), flags_v;
      {
        const int mine = value_size(value), other = __shfl_xor_sync(0xffffffffu, mine, 1), key = key_tile + (lane >> 1);
        const int shift = value_shift(max(mine, other));
        const bool off = (miss >> tile & 1u) || key < lo || key >= len;
        const float fit = exp2i(-shift);
        value = off || mine < 0 ? 0u : pack_f16x2(__uint_as_float(value << 16) * fit, __uint_as_float(value & 0xFFFF0000u) * fit);
        flags_v = off ? kKeyOff : static_cast<uint32_t>(shift) << 8 | static_cast<uint32_t>(mine) >> 31 | static_cast<uint32_t>(other) >> 31 << 1;
      }
      uint32_t out[32], zw[2];
      float fk[2];
#pragma unroll
      for (int i = 0; i < 2; ++i) {
        const float top = fmaxf(fmaxf(fabsf(s[i][0]), fabsf(s[i][1])) * 8.f, fmaxf(fabsf(z[i][0]), fabsf(z[i][1])));
        int e = static_cast<int>((__float_as_uint(top) >> 23) & 255u) - 127;
        e = e < -100 ? -100 : (e > 100 ? 100 : e);
        const float fit = __uint_as_float(static_cast<uint32_t>(127 + 8 - e) << 23);
        const __half2 s0 = __float2half2_rn(s[i][0] * fit), s1 = __float2half2_rn(s[i][1] * fit);
        const __half2 zz = __floats2half2_rn(z[i][0] * fit * 64.f, z[i][1] * fit * 64.f);
        zw[i] = j == 0 ? *reinterpret_cast<const uint32_t*>(&zz) : 0u;
        fk[i] = __uint_as_float(static_cast<uint32_t>(127 - 8 + e) << 23);
#pragma unroll
        for (int x = 0; x < 4; ++x) {
          uint32_t t[4];
          widen_f16(kw[i][x], t);
#pragma unroll
          for (int k = 0; k < 4; ++k) out[2 * (4 * x + k) + i] = hmul2_u(t[k], x < 2 ? s0 : s1);
        }
      }
      __syncwarp();
      if (lane == 0) mbar_arrive(bar(S::RAWFREE + st));
      // S of the block two in front is done, so the softmax is past the fourth in front, and O of the sixth is done: the
      // places of the scales eight in front are free
      if (n >= 2 && !(ok = mbar_wait_warp(bar(S::KFREE + ks), ((n >> 1) - 1) & 1, ctl))) break;
      tc_fence_after();
      float* kfac = reinterpret_cast<float*>(smem + S::oFk + (n % kTtScales * kTtKeys + tile * kTile) * 8);
      if (j == 0) {
#pragma unroll
        for (int i = 0; i < 2; ++i) kfac[2 * (r + 8 * i)] = fk[i];
      }
      if (!(lane & 1)) kfac[lane + 1] = __uint_as_float(flags_v);
      {
        uint16_t* to = reinterpret_cast<uint16_t*>(smem + S::oVs) + (n % kTtScales * 2 + (lane & 1)) * 2 * kTtKeys + tile * kTile + (lane >> 1);
        to[0] = static_cast<uint16_t>(value);
        to[kTtKeys] = static_cast<uint16_t>(value >> 16);
      }
      const uint32_t to = tmem + lanes + (static_cast<uint32_t>(16 * u) << 16) + S::cK + static_cast<uint32_t>(ks) * S::kstep;
      tmem_st_16x128_x16(to, out);
      tmem_st_16x128_x2(to + 64, zw[0], zw[1], 0u, 0u);
      tmem_wait_st();
      tc_fence_before();
      __syncwarp();
      if (lane == 0) {
        mbar_arrive(bar(S::KFULL + ks));
        mbar_arrive(bar(S::SCALES + n % kTtScales));
      }
    }
  } else if (warp < S::mma) {
    // ---------------- values: channels 64 g + 8 r + 4 u + i of quarter q4 = (g, u), all eight tiles ----------------
    const int r = lane >> 2, j = lane & 3, g = q4 >> 1;
    for (int n = 0; n < blocks; ++n) {
      const int st = n % kTtRing, vs = n & 1;
      if (!(ok = mbar_wait_warp(bar(S::RAW + st), (n / kTtRing) & 1, ctl))) break;
      // a place for each of eight blocks: the keys' warps may be some blocks ahead
      if (!(ok = mbar_wait_warp(bar(S::SCALES + n % kTtScales), (n / kTtScales) & 1, ctl))) break;
      if (n >= 2 && !(ok = mbar_wait_warp(bar(S::PVDONE + vs), ((n >> 1) - 1) & 1, ctl))) break;
      tc_fence_after();
      const uint8_t* sc = smem + S::oVs + (n % kTtScales * 2 + g) * 4 * kTtKeys;
#pragma unroll
      for (int t4 = 0; t4 < kTtTiles; t4 += 4) {
        uint32_t out[2][16];
#pragma unroll
        for (int t = 0; t < 4; ++t) {
          const uint8_t* at = smem + S::oRing + st * S::block + (t4 + t) * TB + 8 * D;
#pragma unroll
          for (int half = 0; half < 2; ++half) {
            uint32_t x[4];
            const uint32_t w = *reinterpret_cast<const uint32_t*>(at + (j + 4 * half) * D + r * 16 + q4 * 4);
            const int pair = (t4 + t) * 8 + j + 4 * half;
            const uint32_t s2 = *reinterpret_cast<const uint32_t*>(sc + 4 * pair), z2 = *reinterpret_cast<const uint32_t*>(sc + 2 * kTtKeys + 4 * pair);
            widen_f16(w, x);
#pragma unroll
            for (int i = 0; i < 4; ++i) out[i >> 1][4 * t + 2 * half + (i & 1)] = hfma2_u(x[i], s2, z2);
          }
        }
#pragma unroll
        for (int bl = 0; bl < 2; ++bl)
          tmem_st_16x128_x8(tmem + lanes + (static_cast<uint32_t>(16 * bl) << 16) + S::cV + static_cast<uint32_t>(vs) * S::vstep + t4 * 8, out[bl]);
      }
      tmem_wait_st();
      tc_fence_before();
      __syncwarp();
      if (lane == 0) {
        mbar_arrive(bar(S::VFULL + vs));
        mbar_arrive(bar(S::RAWFREE + st));
      }
    }
  } else if (warp == S::load) {
    // ---------------- loader: pages 32 tiles (4 blocks) ahead of their use ----------------
    const int per_page = a.c.page / kTile;
    const long long head_off = static_cast<long long>(h) * per_page;
    auto look = [&](int i) {                                     // tile t0 + i of the request in the cache, or -1
      const int t = t0 + i;
      if (t >= t1) return -2ll;
      const int pi = t / per_page, pg = a.table[static_cast<long long>(b) * a.max_pages + pi];
      if (pg >= 0 && pg < a.c.n_pages) return static_cast<long long>(pg) * a.c.Hkv * per_page + head_off + (t - pi * per_page);
      return -1ll;
    };
    long long now = look(lane), next = look(32 + lane);
    int n = 0;
    for (; n < blocks; ++n) {
      const int st = n % kTtRing;
      if (n > 0 && (n & 3) == 0) {
        now = next;
        next = look(8 * n + 32 + lane);
      }
      if (n >= kTtRing && !(ok = mbar_wait_warp(bar(S::RAWFREE + st), (n / kTtRing - 1) & 1, ctl))) break;
      const long long at = __shfl_sync(0xffffffffu, now, (8 * n & 31) + (lane & 7));
      const uint32_t there = __ballot_sync(0xffffffffu, at >= 0) & 255u, none = __ballot_sync(0xffffffffu, at == -1) & 255u;
      if (none) bad = DEV_ERR_BOUNDS;
      if (lane == 0) {
        *reinterpret_cast<volatile uint32_t*>(smem + S::oMiss + 4 * st) = there ^ 255u;
        mbar_arrive_expect_tx(bar(S::RAW + st), __popc(there) * TB);
      }
      __syncwarp();
      if (lane < 8 && at >= 0) bulk_load(sbase + S::oRing + st * S::block + lane * TB, a.c.data + at * TB, TB, bar(S::RAW + st));
    }
    // the copies still on their way land before the memory is used again (also where all are issued: the warps that wait
    // for them may have given up)
    for (int i = max(0, n - kTtRing); i < n; ++i) mbar_wait_drain(bar(S::RAW + i % kTtRing), (i / kTtRing) & 1, kDrainLimitNs);
  } else if (warp == S::mma) {
    if (lane == 0) {
      constexpr uint32_t id_s = (1u << 4) | (static_cast<uint32_t>(S::N >> 3) << 17) | (8u << 24);      // fp16, M = 128
      const uint64_t dQ = sdesc_sw128(sbase + S::oQ, 16, 1024);
      auto scores = [&](int n) {
        const int ks = n & 1;
        if (!(ok = mbar_wait(bar(S::KFULL + ks), (n >> 1) & 1, ctl))) return;
        if (n > 0 && !(ok = mbar_wait(bar(S::SFREE), (n - 1) & 1, ctl))) return;
        tc_fence_after();
        const uint32_t ta = tmem + S::cK + static_cast<uint32_t>(ks) * S::kstep;
        static_for<0, 9>([&](auto kc) {
          constexpr int k = decltype(kc)::value;
          umma_ts_imm<id_s, k * 8, (((k >> 2) * S::q_block + (k & 3) * 32) >> 4)>(tmem + S::cS, ta, dQ, k > 0 ? 1u : 0u, 1u);
        });
        umma_commit(bar(S::SFULL));
        umma_commit(bar(S::KFREE + ks));
      };
      for (int n = 0; n < blocks && ok; ++n) scores(n);
      umma_commit(bar(S::FINAL));         // every product issued has completed, after a wait that ran out too
      mbar_wait_drain(bar(S::FINAL), 0, kDrainLimitNs);
    }
  } else if (warp == S::mma_o) {
    if (lane == 0) {
      constexpr uint32_t id_o = (1u << 4) | (1u << 16) | (static_cast<uint32_t>(NR >> 3) << 17) | (8u << 24);    // fp16, P^T by rows
      const uint64_t dP = sdesc_sw128(sbase + S::oP, 16, 1024);
      for (int n = 0; n < blocks; ++n) {
        const int ps = n & 1;
        if (!(ok = mbar_wait(bar(S::VFULL + ps), (n >> 1) & 1, ctl))) break;
        if (!(ok = mbar_wait(bar(S::PFULL + ps), (n >> 1) & 1, ctl))) break;
        tc_fence_after();
        const uint32_t ta = tmem + S::cV + static_cast<uint32_t>(ps) * S::vstep;
        const uint64_t db = sdesc_add(dP, ps * S::p_buf);
        static_for<0, 8>([&](auto kc) {
          constexpr int k = decltype(kc)::value;
          umma_ts_imm<id_o, k * 8, k * 2048 / 16>(tmem + S::cO, ta, db, (n > 0 || k > 0) ? 1u : 0u, 1u);
        });
        umma_commit(bar(S::PVDONE + ps));
      }
      umma_commit(bar(S::FINAL));
      mbar_wait_drain(bar(S::FINAL), 0, kDrainLimitNs);
    }
  }
  __syncwarp();
  if (bad) atomicOr(a.status, bad);
  __syncthreads();                        // (every copy has landed: the loader waited for the last ones)
  tc_fence_after();

  // O^T into rows [row][channel]
  float* jo = reinterpret_cast<float*>(smem + S::oJoin);
  if (warp < S::soft) {
    const int r0 = (warp >> 2) * 32, L = lane & 15;
    const int ch = 64 * (q4 >> 1) + 8 * (L & 7) + 4 * (q4 & 1) + 2 * (lane >> 4) + (L >> 3);
    uint32_t o[32];
    tmem_ld32(tmem + lanes + S::cO + r0, o);
    tmem_wait_ld(o);
#pragma unroll
    for (int i = 0; i < 32; ++i) {
      const bool odd = rownan[r0 + i] >> (q4 >> 1) & 1u;
      jo[(r0 + i) * D + ch] = odd ? __int_as_float(0x7fffffff) : __uint_as_float(o[i]);
    }
  }
  tc_fence_before();
  __syncthreads();
  if (warp == S::mma) tmem_dealloc(tmem, 512);
  auto head_of = [&](int i) {       // index of row i's head in o and lse
    const int row = row_q0 + i;
    return static_cast<long long>(req.row0 + row / G) * a.Hq + h * G + row % G;
  };
  const float* red = reinterpret_cast<const float*>(smem + S::oRed);
  for (int i = warp; i < nq; i += S::warps) {      // a warp a row
    float o[E], top = -rowm[i], sum = (red[i] + red[NR + i]) + (red[2 * NR + i] + red[3 * NR + i]);
    load_vec<E>(jo + i * D + lane * E, o);
    if (rows[i].lo == INT32_MAX) {       // sees nothing: blocks that every other row sees were not masked for it
      top = -1e30f;
      sum = 0.f;
#pragma unroll
      for (int e = 0; e < E; ++e) o[e] = 0.f;
    } else if (fresh[i]) {               // nothing of this chunk: no maximum for the join (its sums are 0, or a key's NaN)
      top = -1e30f;
    }
    tree_row_out<D>(a, chunks, share.ci, share.part0, NR, i, head_of(i), o, top, sum);
  }
  if (chunks == 1) return;
  __syncthreads();
  if (tid == 0) {
    __threadfence();      // after the barrier it covers what the CTA wrote
    flags[1] = atomicAdd(a.count + share.item, 1u) == static_cast<unsigned>(chunks - 1);
  }
  __syncthreads();
  if (!flags[1]) return;
  __threadfence();
  if (tid == 0) a.count[share.item] = 0;        // for the next call
  tree_join<D, 1, 4>(a, chunks, share.part0, NR, warp, S::warps, nq, head_of);
}

}  // namespace kv4
}  // namespace swa
