// Drafted tokens over the 4-bit paged cache: positions and visibility of a
// request's tree of drafted tokens, their attention, and the move of the
// accepted ones to their places.
//
// The tokens of a step lie one request behind the other: those of request b are
// rows cu[b] .. cu[b + 1] - 1 (at most kTreeTokens), and their keys and values
// are in the cache already, as the last tokens of its lens[b], in their order.
// The request's context is what is in front of them.
#pragma once

#include "kv4_attn.cuh"

namespace swa {
namespace kv4 {

constexpr int kTreeTokens = 64;      // drafted tokens of a request: bits of a mask

// ---------------------------------------------------------------------------
// Tree: token i sees itself and what its parent sees; its position is the
// context's length and its depth.
//   pos[i] = ctx + |above(i)| - 1,  seen[i] = bits of above(i),
//   above(i) = {i} and above(parent[i]); parent -1: the context.
// A warp a request; a lane walks up from its two tokens.
// ---------------------------------------------------------------------------
struct TreeArgs {
  int B, N, max_new;                 // N: rows
  const int32_t* parent; const int32_t* cu; const int32_t* lens;
  int32_t* pos; int64_t* seen;       // [N]
  uint32_t* status;                  // or NULL
};

// A request's rows: false where cu is not plausible (and nothing is to be touched).
struct TreeReq {
  int row0, n, ctx;                  // n = 0, all rows hidden: bad
  int rows;                          // rows that are the request's
  bool bad;
};
__device__ __forceinline__ TreeReq tree_req(const int32_t* cu, const int32_t* lens, int b, int N, int max_new, long long cap) {
  TreeReq r{cu[b], 0, 0, 0, false};
  const int end = cu[b + 1], len = lens[b];
  if (r.row0 < 0 || end < r.row0 || end > N) {
    r.bad = true;
    r.row0 = 0;
    return r;
  }
  r.rows = end - r.row0;
  r.ctx = len - r.rows;
  if (len < 0 || len > cap || r.rows > max_new || r.ctx < 0) r.bad = true;
  else r.n = r.rows;
  return r;
}

// Rows in front of the first request; none where its rows are not plausible.
__device__ __forceinline__ int tree_front(const int32_t* cu, int N) {
  const int row0 = cu[0], end = cu[1];
  return row0 > 0 && end >= row0 && end <= N ? row0 : 0;
}

constexpr int kTreeWarps = 4;
__global__ void __launch_bounds__(kTreeWarps * 32) tree_kernel(const __grid_constant__ TreeArgs a) {
  __shared__ int up[kTreeWarps][kTreeTokens];
  const int lane = threadIdx.x & 31, wid = threadIdx.x >> 5;
  const long long stride = static_cast<long long>(gridDim.x) * kTreeWarps;
  uint32_t bad = 0;
  for (long long b = static_cast<long long>(blockIdx.x) * kTreeWarps + wid; b < a.B; b += stride) {
    const TreeReq q = tree_req(a.cu, a.lens, static_cast<int>(b), a.N, a.max_new, INT32_MAX);
    if (q.bad) bad = DEV_ERR_BOUNDS;
    for (int i = lane; i < q.n; i += 32) {
      const int p = a.parent[q.row0 + i];
      up[wid][i] = p >= -1 && p < i ? p : -2;
    }
    __syncwarp();
    for (int i = lane; i < q.rows; i += 32) {
      unsigned long long m = 0;
      if (i < q.n) {
        int t = i;
        while (t >= 0) {               // strictly down: a parent is in front of its child
          m |= 1ull << t;
          t = up[wid][t];
        }
        if (t != -1) {
          m = 0;
          bad = DEV_ERR_BOUNDS;
        }
      }
      a.seen[q.row0 + i] = static_cast<int64_t>(m);
      a.pos[q.row0 + i] = m ? q.ctx + __popcll(m) - 1 : 0;
    }
    __syncwarp();
  }
  // rows of no request: in front of the first and behind the last one
  auto none = [&](long long from, long long to) {
    for (long long i = from + static_cast<long long>(blockIdx.x) * blockDim.x + threadIdx.x; i < to;
         i += static_cast<long long>(gridDim.x) * blockDim.x) {
      a.seen[i] = 0;
      a.pos[i] = 0;
    }
  };
  const int used = a.cu[a.B];
  none(0, tree_front(a.cu, a.N));
  if (used < 0 || used > a.N) bad = DEV_ERR_BOUNDS;
  else none(used, a.N);
  if (bad && a.status) atomicOr(a.status, bad);
}

// ---------------------------------------------------------------------------
// Move: the tokens of slots src[b][t] become those of dst[b][t]. All of a row b
// are read before any is written. A block a (row, kv head). Held by instructions
// more than by bytes (2048 rows of 32 tokens, 4 kv heads of 128: 27 us with a
// thread for every four bytes of a key and two of a value, 16 with 16 bytes each; the
// bytes take 14.5), and by the sectors that 2 bytes of every 4 touch.
// ---------------------------------------------------------------------------
struct MoveArgs {
  Cache c;
  int B, T;
  const int64_t* src; const int64_t* dst;
  uint32_t* status;
};
constexpr int kMoveThreads = 128;

template <int D>
__global__ void __launch_bounds__(kMoveThreads) move_kernel(const __grid_constant__ MoveArgs a) {
  constexpr int SW = D / 64, KU = D / 32, VU = D / 16, UNITS = KU + VU + 2;      // 16-byte pieces of a key and of a pair of values; scales
  __shared__ uint4 held[kTreeTokens * UNITS];
  __shared__ long long from[kTreeTokens], to[kTreeTokens];      // tiles, in bytes; -1: skipped
  __shared__ uint8_t in_from[kTreeTokens], in_to[kTreeTokens];  // tokens of theirs
  const long long slots = static_cast<long long>(a.c.n_pages) * a.c.page;
  const int n = a.T * UNITS;
  // where piece k of token o of a tile starts
  auto piece = [](int k, int o) {
    if (k < KU) return o * (D / 2) + 16 * k;
    if (k < KU + VU) return 8 * D + (o >> 1) * D + 16 * (k - KU);
    return 16 * D + (k - KU - VU) * D + o * (4 * SW);
  };
  uint32_t bad = 0;
  const long long items = static_cast<long long>(a.B) * a.c.Hkv;
  for (long long it = blockIdx.x; it < items; it += gridDim.x) {
    const long long b = it / a.c.Hkv;
    const int h = static_cast<int>(it - b * a.c.Hkv);
    for (int t = threadIdx.x; t < a.T; t += kMoveThreads) {
      const long long s = a.src[b * a.T + t], d = a.dst[b * a.T + t];
      const bool skip = s == -1 || d == -1, out = s < 0 || s >= slots || d < 0 || d >= slots;
      if (!skip && out) bad = DEV_ERR_BOUNDS;
      from[t] = to[t] = -1;
      if (!out && s != d) {
        from[t] = tile_of<D>(a.c, s, h) - a.c.data;
        to[t] = tile_of<D>(a.c, d, h) - a.c.data;
        in_from[t] = static_cast<uint8_t>(s & 15);
        in_to[t] = static_cast<uint8_t>(d & 15);
      }
    }
    __syncthreads();
    // two pieces of a thread in flight
    for (int u0 = threadIdx.x; u0 < n; u0 += 2 * kMoveThreads) {
      uint4 x[2];
#pragma unroll
      for (int i = 0; i < 2; ++i) {
        const int u = u0 + i * kMoveThreads, t = u / UNITS, k = u - t * UNITS;
        x[i] = make_uint4(0u, 0u, 0u, 0u);
        if (u >= n || from[t] < 0) continue;
        const uint8_t* at = a.c.data + from[t] + piece(k, in_from[t]);
        if (k < KU + VU) x[i] = ld16(at);
        else if constexpr (SW == 2) *reinterpret_cast<uint2*>(&x[i]) = *reinterpret_cast<const uint2*>(at);
        else x[i].x = *reinterpret_cast<const uint32_t*>(at);
      }
#pragma unroll
      for (int i = 0; i < 2; ++i)
        if (u0 + i * kMoveThreads < n) held[u0 + i * kMoveThreads] = x[i];
    }
    __syncthreads();
    for (int u = threadIdx.x; u < n; u += kMoveThreads) {
      const int t = u / UNITS, k = u - t * UNITS;
      if (to[t] < 0) continue;
      uint8_t* at = a.c.data + to[t] + piece(k, in_to[t]);
      const uint4 x = held[u];
      if (k < KU) {
        st16(at, x);
      } else if (k < KU + VU) {          // words of a pair of tokens, 16 bits of each: the other's stay as they are
        const int down = 16 * (in_from[t] & 1);
        uint16_t* y = reinterpret_cast<uint16_t*>(at) + (in_to[t] & 1);
        y[0] = static_cast<uint16_t>(x.x >> down);
        y[2] = static_cast<uint16_t>(x.y >> down);
        y[4] = static_cast<uint16_t>(x.z >> down);
        y[6] = static_cast<uint16_t>(x.w >> down);
      } else if constexpr (SW == 2) {
        *reinterpret_cast<uint2*>(at) = make_uint2(x.x, x.y);
      } else {
        *reinterpret_cast<uint32_t*>(at) = x.x;
      }
    }
    __syncthreads();
  }
  if (bad && a.status) atomicOr(a.status, bad);
}

// ---------------------------------------------------------------------------
// Attention of a request's drafted tokens. Row (token i, query head g of the kv
// head's group) sees key j of the context where pos_i - j <= window, and drafted
// token t where bit t of seen_i is set and pos_i - pos_t <= window.
//
// The rows of one (request, kv head) share its keys and values: they are the
// 16-row operand of both products here (S = Q K^T, O += P V), so that each tile
// of the cache is fetched and widened once for 16 rows, and P goes from one
// product's result to the other's operand without an exchange between lanes.
// The cache's words are the eight-column operand as they are (a lane's numbers
// are of key lane / 4, or of channel lane / 4).
//   RW   warps that hold 16 rows each of the same keys (1, 2 or 4); the other
//        4 / RW - 1 groups of warps take other steps of two tiles.
// Precision: q is two fp16 terms (22 bits: lse is an fp32 output; one term left it
// 2e-4 off). P is one bf16 term in bf16 calls, whose o has 8 bits itself (as in the
// training forward; two take 153 us for 134, 16 requests of 32768 and one token),
// and three in fp32 ones. The products with n - 8 are exact,
// steps and centres multiply the sums in fp32.
// ---------------------------------------------------------------------------
struct TreeAttnArgs : AttnArgs {
  int N, max_new;
  const int32_t* cu; const int32_t* pos; const int64_t* seen;
  int slots, setup;                  // CTAs that run at once (0: chunk is given), and their set-up in tiles
};

constexpr int kQTerms = 2;
constexpr int tree_stages(int rw) { return rw == 1 ? 2 : 4; }
constexpr int tree_ctas_per_sm(int d) { return d == 64 && !kThreeTerms ? 4 : 2; }

template <int D, int RW>
struct TreeSmem {
  static constexpr int rows = 16 * RW, groups = kAttnWarps / RW, stages = tree_stages(RW);
  static constexpr int ring1 = stages * 2 * AttnShape<D>::TB;          // of one group of warps
  static constexpr int ring = groups * ring1;
  static constexpr int q = (ring + 15) / 16 * 16;                     // fp16 rows, hi then lo
  static constexpr int q_end = q + rows * kQTerms * D * 2;
  static constexpr int join = kAttnWarps * 16 * (D + 2) * 4;          // over the rings and the queries
  static constexpr int bars = ((q_end > join ? q_end : join) + 127) / 128 * 128;
  static constexpr int qf = bars + groups * stages * 16;                // full and free barriers
  static constexpr int row = qf + rows * 16;                          // first visible key, pos, seen of each row
  static constexpr int tpos = row + rows * 16;                        // positions of the drafted tokens
  static constexpr int flags = tpos + kTreeTokens * 4;
  static constexpr int bytes = flags + 16;
};

struct TreeRow {
  int lo;                            // first key of the context that it sees; INT_MAX: hidden
  int pos;
  unsigned long long seen;
};

// A CTA's share of a call: the chunk'th chunk of `chunk` tiles of group qg of
// request b's rows under kv head h. Either as the host laid them out (grid x of
// chunks, y of kv heads and groups, z of requests: nothing to be computed), or, for
// long contexts, a flat grid whose CTAs look at all the lengths and find the chunk
// for which the call should end first: the host knows only the longest possible
// request, and a batch that is ragged, or far below its tables' width, left most of
// the GPU idle (64 ragged requests of at most 16384 tokens, 16 query heads on 2: 165 us
// against 66; 16 in fp32 of at most 5000: 39 against 25). Every CTA comes to the same answer: integers, and
// fp32 of them.
struct TreeShare {
  int b, h, qg, ci, chunk;
  long long item, part0;             // its counter, and the first of its chunks' rows in part
  bool none;
};
constexpr int kShareB = 128;         // requests of a call whose CTAs do so
constexpr int kShareN = 128;         // chunks of the longest request that are tried
constexpr int kJoinTiles = 8;        // what a join costs, in tiles
constexpr int kShareTiles = 256;     // tables of at least so many tiles a request

template <int NQ, int kThreads>
__device__ __forceinline__ TreeShare tree_share(const TreeAttnArgs& a) {
  TreeShare x;
  x.none = false;
  if (a.slots == 0) {
    x.b = blockIdx.z;
    x.h = blockIdx.y / a.groups;
    x.qg = blockIdx.y - x.h * a.groups;
    x.ci = blockIdx.x;
    x.chunk = a.chunk;
    x.item = (static_cast<long long>(x.b) * a.c.Hkv + x.h) * a.groups + x.qg;
    x.part0 = x.item * a.splits * NQ;
    return x;
  }
  __shared__ int tiles[kShareB], items[kShareB];
  __shared__ float2 bests[kShareN / 32];
  const int tid = threadIdx.x, lane = tid & 31, wid = tid >> 5, G = a.Hq / a.c.Hkv;
  for (int b = tid; b < a.B; b += kThreads) {
    const TreeReq req = tree_req(a.cu, a.lens, b, a.N, a.max_new, static_cast<long long>(a.max_pages) * a.c.page);
    const int len = req.ctx + req.n, lo = a.window >= 0 && req.ctx - a.window > 0 ? req.ctx - a.window : 0;
    tiles[b] = req.n > 0 ? max(1, (len + kTile - 1) / kTile - lo / kTile) : 1;
    items[b] = a.c.Hkv * max(1, (req.n * G + NQ - 1) / NQ);        // (rows to be zeroed take a CTA a kv head)
  }
  __syncthreads();
  // n / c, rounded up, for quotients of a few hundred: the product is off by less than one
  auto div_up = [](int n, int c, float inv) {
    n += c - 1;
    int q = static_cast<int>(static_cast<float>(n) * inv);
    const long long rest = n - static_cast<long long>(q) * c;
    return q + (rest >= c) - (rest < 0);
  };
  int longest = 1;
  float total = 0.f;                 // (the same sum in every lane: the exchange adds the same pairs)
  for (int b = lane; b < a.B; b += 32) {
    longest = max(longest, tiles[b]);
    total += static_cast<float>(tiles[b]) * static_cast<float>(items[b]);
  }
  longest = __reduce_max_sync(0xffffffffu, longest);
#pragma unroll
  for (int o = 16; o > 0; o >>= 1) total += __shfl_xor_sync(0xffffffffu, total, o);
  static_assert(kShareN <= kThreads, "");
  if (tid < kShareN) {               // thread n: the longest request in n + 1 chunks
    const int c = ((longest + tid) / (tid + 1) + 7) / 8 * 8;
    const float inv = 1.0f / static_cast<float>(c);
    int k = 0;
#pragma unroll 4
    for (int b = 0; b < a.B; ++b) k += items[b] * div_up(tiles[b], c, inv);
    const float own = static_cast<float>((c < longest ? c : longest) + a.setup), per = 1.0f / static_cast<float>(a.slots);
    // whole rounds of equal CTAs, or as short ones fill up: both are bounds
    const float even = ceilf(static_cast<float>(k) * per) * own;
    const float filled = (total + static_cast<float>(k) * a.setup) * per + own;
    const int n = div_up(longest, c, inv);
    float t = fminf(even, filled) + (n > 1 ? kJoinTiles + n / 2 : 0);
    if (k > static_cast<int>(gridDim.x)) t = INFINITY;
    const unsigned least = __reduce_min_sync(0xffffffffu, __float_as_uint(t));        // (positive)
    const int at = __ffs(__ballot_sync(0xffffffffu, __float_as_uint(t) == least)) - 1;
    if (lane == at) bests[wid] = make_float2(t, __int_as_float(c));
  }
  __syncthreads();
  float2 best = bests[0];
#pragma unroll
  for (int i = 1; i < kShareN / 32; ++i)
    if (bests[i].x < best.x) best = bests[i];
  x.chunk = __float_as_int(best.y);
  const float inv = 1.0f / static_cast<float>(x.chunk);
  int first = 0;                     // CTAs of the requests in front of b0
  for (int b0 = 0; b0 < a.B; b0 += 32) {
    const int b = b0 + lane, per = b < a.B ? div_up(tiles[b], x.chunk, inv) : 1, k = b < a.B ? items[b] * per : 0;
    int end = k;
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
      const int v = __shfl_up_sync(0xffffffffu, end, o);
      if (lane >= o) end += v;
    }
    const int at = static_cast<int>(blockIdx.x) - first - (end - k);
    const unsigned here = __ballot_sync(0xffffffffu, at >= 0 && at < k);
    if (here) {
      const int src = __ffs(here) - 1, mine = __shfl_sync(0xffffffffu, at, src), p = __shfl_sync(0xffffffffu, per, src);
      x.b = b0 + src;
      const int it = mine / p, groups = items[x.b] / a.c.Hkv;
      x.h = it / groups;
      x.qg = it - x.h * groups;
      x.ci = mine - it * p;
      x.item = static_cast<int>(blockIdx.x) - x.ci;
      x.part0 = x.item * NQ;
      return x;
    }
    first += __shfl_sync(0xffffffffu, end, 31);
  }
  x.none = true;
  return x;
}

// What the CTA's rows see, and the drafted tokens' positions, into shared memory.
template <int NQ, int kThreads>
__device__ __forceinline__ void tree_rows(const TreeAttnArgs& a, const TreeReq& req, int row_q0, int nq, int G, TreeRow* rows, int* tpos,
                                          uint32_t& bad) {
  for (int i = threadIdx.x; i < req.n; i += kThreads) tpos[i] = a.pos[req.row0 + i];
  for (int i = threadIdx.x; i < NQ; i += kThreads) {
    TreeRow x{INT32_MAX, 0, 0};
    if (i < nq) {
      const int at = req.row0 + (row_q0 + i) / G;
      x.pos = a.pos[at];
      x.seen = static_cast<unsigned long long>(a.seen[at]);
      // a row that sees nothing needs no position
      const bool ok = x.pos >= req.ctx && (a.rcos == nullptr || x.pos < a.rows);
      if (x.seen == 0) x.pos = 0;
      else if (!ok) {
        bad = DEV_ERR_BOUNDS;
        x.seen = 0;
        x.pos = 0;
      } else {
        x.lo = a.window >= 0 && x.pos - a.window > 0 ? x.pos - a.window : 0;
      }
    }
    rows[i] = x;
  }
}

// Then, by kWarps warps behind a barrier: of seen only the request's tokens within the
// row's window stay, so that a mask is one bit of it (tested in full per key and row
// it was 2000 clocks of the first step's 3700, and one request of 32 tokens 8.5 us for
// 7.7; of 64 rows in the tcgen05 form 16.4 for 13.2).
template <int NQ, int kWarps>
__device__ __forceinline__ void tree_sight(const TreeAttnArgs& a, const TreeReq& req, TreeRow* rows, const int* tpos, int w) {
  const int lane = threadIdx.x & 31;
  for (int i = w; i < NQ; i += kWarps) {
    auto near = [&](int t) { return t < req.n && (a.window < 0 || static_cast<long long>(rows[i].pos) - tpos[t] <= a.window); };
    const unsigned lo = __ballot_sync(0xffffffffu, near(lane)), hi = __ballot_sync(0xffffffffu, near(lane + 32));
    if (lane == 0) rows[i].seen &= lo | static_cast<unsigned long long>(hi) << 32;
    __syncwarp();
  }
}

// Rows that hold nothing, by the CTA that answers for them: those of a request
// that is refused, those in front of the first one and those behind the last.
template <int D, int kWarps>
__device__ __forceinline__ void tree_zero(const TreeAttnArgs& a, const TreeReq& req, int b, int h, int G) {
  constexpr int E = D / 32;
  const int lane = threadIdx.x & 31, wid = threadIdx.x >> 5;
#pragma unroll 1
  for (int k = 0; k < 3; ++k) {          // (one loop: instructions that few CTAs run are fetched by all)
    int row0 = 0, row1 = 0;
    if (k == 0 && req.bad) {
      row0 = req.row0;
      row1 = row0 + req.rows;
    } else if (k == 1 && b == 0) {
      row1 = req.row0;                   // (0 where cu is not plausible)
    } else if (k == 2 && b == a.B - 1) {
      row0 = a.cu[a.B];
      row1 = row0 >= 0 ? a.N : row0;
    }
    const float z[E] = {};
    for (long long i = wid; i < static_cast<long long>(row1 - row0) * G; i += kWarps) {
      const long long at = (row0 + i / G) * a.Hq + h * G + i % G;
      store_vec<E>(a.o + at * D + lane * E, z);
      if (lane == 0) a.lse[at] = -INFINITY;
    }
  }
}

// A row's sums o (relative to top, base 2), joined over the warps of a CTA by one
// warp: into o and lse, or beside the other chunks'. part0: of the CTA's item.
template <int D>
__device__ __forceinline__ void tree_row_out(const TreeAttnArgs& a, int chunks, int ci, long long part0, int nq_slot, int i, long long head,
                                             float (&o)[D / 32], float top, float sum) {
  constexpr int E = D / 32;
  const int lane = threadIdx.x & 31;
  if (chunks == 1) {
    finish_head<D>(a, head, o, top, sum);
  } else {
    const long long at = part0 + static_cast<long long>(ci) * nq_slot + i;
    store_vec<E>(a.part + at * D + lane * E, o);
    if (lane == 0) a.part_ml[at] = make_float2(top, sum);
  }
}
// Rows i0, i0 + step .. below nq of all chunks, joined in their order by one warp:
// R rows and U chunks of each in flight, since each load waits out the L2's
// latency (32 requests in a window of 1024 keys, three chunks each: 26.6 us with one row
// after the other, 24.4 so).
template <int D, int R, int U, typename Head>
__device__ __forceinline__ void tree_join(const TreeAttnArgs& a, int chunks, long long part0, int nq_slot, int i0, int step, int nq,
                                          Head head_of) {
  constexpr int E = D / 32;
  const int lane = threadIdx.x & 31;
  for (int i = i0; i < nq; i += R * step) {
    float top[R], sum[R], o[R][E];
    long long at[R];
#pragma unroll
    for (int r = 0; r < R; ++r) {
      at[r] = part0 + (i + r * step < nq ? i + r * step : i);
      top[r] = -1e30f;
      sum[r] = 0.f;
#pragma unroll
      for (int e = 0; e < E; ++e) o[r][e] = 0.f;
    }
    for (int k = lane; k < chunks; k += 32)
#pragma unroll
      for (int r = 0; r < R; ++r) top[r] = fmaxf(top[r], __ldcg(a.part_ml + at[r] + static_cast<long long>(k) * nq_slot).x);
#pragma unroll
    for (int r = 0; r < R; ++r)
#pragma unroll
      for (int x = 16; x > 0; x >>= 1) top[r] = fmaxf(top[r], __shfl_xor_sync(0xffffffffu, top[r], x));
    for (int k0 = 0; k0 < chunks; k0 += U) {
      float2 ml[U][R];
      float x[U][R][E];
#pragma unroll
      for (int u = 0; u < U; ++u) {
        const long long k = static_cast<long long>(k0 + u < chunks ? k0 + u : k0) * nq_slot;
#pragma unroll
        for (int r = 0; r < R; ++r) {
          ml[u][r] = __ldcg(a.part_ml + at[r] + k);
          const float* from = a.part + (at[r] + k) * D + lane * E;
          if constexpr (E == 4) {
            const float4 v = __ldcg(reinterpret_cast<const float4*>(from));
            x[u][r][0] = v.x; x[u][r][1] = v.y; x[u][r][2] = v.z; x[u][r][3] = v.w;
          } else {
            const float2 v = __ldcg(reinterpret_cast<const float2*>(from));
            x[u][r][0] = v.x; x[u][r][1] = v.y;
          }
        }
      }
#pragma unroll
      for (int u = 0; u < U; ++u) {
        if (k0 + u >= chunks) continue;
#pragma unroll
        for (int r = 0; r < R; ++r) {
          const float f = ex2_approx(ml[u][r].x - top[r]);
          sum[r] = fmaf(f, ml[u][r].y, sum[r]);
#pragma unroll
          for (int e = 0; e < E; ++e) o[r][e] = fmaf(f, x[u][r][e], o[r][e]);
        }
      }
    }
#pragma unroll
    for (int r = 0; r < R; ++r)
      if (i + r * step < nq) finish_head<D>(a, head_of(i + r * step), o[r], top[r], sum[r]);
  }
}

// Query rows i0, i0 + step .. below i1 by one warp (query_row's arithmetic), the
// next row's loads in flight beside a row's arithmetic. src(i, pos): row i and its
// position; NULL: a row of zeros. Entries times a power of two that brings them
// below 2^14 (up; 0: each row's own): put(i, channel, hi, lo) as two fp16 terms,
// end(i, group, 1 / power, sum) by lane 0 of each group of 64 channels with their
// sum. A loop, for instructions that run once each wait to be fetched: four
// rows unrolled beside each other took 5800 clocks where four in turn take 4100 (one
// request of 32 tokens, the whole kernel: 9.2 us for 8.5).
template <int D, typename Src, typename Put, typename End>
__device__ __forceinline__ void query_rows(const AttnArgs& a, int i0, int i1, int step, float up_all, Src src, Put put, End end) {
  constexpr int E = D / 32;
  const int lane = threadIdx.x & 31, c0 = lane * E;
  struct Row {
    bool on;
    float x[E], y[E], cs[E], sn[E];
  };
  float g[E];
  const bool turned = a.rcos != nullptr && c0 < a.rot;
  const int half = a.rot / 2;
  const bool first = c0 < half;
#pragma unroll
  for (int i = 0; i < E; ++i) g[i] = 1.0f;
  if (a.gq != nullptr) load_vec<E>(a.gq + c0, g);
  auto load = [&](int i) {
    Row r;
    int pos = 0;
    const elem_t* q = src(i, pos);
    r.on = q != nullptr;
#pragma unroll
    for (int k = 0; k < E; ++k) r.x[k] = r.y[k] = r.sn[k] = 0.f, r.cs[k] = 1.f;
    if (!r.on) return r;
    load_vec<E>(q + c0, r.x);
    if (turned) {
      const long long row = static_cast<long long>(pos) * half;
      if (a.interleaved) {
#pragma unroll
        for (int k = 0; k < E / 2; ++k) {
          r.cs[2 * k] = r.cs[2 * k + 1] = a.rcos[row + c0 / 2 + k];
          r.sn[2 * k] = r.sn[2 * k + 1] = a.rsin[row + c0 / 2 + k];
        }
      } else {
        load_vec<E>(q + (first ? c0 + half : c0 - half), r.y);
        load_vec<E>(a.rcos + row + (first ? c0 : c0 - half), r.cs);
        load_vec<E>(a.rsin + row + (first ? c0 : c0 - half), r.sn);
      }
    }
    return r;
  };
  if (i0 >= i1) return;
  Row next = load(i0);
#pragma unroll 1
  for (int i = i0; i < i1; i += step) {
    Row r = next;
    if (i + step < i1) next = load(i + step);
    float down = 1.f, sum = 0.f;
    if (!r.on) {                 // (the warp's lanes alike)
#pragma unroll
      for (int k = 0; k < E; ++k) put(i, c0 + k, __half(0.f), __half(0.f));
    } else {
      if (turned) {
        if (a.interleaved) {
#pragma unroll
          for (int k = 0; k < E; k += 2) {
            const float u = r.x[k], v = r.x[k + 1];
            r.x[k] = fmaf(u, r.cs[k], v * r.sn[k]);
            r.x[k + 1] = fmaf(v, r.cs[k], -u * r.sn[k]);
          }
        } else {
#pragma unroll
          for (int k = 0; k < E; ++k) r.x[k] = fmaf(r.x[k], r.cs[k], (first ? r.y[k] : -r.y[k]) * r.sn[k]);
        }
      }
      float ss = 0.f;
#pragma unroll
      for (int k = 0; k < E; ++k) ss = fmaf(r.x[k], r.x[k], ss);
      ss = warp_sum(ss);
      float eps = a.eps;
      if (ss == INFINITY) {      // the squares pass fp32: the same of 2^-80 of the row
        constexpr float kDown = 0x1p-80f;
        ss = 0.f;
#pragma unroll
        for (int k = 0; k < E; ++k) {
          r.x[k] *= kDown;
          ss = fmaf(r.x[k], r.x[k], ss);
        }
        ss = warp_sum(ss);
        eps = eps * kDown * kDown;
      }
      const float mul = rsqrtf(ss / D + eps) * (a.scale * 1.4426950408889634f);
      float up = up_all;
#pragma unroll
      for (int k = 0; k < E; ++k) r.x[k] *= mul * g[k];
      if (up_all == 0.f) {
        float top = 0.f;
#pragma unroll
        for (int k = 0; k < E; ++k) top = fmaxf(top, fabsf(r.x[k]));
        // (of floats that are not negative the bits are in their order, a NaN above all)
        const unsigned bits = __reduce_max_sync(0xffffffffu, __float_as_uint(top));
        int e = static_cast<int>((bits >> 23) & 255u) - 127;
        e = e < -100 ? -100 : (e > 100 ? 100 : e);
        up = __uint_as_float(static_cast<uint32_t>(127 + 13 - e) << 23);
        down = __uint_as_float(static_cast<uint32_t>(127 - 13 + e) << 23);
      }
#pragma unroll
      for (int k = 0; k < E; ++k) {
        const float v = r.x[k] * up;
        const __half hi = __float2half_rn(v);
        put(i, c0 + k, hi, __float2half_rn(v - __half2float(hi)));
        sum += v;
      }
    }
#pragma unroll
    for (int o = 32 / E; o > 0; o >>= 1) sum += __shfl_xor_sync(0xffffffffu, sum, o);
    if (lane % (64 / E) == 0) end(i, c0 / 64, down, sum);
  }
}

template <int D, int RW, bool kPolled>
__global__ void __launch_bounds__(kAttnWarps * 32, tree_ctas_per_sm(D)) tree_attn_kernel(const __grid_constant__ TreeAttnArgs a) {
  using S = AttnShape<D>;
  using M = TreeSmem<D, RW>;
  constexpr int NG = S::NG, W = S::W, NQ = 16 * RW, KG = kAttnWarps / RW, ST = M::stages, E = D / 32;
  extern __shared__ __align__(128) uint8_t smem[];
  const int tid = threadIdx.x, lane = tid & 31, wid = tid >> 5;
  const int r = lane >> 2, j = lane & 3;
  const int rw = wid % RW, kg = wid / RW;                  // rows 16 rw .., steps kg, kg + KG, ..
  const TreeShare share = tree_share<NQ, kAttnWarps * 32>(a);
  if (share.none) return;
  const int b = share.b, h = share.h, qg = share.qg;
  const int G = a.Hq / a.c.Hkv;
  const long long cap = static_cast<long long>(a.max_pages) * a.c.page;
  uint32_t bad = 0;
  const TreeReq req = tree_req(a.cu, a.lens, b, a.N, a.max_new, cap);
  if (req.bad) bad = DEV_ERR_BOUNDS;

  if (share.ci == 0 && qg == 0) tree_zero<D, kAttnWarps>(a, req, b, h, G);
  if (bad && tid == 0) atomicOr(a.status, bad);
  const int row_q0 = qg * NQ;                              // first (token, head) row of this CTA
  const int nq = min(NQ, req.n * G - row_q0);
  if (nq <= 0) return;
  const int len = req.ctx + req.n;
  const int lo = a.window >= 0 && req.ctx - a.window > 0 ? req.ctx - a.window : 0;
  const int t_lo = lo / kTile, t_hi = (len + kTile - 1) / kTile;     // tiles [t_lo, t_hi)
  const int chunks = max(1, (t_hi - t_lo + share.chunk - 1) / share.chunk);
  if (share.ci >= chunks) return;
  const int t0 = t_lo + share.ci * share.chunk, t1 = min(t_hi, t0 + share.chunk);

  const uint32_t bars = smem_u32(smem + M::bars) + kg * ST * 16, frees = bars + ST * 8;
  uint32_t* flags = reinterpret_cast<uint32_t*>(smem + M::flags);    // [0] abort, [1] last
  if (rw == 0 && lane == 0) {
    for (int s = 0; s < ST; ++s) {
      mbar_init(bars + 8 * s, 1);
      mbar_init(frees + 8 * s, RW);
    }
    fence_mbar_init();
  }
  if (tid == 0) flags[0] = 0;
  __syncwarp();

  // Step n of a group of warps is the tiles t0 + 2 (kg + n KG) and the one
  // behind it, which share a stage; its first warp fetches them. Pages are
  // looked up 32 tiles at a time, a lane a tile.
  const int steps = (t1 - t0 + 1) / 2;
  const int n_mine = steps > kg ? (steps - kg + KG - 1) / KG : 0;
  uint8_t* ring = smem + kg * M::ring1;
  const uint32_t ring_u = smem_u32(ring);
  const int per_page = a.c.page / kTile;
  const long long head_off = static_cast<long long>(h) * per_page;
  long long tile_at = -1;  // of the lane's tile in the cache; -1: none
  uint32_t gone = 0;       // two bits per stage: tiles that are not there
  // every warp of the group looks pages up, so that each knows which are gone
  auto issue = [&](int n) {
    if ((n & 15) == 0) {
      const int t = t0 + 2 * (kg + (n + (lane >> 1)) * KG) + (lane & 1);
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
    const int st = n % ST;
    const long long at = __shfl_sync(0xffffffffu, tile_at, ((2 * n) & 31) + (lane & 1));
    const uint32_t there = __ballot_sync(0xffffffffu, at >= 0) & 3u;
    gone = (gone & ~(3u << (2 * st))) | ((there ^ 3u) << (2 * st));
    if (rw != 0) return;
    if (lane == 0) mbar_arrive_expect_tx(bars + 8 * st, __popc(there) * S::TB);
    __syncwarp();
    if (lane < 2 && at >= 0) bulk_load(ring_u + (st * 2 + lane) * S::TB, a.c.data + at * S::TB, S::TB, bars + 8 * st);
  };
  int issued = 0;
  for (; issued < ST && issued < n_mine; ++issued) issue(issued);

  // rows and queries
  TreeRow* rows = reinterpret_cast<TreeRow*>(smem + M::row);
  int* tpos = reinterpret_cast<int*>(smem + M::tpos);
  __half* qs = reinterpret_cast<__half*>(smem + M::q);
  float* qf = reinterpret_cast<float*>(smem + M::qf);
  tree_rows<NQ, kAttnWarps * 32>(a, req, row_q0, nq, G, rows, tpos, bad);
  __syncthreads();
  tree_sight<NQ, kAttnWarps>(a, req, rows, tpos, wid);
  query_rows<D>(a, wid, NQ, kAttnWarps, 0.f,
      [&](int i, int& pos) -> const elem_t* {
        const int row = row_q0 + i;
        pos = rows[i].pos;
        return rows[i].lo != INT32_MAX ? a.q + (static_cast<long long>(req.row0 + row / G) * a.Hq + h * G + row % G) * D : nullptr;
      },
      [&](int i, int c, __half hi, __half lo) {
        __half* to = qs + i * kQTerms * D + (c & ~7) + (c & 3) * 2 + ((c >> 2) & 1);   // pairs (c, c + 4) side by side
        to[0] = hi;
        to[D] = lo;
      },
      [&](int i, int g, float down, float sum) {
        if (g == 0) qf[i * 4] = down;
        qf[i * 4 + 1 + g] = sum;
      });
  __syncthreads();
  uint32_t qa[kQTerms][2 * W][4];
  float qfac[2], qsum[2][NG];
  TreeRow my[2];
#pragma unroll
  for (int i = 0; i < 2; ++i) {
    const int row = 16 * rw + r + 8 * i;
#pragma unroll
    for (int s = 0; s < kQTerms; ++s) {
#pragma unroll
      for (int w = 0; w < W; ++w) {
        const uint4 c = *reinterpret_cast<const uint4*>(qs + row * kQTerms * D + s * D + (w / 2) * 64 + j * 16 + (w & 1) * 8);
        qa[s][2 * w][i] = c.x; qa[s][2 * w][i + 2] = c.y;
        qa[s][2 * w + 1][i] = c.z; qa[s][2 * w + 1][i + 2] = c.w;
      }
    }
    qfac[i] = qf[row * 4];
#pragma unroll
    for (int g = 0; g < NG; ++g) qsum[i][g] = qf[row * 4 + 1 + g];
    my[i] = rows[row];
  }
  // keys from here on are seen by every row of the warp, up to the context's end
  int all_lo = max(my[0].lo == INT32_MAX ? 0 : my[0].lo, my[1].lo == INT32_MAX ? 0 : my[1].lo);
#pragma unroll
  for (int o = 4; o < 32; o <<= 1) all_lo = max(all_lo, __shfl_xor_sync(0xffffffffu, all_lo, o));

  const WaitCtl<kPolled> ctl{flags, a.status, a.wait_limit_ns};
  float acc[4 * W][4] = {};
  float m[2] = {-1e30f, -1e30f}, l[2] = {}, zs[2][NG] = {};
  int n = 0;
  for (; n < n_mine; ++n) {
    const int st = n % ST;
    if (!mbar_wait_warp(bars + 8 * st, (n / ST) & 1, ctl)) break;
    const uint8_t* tile = ring + st * 2 * S::TB;
    const int key0 = (t0 + 2 * (kg + n * KG)) * kTile;
    const uint32_t miss = gone >> (2 * st) & 3u;
    float s[2][2][4];        // logits (base 2): tile, eight keys, (row, key) as the product leaves them
#pragma unroll
    for (int q = 0; q < 2; ++q) {
#pragma unroll
      for (int t = 0; t < 2; ++t) {
        uint32_t kw[W];
        ld_words<W>(tile + q * S::TB + (r + 8 * t) * (D / 2) + j * (D / 8), kw);
        float d[NG][4] = {};
#pragma unroll
        for (int w = 0; w < W; ++w) {
          uint32_t x[4];
          widen_f16(kw[w], x);
#pragma unroll
          for (int u = kQTerms - 1; u >= 0; --u) {
            const uint32_t(&p)[4] = qa[u][2 * w], (&z)[4] = qa[u][2 * w + 1];
            mma_f16(d[w / 2], p[0], p[1], p[2], p[3], x[0], x[1]);
            mma_f16(d[w / 2], z[0], z[1], z[2], z[3], x[2], x[3]);
          }
        }
#pragma unroll
        for (int e = 0; e < 2; ++e) {
          float sk[NG], zk[NG];
          ld_scales<NG>(tile + q * S::TB + 16 * D + (8 * t + 2 * j + e) * (4 * NG), sk, zk);
#pragma unroll
          for (int i = 0; i < 2; ++i) {
            float v = 0.f;
#pragma unroll
            for (int g = 0; g < NG; ++g) v = fmaf(sk[g], d[g][2 * i + e], fmaf(zk[g], qsum[i][g], v));
            s[q][t][2 * i + e] = v * qfac[i];
          }
        }
      }
    }
    const bool edge = key0 < all_lo || key0 + 2 * kTile > req.ctx || miss;
    if (edge) {
#pragma unroll
      for (int q = 0; q < 2; ++q)
#pragma unroll
        for (int t = 0; t < 2; ++t)
#pragma unroll
          for (int e = 0; e < 2; ++e) {
            const int key = key0 + q * kTile + 8 * t + 2 * j + e, d = key - req.ctx;
#pragma unroll
            for (int i = 0; i < 2; ++i) {
              const bool old = (d < 0) & (key >= my[i].lo);
              const bool drafted = (d >= 0) & (d < kTreeTokens) & static_cast<bool>(my[i].seen >> (d & 63) & 1ull);
              const bool on = (old | drafted) & !(miss >> q & 1u);
              if (!on) s[q][t][2 * i + e] = -INFINITY;
            }
          }
    }
    float top[2];
#pragma unroll
    for (int i = 0; i < 2; ++i)
      top[i] = fmaxf(fmax3(s[0][0][2 * i], s[0][0][2 * i + 1], fmaxf(s[0][1][2 * i], s[0][1][2 * i + 1])),
                     fmax3(s[1][0][2 * i], s[1][0][2 * i + 1], fmaxf(s[1][1][2 * i], s[1][1][2 * i + 1])));
    if (__any_sync(0xffffffffu, top[0] > m[0] + 8.f || top[1] > m[1] + 8.f)) {
#pragma unroll
      for (int i = 0; i < 2; ++i) {
        float x = top[i];
        x = fmaxf(x, __shfl_xor_sync(0xffffffffu, x, 1));
        x = fmaxf(x, __shfl_xor_sync(0xffffffffu, x, 2));
        const float mn = fmaxf(m[i], x), al = ex2_approx(m[i] - mn);
        m[i] = mn;
        l[i] *= al;
#pragma unroll
        for (int g = 0; g < NG; ++g) zs[i][g] *= al;
#pragma unroll
        for (int k = 0; k < 4 * W; ++k) {
          acc[k][2 * i] *= al;
          acc[k][2 * i + 1] *= al;
        }
      }
    }
#pragma unroll
    for (int q = 0; q < 2; ++q) {
      const uint8_t* at = tile + q * S::TB;
      uint32_t pa[kThreeTerms ? 3 : 1][NG][4];     // P times the values' steps, as operand registers
#pragma unroll
      for (int t = 0; t < 2; ++t) {
        float sv[2][NG], zv[2][NG];
        ld_scales<NG>(at + 17 * D + (8 * t + 2 * j) * (4 * NG), sv[0], zv[0]);
        ld_scales<NG>(at + 17 * D + (8 * t + 2 * j + 1) * (4 * NG), sv[1], zv[1]);
#pragma unroll
        for (int i = 0; i < 2; ++i) {
          const float p0 = ex2_approx(s[q][t][2 * i] - m[i]), p1 = ex2_approx(s[q][t][2 * i + 1] - m[i]);
          l[i] += p0 + p1;
#pragma unroll
          for (int g = 0; g < NG; ++g) {
            float w0 = p0 * sv[0][g], w1 = p1 * sv[1][g], z0 = p0 * zv[0][g], z1 = p1 * zv[1][g];
            if (edge) {        // another row may see the key: what it holds, a NaN even, is not this row's
              if (s[q][t][2 * i] == -INFINITY) w0 = z0 = 0.f;
              if (s[q][t][2 * i + 1] == -INFINITY) w1 = z1 = 0.f;
            }
            zs[i][g] += z0 + z1;
            const uint32_t hi = pack_bf16x2(w0, w1);
            pa[0][g][2 * t + i] = hi;
            if constexpr (kThreeTerms) {
              const float e0 = w0 - __uint_as_float(hi << 16), e1 = w1 - __uint_as_float(hi & 0xFFFF0000u);
              const uint32_t mid = pack_bf16x2(e0, e1);
              pa[1][g][2 * t + i] = mid;
              pa[2][g][2 * t + i] = pack_bf16x2(e0 - __uint_as_float(mid << 16), e1 - __uint_as_float(mid & 0xFFFF0000u));
            }
          }
        }
      }
      uint32_t va[W], vb[W];
      ld_words<W>(at + 8 * D + j * D + r * (D / 8), va);
      ld_words<W>(at + 8 * D + (j + 4) * D + r * (D / 8), vb);
#pragma unroll
      for (int w = 0; w < W; ++w) {
        uint32_t x[4], y[4];
        widen_bf16(va[w], x);
        widen_bf16(vb[w], y);
#pragma unroll
        for (int u = (kThreeTerms ? 3 : 1) - 1; u >= 0; --u) {
          const uint32_t(&p)[4] = pa[u][w / 2];
#pragma unroll
          for (int i = 0; i < 4; ++i) mma_bf16(acc[4 * w + i], p[0], p[1], p[2], p[3], x[i], y[i]);
        }
      }
    }
    __syncwarp();
    if constexpr (RW == 1) {
      if (issued < n_mine) issue(issued++);
    } else {
      // a stage is free once every warp of the group is through with it; the one
      // of the step before is filled again, so that the wait is seldom one
      if (lane == 0) mbar_arrive(frees + 8 * st);
      if (n > 0 && issued < n_mine) {
        if (rw == 0 && !mbar_wait_warp(frees + 8 * ((n - 1) % ST), ((n - 1) / ST) & 1, ctl)) {
          ++n;
          break;
        }
        issue(issued++);
      }
    }
  }
  // a wait that ran out: the copies still on their way land before the memory is used again. (Only the warp that asked
  // for them knows which were: a stage that another has counted and this one gave up on never fills.)
  if (rw == 0)
    for (int k = n; k < issued; ++k) mbar_wait_drain(bars + 8 * (k % ST), (k / ST) & 1, kDrainLimitNs);
  if (bad) atomicOr(a.status, bad);

  // join the groups of warps: O, M, L of each row into shared memory
  __syncthreads();
  float* jo = reinterpret_cast<float*>(smem);                    // [warp][16][D]
  float* jm = jo + kAttnWarps * 16 * D;                          // [warp][16][2]: M, L
#pragma unroll
  for (int i = 0; i < 2; ++i) {
    l[i] += __shfl_xor_sync(0xffffffffu, l[i], 1);
    l[i] += __shfl_xor_sync(0xffffffffu, l[i], 2);
#pragma unroll
    for (int g = 0; g < NG; ++g) {
      zs[i][g] += __shfl_xor_sync(0xffffffffu, zs[i][g], 1);
      zs[i][g] += __shfl_xor_sync(0xffffffffu, zs[i][g], 2);
    }
    const int row = wid * 16 + r + 8 * i;
    // channel 64 g + 16 j + 8 e + 4 u + k is entry (2 i + e) of sum 4 (2 g + u) + k
#pragma unroll
    for (int w = 0; w < W; ++w)
#pragma unroll
      for (int e = 0; e < 2; ++e) {
        const float z = zs[i][w / 2];
        const int c = 2 * i + e;
        *reinterpret_cast<float4*>(jo + row * D + (w / 2) * 64 + 16 * j + 8 * e + 4 * (w & 1)) =
            make_float4(acc[4 * w][c] + z, acc[4 * w + 1][c] + z, acc[4 * w + 2][c] + z, acc[4 * w + 3][c] + z);
      }
    if (j == 0) {
      jm[2 * row] = m[i];
      jm[2 * row + 1] = l[i];
    }
  }
  __syncthreads();
  auto head_of = [&](int i) {       // index of row i's head in o and lse
    const int row = row_q0 + i;
    return static_cast<long long>(req.row0 + row / G) * a.Hq + h * G + row % G;
  };
  for (int i = wid; i < nq; i += kAttnWarps) {      // a warp a row, E channels a lane
    float top = -1e30f, sum = 0.f, o[E] = {};
#pragma unroll
    for (int k = 0; k < KG; ++k) top = fmaxf(top, jm[2 * (k * NQ + i)]);
#pragma unroll
    for (int k = 0; k < KG; ++k) {
      const float f = ex2_approx(jm[2 * (k * NQ + i)] - top);
      sum = fmaf(f, jm[2 * (k * NQ + i) + 1], sum);
      float x[E];
      load_vec<E>(jo + (k * NQ + i) * D + lane * E, x);
#pragma unroll
      for (int e = 0; e < E; ++e) o[e] = fmaf(f, x[e], o[e]);
    }
    if (rows[i].lo == INT_MAX) {     // sees nothing: tiles that every other row sees were not masked for it
      top = -1e30f;
      sum = 0.f;
#pragma unroll
      for (int e = 0; e < E; ++e) o[e] = 0.f;
    }
    tree_row_out<D>(a, chunks, share.ci, share.part0, NQ, i, head_of(i), o, top, sum);
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

  tree_join<D, 4, 4>(a, chunks, share.part0, NQ, wid, kAttnWarps, nq, head_of);
}

// Warps over rows, chunks and CTAs of a call, from what the host knows. Partial
// results of split requests have to fit the decode workspace.
struct TreeSplit {
  int nq;                // (token, head) rows of a CTA
  bool tc;               // the tcgen05 form
  int groups, chunk, splits;
  long long items;
  int grid, slots, setup;   // grid > 0: a flat one, whose CTAs find their shares
  long long parts;          // rows of partial results
};
inline TreeSplit tree_split(int B, int Hq, int Hkv, int d, int page, int max_pages, int window, int max_new, long long part_floats) {
  TreeSplit s;
  const int rows = Hq / Hkv * max_new;
  s.tc = !kThreeTerms && d == 128 && rows > 16;
  s.nq = rows <= 16 ? 16 : (rows <= 32 && !s.tc ? 32 : 64);
  s.setup = s.tc ? 48 : 24;          // set-up and end of a CTA, in tiles that it could have done
  const long long nq = s.nq;
  s.groups = static_cast<int>((rows + nq - 1) / nq);
  s.items = static_cast<long long>(B) * Hkv * s.groups;
  const long long cap = static_cast<long long>(max_pages) * page;
  long long keys = cap;
  if (window >= 0 && static_cast<long long>(window) + max_new + kTile < cap) keys = static_cast<long long>(window) + max_new + kTile;
  const long long tiles = (keys + kTile - 1) / kTile;
  const long long slots = 152LL * (s.tc ? 1 : tree_ctas_per_sm(d));
  const long long room = part_floats / (nq * (d + 2));      // partial results of CTAs
  // The CTAs look for their shares where that can spare more than the microsecond
  // that it takes (16 equal requests of 32768: 180 us without, 186 so; of 1500: 19.2,
  // 20.6), and where there is room to split a request.
  s.grid = 0;
  s.slots = 0;
  if (tiles >= kShareTiles && B <= kShareB && s.items < (room < 65536 ? room : 65536 - slots)) {
    s.grid = static_cast<int>(s.items + slots < room ? s.items + slots : room);
    s.slots = static_cast<int>(slots);
    s.chunk = s.splits = 0;
    s.parts = s.grid * nq;
    return s;
  }
  long long best = 0, chunk = tiles;
  for (long long n = 1; n <= kMaxSplits; ++n) {
    const long long c = ((tiles + n - 1) / n + 7) / 8 * 8, real = (tiles + c - 1) / c;
    if (real > 1 && s.items * real > room) break;
    const long long own = (c < tiles ? c : tiles) + s.setup;
    const long long t = (s.items * real + slots - 1) / slots * own + (real > 1 ? kJoinTiles + real / 2 : 0);
    if (n == 1 || t < best) {
      best = t;
      chunk = c;
    }
    if (c == 8) break;
  }
  s.chunk = static_cast<int>(chunk);
  s.splits = static_cast<int>((tiles + chunk - 1) / chunk);
  s.parts = s.items * s.splits * nq;
  return s;
}

}  // namespace kv4
}  // namespace swa
