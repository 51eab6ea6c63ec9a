// Attention of one new token per request over the 4-bit paged cache.
#pragma once

#include "kv4.cuh"

namespace swa {
namespace kv4 {

struct AttnArgs {
  Cache c;
  int B, Hq, max_pages, window;        // window < 0: none
  float scale, eps;
  const elem_t* q;                     // [B, Hq, D]
  const float* gq;
  const float* rcos; const float* rsin; int rows, rot, interleaved;   // rcos NULL: none
  const int32_t* table; const int32_t* lens;
  elem_t* o; float* lse;               // [B, Hq, D], [B, Hq]
  uint32_t* status;
};

// One warp per query head, a key at a time.
template <int D>
__global__ void __launch_bounds__(128) attn_kernel(const __grid_constant__ AttnArgs a) {
  constexpr int NG = D / 64, E = D / 32;
  const int lane = threadIdx.x & 31;
  const int item = blockIdx.x * 4 + (threadIdx.x >> 5);
  if (item >= a.B * a.Hq) return;
  const int b = item / a.Hq, hq = item - b * a.Hq, G = a.Hq / a.c.Hkv, h = hq / G;
  int len = a.lens[b];
  uint32_t bad = 0;
  const long long cap = static_cast<long long>(a.max_pages) * a.c.page;
  if (len < 0 || len > cap) {
    bad = DEV_ERR_BOUNDS;
    len = len < 0 ? 0 : static_cast<int>(cap);
  }
  if (a.rcos != nullptr && len > a.rows) { bad = DEV_ERR_BOUNDS; len = 0; }
  const elem_t* q = a.q + static_cast<long long>(item) * D;
  float x[E], ss = 0.f;
  const int c0 = lane * E;
#pragma unroll
  for (int i = 0; i < E; ++i) {
    const int c = c0 + i;
    x[i] = to_f32(q[c]);
    if (a.rcos != nullptr && c < a.rot && len > 0) {
      const int half = a.rot / 2;
      const int col = a.interleaved ? c / 2 : c % half;
      const int to = a.interleaved ? c ^ 1 : (c < half ? c + half : c - half);
      const bool first = a.interleaved ? (c & 1) == 0 : c < half;
      const long long at = static_cast<long long>(len - 1) * half + col;
      x[i] = x[i] * a.rcos[at] + (first ? 1.f : -1.f) * to_f32(q[to]) * a.rsin[at];
    }
    ss = fmaf(x[i], x[i], ss);
  }
  const float f = rsqrtf(warp_sum(ss) / D + a.eps) * a.scale;
#pragma unroll
  for (int i = 0; i < E; ++i) x[i] *= f * (a.gq ? a.gq[c0 + i] : 1.0f);
  float m = -INFINITY, l = 0.f, acc[E] = {};
  const int g = c0 / 64, x0 = c0 % 64;
  const int lo = a.window >= 0 && len - 1 - a.window > 0 ? len - 1 - a.window : 0;
  for (int j = lo; j < len; ++j) {
    const int pg = a.table[static_cast<long long>(b) * a.max_pages + j / a.c.page];
    if (pg < 0 || pg >= a.c.n_pages) { bad = DEV_ERR_BOUNDS; continue; }
    const uint8_t* tile = tile_of<D>(a.c, static_cast<long long>(pg) * a.c.page + j % a.c.page, h);
    const int t = j % a.c.page % kTile;
    const uint32_t* sc = reinterpret_cast<const uint32_t*>(tile + 16 * D);
    const uint32_t ka = sc[t * NG + g], va = sc[(kTile + t) * NG + g];
    float s = 0.f, v[E];
#pragma unroll
    for (int i = 0; i < E; ++i) {
      const int c = x0 + i;
      const int nk = ((c / 16) * NG + g) * 16 + c % 16;
      const int kn = tile[t * (D / 2) + nk / 2] >> (4 * (nk & 1)) & 15;
      const int nv = (((c / 8) * NG + g) * 2 + (c / 4) % 2) * 8 + (t & 1) * 4 + c % 4;
      const int vn = tile[8 * D + (t / 2) * D + nv / 2] >> (4 * (nv & 1)) & 15;
      s = fmaf(x[i], fmaf(__uint_as_float(ka << 16), static_cast<float>(kn - 8), __uint_as_float(ka & 0xFFFF0000u)), s);
      v[i] = fmaf(__uint_as_float(va << 16), static_cast<float>(vn - 8), __uint_as_float(va & 0xFFFF0000u));
    }
    s = warp_sum(s);
    const float mn = fmaxf(m, s), al = expf(m - mn), p = expf(s - mn);
    l = l * al + p;
#pragma unroll
    for (int i = 0; i < E; ++i) acc[i] = fmaf(p, v[i], acc[i] * al);
    m = mn;
  }
  const float inv = l > 0.f ? 1.0f / l : 0.f;
#pragma unroll
  for (int i = 0; i < E; ++i) a.o[static_cast<long long>(item) * D + c0 + i] = from_f32<elem_t>(acc[i] * inv);
  if (lane == 0) {
    a.lse[item] = l > 0.f ? m + logf(l) : -INFINITY;
    if (bad) atomicOr(a.status, bad);
  }
}

}  // namespace kv4
}  // namespace swa
