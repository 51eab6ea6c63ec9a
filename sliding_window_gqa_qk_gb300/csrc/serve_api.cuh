// Host side of the norm, of the 4-bit projections and of the drafted tokens'
// entry points of include/swa_attn.h: argument checks and launches. Included
// at the end of swa_attn.cu, behind decode_api.cuh, whose helpers it uses.
#pragma once

#include "kv4_tree.cuh"
#include "norm.cuh"
#include "w4.cuh"
#if !defined(SWA_ELEM_FP32)
#include "kv4_tree_tc.cuh"
#include "w4_tc.cuh"
#endif

namespace {

swa_status check_norm(long long rows, int C) {
  if (rows < 0 || C < 8 || C % 8 != 0) return SWA_ERR_INVALID_ARG;
  return C > norm::kMaxC || rows > INT32_MAX ? SWA_ERR_UNSUPPORTED : SWA_OK;
}

swa_status check_w4(int N, int K) {
  if (N < 1 || K < 8 || K % 8 != 0) return SWA_ERR_INVALID_ARG;
  return N > w4::kMaxN || K > w4::kMaxK ? SWA_ERR_UNSUPPORTED : SWA_OK;
}
// Rows of x, whose tiles of up to 256 are counted in 31 bits.
swa_status check_w4_rows(int M) {
  if (M < 0) return SWA_ERR_INVALID_ARG;
  return M > w4::kMaxM ? SWA_ERR_UNSUPPORTED : SWA_OK;
}
long long w4_tiles(int N, int K) {
  return static_cast<long long>((N + w4::kRows - 1) / w4::kRows) * ((K + w4::kCols - 1) / w4::kCols);
}

// Which form a call takes in the bf16 library (GB300, us):
//   up to kFewRows rows   products with the weights as the 16-row operand (32 rows at 8192 x 8192 22.3; the
//                         tcgen05 form takes 22.9 from 33 to 64 rows, and from 9 on)
//   of these, long rows   x in shared memory, K over a cluster: from K = 4096 on (8 rows: 4096 x 4096 6.9 for 7.6,
//                         1536 x 16384 14 for 28; but 16384 x 1536 10.1 for 6.2, 2048 x 2048 5.7 for 4.3), and for
//                         25 to 32 rows of large layers (16384 x 1536 13.6 for 17.6; 2048 x 2048 7.0 for 6.6)
constexpr int kFewRows = 32;
bool wide_form(const w4::LinArgs& a) { return a.K >= 4096 || (a.M > 24 && w4_tiles(a.N, a.K) >= 16384); }

#if !defined(SWA_ELEM_FP32)
template <w4::XKind X, int NT, int PN>
swa_status launch_wide(const w4::LinArgs& l, cudaStream_t st) {
  using S = w4::WideShape<X, NT, PN>;
  const long long groups = (l.N + S::RN - 1) / S::RN;
  const int chunks = (l.K + w4::kChunk - 1) / w4::kChunk;
  w4::WideArgs a{l, 1, 0};
  while (a.splits < 8 && groups * a.splits * 2 <= 2 * 152 && chunks >= 2 * a.splits) a.splits *= 2;
  a.per = (chunks + a.splits - 1) / a.splits;
  auto kern = w4::linear_wide_kernel<X, NT, PN>;
  if (S::bytes > 48 * 1024 && cudaFuncSetAttribute(kern, cudaFuncAttributeMaxDynamicSharedMemorySize, S::bytes) != cudaSuccess) {
    cudaGetLastError();
    return SWA_ERR_CUDA;
  }
  return w4::launch_cluster(kern, groups * a.splits, w4::kWideWarps * 32, S::bytes, a.splits, st, a);
}
#endif

template <w4::XKind X, int NT>
swa_status launch_few(const w4::LinArgs& a, cudaStream_t st) {
  const long long panels = (a.N + w4::kRows - 1) / w4::kRows;
#if !defined(SWA_ELEM_FP32)
  // two panels a warp where the CTAs of their groups still fill the GPU and the sums the registers
  if (a.M <= 8 * NT && wide_form(a)) {
    if constexpr (NT <= 2) {
      if (panels >= 2 * 8 * 19) return launch_wide<X, NT, 2>(a, st);
    }
    return launch_wide<X, NT, 1>(a, st);
  }
#endif
  const long long grid = panels * ((a.M + 8 * NT - 1) / (8 * NT));
  if (grid > INT32_MAX) return SWA_ERR_UNSUPPORTED;
  if (a.K < 32 * w4::kCols) w4::linear_kernel<X, NT, 4><<<static_cast<unsigned>(grid), 128, 0, st>>>(a);
  else w4::linear_kernel<X, NT, 8><<<static_cast<unsigned>(grid), 256, 0, st>>>(a);
  return launched();
}

template <w4::XKind X>
swa_status launch_linear(const w4::LinArgs& a, uint32_t* status, uint64_t wait_ns, cudaStream_t st) {
#if !defined(SWA_ELEM_FP32)
  constexpr bool x8 = X == w4::kX8;
  if (a.M > kFewRows && (!x8 || a.K % 16 == 0)) {      // (e4m3 rows come by TMA, whose strides are multiples of 16 bytes)
    if (a.M <= 64) return w4::launch_linear_tc<64, x8>(a, status, wait_ns, st);
    if (x8 || a.M <= 128) return w4::launch_linear_tc<128, x8>(a, status, wait_ns, st);
    return w4::launch_linear_tc<256, false>(a, status, wait_ns, st);
  }
#endif
  if (a.M <= 8) return launch_few<X, 1>(a, st);
  if (a.M <= 16) return launch_few<X, 2>(a, st);
  if (a.M <= 24) return launch_few<X, 3>(a, st);
  return launch_few<X, 4>(a, st);
}

// swa_w4_linear under a time limit of its pipeline waits (which the form for few rows, and the fp32 library, do not have).
swa_status linear_call(int M, int N, int K, const void* x, const float* x_scale, const void* w4, const void* add, void* y,
                       void* workspace, size_t ws_bytes, uint64_t wait_ns, void* stream) {
  swa_status s = check_w4(N, K);
  if (s != SWA_OK || (s = check_w4_rows(M)) != SWA_OK) return s;
  if ((s = check_header(workspace, ws_bytes)) != SWA_OK) return s;
  if (M == 0) return SWA_OK;
  if (!tensor_ok(x) || !tensor_ok(w4) || !tensor_ok(y) || !aligned(add, 16) || !aligned(x_scale, 4)) return SWA_ERR_INVALID_ARG;
  if (x == y) return SWA_ERR_INVALID_ARG;
  if ((s = check_device()) != SWA_OK) return s;
  const w4::LinArgs a{M, N, K, x, x_scale, static_cast<const uint8_t*>(w4), static_cast<const elem_t*>(add), static_cast<elem_t*>(y)};
  cudaStream_t st = static_cast<cudaStream_t>(stream);
  uint32_t* status = static_cast<uint32_t*>(workspace);
  return x_scale != nullptr ? launch_linear<w4::kX8>(a, status, wait_ns, st) : launch_linear<w4::kXElem>(a, status, wait_ns, st);
}

swa_status check_tokens(int B, int n_tokens, int max_new) {
  if (B < 0 || n_tokens < 0 || max_new < 1) return SWA_ERR_INVALID_ARG;
  if (B == 0 && n_tokens > 0) return SWA_ERR_INVALID_ARG;
  return max_new > kv4::kTreeTokens ? SWA_ERR_UNSUPPORTED : SWA_OK;
}

constexpr long long kTreePartFloats = static_cast<long long>((kKv4Bytes - kKv4Part) / sizeof(float)) - 64;

template <int D, int RW, bool kPolled>
swa_status launch_tree(const kv4::TreeAttnArgs& a, dim3 grid, cudaStream_t st) {
  auto kern = kv4::tree_attn_kernel<D, RW, kPolled>;
  constexpr int smem = kv4::TreeSmem<D, RW>::bytes;
  if (smem > 48 * 1024 && cudaFuncSetAttribute(kern, cudaFuncAttributeMaxDynamicSharedMemorySize, smem) != cudaSuccess) {
    cudaGetLastError();
    return SWA_ERR_CUDA;
  }
  kern<<<grid, kv4::kAttnWarps * 32, smem, st>>>(a);
  return launched();
}
#if !defined(SWA_ELEM_FP32)
template <int NR, bool kPolled>
swa_status launch_tree_tc(const kv4::TreeAttnArgs& a, dim3 grid, cudaStream_t st) {
  using S = kv4::TtShape<NR>;
  auto kern = kv4::tree_tc_kernel<NR, kPolled>;
  if (cudaFuncSetAttribute(kern, cudaFuncAttributeMaxDynamicSharedMemorySize, S::bytes) != cudaSuccess) {
    cudaGetLastError();
    return SWA_ERR_CUDA;
  }
  kern<<<grid, S::warps * 32, S::bytes, st>>>(a);
  return launched();
}
#endif
template <bool kPolled>
swa_status launch_tree(const kv4::TreeAttnArgs& a, int d, const kv4::TreeSplit& sp, cudaStream_t st) {
  const dim3 grid = sp.grid > 0 ? dim3(sp.grid) : dim3(sp.splits, a.c.Hkv * sp.groups, a.B);
#if !defined(SWA_ELEM_FP32)
  if (sp.tc) return launch_tree_tc<64, kPolled>(a, grid, st);
  // (head dim 128 has more rows than 16 in that form only)
  if (d == 128) return launch_tree<128, 1, kPolled>(a, grid, st);
#else
  if (d == 128) return sp.nq == 16 ? launch_tree<128, 1, kPolled>(a, grid, st) : sp.nq == 32 ? launch_tree<128, 2, kPolled>(a, grid, st) : launch_tree<128, 4, kPolled>(a, grid, st);
#endif
  return sp.nq == 16 ? launch_tree<64, 1, kPolled>(a, grid, st) : sp.nq == 32 ? launch_tree<64, 2, kPolled>(a, grid, st) : launch_tree<64, 4, kPolled>(a, grid, st);
}

// Workspace of the serving block: that of the decode attention, then what lies
// between its calls.
struct ServeLayout {
  size_t h, xn, q, k, v, o, lse, end;
};
ServeLayout serve_layout(const swa_params* p, int C, int n) {
  ServeLayout L{};
  const size_t es = sizeof(elem_t), t = static_cast<size_t>(n);
  size_t at = align256(kKv4Bytes);
  auto take = [&](size_t bytes) {
    const size_t x = at;
    at = align256(at + bytes);
    return x;
  };
  L.h = take(t * C * es);
  L.xn = take(t * C * es);
  L.q = take(t * p->Hq * p->d * es);
  L.k = take(t * p->Hkv * p->d * es);
  L.v = take(t * p->Hkv * p->d * es);
  L.o = take(t * p->Hq * p->d * es);
  L.lse = take(t * p->Hq * sizeof(float));
  L.end = at;
  return L;
}
swa_status check_serve(const swa_params* p, int C, int n) {
  swa_status s = check_params(p);
  if (s != SWA_OK) return s;
  if (p->T != 1 || p->causal != 1 || n < 0) return SWA_ERR_INVALID_ARG;
  if ((s = check_norm(n, C)) != SWA_OK || (s = check_w4_rows(n)) != SWA_OK) return s;
  return static_cast<long long>(p->Hq) * p->d > w4::kMaxN ? SWA_ERR_UNSUPPORTED : SWA_OK;
}

}  // namespace

extern "C" {

swa_status swa_rms_norm(long long rows, int C, float eps, const void* x, const void* add, const float* gain, void* h, void* y,
                        void* y8, float* scale, float* rstd, void* stream) {
  swa_status s = check_norm(rows, C);
  if (s != SWA_OK) return s;
  if (!std::isfinite(eps) || eps < 0.f) return SWA_ERR_INVALID_ARG;
  if ((y == nullptr) == (y8 == nullptr) || (y8 != nullptr) != (scale != nullptr)) return SWA_ERR_INVALID_ARG;
  if (rows == 0) return SWA_OK;
  if (x == nullptr || (add != nullptr && h == nullptr) || (h != nullptr && (h == y || h == y8))) return SWA_ERR_INVALID_ARG;
  // (y takes the place of the entries that it is made of; 8-bit rows are shorter, and would lie over other rows)
  if (y8 != nullptr && (y8 == x || y8 == add)) return SWA_ERR_INVALID_ARG;
  if (!aligned(x, 16) || !aligned(add, 16) || !aligned(gain, 16) || !aligned(h, 16) || !aligned(y, 16) || !aligned(y8, 16) ||
      !aligned(scale, 4) || !aligned(rstd, 4))
    return SWA_ERR_INVALID_ARG;
  if ((s = check_device()) != SWA_OK) return s;
  norm::FwdArgs a{};
  a.rows = rows; a.C = C; a.eps = eps;
  a.x = static_cast<const elem_t*>(x); a.add = static_cast<const elem_t*>(add); a.gain = gain;
  a.h = static_cast<elem_t*>(h == x ? (add != nullptr ? h : nullptr) : h);   // h is x already where nothing is added
  a.y = static_cast<elem_t*>(y); a.y8 = static_cast<uint8_t*>(y8); a.scale = scale; a.rstd = rstd;
  const int blocks = norm::row_blocks<false>(rows, C);
  norm::by_width<false>(C, [&](auto tpr, auto vpt) {
    constexpr int T = decltype(tpr)::value, V = decltype(vpt)::value;
    const int threads = T == 32 ? 256 : T;
    if (y8 != nullptr) norm::fwd_kernel<T, V, true><<<blocks, threads, 0, static_cast<cudaStream_t>(stream)>>>(a);
    else norm::fwd_kernel<T, V, false><<<blocks, threads, 0, static_cast<cudaStream_t>(stream)>>>(a);
  });
  return launched();
}

size_t swa_rms_norm_workspace_size(long long rows, int C) {
  if (check_norm(rows, C) != SWA_OK) return 0;
  return (static_cast<size_t>(norm::row_blocks<true>(rows, C)) * C * sizeof(float) + 255) / 256 * 256;
}

swa_status swa_rms_norm_bwd(long long rows, int C, const void* h, const float* rstd, const float* gain, const void* dy,
                            const void* dh, void* dx, float* dgain, void* workspace, size_t ws_bytes, void* stream) {
  swa_status s = check_norm(rows, C);
  if (s != SWA_OK) return s;
  if (!aligned(h, 16) || !aligned(rstd, 4) || !aligned(gain, 16) || !aligned(dy, 16) || !aligned(dh, 16) || !aligned(dx, 16) ||
      !aligned(dgain, 4))
    return SWA_ERR_INVALID_ARG;
  if (rows > 0 && (h == nullptr || rstd == nullptr || dy == nullptr || dx == nullptr)) return SWA_ERR_INVALID_ARG;
  if (dgain != nullptr && rows > 0) {
    if (workspace == nullptr || !aligned(workspace, 256)) return SWA_ERR_INVALID_ARG;
    if (ws_bytes < swa_rms_norm_workspace_size(rows, C)) return SWA_ERR_WORKSPACE;
  }
  cudaStream_t st = static_cast<cudaStream_t>(stream);
  if (rows == 0) {
    if (dgain == nullptr) return SWA_OK;
    cudaMemsetAsync(dgain, 0, static_cast<size_t>(C) * sizeof(float), st);
    return launched();
  }
  if ((s = check_device()) != SWA_OK) return s;
  norm::BwdArgs a{};
  a.rows = rows; a.C = C;
  a.h = static_cast<const elem_t*>(h); a.rstd = rstd; a.gain = gain;
  a.dy = static_cast<const elem_t*>(dy); a.dh = static_cast<const elem_t*>(dh); a.dx = static_cast<elem_t*>(dx);
  a.part = dgain != nullptr ? static_cast<float*>(workspace) : nullptr;
  const int blocks = norm::row_blocks<true>(rows, C);
  norm::by_width<true>(C, [&](auto tpr, auto vpt) {
    constexpr int T = decltype(tpr)::value, V = decltype(vpt)::value;
    norm::bwd_kernel<T, V><<<blocks, T == 32 ? 256 : T, T == 32 ? C * sizeof(float) : 0, st>>>(a);
  });
  if ((s = launched()) != SWA_OK || dgain == nullptr) return s;
  norm::gain_kernel<<<(C + 31) / 32, 256, 0, st>>>(a.part, blocks, C, dgain);
  return launched();
}

size_t swa_w4_size(int N, int K) { return check_w4(N, K) != SWA_OK ? 0 : static_cast<size_t>(w4_tiles(N, K)) * w4::kTileBytes; }

swa_status swa_w4_pack(int N, int K, const void* w, void* w4, void* stream) {
  swa_status s = check_w4(N, K);
  if (s != SWA_OK) return s;
  if (!tensor_ok(w) || !tensor_ok(w4)) return SWA_ERR_INVALID_ARG;
  if ((s = check_device()) != SWA_OK) return s;
  const w4::PackArgs a{N, K, static_cast<const elem_t*>(w), static_cast<uint8_t*>(w4)};
  w4::pack_kernel<<<flat_grid(w4_tiles(N, K), 8, num_sms() * 8LL), 256, 0, static_cast<cudaStream_t>(stream)>>>(a);
  return launched();
}

swa_status swa_w4_unpack(int N, int K, const void* w4, void* w, void* stream) {
  swa_status s = check_w4(N, K);
  if (s != SWA_OK) return s;
  if (!tensor_ok(w) || !tensor_ok(w4)) return SWA_ERR_INVALID_ARG;
  if ((s = check_device()) != SWA_OK) return s;
  w4::unpack_kernel<<<flat_grid(w4_tiles(N, K), 8, num_sms() * 8LL), 256, 0, static_cast<cudaStream_t>(stream)>>>(
      N, K, static_cast<const uint8_t*>(w4), static_cast<elem_t*>(w));
  return launched();
}

swa_status swa_w4_linear(int M, int N, int K, const void* x, const float* x_scale, const void* w4, const void* add, void* y,
                         void* workspace, size_t ws_bytes, void* stream) {
  return linear_call(M, N, K, x, x_scale, w4, add, y, workspace, ws_bytes, kWaitLimitNs, stream);
}

swa_status swa_kv4_tree(int B, int n_tokens, int max_new, const int32_t* parent, const int32_t* cu, const int32_t* lens,
                        int32_t* pos, int64_t* seen, void* workspace, size_t ws_bytes, void* stream) {
  swa_status s = check_tokens(B, n_tokens, max_new);
  if (s != SWA_OK) return s;
  if (!aligned(parent, 4) || !aligned(cu, 4) || !aligned(lens, 4) || !aligned(pos, 4) || !aligned(seen, 8)) return SWA_ERR_INVALID_ARG;
  if ((s = check_header(workspace, ws_bytes)) != SWA_OK) return s;
  if (n_tokens == 0) return SWA_OK;
  if (parent == nullptr || cu == nullptr || lens == nullptr || pos == nullptr || seen == nullptr) return SWA_ERR_INVALID_ARG;
  if ((s = check_device()) != SWA_OK) return s;
  const kv4::TreeArgs a{B, n_tokens, max_new, parent, cu, lens, pos, seen, static_cast<uint32_t*>(workspace)};
  kv4::tree_kernel<<<flat_grid(B, kv4::kTreeWarps, num_sms() * 8LL), kv4::kTreeWarps * 32, 0, static_cast<cudaStream_t>(stream)>>>(a);
  return launched();
}

swa_status swa_kv4_move(const swa_params* p, const swa_kv4_cache* c, const int64_t* src, const int64_t* dst, void* workspace,
                        size_t ws_bytes, void* stream) {
  swa_status s = check_rows(p);
  if (s != SWA_OK) return s;
  kv4::MoveArgs a{};
  if ((s = check_cache(p, c, a.c)) != SWA_OK) return s;
  if (p->T > kv4::kTreeTokens) return SWA_ERR_UNSUPPORTED;
  if (!aligned(src, 8) || !aligned(dst, 8)) return SWA_ERR_INVALID_ARG;
  if ((s = check_header(workspace, ws_bytes)) != SWA_OK) return s;
  if (p->B == 0 || p->T == 0) return SWA_OK;
  if (src == nullptr || dst == nullptr) return SWA_ERR_INVALID_ARG;
  if ((s = check_device()) != SWA_OK) return s;
  a.B = p->B; a.T = p->T; a.src = src; a.dst = dst;
  a.status = static_cast<uint32_t*>(workspace);
  const int grid = flat_grid(static_cast<long long>(p->B) * p->Hkv, 1, num_sms() * 64LL);
  by_head_dim(p->d, [&] { kv4::move_kernel<64><<<grid, kv4::kMoveThreads, 0, static_cast<cudaStream_t>(stream)>>>(a); },
              [&] { kv4::move_kernel<128><<<grid, kv4::kMoveThreads, 0, static_cast<cudaStream_t>(stream)>>>(a); });
  return launched();
}

swa_status swa_kv4_tree_attn(const swa_params* p, const swa_extras* ex, const swa_kv4_cache* c, const swa_rope* r,
                             int n_tokens, int max_new, const void* q, const float* gq, const int32_t* table, int max_pages,
                             const int32_t* lens, const int32_t* cu, const int32_t* pos, const int64_t* seen, void* o,
                             float* lse, void* workspace, size_t ws_bytes, void* stream) {
  swa_status s = check_params(p);
  if (s != SWA_OK) return s;
  if (p->T != 1 || p->causal != 1) return SWA_ERR_INVALID_ARG;
  if ((s = check_tokens(p->B, n_tokens, max_new)) != SWA_OK) return s;
  kv4::TreeAttnArgs a{};
  if ((s = check_cache(p, c, a.c)) != SWA_OK) return s;
  bool rope = false;
  if ((s = check_rope(r, p->d, rope)) != SWA_OK) return s;
  if (ex != nullptr && (ex->rope_cos != nullptr || ex->rope_sin != nullptr)) return SWA_ERR_INVALID_ARG;
  if (!width_ok(max_pages, c->page)) return SWA_ERR_INVALID_ARG;
  if (workspace == nullptr || !aligned(workspace, 256)) return SWA_ERR_INVALID_ARG;
  if (ws_bytes < kKv4Bytes) return SWA_ERR_WORKSPACE;
  if (n_tokens == 0) return SWA_OK;
  if (!tensor_ok(q) || !tensor_ok(o) || lse == nullptr || table == nullptr || lens == nullptr || cu == nullptr || pos == nullptr ||
      seen == nullptr)
    return SWA_ERR_INVALID_ARG;
  if (!aligned(lse, 4) || !aligned(table, 4) || !aligned(lens, 4) || !aligned(gq, 16) || !aligned(cu, 4) || !aligned(pos, 4) ||
      !aligned(seen, 8))
    return SWA_ERR_INVALID_ARG;
  const kv4::TreeSplit sp = kv4::tree_split(p->B, p->Hq, p->Hkv, p->d, c->page, max_pages, p->window, max_new, kTreePartFloats);
  // (groups of at least 64 rows of at most 64 tokens: no more items than B * Hq, and than the workspace's counters)
  if ((s = check_device()) != SWA_OK) return s;
  a.B = p->B; a.Hq = p->Hq; a.max_pages = max_pages; a.window = p->window;
  a.scale = p->softmax_scale > 0.f ? p->softmax_scale : 1.0f / std::sqrt(static_cast<float>(p->d));
  a.eps = p->eps;
  a.q = static_cast<const elem_t*>(q); a.gq = gq;
  if (rope) {
    a.rcos = r->cos; a.rsin = r->sin; a.rows = r->rows; a.rot = r->rot; a.interleaved = r->interleaved;
  }
  a.table = table; a.lens = lens; a.cu = cu; a.pos = pos; a.seen = seen;
  a.N = n_tokens; a.max_new = max_new;
  a.o = static_cast<elem_t*>(o); a.lse = lse;
  a.status = static_cast<uint32_t*>(workspace);
  a.chunk = sp.chunk; a.splits = sp.splits; a.groups = sp.groups;
  a.slots = sp.slots; a.setup = sp.setup;
  a.count = reinterpret_cast<unsigned*>(static_cast<uint8_t*>(workspace) + kKv4Count);
  a.part = reinterpret_cast<float*>(static_cast<uint8_t*>(workspace) + kKv4Part);
  a.part_ml = reinterpret_cast<float2*>(a.part + sp.parts * p->d);
  a.wait_limit_ns = ex != nullptr && ex->wait_limit_ns != 0 ? ex->wait_limit_ns : kWaitLimitNs;
  cudaStream_t st = static_cast<cudaStream_t>(stream);
  return a.wait_limit_ns < kPollBelowNs ? launch_tree<true>(a, p->d, sp, st) : launch_tree<false>(a, p->d, sp, st);
}

size_t swa_kv4_block_workspace_size(const swa_params* p, int C, int n_tokens) {
  return check_serve(p, C, n_tokens) == SWA_OK ? serve_layout(p, C, n_tokens).end : 0;
}

swa_status swa_kv4_block(const swa_params* p, const swa_extras* ex, const swa_kv4_cache* c, const swa_rope* r,
                         const swa_kv4_weights* w, int n_tokens, int max_new, const void* x, const void* add, const float* gain,
                         const float* gq, const float* gk, const void* ve, const int32_t* tok, const int64_t* slot,
                         const int32_t* pos, const int32_t* cu, const int64_t* seen, const int32_t* table, int max_pages,
                         const int32_t* lens, void* out, void* workspace, size_t ws_bytes, void* stream) {
  if (p == nullptr || w == nullptr) return SWA_ERR_INVALID_ARG;
  swa_status s = check_serve(p, w->C, n_tokens);
  if (s != SWA_OK) return s;
  const bool tree = seen != nullptr || cu != nullptr;
  if ((seen == nullptr) != (cu == nullptr) || (!tree && n_tokens != p->B)) return SWA_ERR_INVALID_ARG;
  if (ex != nullptr && (ex->gate_x != nullptr || ex->rope_cos != nullptr || ex->rope_sin != nullptr)) return SWA_ERR_INVALID_ARG;
  if (ex != nullptr && ex->gate_w != nullptr && ex->gate_ch > w->C) return SWA_ERR_INVALID_ARG;
  if (workspace == nullptr || !aligned(workspace, 256)) return SWA_ERR_INVALID_ARG;
  const ServeLayout L = serve_layout(p, w->C, n_tokens);
  if (ws_bytes < L.end) return SWA_ERR_WORKSPACE;
  if (n_tokens == 0) return SWA_OK;
  if (!tensor_ok(x) || !tensor_ok(out) || out == x || (add != nullptr && out == add)) return SWA_ERR_INVALID_ARG;
  for (const void* m : {w->wq, w->wk, w->wv, w->wo})
    if (!tensor_ok(m)) return SWA_ERR_INVALID_ARG;
  uint8_t* ws = static_cast<uint8_t*>(workspace);
  const void* h = add != nullptr ? ws + L.h : x;
  // everything that can be refused is, before the first launch: the calls below have their own checks, which these
  // arguments pass, and those of the append and the attention come from outside
  {
    kv4::Cache cache{};
    bool rope = false;
    if ((s = check_cache(p, c, cache)) != SWA_OK || (s = check_rope(r, p->d, rope)) != SWA_OK) return s;
    if ((s = check_tokens(p->B, n_tokens, tree ? max_new : 1)) != SWA_OK) return s;
    if (!width_ok(max_pages, c->page) || slot == nullptr || pos == nullptr || table == nullptr || lens == nullptr) return SWA_ERR_INVALID_ARG;
    if (!aligned(add, 16) || !aligned(gain, 16) || !aligned(gq, 16) || !aligned(gk, 4) || !aligned(tok, 4) || !aligned(slot, 8) ||
        !aligned(pos, 4) || !aligned(cu, 4) || !aligned(seen, 8) || !aligned(table, 4) || !aligned(lens, 4))
      return SWA_ERR_INVALID_ARG;
    if (ve != nullptr && (!aligned(ve, 16) || tok == nullptr || p->vocab < 1)) return SWA_ERR_INVALID_ARG;
    if (ex != nullptr && ex->gate_w != nullptr && (ex->gate_ch < 1 || ex->gate_ch > kMaxGateCh || p->Hkv > kMaxGateHeads))
      return SWA_ERR_INVALID_ARG;
  }
  if ((s = swa_rms_norm(n_tokens, w->C, p->eps, x, add, gain, add != nullptr ? ws + L.h : nullptr, ws + L.xn, nullptr, nullptr,
                        nullptr, stream)) != SWA_OK)
    return s;
  const int nq = p->Hq * p->d, nk = p->Hkv * p->d;
  swa_extras wait{};
  wait.wait_limit_ns = ex != nullptr ? ex->wait_limit_ns : 0;
  const uint64_t wait_ns = wait.wait_limit_ns != 0 ? wait.wait_limit_ns : kWaitLimitNs;
  const struct { const void* w; int n; size_t to; } proj[] = {{w->wq, nq, L.q}, {w->wk, nk, L.k}, {w->wv, nk, L.v}};
  for (const auto& m : proj)
    if ((s = linear_call(n_tokens, m.n, w->C, ws + L.xn, nullptr, m.w, nullptr, ws + m.to, workspace, ws_bytes, wait_ns, stream)) != SWA_OK)
      return s;
  swa_params rows = *p;          // the tokens as rows of one, for the append
  rows.B = n_tokens;
  rows.Hq = p->Hkv;
  swa_extras gate{};
  if (ex != nullptr && ex->gate_w != nullptr && ve != nullptr) {
    gate.gate_x = ws + L.xn;
    gate.gate_x_stride = w->C;
    gate.gate_w = ex->gate_w;
    gate.gate_ch = ex->gate_ch;
  }
  if ((s = swa_kv4_append(&rows, gate.gate_w != nullptr ? &gate : nullptr, c, r, ws + L.k, ws + L.v, gk, ve, tok, nullptr, pos, slot,
                          workspace, ws_bytes, stream)) != SWA_OK)
    return s;
  float* lse = reinterpret_cast<float*>(ws + L.lse);
  s = tree ? swa_kv4_tree_attn(p, &wait, c, r, n_tokens, max_new, ws + L.q, gq, table, max_pages, lens, cu, pos, seen, ws + L.o, lse,
                               workspace, ws_bytes, stream)
           : swa_kv4_attn(p, &wait, c, r, ws + L.q, gq, table, max_pages, lens, ws + L.o, lse, workspace, ws_bytes, stream);
  if (s != SWA_OK) return s;
  return linear_call(n_tokens, w->C, nq, ws + L.o, nullptr, w->wo, h, out, workspace, ws_bytes, wait_ns, stream);
}

}  // extern "C"
