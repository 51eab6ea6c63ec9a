// Host side of the rotary and decode entry points of include/swa_attn.h:
// argument checks and launches. Included at the end of swa_attn.cu, whose
// helpers (check_params, aligned, launched, ...) it uses.
#pragma once

#include "kv4.cuh"
#include "kv4_attn.cuh"
#include "rope.cuh"

namespace {

constexpr int kMaxRowHeads = 65535;

// The problem of the calls whose kernels walk flat lists of rows (rotation,
// append, read): any number of tokens, in any shape. The rotation of few
// tokens counts batches of three heads and more of q and k in grid y.
swa_status check_rows(const swa_params* p) {
  const swa_status s = check_problem(p);
  if (s != SWA_OK) return s;
  return p->Hq > kMaxRowHeads ? SWA_ERR_UNSUPPORTED : SWA_OK;
}

// Rotary tables of the rope and decode calls: r NULL, or both tables NULL:
// none (on = false).
swa_status check_rope(const swa_rope* r, int d, bool& on) {
  on = false;
  if (r == nullptr || (r->cos == nullptr && r->sin == nullptr)) return SWA_OK;
  if (r->cos == nullptr || r->sin == nullptr || !aligned(r->cos, 16) || !aligned(r->sin, 16) || r->rows < 1 ||
      r->rot < 16 || r->rot > d || r->rot % 16 != 0 || (r->interleaved != 0 && r->interleaved != 1))
    return SWA_ERR_INVALID_ARG;
  on = true;
  return SWA_OK;
}

// The workspace of calls that need only its status word: NULL (device checks
// are not reported) or at least the header.
swa_status check_header(void* ws, size_t bytes) {
  if (ws == nullptr) return SWA_OK;
  if (!aligned(ws, 256)) return SWA_ERR_INVALID_ARG;
  return bytes < 256 ? SWA_ERR_WORKSPACE : SWA_OK;
}

constexpr int kMaxPage = 1 << 20;

swa_status check_pages(int n_pages, int page) {
  if (n_pages < 1 || page < kv4::kTile || page % kv4::kTile != 0) return SWA_ERR_INVALID_ARG;
  // tiles are counted in 31 bits (2^31 of them are 2.4 TB and more)
  if (page > kMaxPage || static_cast<long long>(n_pages) * (page / kv4::kTile) > INT32_MAX) return SWA_ERR_UNSUPPORTED;
  return SWA_OK;
}

// A table row's tokens: positions a step or two past them still fit 32 bits.
bool width_ok(int max_pages, int page) {
  return max_pages >= 1 && static_cast<long long>(max_pages) * page <= INT32_MAX - 64;
}

swa_status check_cache(const swa_params* p, const swa_kv4_cache* c, kv4::Cache& out) {
  if (c == nullptr || c->data == nullptr || !aligned(c->data, 16)) return SWA_ERR_INVALID_ARG;
  const swa_status s = check_pages(c->n_pages, c->page);
  if (s != SWA_OK) return s;
  out.data = static_cast<uint8_t*>(c->data);
  out.n_pages = c->n_pages;
  out.page = c->page;
  out.Hkv = p->Hkv;
  out.per_page = kv4::fast_div(static_cast<uint32_t>(c->page / kv4::kTile));
  return SWA_OK;
}

// Blocks of a flat list of `items` for blocks of `per` items, at most `cap`.
int flat_grid(long long items, long long per, long long cap) {
  const long long n = (items + per - 1) / per;
  return static_cast<int>(n < 1 ? 1 : (n < cap ? n : cap));
}

constexpr int kKv4BlocksPerSm = 8;
constexpr long long kFewThreads = 512;   // per SM
constexpr int kAppendBlocksPerSm = 64;

// Workspace of the decode attention: header, counters of finished chunks,
// partial results; one size for every call. Calls of any shape may follow one
// another on a workspace, so the counters, which each call leaves at zero,
// have a place of their own (a call has at most B * Hq <= 65535 of them),
// where no call's partial results ever lie.
constexpr size_t kKv4Count = 256, kKv4Part = kKv4Count + 65536 * sizeof(unsigned);
constexpr size_t kv4_ws_bytes() {
  long long most = 0;
  for (int d = 64; d <= 128; d += 64)
    for (int operands = 1; operands <= 2; ++operands) {
      const long long n = kv4::attn_part_floats(d, operands);
      most = n > most ? n : most;
    }
  return (kKv4Part + static_cast<size_t>(most) * sizeof(float) + 255) / 256 * 256;
}
constexpr size_t kKv4Bytes = kv4_ws_bytes();

template <int D, int NT, bool kPolled>
swa_status launch_attn(const kv4::AttnArgs& a, int heads_kv, cudaStream_t st) {
  auto kern = kv4::attn_kernel<D, NT, kPolled>;
  constexpr int smem = kv4::AttnSmem<D, NT>::bytes;
  static_assert(smem <= 48 * 1024, "within what a launch gets unasked");
  kern<<<dim3(a.splits, heads_kv * a.groups, a.B), kv4::kAttnWarps * 32, smem, st>>>(a);
  return launched();
}
template <bool kPolled>
swa_status launch_attn(const kv4::AttnArgs& a, int d, int heads, int heads_kv, cudaStream_t st) {
  if (d == 64)
    return heads == kv4::kColQ ? launch_attn<64, 1, kPolled>(a, heads_kv, st) : launch_attn<64, 2, kPolled>(a, heads_kv, st);
  return heads == kv4::kColQ ? launch_attn<128, 1, kPolled>(a, heads_kv, st) : launch_attn<128, 2, kPolled>(a, heads_kv, st);
}

template <typename F64, typename F128>
void by_head_dim(int d, F64 f64, F128 f128) {
  if (d == 64) f64(); else f128();
}

// Shared memory of a plan of B requests. The limit that the kernel is given
// is that of the largest plan whatever B is: it holds for the device, and
// another thread's call may lie between a call's asking and its launch.
constexpr size_t plan_smem(int B) { return (static_cast<size_t>(B) * 3 + 1) * sizeof(int); }

// Tokens of one launch of the row kernels, whose rows count in 31 bits.
long long launch_tokens(int Hkv) { return (1LL << 30) / Hkv; }

}  // namespace

extern "C" {

swa_status swa_rope_tables(const swa_rope_freq* f, int first, int rows, float* cos, float* sin, void* stream) {
  if (f == nullptr || first < 0 || rows < 0 || f->rot < 16 || f->rot > kMaxRot || f->rot % 16 != 0)
    return SWA_ERR_INVALID_ARG;
  if (static_cast<long long>(first) + rows > INT32_MAX) return SWA_ERR_INVALID_ARG;
  if (!std::isfinite(f->base) || f->base < 1.0 || !std::isfinite(f->amplitude) || f->amplitude < 0.0)
    return SWA_ERR_INVALID_ARG;
  if (f->scaling < SWA_ROPE_PLAIN || f->scaling > SWA_ROPE_BY_PARTS) return SWA_ERR_INVALID_ARG;
  if (f->scaling != SWA_ROPE_PLAIN && (!std::isfinite(f->factor) || f->factor < 1.0)) return SWA_ERR_INVALID_ARG;
  if (f->scaling == SWA_ROPE_BY_PARTS &&
      (!std::isfinite(f->orig_len) || f->orig_len <= 0.0 || !std::isfinite(f->slow) || !std::isfinite(f->fast) ||
       f->slow < 0.0 || f->fast <= f->slow))
    return SWA_ERR_INVALID_ARG;
  if (cos == nullptr || sin == nullptr || !aligned(cos, 16) || !aligned(sin, 16)) return SWA_ERR_INVALID_ARG;
  if (rows == 0) return SWA_OK;
  const swa_status s = check_device();
  if (s != SWA_OK) return s;
  RopeTableArgs a{};
  const double two_pi = 6.283185307179586476925286766559;
  const double rot = f->rot;
  const double base = f->scaling == SWA_ROPE_NTK ? f->base * std::pow(f->factor, rot / (rot - 2.0)) : f->base;
  a.half = f->rot / 2;
  for (int c = 0; c < a.half; ++c) {
    double th = std::pow(base, -2.0 * c / rot);
    if (f->scaling == SWA_ROPE_LINEAR) th /= f->factor;
    if (f->scaling == SWA_ROPE_BY_PARTS) {
      double keep = (f->orig_len * th / two_pi - f->slow) / (f->fast - f->slow);
      keep = keep < 0.0 ? 0.0 : (keep > 1.0 ? 1.0 : keep);
      th = th * keep + th / f->factor * (1.0 - keep);
    }
    a.turn[c] = static_cast<unsigned long long>(std::ldexp(th / two_pi, 64));   // theta <= 1: below 2^62
  }
  a.cos = cos; a.sin = sin;
  a.n = static_cast<long long>(rows) * a.half / 4;
  a.first = static_cast<unsigned>(first);
  a.amplitude = f->amplitude > 0.0 ? static_cast<float>(f->amplitude) : 1.0f;
  rope_table_kernel<<<flat_grid(a.n, kTableThreads, num_sms() * 8LL), kTableThreads, 0,
                      static_cast<cudaStream_t>(stream)>>>(a);
  return launched();
}

swa_status swa_rope_apply(const swa_params* p, const swa_rope* r, const int32_t* pos, const void* q, const void* k,
                          void* q_out, void* k_out, int inverse, void* workspace, size_t ws_bytes, void* stream) {
  swa_status s = check_rows(p);
  if (s != SWA_OK) return s;
  bool on = false;
  if ((s = check_rope(r, p->d, on)) != SWA_OK) return s;
  const bool fresh = (inverse & SWA_ROPE_NEW_OUTPUTS) != 0;
  inverse &= ~SWA_ROPE_NEW_OUTPUTS;
  if (!on || (inverse != 0 && inverse != 1)) return SWA_ERR_INVALID_ARG;
  if ((q == nullptr) != (q_out == nullptr) || (k == nullptr) != (k_out == nullptr)) return SWA_ERR_INVALID_ARG;
  if (fresh && ((q != nullptr && q == q_out) || (k != nullptr && k == k_out))) return SWA_ERR_INVALID_ARG;
  if (!aligned(q, 16) || !aligned(k, 16) || !aligned(q_out, 16) || !aligned(k_out, 16) || !aligned(pos, 4))
    return SWA_ERR_INVALID_ARG;
  if (pos == nullptr && r->rows < p->T) return SWA_ERR_INVALID_ARG;
  if ((s = check_header(workspace, ws_bytes)) != SWA_OK) return s;
  if (p->B == 0 || p->T == 0 || (q == nullptr && k == nullptr)) return SWA_OK;
  if ((s = check_device()) != SWA_OK) return s;
  constexpr int EPL = 16 / static_cast<int>(sizeof(elem_t));
  RopeArgs a{};
  a.q = static_cast<const elem_t*>(q); a.k = static_cast<const elem_t*>(k);
  a.qo = static_cast<elem_t*>(q_out); a.ko = static_cast<elem_t*>(k_out);
  a.cos = r->cos; a.sin = r->sin; a.pos = pos;
  a.N = static_cast<long long>(p->B) * p->T;
  a.T = p->T; a.rows = r->rows; a.d = p->d; a.rot = r->rot;
  a.Hq = q != nullptr ? p->Hq : 0;
  a.Hkv = k != nullptr ? p->Hkv : 0;
  a.turned = (r->interleaved ? r->rot : r->rot / 2) / EPL;
  const bool in_place = (q == nullptr || q == q_out) && (k == nullptr || k == k_out);
  a.units = a.turned + (in_place ? 0 : (p->d - r->rot) / EPL);
  a.sgn = inverse ? -1.f : 1.f;
  a.fresh = fresh;
  a.status = static_cast<uint32_t*>(workspace);
  const int H = a.Hq + a.Hkv;
  const long long threads = a.N * a.units;
  if (threads / kRopeThreads >= INT32_MAX) return SWA_ERR_UNSUPPORTED;
  // One thread for all heads of its unit reads the angles once; few positions
  // are spread over the heads instead, so that no thread goes round twice.
  a.heads = threads >= num_sms() * kFewThreads ? H : kRopeBatch[r->interleaved];
  const dim3 grid(static_cast<unsigned>((threads + kRopeThreads - 1) / kRopeThreads), (H + a.heads - 1) / a.heads);
  if (r->interleaved)
    rope_kernel<true><<<grid, kRopeThreads, 0, static_cast<cudaStream_t>(stream)>>>(a);
  else
    rope_kernel<false><<<grid, kRopeThreads, 0, static_cast<cudaStream_t>(stream)>>>(a);
  return launched();
}

size_t swa_kv4_cache_size(const swa_params* p, int n_pages, int page) {
  if (check_rows(p) != SWA_OK || check_pages(n_pages, page) != SWA_OK) return 0;
  return static_cast<size_t>(n_pages) * p->Hkv * (page / kv4::kTile) * kv4::tile_bytes(p->d);
}

swa_status swa_kv4_plan(int n_pages, int page, int B, int max_pages, const int32_t* lens, const int32_t* new_lens,
                        int32_t* table, const int32_t* free_pages, int n_free, const int32_t* free_head, int n_tokens,
                        int64_t* slot, int32_t* pos, int32_t* row, int32_t* cu, int32_t* lens_out, int32_t* head_out,
                        void* workspace, size_t ws_bytes, void* stream) {
  swa_status s = check_pages(n_pages, page);
  if (s != SWA_OK) return s;
  if (B < 0 || !width_ok(max_pages, page) || n_free < 0 || n_tokens < 0 || n_tokens > INT32_MAX - kv4::kPlanTokens)
    return SWA_ERR_INVALID_ARG;
  if (B > kv4::kPlanMaxB) return SWA_ERR_UNSUPPORTED;
  if (free_head == nullptr || head_out == nullptr || cu == nullptr || (n_free > 0 && free_pages == nullptr))
    return SWA_ERR_INVALID_ARG;
  if (B > 0 && (lens == nullptr || table == nullptr || lens_out == nullptr)) return SWA_ERR_INVALID_ARG;
  if (n_tokens > 0 && (slot == nullptr || pos == nullptr || row == nullptr)) return SWA_ERR_INVALID_ARG;
  if (!aligned(slot, 16) || !aligned(pos, 16) || !aligned(row, 16)) return SWA_ERR_INVALID_ARG;
  for (const void* x : {static_cast<const void*>(lens), static_cast<const void*>(new_lens), static_cast<const void*>(table),
                        static_cast<const void*>(free_pages), static_cast<const void*>(free_head),
                        static_cast<const void*>(cu), static_cast<const void*>(lens_out),
                        static_cast<const void*>(head_out)})
    if (!aligned(x, 4)) return SWA_ERR_INVALID_ARG;
  // every block reads the inputs for itself while block 0 writes the outputs
  if ((B > 0 && (lens_out == lens || lens_out == new_lens)) || head_out == free_head) return SWA_ERR_INVALID_ARG;
  if ((s = check_header(workspace, ws_bytes)) != SWA_OK) return s;
  if ((s = check_device()) != SWA_OK) return s;
  kv4::PlanArgs a{};
  a.B = B; a.page = page; a.n_pages = n_pages; a.max_pages = max_pages; a.n_free = n_free; a.n_tokens = n_tokens;
  a.lens = lens; a.new_lens = new_lens; a.table = table; a.free_pages = free_pages; a.head = free_head;
  a.slot = slot; a.pos = pos; a.row = row; a.cu = cu; a.lens_out = lens_out; a.head_out = head_out;
  a.status = static_cast<uint32_t*>(workspace);
  const size_t smem = plan_smem(B);
  if (smem > 48 * 1024 - 1024 &&     // what a launch gets unasked, less the kernel's own arrays
      cudaFuncSetAttribute(kv4::plan_kernel, cudaFuncAttributeMaxDynamicSharedMemorySize,
                           static_cast<int>(plan_smem(kv4::kPlanMaxB))) != cudaSuccess) {
    cudaGetLastError();   // told here, and not again by the next launch
    return SWA_ERR_CUDA;
  }
  // as many blocks as the tokens want, or the requests: two to a warp, for their new pages
  const int by_tokens = flat_grid(n_tokens, kv4::kPlanThreads * kv4::kPlanTokens, num_sms());
  const int by_requests = flat_grid(B, kv4::kPlanThreads / 16, num_sms());
  const int grid = by_tokens > by_requests ? by_tokens : by_requests;
  kv4::plan_kernel<<<grid, kv4::kPlanThreads, smem, static_cast<cudaStream_t>(stream)>>>(a);
  return launched();
}

swa_status swa_kv4_append(const swa_params* p, const swa_extras* ex, const swa_kv4_cache* c, const swa_rope* r,
                          const void* k, const void* v, const float* gk, const void* ve, const int32_t* tok,
                          const float* ve_gate, const int32_t* pos, const int64_t* slot, void* workspace,
                          size_t ws_bytes, void* stream) {
  swa_status s = check_rows(p);
  if (s != SWA_OK) return s;
  kv4::AppendArgs a{};
  if ((s = check_cache(p, c, a.c)) != SWA_OK) return s;
  bool rope = false;
  if ((s = check_rope(r, p->d, rope)) != SWA_OK) return s;
  if (rope && pos == nullptr && r->rows < p->T) return SWA_ERR_INVALID_ARG;
  if (!aligned(pos, 4) || !aligned(slot, 8) || !aligned(gk, 4) || !aligned(tok, 4) || !aligned(ve_gate, 4))
    return SWA_ERR_INVALID_ARG;
  if (ex != nullptr && (ex->rope_cos != nullptr || ex->rope_sin != nullptr)) return SWA_ERR_INVALID_ARG;
  Call call;
  call.p = *p;
  if ((s = set_extras(call, ex, ve_gate)) != SWA_OK) return s;
  if (ve != nullptr && (!aligned(ve, 16) || tok == nullptr || p->vocab < 1)) return SWA_ERR_INVALID_ARG;
  if ((s = check_header(workspace, ws_bytes)) != SWA_OK) return s;
  if (p->B == 0 || p->T == 0) return SWA_OK;
  if (!tensor_ok(k) || !tensor_ok(v) || slot == nullptr) return SWA_ERR_INVALID_ARG;
  if ((s = check_device()) != SWA_OK) return s;
  a.heads = kv4::fast_div(static_cast<uint32_t>(p->Hkv));
  a.seq = kv4::fast_div(static_cast<uint32_t>(p->T));
  a.eps = p->eps; a.ve_scale = p->ve_scale; a.vocab = p->vocab;
  a.gk = gk;
  if (ve != nullptr) {
    a.ve = static_cast<const elem_t*>(ve);
    a.gx_stride = call.gx_stride; a.gw = call.gw; a.gch = call.gch;
  }
  if (rope) {
    a.rcos = r->cos; a.rsin = r->sin; a.rows = r->rows; a.rot = r->rot; a.interleaved = r->interleaved;
  }
  a.status = static_cast<uint32_t*>(workspace);
  cudaStream_t st = static_cast<cudaStream_t>(stream);
  const long long cap = static_cast<long long>(num_sms()) * kAppendBlocksPerSm;
  const long long tokens = static_cast<long long>(p->B) * p->T, step = launch_tokens(p->Hkv);
  for (long long n0 = 0; n0 < tokens; n0 += step) {
    a.N = static_cast<uint32_t>(tokens - n0 < step ? tokens - n0 : step);
    a.t0 = static_cast<uint32_t>(n0 % p->T);
    const long long row0 = n0 * p->Hkv * p->d;
    a.k = static_cast<const elem_t*>(k) + row0; a.v = static_cast<const elem_t*>(v) + row0;
    a.pos = pos ? pos + n0 : nullptr; a.slot = slot + n0;
    if (ve != nullptr) {
      a.tok = tok + n0;
      a.gate = ve_gate ? ve_gate + n0 * p->Hkv : nullptr;
      a.gx = call.gx ? call.gx + n0 * call.gx_stride : nullptr;
    }
    const long long rows = static_cast<long long>(a.N) * p->Hkv;
    auto launch = [&](auto kern, int rpi) { kern<<<flat_grid(rows, kv4::kAppendWarps * rpi, cap), kv4::kAppendWarps * 32, 0, st>>>(a); };
    by_head_dim(p->d,
        [&] { ve ? launch(kv4::append_kernel<64, true>, RowMap<64>::RPI) : launch(kv4::append_kernel<64, false>, RowMap<64>::RPI); },
        [&] { ve ? launch(kv4::append_kernel<128, true>, RowMap<128>::RPI) : launch(kv4::append_kernel<128, false>, RowMap<128>::RPI); });
    if ((s = launched()) != SWA_OK) return s;
  }
  return SWA_OK;
}

swa_status swa_kv4_read(const swa_params* p, const swa_kv4_cache* c, const int64_t* slot, void* k_out, void* v_out,
                        void* workspace, size_t ws_bytes, void* stream) {
  swa_status s = check_rows(p);
  if (s != SWA_OK) return s;
  kv4::ReadArgs a{};
  if ((s = check_cache(p, c, a.c)) != SWA_OK) return s;
  if ((s = check_header(workspace, ws_bytes)) != SWA_OK) return s;
  if (!aligned(slot, 8)) return SWA_ERR_INVALID_ARG;
  if (p->B == 0 || p->T == 0) return SWA_OK;
  if (!tensor_ok(k_out) || !tensor_ok(v_out) || slot == nullptr) return SWA_ERR_INVALID_ARG;
  if ((s = check_device()) != SWA_OK) return s;
  a.heads = kv4::fast_div(static_cast<uint32_t>(p->Hkv));
  a.status = static_cast<uint32_t*>(workspace);
  cudaStream_t st = static_cast<cudaStream_t>(stream);
  const long long cap = static_cast<long long>(num_sms()) * kKv4BlocksPerSm;
  const long long tokens = static_cast<long long>(p->B) * p->T, step = launch_tokens(p->Hkv);
  for (long long n0 = 0; n0 < tokens; n0 += step) {
    a.N = static_cast<uint32_t>(tokens - n0 < step ? tokens - n0 : step);
    a.slot = slot + n0;
    a.k = static_cast<elem_t*>(k_out) + n0 * p->Hkv * p->d;
    a.v = static_cast<elem_t*>(v_out) + n0 * p->Hkv * p->d;
    const long long rows = static_cast<long long>(a.N) * p->Hkv;
    auto launch = [&](auto kern, int rpi) { kern<<<flat_grid(rows, kRowWarps * rpi, cap), kRowWarps * 32, 0, st>>>(a); };
    by_head_dim(p->d, [&] { launch(kv4::read_kernel<64>, RowMap<64>::RPI); }, [&] { launch(kv4::read_kernel<128>, RowMap<128>::RPI); });
    if ((s = launched()) != SWA_OK) return s;
  }
  return SWA_OK;
}

size_t swa_kv4_workspace_size(const swa_params* p, int page, int max_pages) {
  if (check_params(p) != SWA_OK || check_pages(1, page) != SWA_OK || !width_ok(max_pages, page)) return 0;
  return kKv4Bytes;
}

swa_status swa_kv4_workspace_init(void* workspace, size_t ws_bytes, void* stream) {
  if (workspace == nullptr || !aligned(workspace, 256)) return SWA_ERR_INVALID_ARG;
  if (ws_bytes < kKv4Bytes) return SWA_ERR_WORKSPACE;
  if (cudaMemsetAsync(workspace, 0, kKv4Part, static_cast<cudaStream_t>(stream)) != cudaSuccess) return SWA_ERR_CUDA;
  return SWA_OK;
}

swa_status swa_kv4_attn(const swa_params* p, const swa_extras* ex, const swa_kv4_cache* c, const swa_rope* r,
                        const void* q, const float* gq, const int32_t* table, int max_pages, const int32_t* lens,
                        void* o, float* lse, void* workspace, size_t ws_bytes, void* stream) {
  swa_status s = check_params(p);
  if (s != SWA_OK) return s;
  if (p->T != 1 || p->causal != 1) return SWA_ERR_INVALID_ARG;
  kv4::AttnArgs a{};
  if ((s = check_cache(p, c, a.c)) != SWA_OK) return s;
  bool rope = false;
  if ((s = check_rope(r, p->d, rope)) != SWA_OK) return s;
  if (ex != nullptr && (ex->rope_cos != nullptr || ex->rope_sin != nullptr)) return SWA_ERR_INVALID_ARG;
  if (!width_ok(max_pages, c->page)) return SWA_ERR_INVALID_ARG;
  if (workspace == nullptr || !aligned(workspace, 256)) return SWA_ERR_INVALID_ARG;
  const kv4::AttnSplit sp = kv4::attn_split(p->B, p->Hq, p->Hkv, p->d, c->page, max_pages, p->window);
  if (ws_bytes < kKv4Bytes) return SWA_ERR_WORKSPACE;
  if (p->B == 0) return SWA_OK;
  if (!tensor_ok(q) || !tensor_ok(o) || lse == nullptr || table == nullptr || lens == nullptr) return SWA_ERR_INVALID_ARG;
  if (!aligned(lse, 4) || !aligned(table, 4) || !aligned(lens, 4) || !aligned(gq, 16)) return SWA_ERR_INVALID_ARG;
  if ((s = check_device()) != SWA_OK) return s;
  a.B = p->B; a.Hq = p->Hq; a.max_pages = max_pages; a.window = p->window;
  a.scale = p->softmax_scale > 0.f ? p->softmax_scale : 1.0f / std::sqrt(static_cast<float>(p->d));
  a.eps = p->eps;
  a.q = static_cast<const elem_t*>(q); a.gq = gq;
  if (rope) {
    a.rcos = r->cos; a.rsin = r->sin; a.rows = r->rows; a.rot = r->rot; a.interleaved = r->interleaved;
  }
  a.table = table; a.lens = lens;
  a.o = static_cast<elem_t*>(o); a.lse = lse;
  a.status = static_cast<uint32_t*>(workspace);
  a.chunk = sp.chunk; a.splits = sp.splits; a.groups = sp.groups;
  a.count = reinterpret_cast<unsigned*>(static_cast<uint8_t*>(workspace) + kKv4Count);
  a.part = reinterpret_cast<float*>(static_cast<uint8_t*>(workspace) + kKv4Part);
  a.part_ml = reinterpret_cast<float2*>(a.part + sp.items * sp.splits * sp.heads * p->d);
  a.wait_limit_ns = ex != nullptr && ex->wait_limit_ns != 0 ? ex->wait_limit_ns : kWaitLimitNs;
  cudaStream_t st = static_cast<cudaStream_t>(stream);
  return a.wait_limit_ns < kPollBelowNs ? launch_attn<true>(a, p->d, sp.heads, p->Hkv, st)
                                        : launch_attn<false>(a, p->d, sp.heads, p->Hkv, st);
}

}  // extern "C"
