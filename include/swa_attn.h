/*
 * swa_attn.h - C ABI of the GB300 (sm_103a) attention-block library.
 *
 * The block computed here is the attention of the autoresearch GPT training
 * script as its pages describe it:
 *   - QK-norm: RMSNorm of queries and keys right before the attention dot
 *     product (autoresearch train.py walkthrough post, model paragraph;
 *     "autoresearch Administrator & Developer Guide" §8.2.1, F.rms_norm row),
 *     here with optional learned per-channel gains gq, gk of shape [d];
 *   - grouped-query attention, n_kv_head <= n_head (Guide §8.2.1, GQA row;
 *     §6.3 techniques table): query head h reads kv head h / (Hq / Hkv);
 *   - a causal sliding window or full causal mask per layer, chosen by the
 *     "SSSL" window pattern (post, model paragraph; Guide §3.4 WINDOW_PATTERN);
 *   - on value-embedding layers, v_eff = v + ve_scale * gate * VE[token]
 *     (Guide §8.2.1, value-embedding row and its gate snippet).
 *
 * Two shared libraries export these symbols:
 *   libswaattn.so       bf16 tensors, tcgen05 tensor-core kernels (the product path);
 *   libswaattn_fp32.so  fp32 tensors, SIMT FFMA kernels (a debug build with
 *                       the same band schedule, used to check the method at
 *                       fp32 precision).
 * "elem" below is bf16 (raw 16-bit bit patterns) in the first, float in the
 * second. Gains, LSE, gate and all gradients of shared parameters are fp32 in
 * both.
 *
 * Conventions common to every call:
 *   - All tensor pointers are DEVICE pointers of the current CUDA device; the
 *     caller owns every buffer, including the workspace. The library never
 *     allocates or frees device memory.
 *   - Layouts are dense row-major:
 *       q, o, dO, dq       [B, T, Hq,  d]   elem
 *       k, v, dk, dv       [B, T, Hkv, d]   elem
 *       lse                [B, Hq, T]       fp32, natural-log sum of exp of the
 *                                           scaled, masked logits of each row
 *       gq, gk, dgq, dgk   [d]              fp32
 *       ve, dve            [vocab, Hkv*d]   elem (ve) / fp32 (dve)
 *       tok                [B, T]           int32
 *       ve_gate            [B, T, Hkv]      fp32
 *   - Tensor pointers must be 16-byte aligned; the workspace 256-byte aligned.
 *   - Calls are asynchronous on `stream` (a cudaStream_t; NULL = legacy default
 *     stream). SWA_ERR_INVALID_ARG, SWA_ERR_WORKSPACE and the unsupported-
 *     size checks come before the first launch: nothing was launched. A
 *     failing CUDA call inside a call (SWA_ERR_CUDA) can come after earlier
 *     launches of that call; its outputs are then undefined. Errors found on the device (a bounded wait that ran
 *     out, a token id outside [0, vocab)) are OR-ed into a status word in the
 *     workspace header and read back by swa_attn_check_status().
 *   - B == 0 or T == 0 is a valid empty problem: nothing is computed; the
 *     backward still zero-fills dgq, dgk and dve.
 */
#ifndef SWA_ATTN_H
#define SWA_ATTN_H

#include <stddef.h>
#include <stdint.h>

#ifdef __cplusplus
extern "C" {
#endif

typedef enum swa_status {
  SWA_OK = 0,
  SWA_ERR_INVALID_ARG = 1,  /* bad shape, NULL pointer, misalignment, bad flag   */
  SWA_ERR_UNSUPPORTED = 2,  /* valid but not built: d not in {64,128}, wrong GPU  */
  SWA_ERR_CUDA = 3,         /* a CUDA runtime/driver call failed                  */
  SWA_ERR_TIMEOUT = 4,      /* device: a bounded pipeline wait ran out            */
  SWA_ERR_WORKSPACE = 5,    /* workspace too small for this problem               */
  SWA_ERR_DEVICE_CHECK = 6  /* device: a token id outside [0, vocab) was skipped; in
                               the rotary and decode calls also a position, slot,
                               page, length or request that was refused           */
} swa_status;

/* Problem description shared by every call. */
typedef struct swa_params {
  int B, T;         /* batch, sequence length (>= 0)                              */
  int Hq, Hkv;      /* query heads, kv heads; Hq % Hkv == 0                       */
  int d;            /* head dim: 64 or 128                                         */
  int window;       /* -1: no window. Else, causal: key j visible to query i iff
                       i - window <= j <= i; non-causal: iff |i - j| <= window.
                       window >= T - 1 is the same as -1.                          */
  int causal;       /* 1: causal (every layer of the SSSL stack); 0: bidirectional */
  float softmax_scale; /* 0: 1/sqrt(d)                                             */
  float eps;        /* RMSNorm epsilon, >= 0 (the script's F.rms_norm default is
                       used by callers that pass 1e-6)                             */
  float ve_scale;   /* multiplies gate * VE[tok]; ignored when ve == NULL          */
  int vocab;        /* rows of the VE table; ignored when ve == NULL               */
} swa_params;

/* flags */
#define SWA_REUSE_PROLOGUE 1u  /* the workspace still holds this problem's QK-norm /
                                  VE-mix outputs from an earlier call with the same
                                  inputs: skip recomputing them                       */
#define SWA_BWD_STAGE_PRE 2u   /* backward stages to run; none of the three bits set */
#define SWA_BWD_STAGE_MAIN 4u  /* means all of them. PRE: D = rowsum(dO * O), clear   */
#define SWA_BWD_STAGE_POST 8u  /* the accumulators unless the forward left them
                                  zeroed (and dve); MAIN: the attention
                                  backward with the key-side RMSNorm backward (dk,
                                  dv, dve); POST: query-side RMSNorm backward and
                                  the gain gradients.
                                  Running them one call at a time, in this order,
                                  gives the same result as one call with all three.  */

/*
 * Bytes of workspace a problem needs (forward only, or forward + backward).
 * Returns 0 when the parameters are invalid. The workspace holds a 256-byte
 * header (device status word, record of a zeroed dQ accumulator), the
 * QK-norm outputs qn, kn and their inverse
 * RMS, v_eff on VE layers, and for the backward the fp32 accumulators.
 * A fresh workspace must be initialised once with swa_attn_workspace_init().
 */
size_t swa_attn_workspace_size(const swa_params* p, int for_backward);

/* Zeroes the workspace header (status word) on `stream`. */
swa_status swa_attn_workspace_init(void* workspace, size_t ws_bytes, void* stream);

/*
 * Forward: o = softmax(scale * qn kn^T + mask) v_eff and lse, where
 * qn = gq * q / sqrt(mean(q^2) + eps) (likewise kn) and v_eff = v on plain
 * layers, v + ve_scale * gate * VE[tok] on value-embedding layers.
 *   gq, gk   may be NULL (unit gains).
 *   ve       NULL: no value embedding (tok, ve_gate ignored). Else tok is
 *            required and ve_gate may be NULL (gate = 1, the pages' gate at
 *            initialisation: 2 * sigmoid(0)).
 *   flags    0 or SWA_REUSE_PROLOGUE.
 * Writes o and lse, and the prologue outputs into the workspace (kept for the
 * backward's SWA_REUSE_PROLOGUE). When ws_bytes is at least the backward
 * size (swa_attn_workspace_size(p, 1)) and Hq / Hkv is even, the forward
 * kernel also zeroes the backward's fp32 dQ accumulator and records that in
 * the workspace header; the next backward of the same problem on this
 * workspace then skips that clear. Any later call that may overwrite the
 * accumulator drops the record (a forward that does not zero it, the
 * backward's main stage).
 */
swa_status swa_attn_fwd(const swa_params* p, const void* q, const void* k, const void* v,
                        const float* gq, const float* gk, const void* ve, const int32_t* tok,
                        const float* ve_gate, void* o, float* lse, void* workspace,
                        size_t ws_bytes, unsigned flags, void* stream);

/*
 * Backward of the forward for the loss <o, dO>: gradients of q, k, v, the
 * gains and the VE table. Inputs as in swa_attn_fwd plus the forward's o and
 * lse and the upstream gradient dO. Outputs (overwritten, not accumulated):
 *   dq, dk, dv       required.
 *   dgq, dgk         may be NULL (not computed); when non-NULL they receive
 *                    the full gain gradient (summed over batch, time, heads).
 *                    With gq (gk) NULL the gain is 1 and dgq (dgk) is still the
 *                    gradient with respect to it.
 *   dve              may be NULL; when non-NULL (and ve != NULL) it receives
 *                    the gradient of the VE table, zero in rows no token used.
 * The gradient of a given ve_gate is not produced (it is an input); the
 * learned gate of swa_attn_bwd_ex produces its own gradients.
 * flags: SWA_REUSE_PROLOGUE and the SWA_BWD_STAGE_* bits.
 */
swa_status swa_attn_bwd(const swa_params* p, const void* q, const void* k, const void* v,
                        const float* gq, const float* gk, const void* ve, const int32_t* tok,
                        const float* ve_gate, const void* o, const float* lse, const void* dO,
                        void* dq, void* dk, void* dv, float* dgq, float* dgk, float* dve,
                        void* workspace, size_t ws_bytes, unsigned flags, void* stream);

/*
 * Extras of the _ex entry points (each part optional; all-NULL extras, or a
 * NULL pointer, make them identical to swa_attn_fwd / swa_attn_bwd).
 *
 * Rotary position embedding, fused into the QK-norm prologue (rotation
 * first, then the norm, so the norm comes right before the dot product, as
 * in the autoresearch train.py walkthrough post, model paragraph; the
 * Administrator & Developer Guide §8.2.1 model table, "Rotary embeddings"
 * row, has the cos / sin tables precomputed once by the caller). The pages
 * print neither the channel pairing nor the sign; this library pairs channel
 * c with c + d/2 and turns the pair of position t by the angle of row t,
 * column c:
 *   y_c       =  x_c cos[t][c] + x_{c+d/2} sin[t][c]
 *   y_{c+d/2} = -x_c sin[t][c] + x_{c+d/2} cos[t][c]        (c < d/2)
 *   rope_cos, rope_sin  fp32 [rope_rows][d/2] row-major, 16-byte aligned,
 *                       rope_rows >= T (row t is position t); both NULL: none.
 *
 * Learned value-embedding gate (Guide §8.2.1, the gate snippet): on VE
 * calls, gate[b,t,h] = 2 * sigmoid(sum_c gate_w[h][c] * gate_x[b,t,c]), used
 * in place of the ve_gate argument (which must then be NULL):
 *   gate_x         elem (bf16 / fp32 per library) rows of the block input;
 *                  channel c of position (b, t) at gate_x[(b*T + t)*gate_x_stride + c]
 *   gate_x_stride  elements between consecutive (b, t) rows (>= gate_ch)
 *   gate_w         fp32 [Hkv][gate_ch]; NULL: no learned gate
 *   gate_ch        1 .. 32 channels (32 in the pages); Hkv <= 32
 *   d_gate_w       backward output, fp32 [Hkv][gate_ch] (overwritten), or NULL
 *   d_gate_x       backward output, fp32 [B, T, gate_ch] (overwritten): the
 *                  gradient of the channels read (the caller adds it into
 *                  its gradient of the block input), or NULL
 * The forward keeps the gate values in the workspace for the backward.
 *
 * Time limit of the kernels' pipeline waits (not from the pages: a property
 * of this library's kernels, whose warps hand work to each other through
 * shared-memory barriers):
 *   wait_limit_ns  0: the default, 2 s per wait. Else the limit of every
 *                  pipeline wait of this call's tensor-core kernels. A wait
 *                  that runs out makes its CTA give up: it records
 *                  SWA_ERR_TIMEOUT in the workspace status word, lets the
 *                  copies and MMAs it issued land (those waits keep their
 *                  own 2 s limit), and returns; the call's outputs are then
 *                  undefined. A short limit is how a caller (or a test) can
 *                  make this path run. Limits below 1 ms are kept by polling
 *                  the barrier without suspending; longer ones by the
 *                  barrier's suspending wait, with the clock read every 64
 *                  polls. The fp32 debug build has no such waits and ignores
 *                  the field.
 */
typedef struct {
  const float* rope_cos;
  const float* rope_sin;
  int rope_rows;
  const void* gate_x;
  long long gate_x_stride;
  const float* gate_w;
  int gate_ch;
  float* d_gate_w;
  float* d_gate_x;
  unsigned long long wait_limit_ns;
} swa_extras;

/* swa_attn_fwd with extras (arguments otherwise identical). */
swa_status swa_attn_fwd_ex(const swa_params* p, const swa_extras* ex, const void* q, const void* k,
                           const void* v, const float* gq, const float* gk, const void* ve,
                           const int32_t* tok, const float* ve_gate, void* o, float* lse,
                           void* workspace, size_t ws_bytes, unsigned flags, void* stream);

/* swa_attn_bwd with extras: with rotary, dq and dk are the gradients of the
 * unrotated q and k (the transposed rotation of the norm backward's result);
 * with the learned gate, d_gate_w and d_gate_x as above (written by the POST
 * stage). A backward with SWA_REUSE_PROLOGUE needs the same extras as its
 * forward. */
swa_status swa_attn_bwd_ex(const swa_params* p, const swa_extras* ex, const void* q, const void* k,
                           const void* v, const float* gq, const float* gk, const void* ve,
                           const int32_t* tok, const float* ve_gate, const void* o,
                           const float* lse, const void* dO, void* dq, void* dk, void* dv,
                           float* dgq, float* dgk, float* dve, void* workspace, size_t ws_bytes,
                           unsigned flags, void* stream);

/*
 * Forward without a caller-provided workspace: the same computation and
 * outputs as swa_attn_fwd (flags 0), but its scratch (QK-norm / VE-mix
 * outputs and the status word) lives in one fixed array of
 * SWA_NOALLOC_SCRATCH_BYTES of device memory inside the library. The pages
 * have no counterpart of this call; it exists for callers that cannot
 * allocate device memory at the point where they run the attention: a
 * plug-in whose host framework owns every allocation, a service that must not
 * grow its memory after start-up, or a latency-critical path that cannot
 * afford cudaMalloc's implicit device synchronisation.
 *   - Allocates nothing: no cudaMalloc, no cudaFree, no allocating library
 *     routine. The array is part of the library's device code, so every GPU
 *     that loads the library holds it until the process exits.
 *   - The first call on a device looks up the array's device address (once
 *     per device, with that device current), and a call looks it up again
 *     when the calling thread's current CUDA context is not the one of that
 *     lookup (after cudaDeviceReset, or under a context the caller made
 *     current); make the first call on a device, and the first after such a
 *     change, before any stream capture begins.
 *   - Problems whose forward workspace (swa_attn_workspace_size(p, 0)) is
 *     larger than the array are rejected with SWA_ERR_WORKSPACE, launching
 *     nothing.
 *   - Every call, from any stream or thread, shares the one array and it
 *     keeps the last call's contents: calls that overlap on the GPU race and
 *     corrupt each other's results; order them (same stream or events).
 *     Nothing in it has to start at zero (the prologue writes every value the
 *     forward reads).
 *   - Device-side checks are not reported: when one fires (a token id outside
 *     [0, vocab), a pipeline wait that ran out) this call still returns
 *     SWA_OK, and o and lse are undefined. Callers that need to see those
 *     checks use swa_attn_fwd with a workspace and swa_attn_check_status.
 */
#define SWA_NOALLOC_SCRATCH_BYTES (32u * 1024u * 1024u)
swa_status swa_attn_fwd_noalloc(const swa_params* p, const void* q, const void* k,
                                const void* v, const float* gq, const float* gk, const void* ve,
                                const int32_t* tok, const float* ve_gate, void* o, float* lse,
                                void* stream);

/*
 * One training step of one attention call with every tensor in HOST memory:
 * the inputs are copied host -> device, the forward and the backward run
 * (the backward reusing the forward's QK-norm / VE-mix outputs), and o, lse
 * and the gradients are copied device -> host, all enqueued on `stream` in
 * that order; the call returns without waiting (synchronize the stream, or
 * record an event after it, before reading the outputs). The pages have no
 * counterpart of this call: it is the library's end-to-end path for callers
 * whose data lives on the host.
 *   q, k, v, dO, gq, gk, ve, tok, ve_gate   host inputs, the layouts and
 *                  meanings of swa_attn_fwd / swa_attn_bwd (gq, gk, ve, tok,
 *                  ve_gate may be NULL as there)
 *   o, lse, dq, dk, dv, dgq, dgk, dve        host outputs, as there
 *                  (dgq, dgk, dve may be NULL: not computed, not copied)
 *   ex             as for the _ex calls; its rotary tables and gate weights
 *                  are DEVICE pointers (not copied)
 *   device_buffer  device memory of at least swa_attn_step_host_size(p)
 *                  bytes, 256-byte aligned, passed to swa_attn_workspace_init
 *                  once before its first use; it holds the attention's
 *                  workspace (so swa_attn_check_status reads it) and the
 *                  device copies of every input and output. Reusing it on the
 *                  same stream is safe (stream order); on several streams at
 *                  once, give each its own buffer.
 * Copies from and to pageable host memory make the CUDA runtime stage them
 * and block the calling thread; page-locked (pinned) host buffers let them
 * run asynchronously and overlap work on other streams. Each copy is one
 * cudaMemcpyAsync. Errors: SWA_ERR_INVALID_ARG for a NULL required pointer
 * or a misaligned device buffer, SWA_ERR_WORKSPACE for a buffer too small,
 * both before anything is enqueued; then those of swa_attn_fwd and
 * swa_attn_bwd, and SWA_ERR_CUDA when a copy cannot be enqueued (the outputs
 * are then undefined).
 */
size_t swa_attn_step_host_size(const swa_params* p);
swa_status swa_attn_step_host(const swa_params* p, const swa_extras* ex, const void* q,
                              const void* k, const void* v, const float* gq, const float* gk,
                              const void* ve, const int32_t* tok, const float* ve_gate,
                              const void* dO, void* o, float* lse, void* dq, void* dk, void* dv,
                              float* dgq, float* dgk, float* dve, void* device_buffer,
                              size_t device_bytes, void* stream);

/*
 * The whole attention block around the core: the block's pre-norm, the four
 * bias-free projections c_q, c_k, c_v, c_proj and the residual
 * (autoresearch Administrator & Developer Guide §8.2.1 model table,
 * "Pre-norm + residual": x = x + attn(norm(x)); train.py walkthrough post,
 * model paragraph: RMSNorm on the block inputs):
 *   xn  = x / sqrt(mean_c(x^2) + eps)               (no gain; eps of swa_params)
 *   q   = xn wq^T, k = xn wk^T, v = xn wv^T         (viewed as [B, T, H, d])
 *   o   = the attention of swa_attn_fwd_ex on (q, k, v), with the learned
 *         gate (if any) reading the first gate_ch channels of xn
 *   out = x + o wo^T                                (o viewed as [B, T, Hq*d])
 * Weights use the torch.nn.Linear layout [out_features][in_features], elem:
 *   wq [Hq*d][C], wk and wv [Hkv*d][C], wo [C][Hq*d];  x, out, dout, dx
 *   [B, T, C] elem;  weight gradients dwq, dwk, dwv, dwo fp32, same shapes
 *   as the weights (overwritten; NULL skips one).
 * C (the model width) is a multiple of 8, at most 65536; B*T < 2^31.
 * Extras: rotary tables and gate_w / gate_ch / d_gate_w as for the _ex
 * calls; gate_x and d_gate_x must be NULL (the block supplies the gate's
 * input and adds the gradient of the channels it read into dx); gate_ch <= C.
 * As in the attention calls, the gate applies on value-embedding calls only
 * (ve != NULL); without a VE table it is ignored and d_gate_w is not written.
 * The projections run on this library's own GEMM kernels (tcgen05 tensor
 * cores with bf16 operands and fp32 accumulation in the bf16 library, fp32
 * SIMT in the fp32 debug library); the weight gradients split B*T over
 * several CTAs and add their fp32 partial sums into dwq, dwk, dwv and dwo,
 * so their last bits can differ from run to run. The workspace
 * (swa_block_workspace_size) holds the attention's workspace first (so
 * swa_attn_check_status reads the block workspace too),
 * then the forward's saved tensors (xn, q, k, v, o, lse) and a transposed
 * copy of the rotary tables; swa_block_bwd needs the workspace that
 * swa_block_fwd filled for the same inputs.
 */
typedef struct {
  int C;              /* model width: channels of x                         */
  const void* wq;     /* [Hq*d][C]  elem                                     */
  const void* wk;     /* [Hkv*d][C] elem                                     */
  const void* wv;     /* [Hkv*d][C] elem                                     */
  const void* wo;     /* [C][Hq*d]  elem                                     */
} swa_block_weights;

/* Bytes of workspace for swa_block_fwd (for_backward = 0) or for the pair
 * swa_block_fwd + swa_block_bwd (for_backward = 1); 0 for invalid arguments. */
size_t swa_block_workspace_size(const swa_params* p, int C, int for_backward);

/* out = x + c_proj(attention(c_q, c_k, c_v of the normed x)). */
swa_status swa_block_fwd(const swa_params* p, const swa_extras* ex, const swa_block_weights* w,
                         const void* x, const float* gq, const float* gk, const void* ve,
                         const int32_t* tok, void* out, void* workspace, size_t ws_bytes, void* stream);

/* Gradients of <out, dout>: dx (elem, including the residual's dout), the
 * weight gradients, and the attention's dgq, dgk, dve, d_gate_w as in
 * swa_attn_bwd_ex. */
swa_status swa_block_bwd(const swa_params* p, const swa_extras* ex, const swa_block_weights* w,
                         const void* x, const float* gq, const float* gk, const void* ve,
                         const int32_t* tok, const void* dout, void* dx, float* dwq, float* dwk,
                         float* dwv, float* dwo, float* dgq, float* dgk, float* dve, void* workspace,
                         size_t ws_bytes, void* stream);

/*
 * Rotary positions as operators of their own. The _ex and block calls fuse
 * one form of them (whole heads, channels c and c + d/2 paired, positions
 * counted from 0); these calls build the tables that form reads, and rotate q
 * and k in every form: of the whole head or its first `rot` channels, paired
 * as two halves or side by side, at positions of the caller's. With a
 * rotation of its own, the attention is called without rotary tables:
 * swa_rope_apply, swa_attn_fwd, swa_attn_bwd, then swa_rope_apply with
 * inverse = 1 on dq and dk (the rotation's transpose is its backward).
 *
 * swa_rope_tables writes, for the rows t = first .. first + rows - 1,
 *   cos[t - first][c] = amplitude * cos(t * theta_c), sin likewise,
 *   fp32 [rows][rot/2], 16-byte aligned, c < rot/2, theta_c = base^(-2c/rot),
 * with the frequencies scaled for contexts longer than those trained on:
 *   SWA_ROPE_PLAIN     as they are (factor is not read)
 *   SWA_ROPE_LINEAR    theta_c / factor (positions interpolated)
 *   SWA_ROPE_NTK       base * factor^(rot / (rot - 2)) in place of base
 *   SWA_ROPE_BY_PARTS  (YaRN, Peng et al. 2023, "NTK-by-parts") a column
 *                      that makes n = orig_len * theta_c / (2 pi) turns over
 *                      the original context keeps theta_c for n >= fast, gets
 *                      theta_c / factor for n <= slow, and in between the two
 *                      mixed by (n - slow) / (fast - slow)
 * Angles are reduced exactly in 64-bit fixed point: far positions are as
 * accurate as near ones. Limits: rot a multiple of 16, 16 .. 128; base >= 1;
 * factor >= 1; 0 <= slow < fast; first + rows < 2^31; amplitude 0 counts as 1
 * (after a QK-norm a common amplitude cancels when whole heads are turned).
 */
#define SWA_ROPE_PLAIN 0
#define SWA_ROPE_LINEAR 1
#define SWA_ROPE_NTK 2
#define SWA_ROPE_BY_PARTS 3
typedef struct {
  int rot;
  int scaling;
  double base, factor, orig_len, slow, fast, amplitude;
} swa_rope_freq;
swa_status swa_rope_tables(const swa_rope_freq* f, int first, int rows, float* cos, float* sin,
                           void* stream);

/*
 * Rotary tables as the calls below read them: row t is position t. rot (a
 * multiple of 16, at most d) channels are turned, the rest are left alone.
 * interleaved 0: channel c < rot/2 pairs with c + rot/2; 1: 2c with 2c + 1.
 * The pair (a, b) of column c becomes (a cos + b sin, b cos - a sin), as in
 * swa_extras.
 */
typedef struct {
  const float* cos;   /* fp32 [rows][rot/2], 16-byte aligned */
  const float* sin;
  int rows;
  int rot;
  int interleaved;
} swa_rope;

/*
 * Rotates q [B, T, Hq, d] into q_out and k [B, T, Hkv, d] into k_out (each
 * pair may be NULL, and an output may be its input: in place; any other
 * overlap is undefined). Of p, B, T, Hq, Hkv and d are read (and all checked).
 *   pos      int32 [B, T] positions, or NULL: row t of the sequence is position
 *            t (then rows >= T). A token whose position is outside the tables
 *            keeps its output rows as they were and is reported.
 *   inverse  1: the transposed rotation, the backward of the forward's; 0: the
 *            rotation. SWA_ROPE_NEW_OUTPUTS may be added: the outputs hold
 *            nothing yet (neither may be its input), and the rows of such
 *            tokens are set to zero
 *   workspace  at least its 256-byte header, where device checks are reported
 *            (swa_attn_check_status); NULL: they are not
 * Sums are fp32, rounded once to elem. Limit: Hq <= 65535, here and in the
 * append, the read and swa_kv4_cache_size, which take any number of tokens B * T.
 */
#define SWA_ROPE_NEW_OUTPUTS 4
swa_status swa_rope_apply(const swa_params* p, const swa_rope* r, const int32_t* pos, const void* q,
                          const void* k, void* q_out, void* k_out, int inverse, void* workspace,
                          size_t ws_bytes, void* stream);

/*
 * The decode path: the same attention for one new token per request, over a
 * paged cache that holds keys (rotated and normed) and values (with their
 * value embedding) in 4 bits. The pages have no counterpart of these calls:
 * the script only trains.
 *
 * The cache is one buffer of swa_kv4_cache_size bytes, 16-byte aligned:
 * [n_pages][Hkv][page/16] tiles of 18 d bytes, page a multiple of 16 tokens.
 * A tile holds 16 consecutive tokens of one kv head:
 *   8 d bytes  keys, token by token, d/2 bytes each
 *   8 d bytes  values, token pair by token pair, d bytes each
 *   d bytes    the keys' scales: [16 tokens][d/64] pairs (s, z) of bf16
 *   d bytes    the values' scales, likewise
 * A number n = 0..15 of 64-channel group g stands for s (n - 8) + z, where
 *   s = bf16((max - min) / 15), z = bf16(min + 8 s) over the group,
 *   n = floor((x - z) / s + 8.5) kept within 0..15, 8 where s = 0.
 * Keys, and values with an embedding, come out of fp32 arithmetic: the z of one
 * may be bf16's other neighbour of min + 8 s where no number depends on it. (A
 * group that holds an infinity or a NaN, or whose span overflows fp32, is held
 * as NaN; steps below 1e-36 count as 0.) Low nibble first, the numbers of a row
 * are in the order
 *   keys    [j 0..3][g][i 0..15]:          channel 64 g + 16 j + i
 *   values  [r 0..7][g][u 0..1][token of the pair][i 0..3]:
 *                                          channel 64 g + 8 r + 4 u + i
 * in which the attention's matrix instructions take them.
 *
 * A slot is page * (page size) + offset, int64; slot -1 is no slot: padding.
 * Every number read from device memory (slots, pages, lengths, positions,
 * token ids) is checked on the device: one out of range is reported in the
 * workspace status word and skipped as stated, never followed. `workspace` of
 * plan, append and read is as in swa_rope_apply.
 */
typedef struct {
  void* data;
  int n_pages;
  int page;
} swa_kv4_cache;
size_t swa_kv4_cache_size(const swa_params* p, int n_pages, int page);

/*
 * The plan of a step: which pages the requests get, and where each new token
 * goes, from the requests' lengths, without the host reading any of them.
 * Request b holds lens[b] tokens and gets new_lens[b] more (NULL: one each).
 *   table      int32 [B][max_pages], the pages of each request in order; the
 *              first ceil(lens[b] / page) are read, new ones are written
 *              behind them, and the rest is left as it was
 *   free_pages int32 [n_free]; entries from *free_head on are free. Requests
 *              take what they need from it in order.
 *   slot (int64), pos, row (int32)  [n_tokens]: slot, position and request of
 *              each new token, requests one after the other; behind the last
 *              token slot = -1, pos = 0, row = -1. 16-byte aligned.
 *   cu         int32 [B + 1]: first token of each request, and their number
 *              (at most 2^31 - 1)
 *   lens_out   int32 [B], head_out int32: lengths and list head afterwards
 *              (not lens, new_lens and free_head themselves, which every block
 *              reads)
 * A request is refused, and reported, when the pages left do not suffice
 * (requests behind it that need no page still go), when it would pass
 * max_pages, when its tokens pass n_tokens, or when its numbers are negative
 * (a negative count takes no tokens): its tokens get slot -1, its length and
 * table row stay, and it takes no page (pos is 0 where it would pass the
 * table row, or the length is negative). A page id outside [0, n_pages) gives
 * slot -1 and is reported. Limits: B <= 8192, max_pages * page < 2^31 - 64 (in
 * the attention too).
 */
swa_status swa_kv4_plan(int n_pages, int page, int B, int max_pages, const int32_t* lens,
                        const int32_t* new_lens, int32_t* table, const int32_t* free_pages, int n_free,
                        const int32_t* free_head, int n_tokens, int64_t* slot, int32_t* pos,
                        int32_t* row, int32_t* cu, int32_t* lens_out, int32_t* head_out,
                        void* workspace, size_t ws_bytes, void* stream);

/*
 * Puts new rows into the cache: k [B, T, Hkv, d] is rotated (r, NULL: not; at
 * pos int32 [B, T], NULL: position t), normed and multiplied by gk as in
 * swa_attn_fwd_ex; v gets its value embedding (ve, tok, ve_gate, or the
 * learned gate of ex, as there; ex's own rotary tables must be NULL); both
 * are quantised from fp32 into slot int64 [B, T]. Tokens with slot -1 are
 * skipped; tokens with a slot outside the cache or (with r) a position
 * outside the tables are skipped and reported; a token id outside [0, vocab)
 * is reported and adds no embedding. Two tokens with the same slot in one
 * call leave that slot's content undefined. A key whose squares pass fp32's
 * range is normed all the same.
 */
swa_status swa_kv4_append(const swa_params* p, const swa_extras* ex, const swa_kv4_cache* c,
                          const swa_rope* r, const void* k, const void* v, const float* gk,
                          const void* ve, const int32_t* tok, const float* ve_gate,
                          const int32_t* pos, const int64_t* slot, void* workspace, size_t ws_bytes,
                          void* stream);

/*
 * The keys and values of slots, as the numbers they stand for (keys rotated
 * and normed): k_out, v_out [B, T, Hkv, d] elem. Rows of slot -1, and of
 * slots outside the cache (reported), are zero.
 */
swa_status swa_kv4_read(const swa_params* p, const swa_kv4_cache* c, const int64_t* slot, void* k_out,
                        void* v_out, void* workspace, size_t ws_bytes, void* stream);

/*
 * Attention of one token per request: q [B, Hq, d] is the token at position
 * lens[b] - 1 (whose key and value are in the cache already), rotated there
 * (r, NULL: not), normed and multiplied by gq; it sees the cache's keys j with
 * lens[b] - 1 - window <= j < lens[b] (window -1: all). p->T must be 1 and
 * p->causal 1, B * Hq at most 65535; window, softmax_scale and eps as in
 * swa_attn_fwd. gq is 16-byte aligned.
 *   table    int32 [B][max_pages]; entries behind ceil(lens[b] / page) and in
 *            front of the window are not read
 *   lens     int32 [B]; 0: the request's rows of o are 0 and of lse -infinity
 *   o, lse   [B, Hq, d] elem, [B, Hq] fp32 (natural log)
 *   ex       NULL, or its wait_limit_ns
 * A length below 0 counts as 0, one above max_pages * page as that, one
 * above the rotary tables' rows as 0; keys of a page outside [0, n_pages) are
 * left out; all four are reported. Several query tokens of one request are as
 * many rows of B, with the same table row and lengths one apart.
 *
 * The workspace (256-byte aligned, passed to swa_kv4_workspace_init once
 * before its first use) holds the status word, counters, and the partial
 * results of long requests that several CTAs share (10 MB). Its size,
 * swa_kv4_workspace_size, is the same for every valid call: calls of any
 * shapes, layers and windows, and captured graphs of them, may share one as
 * long as they run one after the other (one stream, or events); calls that can
 * overlap need one each. The partial results of a request are joined in a
 * fixed order: a call gives the same bits every time.
 */
size_t swa_kv4_workspace_size(const swa_params* p, int page, int max_pages);
swa_status swa_kv4_workspace_init(void* workspace, size_t ws_bytes, void* stream);
swa_status swa_kv4_attn(const swa_params* p, const swa_extras* ex, const swa_kv4_cache* c,
                        const swa_rope* r, const void* q, const float* gq, const int32_t* table,
                        int max_pages, const int32_t* lens, void* o, float* lse, void* workspace,
                        size_t ws_bytes, void* stream);

/*
 * Several drafted tokens of a request at once (speculative decoding): a tree of
 * them, each the continuation of its parent. A step's tokens lie one request
 * behind the other, as swa_kv4_plan lays them out: those of request b are rows
 * cu[b] .. cu[b + 1] - 1 (at most max_new, 1 .. 64), their slots are the last ones
 * of its lens[b], in order. The rest of lens[b] is its context. Rows in front of
 * cu[0] and behind cu[B] are padding.
 *
 * swa_kv4_tree: what the tokens see, and where they stand, from their parents.
 *   parent  int32 [n_tokens], the index of the token's parent among its request's
 *           (in front of it), or -1: it follows the context
 *   pos     int32 [n_tokens]: the context's length and the token's depth. Both
 *           swa_kv4_append (with the plan's slots) and the attention rotate there.
 *   seen    int64 [n_tokens]: bit t set: the token sees the request's token t
 *           (itself and those above it)
 * Padding, tokens whose parent is not in front of them, those below these, and
 * the tokens of a request that is refused get seen 0 and pos 0; all but the padding
 * are reported. A request is refused when it has more than max_new tokens, or
 * more than lens[b], or when lens[b] is negative; where cu itself is not
 * plausible (negative, falling, beyond n_tokens), its rows are not touched.
 *
 * swa_kv4_tree_attn: their attention; q [n_tokens, Hq, d] is rotated at pos,
 * normed and multiplied by gq as in swa_kv4_attn, whose arguments the others are
 * (p->T must be 1; p->B counts requests). A token sees its whole context and the
 * drafted tokens of seen (bits behind the request's last token count nothing),
 * both only where their position is at least pos - window. seen and pos need not
 * come from a tree. A row of seen 0 sees nothing, not even the context: o is 0, lse
 * -infinity, as for padding. So are, and are reported, rows whose position lies
 * in front of the context's end or outside the rotary tables, and those of refused
 * requests (as above, or lens[b] > max_pages * page). Keys of a page outside
 * [0, n_pages) are left out and reported. What a token does not see changes
 * nothing of its row, a NaN even. The workspace is that of swa_kv4_attn
 * (swa_kv4_workspace_size, and what is said there of sharing one). Limit: B * Hq
 * at most 65535.
 * Rounding: in bf16 calls the probabilities count 8 bits where they multiply
 * the values (not in their sum, nor in lse; swa_kv4_attn keeps 16, so a single
 * drafted token's o is less exact than plain decoding's). With d = 128 and more than
 * 16 (token, head) rows of a kv head they count 11 bits, and the values 11 (of a
 * key's largest; values below 2^-97 lose more). Sums are fp32, joined in a fixed order.
 *
 * swa_kv4_move: the tokens of slots src[b][t] become those of dst[b][t] (int64 [p->B,
 * p->T], T <= 64), in the whole cache of a layer: the accepted path of a tree put
 * in order behind its context. All of row b are read before any is written; slots
 * that one row writes and another row reads or writes leave those undefined, as
 * does the same dst twice in a row. Pairs with a -1 are skipped; with a slot outside
 * the cache skipped and reported.
 */
swa_status swa_kv4_tree(int B, int n_tokens, int max_new, const int32_t* parent, const int32_t* cu, const int32_t* lens,
                        int32_t* pos, int64_t* seen, void* workspace, size_t ws_bytes, void* stream);
swa_status swa_kv4_tree_attn(const swa_params* p, const swa_extras* ex, const swa_kv4_cache* c, const swa_rope* r,
                             int n_tokens, int max_new, const void* q, const float* gq, const int32_t* table, int max_pages,
                             const int32_t* lens, const int32_t* cu, const int32_t* pos, const int64_t* seen, void* o,
                             float* lse, void* workspace, size_t ws_bytes, void* stream);
swa_status swa_kv4_move(const swa_params* p, const swa_kv4_cache* c, const int64_t* src, const int64_t* dst, void* workspace,
                        size_t ws_bytes, void* stream);

/*
 * The norm in front of a layer, with the residual's addition, as an operator of
 * its own (the block calls have one without gain inside):
 *   h = x + add (rounded to elem),  rstd = 1 / sqrt(mean_c(h^2) + eps),  y = gain h rstd
 * over rows of C channels (a multiple of 8, at most 65536).
 *   add    NULL: h = x
 *   gain   fp32 [C], or NULL (1)
 *   h      elem [rows, C]; NULL only where add is NULL. May be x or add.
 *   y      elem [rows, C], may be x or add; or
 *   y8, scale  y in 8 bits: e4m3 numbers [rows, C], fp32 [rows]; y ~ y8 * scale. y8 is
 *          none of x, add and h.
 *          y8 = e4m3(448 u / max|u|), scale = max|u| rstd / 448 with u = gain h,
 *          to nearest, ties to even, exactly so. A row that holds a NaN or an
 *          infinity is NaN in both; one whose entries are all 0 is 0 in both (so is one
 *          whose gains bring max|u| 2^60 below the entries' own size and fp32's end).
 *   rstd   fp32 [rows] or NULL (the backward wants it)
 * Sums are fp32; squares that leave its range are summed of the row times a
 * power of two.
 *
 * swa_rms_norm_bwd, for the loss <y, dy> + <h, dh>:
 *   dx     elem [rows, C]: gradient of x and of add; may be dy, dh or h
 *   dgain  fp32 [C] (overwritten), or NULL. It wants the workspace
 *          (swa_rms_norm_workspace_size, 256-byte aligned; nothing in it is kept or has
 *          to be set): partial sums, added in a fixed order.
 *   dh     NULL: h is not used elsewhere
 * rows == 0 clears dgain.
 */
swa_status swa_rms_norm(long long rows, int C, float eps, const void* x, const void* add, const float* gain, void* h, void* y,
                        void* y8, float* scale, float* rstd, void* stream);
size_t swa_rms_norm_workspace_size(long long rows, int C);
swa_status swa_rms_norm_bwd(long long rows, int C, const void* h, const float* rstd, const float* gain, const void* dy,
                            const void* dh, void* dx, float* dgain, void* workspace, size_t ws_bytes, void* stream);

/*
 * Projections whose weights are held in 4 bits, for serving:
 *   y[m][n] = x_scale[m] sum_k x[m][k] W[n][k] + add[m][n]
 * K a multiple of 8; N, K at most 2^24, M at most 2^31 - 256. The weights are swa_w4_size(N, K) bytes,
 * 16-byte aligned: [ceil(N / 16)][ceil(K / 64)] tiles of 544 bytes, 512 of numbers
 * and 16 steps (bf16). A number n = 0..15 stands for s (n - 8), with a step s per
 * row and 64 columns. Lane = 4 r + j (r 0..7, j 0..3) of a tile has its bytes 16
 * lane ..; their 32-bit word w has, low nibble first, for e = 0, 1, q = 0, 1, hi
 * = 0, 1 the number of row r + 8 hi, column 16 j + 4 w + 2 q + e. Step 2 r + hi is
 * that of row r + 8 hi.
 *
 * swa_w4_pack makes them of w [N][K] elem (torch.nn.Linear layout):
 *   s = bf16(max|w| / 7) (the quotient in fp32) over the group, n = floor(w / s +
 *   8.5) kept within 0..15, exactly so; n = 8 where s is below 1e-36 (it is 0 then).
 * A group that holds a NaN or an infinity is NaN. Beyond N and K numbers are 8 and
 * steps 0. swa_w4_unpack gives w as the numbers it is held as, rounded to elem.
 *
 * swa_w4_linear: x [M][K] elem, or e4m3 where x_scale (fp32 [M]) is given: the pair
 * that swa_rms_norm makes. add [M][N] or NULL; it may be y. x, add and y are 16-byte
 * aligned. Sums are fp32. Products are exact in calls of up to 32 rows and in the
 * fp32 library; in larger bf16 calls a weight s (n - 8) enters rounded to bf16 (2^-8
 * of it, so of the sum of sizes |x W|: a row's result may change with M).
 * workspace: as in swa_rope_apply (the pipeline waits of larger bf16 calls report
 * there). K is cut into parts that are added in a fixed order.
 */
size_t swa_w4_size(int N, int K);
swa_status swa_w4_pack(int N, int K, const void* w, void* w4, void* stream);
swa_status swa_w4_unpack(int N, int K, const void* w4, void* w, void* stream);
swa_status swa_w4_linear(int M, int N, int K, const void* x, const float* x_scale, const void* w4, const void* add, void* y,
                         void* workspace, size_t ws_bytes, void* stream);

/*
 * A step of serving through the whole attention block (swa_block_fwd's, whose
 * weights are held in 4 bits here): the tokens' norm, projections, append,
 * attention and residual, as one call of the calls above:
 *   h   = x + add                      [n_tokens, C] elem; add NULL: h = x
 *   xn  = swa_rms_norm of h with `gain` (NULL: none, as in swa_block_fwd)
 *   q, k, v = xn wq^T, xn wk^T, xn wv^T          (swa_w4_linear)
 *   swa_kv4_append of k, v at slot, pos, with gk, ve, tok, and the learned gate of
 *         ex (gate_w, gate_ch <= C; it reads xn's first channels; gate_x NULL)
 *   o   = swa_kv4_attn of q, one token a request (cu and seen NULL, n_tokens = p->B;
 *         its position in pos is lens[b] - 1), or swa_kv4_tree_attn (cu, seen, pos)
 *   out = h + o wo^T
 * p, c, r, gq, table, max_pages, lens, max_new are those of the attention (p->T 1).
 * ex's wait_limit_ns holds for the projections too. out is none of x and add. lens counts the tokens of the
 * call. The workspace: swa_kv4_block_workspace_size bytes for n_tokens or more,
 * passed to swa_kv4_workspace_init once; it may serve the other decode calls too.
 */
typedef struct {
  int C;                 /* model width                                        */
  const void* wq;        /* swa_w4_pack of [Hq*d][C]                            */
  const void* wk;        /* of [Hkv*d][C]                                       */
  const void* wv;        /* of [Hkv*d][C]                                       */
  const void* wo;        /* of [C][Hq*d]                                        */
} swa_kv4_weights;
size_t swa_kv4_block_workspace_size(const swa_params* p, int C, int n_tokens);
swa_status swa_kv4_block(const swa_params* p, const swa_extras* ex, const swa_kv4_cache* c, const swa_rope* r,
                         const swa_kv4_weights* w, int n_tokens, int max_new, const void* x, const void* add, const float* gain,
                         const float* gq, const float* gk, const void* ve, const int32_t* tok, const int64_t* slot,
                         const int32_t* pos, const int32_t* cu, const int64_t* seen, const int32_t* table, int max_pages,
                         const int32_t* lens, void* out, void* workspace, size_t ws_bytes, void* stream);

/*
 * Synchronises `stream`, reads the workspace status word, clears it, and
 * returns SWA_OK, SWA_ERR_TIMEOUT or SWA_ERR_DEVICE_CHECK (timeout wins).
 * After a timeout it also drops the record of a zeroed dQ accumulator (a
 * forward that gave up may not have zeroed it), so the next backward clears
 * the accumulator itself.
 */
swa_status swa_attn_check_status(void* workspace, void* stream);

/*
 * Window of layer `layer` of an `n_layer` stack under a window pattern of
 * 'S' (sliding, window T/2) and 'L' (full) characters, e.g. "SSSL": the
 * layer's character is pattern[layer % strlen(pattern)] and the last layer is
 * always full (post, model paragraph; Guide §3.4). Returns T/2 or -1; -2 on
 * invalid arguments (NULL/empty pattern, a character other than S/L, layer
 * out of [0, n_layer)).
 */
int swa_sssl_window(int layer, int n_layer, const char* pattern, int T);

/*
 * 1 if layer `layer` of an `n_layer` stack mixes value embeddings into v:
 * alternating layers, the last always included (Guide §8.2.1, has_ve); 0 if
 * not; -1 on invalid arguments.
 */
int swa_has_ve(int layer, int n_layer);

/* Static, human-readable text of a status code. */
const char* swa_strerror(swa_status s);

/* Static text naming the build: element type and kernel family. */
const char* swa_build_info(void);

#ifdef __cplusplus
}
#endif

#endif /* SWA_ATTN_H */
