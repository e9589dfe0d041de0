/* gdn.h -- C ABI of libgdn.so, the MI355X (gfx950) GDN linear-attention layer.
 *
 * The layer is the Gated DeltaNet ("gated delta rule") linear attention that a
 * hybrid full-attention + GDN model reaches through
 * HybridAttnBackend.forward_gdn(layer, forward_batch, mixed_qkv, a, b)
 * (pymllm.layers.attention.hybrid_backend API page, HybridAttnBackend.forward_gdn:
 * "delegate GDN computation to the GDN backend").  The recurrence, per sequence and
 * v-head, with q and k L2-normalised per head, is
 *
 *     S_t = g_t S_{t-1} (I - beta_t k_t k_t^T) + beta_t v_t k_t^T,   o_t = scale S_t q_t
 *     g_t = exp(-exp(A_log) softplus(a_t + dt_bias)),                beta_t = sigmoid(b_t)
 *
 * (Yang, Kautz & Hatamizadeh, Gated Delta Networks, ICLR 2025).  A delta-off mode
 * computes the Mamba2 SSD scan of flashinfer.mamba.ssd_combined_fwd (parameter
 * list of that page): S_t = exp(dt'_t A) S_{t-1} + dt'_t x_t B_t^T,
 * y_t = S_t C_t + D x_t, out_t = y_t silu(z_t).
 *
 * Conventions shared by every call
 *   - Every pointer in an args struct is DEVICE memory owned by the caller.  The
 *     library allocates nothing, keeps no state between calls (gdn_extend_noalloc's
 *     static scratch aside) and never synchronises: work is enqueued on `stream` (a
 *     hipStream_t; NULL = the legacy default stream) and the call returns at once.
 *   - Strides and sizes are in elements, not bytes.  Within a token, heads are
 *     contiguous: element (t, head, i) of q is q[t * q_stride + head * d_k + i].
 *   - Rows are accessed 4 elements at a time: q, k, v, z and out must be aligned
 *     to 4 elements of their dtype (8 bytes bf16, 16 bytes fp32), the pool to 16
 *     bytes, and every token stride must be a multiple of 4; otherwise GDN_E_SHAPE.
 *   - Host-side validation runs first; on any error the call returns a nonzero
 *     gdn_status, launches nothing and touches no buffer.  A failed launch returns
 *     GDN_E_HIP; gdn_last_hip_error() then gives the hipError_t (per thread).
 *   - Device-resident index data (cu_seqlens, slot, has_init) is trusted: checking
 *     it would need a host synchronisation.  Out-of-range or duplicate slots are
 *     undefined behaviour; gdn_validate_slots() is the opt-in device-side check.
 *   - A negative slot disables its sequence: no output row and no pool slot is
 *     touched (after the "negative entries disable" rule of the checkpoint
 *     arguments on the flashinfer.mamba.ssd_combined_fwd page).
 *   - Two calls that write the same pool slot must be ordered by the caller.
 */
#ifndef GDN_H
#define GDN_H

#include <stdint.h>

#ifdef __cplusplus
extern "C" {
#endif

#define GDN_ABI_VERSION 11

typedef enum gdn_status {
  GDN_OK = 0,
  GDN_E_NULL = 1,        /* a required pointer is NULL                        */
  GDN_E_SHAPE = 2,       /* inconsistent sizes / strides                      */
  GDN_E_DTYPE = 3,       /* unsupported dtype combination                     */
  GDN_E_UNSUPPORTED = 4, /* valid request this build has no kernel for        */
  GDN_E_INDEX = 5,       /* index argument out of range (host-checkable ones) */
  GDN_E_HIP = 6,         /* the HIP runtime reported an error at launch        */
  GDN_E_SCRATCH = 7      /* gdn_extend_noalloc: needs more than its static scratch */
} gdn_status;

typedef enum gdn_dtype { GDN_F32 = 0, GDN_BF16 = 1, GDN_E4M3 = 2 /* gdn_rms_norm outputs */ } gdn_dtype;

enum { GDN_MODE_GDN = 0, GDN_MODE_SSD = 1 };

/* ---------------------------------------------------------------- gdn_gate
 * a, b -> log g, beta for every (token, head).
 *   GDN mode: log_g = -exp(A[h]) * softplus(a[t,h] + dt_bias[h]); beta = sigmoid(b[t,h]).
 *             A holds A_log.  dt_softplus, dt_min, dt_max are ignored.
 *   SSD mode: dt' = a[t,h] + dt_bias[h], softplus'd when dt_softplus != 0, then
 *             clamped to [dt_min, dt_max] (inclusive, ssd_combined_fwd dt_limit);
 *             log_g = dt' * A[h] (A < 0); beta = dt'.  b must be NULL.
 * The decay is returned as log g (<= 0, fp32) because the chunked extend works with
 * in-chunk cumulative sums of it; g = exp(log_g).
 * Outputs log_g and beta are fp32 [T, H], row stride H (contiguous).  dt_bias may
 * be NULL (zero bias).  T = 0 is a no-op. */
typedef struct gdn_gate_args {
  int32_t mode;          /* GDN_MODE_GDN | GDN_MODE_SSD                 */
  int32_t in_dtype;      /* gdn_dtype of a and b                        */
  int64_t T;             /* tokens                                      */
  int32_t H;             /* heads (v-heads)                             */
  int32_t _pad0;
  const void* a;         /* [T, H], row stride a_stride (GDN: a; SSD: dt) */
  int64_t a_stride;
  const void* b;         /* [T, H], row stride b_stride (GDN only)      */
  int64_t b_stride;
  const float* A;        /* [H] fp32: GDN A_log, SSD A                  */
  const float* dt_bias;  /* [H] fp32 or NULL                            */
  int32_t dt_softplus;   /* SSD only                                    */
  float dt_min, dt_max;  /* SSD only; use 0 and +inf for "no limit"     */
  int32_t _pad1;
  float* log_g;          /* out [T, H] fp32                             */
  float* beta;           /* out [T, H] fp32                             */
} gdn_gate_args;

/* ---------------------------------------------------------------- gdn_extend
 * Packed-varlen prefill / extend.  Sequence n owns tokens [cu_seqlens[n],
 * cu_seqlens[n+1]) (cu_seqlens[0] = 0, non-decreasing, last <= T: tokens after the
 * last sequence are padding of a static buffer, e.g. under graph capture, and their
 * output rows are not written).  It starts from
 * pool[slot[n]] when has_init[n] != 0 (has_init NULL = all 1) and from zeros
 * otherwise, and writes its final state to pool[slot[n]] -- also for a
 * zero-length sequence, which writes its start state back.  slot[n] < 0 skips it.
 *
 *   q, k : [T, H_qk, d_k] (token stride q_stride / k_stride, heads contiguous)
 *   v    : [T, H_v, d_v]  (token stride v_stride)
 *   log_g, beta : [T, H_v] fp32 from gdn_gate
 *   pool : fp32 [num_slots, H_v, d_v, d_k] -- one [d_v, d_k] matrix S per
 *          (slot, v-head), d_k fastest; read and written in place
 *   out  : [T, H_v, d_v] in out_dtype (token stride out_stride), RNE rounding
 * v-head h reads qk-head h / (H_v / H_qk).  GDN mode L2-normalises q and k
 * (q / sqrt(|q|^2 + 1e-6)) and uses `scale`; SSD mode does not normalise, ignores
 * scale (1), and applies the D skip (D_per_dim ? D[h, i] : D[h]) and the silu(z)
 * gate when D / z are non-NULL (D and z in in_dtype, z laid out like v).
 * In SSD mode q = C, k = B (H_qk = ngroups, d_k = dstate), v = x (d_v = headdim),
 * log_g / beta from gdn_gate in SSD mode.
 *
 * Supported: d_k, d_v in {64, 128}; H_v % H_qk == 0; in_dtype bf16 or fp32 with
 * out_dtype bf16 or fp32.  bf16 inputs use the chunked MFMA kernels, fp32 inputs and
 * short batches (max_seqlen in 1..8) the token-recurrent kernel; gdn_extend_kernel()
 * tells which kernel a call takes and why.  max_seqlen is a host-side hint (an upper
 * bound of the longest sequence, 0 = unknown); a wrong hint changes speed, never
 * results.
 *   chunk, GDN mode : 0 (default) or 64 (the chunk-64 kernel; d_k = d_v = 128).
 *   chunk, SSD mode : 64, 128 or 0 (default: 128 when the call can take it, else 64).
 *     The chunk-128 delta-off kernel (d_k = dstate = 128, d_v = headdim = 64, the
 *     ssd_combined_fwd chunk size) needs a caller workspace: fp16 copies of B and C
 *     and the chunks' C B^T tiles (every head of a group reads them) and, to run the
 *     segments of a sequence in parallel, their states.  gdn_extend_workspace_size() gives the bytes it wants;
 *     a smaller workspace (at least the size for one segment) means fewer segments,
 *     i.e. speed only.  chunk = 128 without a usable workspace: GDN_E_NULL (none) or
 *     GDN_E_SHAPE (too small for one segment).  Its fp16 operands need |C.B|, |dt' x|
 *     and the state below 65504 (beyond that the outputs turn inf / NaN).  It reads z
 *     and writes out in 16-byte pieces: with z or out not 16-byte aligned, or a row
 *     stride of either that is not a multiple of 16 bytes, chunk 0 takes the chunk-64
 *     kernel and chunk 128 returns GDN_E_UNSUPPORTED.
 *
 * State checkpoints (optional; the checkpoint_token_indices / checkpoint_state_slots
 * / checkpoint_states arguments of the ssd_combined_fwd page, in both modes):
 *   ckpt_token  : int32 [N], one exclusive token boundary per sequence: absolute
 *                 packed-token index, or relative to the sequence's first token
 *                 when ckpt_relative != 0; negative disables the sequence's capture
 *   ckpt_slot   : int32 [N], row of ckpt_states; negative disables
 *   ckpt_states : fp32 [num_ckpt, H_v, d_v, d_k] (the pool's layout), caller-owned
 * Sequence n (slot[n] >= 0) with a boundary b inside [its first token, its end]
 * writes the state after its tokens before b to ckpt_states[ckpt_slot[n]]: its start
 * state for b at the first token, its final state for b at the end.  A boundary
 * outside the sequence captures nothing.  The three pointers are given together or
 * not at all (else GDN_E_NULL); num_ckpt >= 0.  As for the pool, ckpt_slot values
 * are device data and not range-checked: they must be < num_ckpt and distinct among
 * capturing sequences.
 *
 * Target-verify states (optional; the speculative state buffer of the target-verify
 * path in the SGLang GDN test article, chains and EAGLE trees):
 *   spec_states : fp32 [num_spec, spec_steps, H_v, d_v, d_k], caller-owned
 *   spec_slot   : int32 [N], row of spec_states; negative: the sequence records nothing
 *   spec_parent : int32 [T] or NULL; token tree: token i of a sequence (index within
 *                 it) starts from the state after its token spec_parent[t] (an earlier
 *                 index), or from the sequence's start state for -1; NULL = a chain.
 *                 A parent outside [0, i) or not below spec_steps counts as -1 (the
 *                 rule of gdn_conv1d's parent), so only recorded rows are ever read; a
 *                 sequence without a speculative row (spec_slot[n] < 0) runs as a chain
 *   keep_pool   : non-zero leaves the pool unwritten (read only)
 * Sequence n with spec_slot[n] >= 0 writes the state after its token i to
 * spec_states[spec_slot[n], i] for i < spec_steps.  With spec_parent every sequence
 * with tokens needs spec_slot[n] >= 0 and at most spec_steps tokens (device data, not
 * checked).  The pool receives the state after the sequence's last token (a chain's
 * final state) unless keep_pool.  spec_states and spec_slot go together, spec_parent
 * needs them (else GDN_E_NULL); spec_steps >= 1 with them.  Calls with target-verify
 * states run the token-recurrent kernel (verify batches are a few tokens per
 * sequence). */
typedef struct gdn_extend_args {
  int32_t mode;          /* GDN_MODE_GDN | GDN_MODE_SSD          */
  int32_t in_dtype;      /* q, k, v (and D, z)                   */
  int32_t out_dtype;
  int32_t N;             /* sequences                            */
  int64_t T;             /* packed tokens                        */
  int32_t H_qk, H_v, d_k, d_v;
  int32_t chunk;         /* 0 = default                          */
  int32_t max_seqlen;    /* hint, 0 = unknown                    */
  const void* q;
  int64_t q_stride;
  const void* k;
  int64_t k_stride;
  const void* v;
  int64_t v_stride;
  const float* log_g;
  const float* beta;
  const int32_t* cu_seqlens; /* [N+1]                            */
  const int32_t* slot;       /* [N]                              */
  const int32_t* has_init;   /* [N] or NULL                      */
  float* pool;
  int64_t num_slots;
  void* out;
  int64_t out_stride;
  float scale;
  int32_t D_per_dim;
  const void* D;         /* SSD only, or NULL                    */
  const void* z;         /* SSD only, or NULL                    */
  int64_t z_stride;
  const int32_t* ckpt_token; /* [N] or NULL (no checkpoints)     */
  const int32_t* ckpt_slot;  /* [N] or NULL                      */
  float* ckpt_states;        /* [num_ckpt, H_v, d_v, d_k] or NULL */
  int64_t num_ckpt;
  int32_t ckpt_relative;     /* boundaries relative to each sequence's first token */
  int32_t keep_pool;         /* non-zero: the pool is not written   */
  float* spec_states;        /* [num_spec, spec_steps, H_v, d_v, d_k] or NULL */
  const int32_t* spec_slot;  /* [N] or NULL                      */
  const int32_t* spec_parent;/* [T] or NULL (chain)              */
  int64_t num_spec;
  int32_t spec_steps;
  int32_t _pad_spec;
  void* workspace;           /* device scratch of the chunk-128 delta-off kernel, or NULL */
  int64_t workspace_bytes;
} gdn_extend_args;

/* Workspace bytes the chunk-128 delta-off kernel wants for a gdn_extend (gate NULL) or
 * gdn_extend_gated call with these arguments (fp16 B and C copies, the C B^T tiles of
 * every chunk, and the states of the pieces of the segments the library would run: it
 * grows with T and with N x H_v x pieces), or
 * 0 when the call would run another kernel or is invalid.  Host-side, launches nothing;
 * args->workspace / workspace_bytes are ignored.  The workspace must be 256-byte
 * aligned (else GDN_E_SHAPE) and is overwritten by the call (its contents need not be
 * initialised and mean nothing afterwards); calls in flight at once need their own. */
int64_t gdn_extend_workspace_size(const gdn_extend_args* args, const gdn_gate_args* gate);

/* Kernels of gdn_extend / gdn_extend_gated, and what keeps a call from a faster one. */
enum {
  GDN_KERNEL_RECURRENT = 1,   /* token-recurrent (decode kernel, a token at a time)   */
  GDN_KERNEL_CHUNKED = 2,     /* chunk-64 MFMA kernel                                 */
  GDN_KERNEL_SSD_CHUNKED = 3  /* chunk-128 delta-off MFMA kernel                      */
};
enum {
  GDN_WHY_FP32 = 1 << 0,        /* fp32 inputs                                          */
  GDN_WHY_SHORT = 1 << 1,       /* max_seqlen hint in 1..8 (short or verify batches)    */
  GDN_WHY_VERIFY = 1 << 2,      /* target-verify states requested                       */
  GDN_WHY_HEAD_DIMS = 1 << 3,   /* head sizes without a chunked tile plan               */
  GDN_WHY_ALIGN = 1 << 4,       /* rows not 16-byte aligned or strides not multiples of 8 */
  GDN_WHY_STRIDE = 1 << 5,      /* token strides beyond 32-bit in-chunk offsets         */
  GDN_WHY_BATCH = 1 << 6,       /* more than 65535 sequences                            */
  GDN_WHY_GATE_ALIGN = 1 << 7,  /* folded gate (GDN): a, b not 4-byte aligned, odd strides */
  GDN_WHY_WORKSPACE = 1 << 8,   /* delta-off: no workspace for the chunk-128 kernel     */
  GDN_WHY_CHUNK = 1 << 9        /* delta-off: chunk 64 requested                        */
};
/* The kernel a gdn_extend (gate NULL) or gdn_extend_gated call with these arguments
 * runs, decided on the host exactly as the call decides it; launches nothing.
 * Returns GDN_KERNEL_* (> 0), or minus the gdn_status the call would return.  *why
 * (may be NULL) receives the GDN_WHY_* bits of everything that keeps the call from
 * the fastest kernel of its mode (0 when it takes that kernel). */
int gdn_extend_kernel(const gdn_extend_args* args, const gdn_gate_args* gate, int32_t* why);

/* ---------------------------------------------------------------- gdn_decode
 * One token per sequence: token b belongs to sequence b, which always starts from
 * pool[slot[b]] and writes it back in place (state read-modify-write).  slot[b] < 0
 * marks a padding row: its output row and every pool slot stay untouched.
 * Layouts as gdn_extend with T = B; log_g / beta are [B, H_v].  GDN mode only. */
typedef struct gdn_decode_args {
  int32_t in_dtype;
  int32_t out_dtype;
  int32_t B;
  int32_t H_qk, H_v, d_k, d_v;
  int32_t _pad0;
  const void* q;
  int64_t q_stride;
  const void* k;
  int64_t k_stride;
  const void* v;
  int64_t v_stride;
  const float* log_g;
  const float* beta;
  const int32_t* slot;   /* [B] */
  float* pool;
  int64_t num_slots;
  void* out;
  int64_t out_stride;
  float scale;
  int32_t _pad1;
} gdn_decode_args;

/* `stream` is a hipStream_t passed as void* so this header needs no HIP include. */
int gdn_gate(const gdn_gate_args* args, void* stream);
int gdn_extend(const gdn_extend_args* args, void* stream);
int gdn_decode(const gdn_decode_args* args, void* stream);

/* ---------------------------------------------------------------- gated calls
 * gdn_extend / gdn_decode with the gate folded in: the kernels compute log g and
 * beta from the raw gate inputs that `gate` describes, with the arithmetic of
 * gdn_gate, instead of reading args->log_g / args->beta (ignored, may be NULL).
 * This is the same computation as gdn_gate followed by gdn_extend / gdn_decode,
 * bit for bit (one shared definition of the gate functions), with one launch and
 * the fp32 [T, H_v] round trip fewer: the shape of forward_gdn(layer,
 * forward_batch, mixed_qkv, a, b) on the hybrid_backend page, whose a, b are the
 * gate inputs.  The chunked kernel reads bf16 a, b as aligned 32-bit words: with a,
 * b not 4-byte aligned or an odd row stride the call runs the token-recurrent
 * kernel instead (speed only).
 *   gate->mode     : args->mode (extend) / GDN_MODE_GDN (decode), else
 *                    GDN_E_UNSUPPORTED
 *   gate->in_dtype : args->in_dtype, else GDN_E_DTYPE
 *   gate->T, H     : args->T (extend) or args->B (decode), and args->H_v, else
 *                    GDN_E_SHAPE
 *   gate->a, b, A, dt_bias, dt_softplus, dt_min, dt_max : as for gdn_gate
 *   gate->log_g, beta : not written, may be NULL
 * A NULL `gate` returns GDN_E_NULL; everything else is validated as for the
 * ungated call. */
int gdn_extend_gated(const gdn_extend_args* args, const gdn_gate_args* gate, void* stream);
int gdn_decode_gated(const gdn_decode_args* args, const gdn_gate_args* gate, void* stream);

/* ---------------------------------------------------------------- extend without allocation
 * For callers that cannot allocate device memory: code under HIP graph capture, tight
 * serving loops, harnesses that forbid hipMalloc.  gdn_extend_gated (gate may be NULL:
 * then gdn_extend) with the chunk-128 delta-off kernel's workspace taken from a static
 * device array of the library, GDN_NOALLOC_SCRATCH_BYTES per device, instead of from
 * args->workspace, which must be NULL with workspace_bytes 0 (else GDN_E_SHAPE).  The
 * call allocates and frees nothing.
 *   - A call whose chunk-128 kernel needs more than the array holds at one segment per
 *     sequence (about T x H_qk > 99000 token-groups: 672 bytes per token and group)
 *     returns GDN_E_SCRATCH and launches nothing; gdn_extend_gated with a workspace of
 *     gdn_extend_workspace_size bytes runs it.  A need between one segment's and gdn_extend_workspace_size's means
 *     fewer segments per sequence (speed only).
 *   - The first call on a device, with that device current, resolves the device's copy
 *     of the array (a failure returns GDN_E_HIP); the copy stays allocated until the
 *     process ends.
 *   - Every call on one device shares its copy, which keeps the last call's contents:
 *     calls that overlap in time on one device (two streams, two threads) race and give
 *     undefined results, so the caller orders them.  No part of it needs to start at
 *     zero: a call writes every byte it reads before reading it, in stream order.
 * Every other argument, result and error as gdn_extend_gated. */
#define GDN_NOALLOC_SCRATCH_BYTES (64ll << 20)
int gdn_extend_noalloc(const gdn_extend_args* args, const gdn_gate_args* gate, void* stream);

/* ---------------------------------------------------------------- short causal conv
 * The depthwise causal conv1d of width K (and SiLU) that turns the input projection
 * into mixed_qkv in front of the layer, with each sequence's last K - 1 inputs kept
 * per slot in a conv-state pool: the per-layer conv state that sits next to the
 * temporal state in the hybrid model's memory pool (SGLang GDN test-matrix article,
 * framerc.cn, memory-pool section, its conv[0] buffer).  Channel c of sequence n
 * sees the window  w = (has_init[n] ? pool[slot[n]][c] : zeros) || its own inputs,
 * and its token i (= t - cu_seqlens[n]) gives
 *     out[t, c] = act(bias[c] + sum_{j < K} weight[c, j] * w[i + j])
 *     act(y) = y * sigmoid(y) when activation != 0, y otherwise
 * (the causal convolution: weight[c, K - 1] multiplies the current input).  The
 * slot's new state is the last K - 1 entries of w: partly the old state for a
 * sequence shorter than K - 1, the start state for an empty one.
 *   x      : bf16 [T, D], token stride x_stride (the projected mixed_qkv, before the conv)
 *   weight : bf16 [D, K], a channel's K taps contiguous, oldest input first
 *   bias   : bf16 [D], or NULL for none
 *   pool   : bf16 [num_slots, D, K - 1] with slot stride pool_stride (>= D (K - 1)),
 *            a channel's entries contiguous, oldest first; read, and written in place
 *            unless keep_pool != 0 (then only read: target-verify passes whose
 *            accepted prefix the caller commits later)
 *   out    : bf16 [T, D], token stride out_stride; the fp32 result rounded to nearest even
 *   parent : int32 [T] or NULL (gdn_conv1d only): a target-verify token tree, in the
 *            convention of gdn_extend's spec_parent (token i of a sequence continues
 *            its token parent[t], an earlier index, or the state for -1); the window of
 *            a token is then the state followed by the inputs along its root path.  A
 *            parent outside [0, i) counts as -1.  Requires keep_pool != 0 (which branch
 *            to keep is the caller's choice), else GDN_E_SHAPE.
 * cu_seqlens, slot, has_init (NULL = all 1) and num_slots follow gdn_extend, with
 * the same rules for negative slots, padding tokens after the last sequence and
 * device-resident indices.
 * Supported: dtype GDN_BF16 (else GDN_E_DTYPE); K in {2, 3, 4} (else
 * GDN_E_UNSUPPORTED).  D >= 8 and a multiple of 8; x, out, weight, bias and pool
 * 16-byte aligned; x_stride, out_stride >= D and pool_stride multiples of 8
 * (else GDN_E_SHAPE).  The fp32 arithmetic: the K products and the bias summed in
 * fp32, then the activation. */
typedef struct gdn_conv_args {
  int32_t dtype;
  int32_t K;
  int32_t activation;
  int32_t N;             /* sequences (gdn_conv1d) or rows (gdn_conv1d_update) */
  int64_t T;             /* tokens; gdn_conv1d_update: must equal N */
  int64_t D;             /* channels */
  const void* x;
  int64_t x_stride;
  const void* weight;
  const void* bias;
  const int32_t* cu_seqlens; /* [N + 1]; ignored by gdn_conv1d_update */
  const int32_t* slot;       /* [N] */
  const int32_t* has_init;   /* [N] or NULL; ignored by gdn_conv1d_update */
  void* pool;
  int64_t num_slots;
  int64_t pool_stride;
  void* out;
  int64_t out_stride;
  int32_t keep_pool;
  int32_t _pad0;
  const int32_t* parent;     /* [T] or NULL; ignored by gdn_conv1d_update */
} gdn_conv_args;

/* Packed varlen (prefill / extend): two launches on `stream`, the outputs (which
 * read the old states) and then the new states.  out must not overlap x or the pool
 * (else GDN_E_SHAPE).  T = 0 launches only the state pass (empty sequences keep or
 * clear their slot as above); N = 0 launches nothing. */
int gdn_conv1d(const gdn_conv_args* args, void* stream);
/* Decode: one token per row (T = N = rows), row b always starts from pool[slot[b]]
 * (cu_seqlens, has_init ignored); slot[b] < 0 marks a padding row whose output row
 * and slot stay untouched.  One launch; out may be x itself (same rows). */
int gdn_conv1d_update(const gdn_conv_args* args, void* stream);

/* ---------------------------------------------------------------- softmax attention
 * The full-attention half of the hybrid model: the layer that RadixAttention stands for
 * on the radix_attention page (num_heads, num_kv_heads, head_dim, scaling, logit_cap,
 * sliding_window_size; forward(q, k, v, forward_batch, save_kv_cache)), with its keys
 * and values in a paged 8-bit cache.  With p_i, p_j the positions of a query and a key,
 * query head h reading kv head h / (H / H_kv):
 *     s_ij = scale q_i.k_j;  softcap > 0: s_ij = softcap tanh(s_ij / softcap);
 *     slopes: s_ij -= slopes[h] |p_i - p_j|
 *     o_i  = sum_j exp(s_ij) v_j / sum_j exp(s_ij)  over the keys j that i sees
 * and o_i = 0 for a query that sees nothing.  bf16 inputs and outputs, d in {64, 128,
 * 256}, fp32 scores, softmax statistics and sums; the softmax weights are rounded to
 * bf16 for the product with the values.  A value that a query does not see does not
 * reach it, whatever it holds (NaN and infinities too).  Positions, given or from lengths,
 * lie in [0, 2^30); softcap is at most 8192 (GDN_E_UNSUPPORTED: near 0 the tanh is off by
 * softcap 2^-22).  Calls whose launch would have 2^32 threads or more in a dimension are
 * GDN_E_UNSUPPORTED.
 *
 * The cache.  Pages of `page` rows; row r of a sequence is row r % page of the page
 * block_table[n, r / page] (row stride table_stride, table_width entries per sequence).
 * A cached value is code * scale: codes in OCP e4m3, the scale a power of two per (page,
 * kv head), the smallest with max |x| <= 448 scale over the rows written, at least
 * 2^-64.  Page ids are device data that the kernels bound: rows on a page outside
 * [0, num_pages), and rows past table_width * page, are neither read nor written (as
 * keys they are not seen). */
typedef struct gdn_kv_cache {
  void* k;               /* e4m3 [num_pages, H_kv, page, d], 16-byte aligned    */
  void* v;               /* like k                                              */
  float* k_scale;        /* fp32 [num_pages, H_kv]                              */
  float* v_scale;
  int32_t* pos;          /* int32 [num_pages, H_kv, page], 16-byte aligned: the rows' positions;
                            NULL: a row's position is its index                 */
  float* weight;         /* fp32 like pos: accumulated softmax weights; or NULL */
  int64_t num_pages;
  int32_t page;          /* 16, 32, 64 or 128                                   */
  int32_t H_kv;
  int32_t d;             /* 64, 128 or 256                                      */
  int32_t _pad0;
} gdn_kv_cache;

/* gdn_kv_store: quantise the new tokens' keys and values into the cache.  Sequence n's
 * tokens [cu_seqlens[n], cu_seqlens[n+1]) (cu_seqlens NULL: token n alone, T = N) become
 * its rows cache_len[n], cache_len[n] + 1, ...; cache_len[n] < 0 skips the sequence.  A
 * page that holds earlier rows of the sequence keeps the larger of its scale and the new
 * rows' need; where the scale grows, the earlier codes are rounded to it.  A page that
 * starts with the new rows takes their scale.  NaN and infinities are stored as NaN and
 * do not count for the scale.  (Finite values past 31 2^123, near bf16's largest, may round
 * to 2^128, which is infinite.)  Rows behind the last one written are left as they are.
 * With cache.pos the rows' positions become start[n], start[n] + 1, ... (start NULL:
 * cache_len[n]); with cache.weight their weights become 0.  k, v: bf16 [T, H_kv, d],
 * 16-byte aligned rows (strides multiples of 8).  Two sequences of one call must not
 * write the same page.  One launch. */
typedef struct gdn_kv_store_args {
  gdn_kv_cache cache;
  int32_t in_dtype;            /* GDN_BF16                         */
  int32_t N;
  int64_t T;
  const void* k;
  int64_t k_stride;
  const void* v;
  int64_t v_stride;
  const int32_t* cu_seqlens;   /* [N + 1] or NULL                  */
  const int32_t* cache_len;    /* [N] rows already held            */
  const int32_t* start;        /* [N] or NULL                      */
  const int32_t* block_table;  /* [N, table_width]                 */
  int64_t table_stride;
  int32_t table_width;
  int32_t _pad0;
} gdn_kv_store_args;
int gdn_kv_store(const gdn_kv_store_args* args, void* stream);

/* gdn_attn_extend: attention of packed new tokens (prefill, chunked prefill, verify) over
 * their own keys and values and, with a cache (cache.k non-NULL), the cache_len[n] rows
 * that sequence n already holds there (cache_len[n] < 0 skips the sequence: its output
 * rows are left as they are).  Token i of sequence n has the position start[n] + i (start
 * NULL: cache_len[n] + i, or i without a cache); a cached row has cache.pos, or its index.
 * Token i sees its own sequence's token j when all of these hold:
 *   - causal = 0, or j <= i, or j < visible[n] (prefix mask: the first visible[n] tokens
 *     are seen by every token; NULL: none);
 *   - window = 0, or |i - j| < window;
 *   - doc = NULL, or doc[i] == doc[j] and doc[i] >= 0 (document mask over the packed
 *     tokens; tokens with a negative id see nothing and are not seen).
 * and a cached row when window = 0 or the positions are less than `window` apart.  doc
 * cannot be combined with a cache (GDN_E_UNSUPPORTED).
 *   q, out : bf16 [T, H, d]; k, v : bf16 [T, H_kv, d]; heads contiguous, 16-byte aligned
 *   rows (strides multiples of 8, at most 2^22).
 * cu_seqlens follows gdn_extend: cu_seqlens[N] <= T, rows behind the last sequence are
 * not written.  out must not overlap an input.  The new tokens are not stored (gdn_kv_store).
 * T * (H / H_kv) must stay below 2^31 - 1024 (GDN_E_UNSUPPORTED).
 * With few rows the keys are split over workgroups, whose parts stand in a workspace of
 * gdn_attn_extend_workspace_size bytes (0: none), 256-byte aligned, with any contents (calls in
 * flight at once need their own); without one (NULL) they are not split.  The split goes by
 * the table's width, or by max_cached, a host hint of the longest cache_len (0 = unknown):
 * speed only, but for the workspace.  One launch, two with a split. */
typedef struct gdn_attn_extend_args {
  gdn_kv_cache cache;
  int32_t in_dtype;            /* GDN_BF16                         */
  int32_t out_dtype;           /* GDN_BF16                         */
  int32_t N;
  int32_t H, H_kv, d;
  int64_t T;
  const void* q;
  int64_t q_stride;
  const void* k;
  int64_t k_stride;
  const void* v;
  int64_t v_stride;
  void* out;
  int64_t out_stride;
  const int32_t* cu_seqlens;   /* [N + 1]                          */
  const int32_t* cache_len;    /* [N]; required with a cache, NULL without */
  const int32_t* start;        /* [N] or NULL                      */
  const int32_t* block_table;  /* [N, table_width]                 */
  int64_t table_stride;
  int32_t table_width;
  int32_t causal;
  const int32_t* visible;      /* [N] or NULL                      */
  const int32_t* doc;          /* [T] or NULL                      */
  const float* slopes;         /* [H] or NULL                      */
  int32_t window;              /* 0 = none                         */
  float scale;
  float softcap;               /* 0 = none                         */
  int32_t max_cached;          /* 0 = unknown                      */
  void* workspace;             /* or NULL                          */
  int64_t workspace_bytes;
} gdn_attn_extend_args;
int gdn_attn_extend(const gdn_attn_extend_args* args, void* stream);
/* Workspace bytes with which a gdn_attn_extend call with these arguments splits its keys,
 * or minus the gdn_status of a call that would be refused. */
int64_t gdn_attn_extend_workspace_size(const gdn_attn_extend_args* args);

/* gdn_attn_decode: one token per sequence over the rows 0 .. kv_len[n] - 1 of the cache
 * (its own row among them: gdn_kv_store first).  kv_len[n] = 0 writes zeros, kv_len[n] < 0
 * marks a padding row: its output row is left as it is.  The query's position is q_pos[n]
 * (NULL: kv_len[n] - 1); with a window only rows closer than it are seen.  accumulate != 0
 * adds to cache.weight of every row of the sequence the sum of the softmax weights that
 * the kv head's H / H_kv query heads give it; sequences of one call must then not share
 * pages.  N is at most 65535.  max_kvlen is a host hint of the longest kv_len (0 = unknown): speed only.
 * With cache.pos a window is looked up row by row: all kv_len[n] rows are read.
 * The rows are split over workgroups, whose partial results a second launch joins; they
 * stand in a workspace of gdn_attn_decode_workspace_size bytes (0: none needed), 256-byte
 * aligned, with any contents; calls in flight at once need their own.  accumulate takes 4
 * bytes of it per query head and row of the table, whatever max_kvlen says. */
typedef struct gdn_attn_decode_args {
  gdn_kv_cache cache;
  int32_t in_dtype;            /* GDN_BF16                         */
  int32_t out_dtype;           /* GDN_BF16                         */
  int32_t N;
  int32_t H;
  const void* q;               /* bf16 [N, H, d]                   */
  int64_t q_stride;
  void* out;                   /* bf16 [N, H, d]                   */
  int64_t out_stride;
  const int32_t* kv_len;       /* [N]                              */
  const int32_t* q_pos;        /* [N] or NULL                      */
  const int32_t* block_table;  /* [N, table_width]                 */
  int64_t table_stride;
  int32_t table_width;
  int32_t max_kvlen;
  const float* slopes;         /* [H] or NULL                      */
  int32_t window;              /* 0 = none                         */
  float scale;
  float softcap;               /* 0 = none                         */
  int32_t accumulate;
  void* workspace;
  int64_t workspace_bytes;
} gdn_attn_decode_args;
int gdn_attn_decode(const gdn_attn_decode_args* args, void* stream);
/* Workspace bytes of a gdn_attn_decode call with these arguments, or minus the gdn_status
 * it would return (the workspace fields are ignored).  Host-side, launches nothing. */
int64_t gdn_attn_decode_workspace_size(const gdn_attn_decode_args* args);

/* gdn_kv_evict: cut every sequence to at most `budget` rows per kv head, in place.  Of a
 * sequence of kv_len[n] > budget rows, each kv head keeps the rows with pos > (its largest
 * pos) - recent, then those of largest weight; ties go to the lowest row, a NaN weight
 * ranks below all others, and never more than `budget` rows are kept.  (Weights come from
 * gdn_attn_decode alone: rows that no decode step has attended to yet are ties.)  The kept rows at
 * or past `budget` move, in order, into the dropped rows before it, in order, with their
 * pos and weight; the others stay.  (Attention does not depend on the order of rows, only
 * on their pos.)  The scale of a page that receives rows becomes the largest of its own
 * and those of the rows' pages, and its rows before `budget` are rounded to it.
 * new_len[n] = min(kv_len[n], budget) (may be kv_len itself; kv_len[n] < 0 is copied).
 * Rows at or past new_len mean nothing afterwards.  The cache needs pos and weight.
 * A sequence with an id out of range among its pages' first kv_len[n] rows is left as it
 * is, with new_len[n] = kv_len[n].  Sequences must not share pages.  0 <= recent <= budget,
 * budget >= 1 (a budget past the table's rows counts as those), N at most 65535, fewer
 * than 2^31 rows (num_pages * page) in the cache (GDN_E_UNSUPPORTED).  Two launches;
 * workspace as for gdn_attn_decode. */
typedef struct gdn_kv_evict_args {
  gdn_kv_cache cache;
  int32_t N;
  int32_t budget;
  int32_t recent;
  int32_t table_width;
  const int32_t* kv_len;       /* [N]                              */
  int32_t* new_len;            /* [N]                              */
  const int32_t* block_table;  /* [N, table_width]                 */
  int64_t table_stride;
  void* workspace;
  int64_t workspace_bytes;
} gdn_kv_evict_args;
int gdn_kv_evict(const gdn_kv_evict_args* args, void* stream);
int64_t gdn_kv_evict_workspace_size(const gdn_kv_evict_args* args);

/* ---------------------------------------------------------------- selective scan
 * The state space scan whose decay is a matrix (one per channel and state; the delta-off
 * mode above has one decay per head).  Channel c, of group g = c / (D / G), has a state h
 * of `states` values; token by token
 *     delta = dt[t, c] + dt_bias[c], softplus'd when dt_softplus != 0
 *     h[i]  = exp(delta A[c, i]) h[i] + delta x[t, c] B[t, g, i]
 *     y     = sum_i C[t, g, i] h[i] + D_skip[c] x[t, c]
 *     out[t, c] = z ? y z[t, c] sigmoid(z[t, c]) : y
 * in fp32, rounded once (nearest even) to out_dtype.
 *   x, dt, z, out : [T, D]; B, C : [T, G, states], groups contiguous; token strides of
 *                   at least a row; aligned to their element.  x, dt, B, C, z: in_dtype
 *   A             : fp32 [D, states], 16-byte aligned (the exponent's factor itself, negative
 *                   in such layers, not its logarithm)
 *   D_skip, dt_bias : fp32 [D] or NULL (zero)
 *   pool          : fp32 [num_slots, D, states], 16-byte aligned, read and written in place
 * Supported: states in {8, 16, 32, 64, 128} (else GDN_E_UNSUPPORTED), D % G == 0, in_dtype
 * and out_dtype bf16 or fp32.  out must not overlap x, dt, B, C, z or the pool (address
 * ranges, else GDN_E_SHAPE).  D is at most 2^24; calls whose launch would have 2^32 threads
 * or more (512 for each 64 channels of a group, sequence and segment; segments are left out
 * first) are GDN_E_UNSUPPORTED.
 *
 * gdn_selective_scan: packed prompts.  cu_seqlens, slot, has_init (NULL = all 1), padding
 * tokens, skipped and empty sequences as gdn_extend; keep_pool != 0 leaves the pool as it
 * is.  max_seqlen is a host hint (an upper bound of the longest sequence, 0 = unknown): it
 * changes the split over workgroups, never what is computed: long sequences in few
 * workgroups are cut into segments, whose states a first launch prepares in a workspace of
 * gdn_selective_scan_workspace_size bytes (0: no segments), 256-byte aligned, with any
 * contents (calls in flight at once need their own); without one (NULL) there are none.
 * A segment's start state is folded from those before it, which rounds differently (and
 * makes an infinite state NaN where the factors' product leaves fp32's range).  No
 * sequence of GDN_SELECTIVE_UNCUT tokens or fewer is cut (T up to it: no workspace).
 * gdn_selective_update: one token per row (T = N), row b continues pool[slot[b]], negative
 * slots as gdn_decode; cu_seqlens, has_init, max_seqlen, keep_pool, workspace ignored. */
#define GDN_SELECTIVE_UNCUT 112
typedef struct gdn_selective_args {
  int32_t in_dtype;
  int32_t out_dtype;
  int32_t N;             /* sequences (scan) or rows (update)    */
  int32_t G;
  int64_t T;
  int64_t D;
  int32_t states;
  int32_t dt_softplus;
  const void* x;
  int64_t x_stride;
  const void* dt;
  int64_t dt_stride;
  const void* B;
  int64_t B_stride;
  const void* C;
  int64_t C_stride;
  const void* z;             /* or NULL                          */
  int64_t z_stride;
  const float* A;
  const float* D_skip;       /* [D] or NULL                      */
  const float* dt_bias;      /* [D] or NULL                      */
  const int32_t* cu_seqlens; /* [N + 1]                          */
  const int32_t* slot;       /* [N]                              */
  const int32_t* has_init;   /* [N] or NULL                      */
  float* pool;
  int64_t num_slots;
  void* out;
  int64_t out_stride;
  int32_t max_seqlen;
  int32_t keep_pool;
  void* workspace;
  int64_t workspace_bytes;
} gdn_selective_args;
int gdn_selective_scan(const gdn_selective_args* args, void* stream);
/* Workspace bytes with which a gdn_selective_scan call with these arguments cuts its
 * sequences, or minus the gdn_status of a call that would be refused. */
int64_t gdn_selective_scan_workspace_size(const gdn_selective_args* args);
int gdn_selective_update(const gdn_selective_args* args, void* stream);

/* ---------------------------------------------------------------- root-mean-square norm
 * The norm in front of a layer (with the residual's addition) and behind a linear-attention
 * layer (per head, gated), with an output that the next matrix product takes in 8 bits.
 * A token's row is H parts of d values, each normalised by itself:
 *     u = x;  residual: u = x + residual, and residual becomes u (rounded to its type);
 *     gate and gate_first: u = x g sigmoid(g)
 *     y = u / sqrt(mean(u^2) + eps) (weight + offset);  gate and not gate_first: y g sigmoid(g)
 * in fp32 (whose range the sum of u^2 must not leave), from the sum x + residual before its
 * rounding.  weight [d] is shared by the H parts (NULL: y
 * without it and offset).  out: bf16 or fp32, or e4m3 codes with y = code * scale:
 * scale[t, k] belongs to the k-th `group` values of the token's H d (the last group may be
 * shorter; group 0: the whole row) and is max |y| / 448, at least 2^-64; a code is the fp32
 * quotient y / scale rounded to nearest even.  Values that are not finite do not count for the scale, and are
 * stored as NaN.
 *   x, gate : in_dtype [T, H, d]; residual : bf16 or fp32 [T, H, d]; out [T, H, d]; a row's
 *   H d values contiguous, token strides of at least H d; aligned to their element
 *   scale : fp32 [T, ceil(H d / group)], contiguous (e4m3 only, else ignored)
 * Supported: bf16 or fp32 x, weight and residual; group 0, 64 or 128 (else
 * GDN_E_UNSUPPORTED); H at most 8192, H d at most 2^20; T below 2^24 (2^22 where H d is
 * 8193 to 32768 and d at least 8, or H 1: a launch has fewer than 2^32 threads) and not both a
 * gate and a residual (else GDN_E_UNSUPPORTED).
 * out, scale and residual must not overlap each other or an input (address ranges, else
 * GDN_E_SHAPE).  One launch. */
typedef struct gdn_rms_norm_args {
  int32_t in_dtype;
  int32_t out_dtype;         /* GDN_F32, GDN_BF16 or GDN_E4M3    */
  int32_t weight_dtype;
  int32_t residual_dtype;
  int64_t T;
  int32_t H, d;
  const void* x;
  int64_t x_stride;
  const void* gate;          /* or NULL                          */
  int64_t gate_stride;
  void* residual;            /* or NULL                          */
  int64_t residual_stride;
  const void* weight;        /* [d] or NULL                      */
  void* out;
  int64_t out_stride;
  float* scale;              /* e4m3 only                        */
  float eps, offset;
  int32_t gate_first;
  int32_t group;
} gdn_rms_norm_args;
int gdn_rms_norm(const gdn_rms_norm_args* args, void* stream);

/* ---------------------------------------------------------------- pages of a step
 * The lengths, block-table entries and slot maps that a step's other calls read, formed on
 * the GPU from the requests' lengths: a program whose lengths live there (sampled ends,
 * accepted drafts, replayed graphs) needs no copy to the host.  The free pages are a
 * stack in device memory:
 *   pool : int32 [2 + capacity]: the number of free pages, 0 (the library's own), and the
 *          stack, whose top is pool[1 + pool[0]]
 * (With `page` larger than any sequence the same calls hand out state slots, one each.)
 *
 * gdn_plan_pages: request n holds held[n] rows and brings new_len[n] tokens.  It takes the
 * pages ceil(held / page) .. ceil((held + new) / page) - 1 of its row of block_table from
 * the top of the stack, requests and pages in order.  A request is served when
 *   - held[n] >= 0 and new_len[n] >= 0 (otherwise it is a padding row without tokens),
 *   - its table has room for held + new rows, fewer than 2^31 (otherwise it takes no page), and
 *   - the pages and the tokens up to its end fit into the stack and into T (so that from the
 *     first request that does not fit on none is served).
 * Outputs, all written whole:
 *   cu_seqlens [N + 1] : tokens before each request, served or not, at most T (so that a layer's
 *     slot of a request with a negative cache_len has to be negative too: its tokens may be cut)
 *   cache_len [N]      : held[n], or -1 where the request is not served
 *   kv_len [N]         : held[n] + new_len[n], or -1
 *   slots, positions, seq [T] : of a served request's i-th token, with row r = held + i:
 *     page id * page + r % page (-1 where the table holds a negative id), start[n] + i
 *     (start NULL: r), and n; -1 for every other token.  Each may be NULL.
 * Entries of block_table that no new page takes are left as they are.  Page ids are handed
 * out as they stand on the stack; a number of free pages outside [0, capacity] counts as the
 * nearer end.  N at most 65535, 1 <= page <= 2^30, T below 2^31.
 *
 * gdn_release_pages: request n keeps its first keep[n] rows of held[n]: the pages
 * ceil(keep / page) .. ceil(held / page) - 1 of its table go back on the stack, requests and
 * pages in order, as far as `capacity` goes; keep[n] < 0 or held[n] <= keep[n]: none.  Negative
 * entries are no pages and are passed over.  Table entries are left as they are.
 *
 * Every output must be apart from every input and output (address ranges, else
 * GDN_E_SHAPE), but for block_table and pool, which are both.  Calls on one pool are
 * ordered by the caller.  One launch each. */
typedef struct gdn_plan_pages_args {
  int32_t* pool;
  int64_t capacity;
  int32_t N;
  int32_t page;
  int64_t T;
  const int32_t* held;       /* [N]                              */
  const int32_t* new_len;    /* [N]                              */
  const int32_t* start;      /* [N] or NULL                      */
  int32_t* block_table;      /* [N, table_width]                 */
  int64_t table_stride;
  int32_t table_width;
  int32_t _pad0;
  int32_t* cu_seqlens;       /* [N + 1]                          */
  int32_t* cache_len;        /* [N]                              */
  int32_t* kv_len;           /* [N]                              */
  int64_t* slots;            /* [T] or NULL                      */
  int32_t* positions;        /* [T] or NULL                      */
  int32_t* seq;              /* [T] or NULL                      */
} gdn_plan_pages_args;
int gdn_plan_pages(const gdn_plan_pages_args* args, void* stream);

typedef struct gdn_release_pages_args {
  int32_t* pool;
  int64_t capacity;
  int32_t N;
  int32_t page;
  const int32_t* keep;       /* [N]                              */
  const int32_t* held;       /* [N]                              */
  const int32_t* block_table;
  int64_t table_stride;
  int32_t table_width;
  int32_t _pad0;
} gdn_release_pages_args;
int gdn_release_pages(const gdn_release_pages_args* args, void* stream);

/* Device-side check of slot[0..n): *flag (device int32) receives 0 when every
 * non-negative slot is < num_slots and no non-negative slot repeats, 1 when one
 * is out of range, 2 when one repeats (3 when both).  Negative slots are padding
 * and may repeat.  Asynchronous like the others; O(n^2) comparisons. */
int gdn_validate_slots(const int32_t* slot, int32_t n, int64_t num_slots, int32_t* flag,
                       void* stream);

/* Measurement helpers, not part of the layer: they give the achievable peaks of the
 * running GPU that the layer's kernels are reported against, beside the published ones.
 *
 * gdn_probe_copy: copies `bytes` bytes from src to dst (device pointers, 16-byte
 * aligned, bytes a positive multiple of 16; dst either equal to src -- in place, every
 * element read and rewritten -- or not overlapping it) with a streaming kernel; the
 * caller times it.  HBM traffic: 2 x bytes.
 * gdn_probe_mfma: `blocks` workgroups of four waves (1 <= blocks <= 65536), each wave
 * four chains of `iters` (1 <= iters <= 1 << 20) dependent 32x32x16 bf16 MFMAs with
 * fp32 accumulation: blocks x 4 x 4 x iters x 32768 flop.  out (device, blocks x 256
 * floats, caller-owned) receives one finite sum per thread.
 * Both are asynchronous on `stream`; GDN_E_NULL / GDN_E_SHAPE on bad arguments. */
int gdn_probe_copy(const void* src, void* dst, int64_t bytes, void* stream);
int gdn_probe_mfma(float* out, int32_t blocks, int32_t iters, void* stream);

const char* gdn_status_str(int status);
int gdn_last_hip_error(void);
int gdn_abi_version(void);

#ifdef __cplusplus
}
#endif

#endif /* GDN_H */
