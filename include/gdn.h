/*
 * gdn.h -- C ABI of the GB300 gated delta-rule library (libgdn.so).
 *
 * Four operations of the gated delta-rule recurrence, each a set of hand-written CUDA kernels for
 * sm_103a:
 *   gdn_decode_step      one-token GDN step with key sharing (Hv value heads over Hk key heads)
 *   gdn_decode_step_pooled  the same on a pooled state indexed by cache_indices
 *   gdn_decode_multi     T consecutive decode steps with the state held on chip
 *   comba_decode_step    one-token Comba step (state read with key p, written with key k)
 *   comba_forward        the Comba recurrence over T tokens with the state held on chip
 *   gdn_prefill_chunked  varlen chunkwise-WY prefill over a pooled state, gates derived in-kernel
 *   gdn_prefill_chunked_f16  the same with IEEE binary16 token arrays
 *   gdn_prefill_chunked_noalloc  the same with the library's own fixed-size workspace
 *   comba_prefill_chunked  varlen chunkwise-WY prefill of the Comba recurrence over a pooled state
 *   gdn_window_fused     fused decode window: conv + SiLU, L2 norm, gates, recurrence over ntok
 *                        tokens, gated RMSNorm, with verify / commit / partial commit
 * and the operations of the attention layers and of the drafted decoding around them:
 *   attn_paged           causal attention of each sequence's new tokens over its paged cache
 *   attn_cache_write     keys and values into the paged cache, quantised to 8 bits or as they are
 *   attn_cache_read      cached keys and values back to dense rows
 *   draft_verify         which drafted tokens the target accepts, and the token that follows them
 *
 * Conventions shared by every entry point
 *   - Every tensor argument is a DEVICE pointer to dense, contiguous, row-major memory in the layout
 *     given beside it.  "bf16" is IEEE bfloat16 (the upper half of a float32); "f16" is IEEE
 *     binary16; "f32" is IEEE float.
 *   - The caller owns every buffer, including the prefill workspace.  The library allocates no
 *     device memory and keeps no global state besides a per-device table of kernel attributes and
 *     the fixed 64 MiB device scratch array of gdn_prefill_chunked_noalloc.
 *   - Calls are asynchronous on `stream` (a cudaStream_t; NULL is the legacy default stream).
 *     Results are valid once the stream has been synchronised.
 *   - Arguments are validated on the host before anything is launched.  A rejected call returns
 *     GDN_ERR_INVALID_ARG or GDN_ERR_UNSUPPORTED and writes nothing.  A failed launch returns
 *     GDN_ERR_CUDA.  gdn_last_error() gives a human-readable reason for the last failure on the
 *     calling thread.
 *   - Sizes of zero are legal no-ops (nothing is launched; pointers may then be NULL).
 *
 * Sources (page title and section) of what each operation computes:
 *   [gated_delta.rs]  metaltile-std, src/ffai/gated_delta.rs: module doc "Recurrence per step",
 *                     "Layouts", "DISPATCH INVARIANTS".
 *   [comba spec]      KBench, specs/comba_decode_step.py: signature, spec_md, contract_md,
 *                     precision_md.
 *   [gdn_chunkwise]   pymllm, gdn_chunkwise: module doc "Algorithm (per chunk of C tokens)",
 *                     gdn_extend_chunkwise parameters.
 *   [gdn.metal]       regolith, baseline-kernels/gdn.metal: header comment and GdnArgs.
 */
#ifndef GDN_H
#define GDN_H

#include <stddef.h>
#include <stdint.h>

#ifdef __cplusplus
extern "C" {
#endif

typedef enum gdn_status {
    GDN_OK = 0,
    GDN_ERR_INVALID_ARG = 1, /* null pointer, negative size, bad layout or overlap */
    GDN_ERR_UNSUPPORTED = 2, /* a valid request outside the shapes the kernels are built for */
    GDN_ERR_CUDA = 3,        /* a CUDA runtime or driver call failed (see gdn_last_error) */
    GDN_ERR_TIMEOUT = 4      /* reserved for bounded device-side waits that gave up */
} gdn_status;

typedef enum gdn_dtype {
    GDN_BF16 = 0,
    GDN_F32 = 1,
    GDN_F16 = 2, /* IEEE binary16 */
    GDN_E4M3 = 3 /* 8-bit float: 4 exponent bits, 3 of significand, largest 448, no infinity */
} gdn_dtype;

/* A cudaStream_t, passed opaquely so that this header needs no CUDA header. */
typedef void* gdn_stream_t;

/* Bits of the device status word (the entry points that take dev_status). */
#define GDN_STATUS_BAD_CACHE_INDEX 1 /* a cache_indices entry outside [0, pool_size); a page or slot outside the cache */
#define GDN_STATUS_BAD_SEQLENS 2     /* cu_seqlens[n] < 0, decreasing, or beyond T; a length its page table cannot hold */
#define GDN_STATUS_TIMEOUT 4         /* a bounded wait for the tensor core or a copy gave up */
#define GDN_STATUS_BAD_PROBS 8       /* draft_verify: a distribution to draw from has no mass */
#define GDN_STATUS_BAD_TOKEN 16      /* draft_verify: a drafted token outside [0, V) */

/*
 * gdn_decode_step -- one GDN decode step for B sequences.  [gated_delta.rs] "Recurrence per step":
 *     S' = g S;  kv = S' k (sum over Dk);  delta = (v - kv) beta;  S_new = S' + delta (x) k;
 *     y = scale * S_new q (sum over Dk).
 * Value head hv reads key head hv / (Hv / Hk) ([gated_delta.rs] DISPATCH INVARIANTS).
 *
 *   state_in   f32  [B, Hv, Dv, Dk]  (Dk contiguous)      read
 *   state_out  f32  [B, Hv, Dv, Dk]                       written; may equal state_in (in place),
 *                                                         must not partially overlap it
 *   q, k       bf16 [B, Hk, Dk]                           k is used as given (no normalisation)
 *   v          bf16 [B, Hv, Dv]
 *   g          f32  [B, Hv]   linear forget gate (not its log)
 *   beta       bf16 [B, Hv]
 *   y          [B, Hv, Dv] of y_dtype (GDN_BF16: round to nearest even; GDN_F32)
 *   scale      readout scale (Dk^-0.5 is the usual choice; 1 reproduces the page exactly)
 * Supported: Dk in {64, 128, 256}, any Dv >= 1, Hk >= 1, Hv % Hk == 0.
 * All state arithmetic is f32; bf16 inputs are widened exactly.
 */
gdn_status gdn_decode_step(const float* state_in, float* state_out, const void* q, const void* k,
                           const void* v, const float* g, const void* beta, void* y,
                           gdn_dtype y_dtype, int B, int Hk, int Hv, int Dk, int Dv, float scale,
                           gdn_stream_t stream);

/*
 * gdn_decode_multi -- T consecutive GDN decode steps for B sequences in one call: the state stays
 * in registers across the tokens and crosses HBM once ([gated_delta.rs] mt_gated_delta_chunk:
 * the same recurrence as gdn_decode_step, wrapped in a loop over t).
 *
 *   state_in, state_out  f32 [B, Hv, Dv, Dk]   as gdn_decode_step (state_out after the T tokens)
 *   q, k       bf16 [B, T, Hk, Dk]
 *   v          bf16 [B, T, Hv, Dv]
 *   g          f32  [B, T, Hv]   linear gates
 *   beta       bf16 [B, T, Hv]
 *   y          [B, T, Hv, Dv] of y_dtype
 * Supported: as gdn_decode_step, any T >= 0 (T = 0 copies nothing and writes nothing).
 */
gdn_status gdn_decode_multi(const float* state_in, float* state_out, const void* q, const void* k,
                            const void* v, const float* g, const void* beta, void* y,
                            gdn_dtype y_dtype, int B, int T, int Hk, int Hv, int Dk, int Dv,
                            float scale, gdn_stream_t stream);

/*
 * gdn_decode_step_pooled -- the same decode step on a pooled state: batch row b reads and writes,
 * in place, slot cache_indices[b] of state_pool (the cache_indices / state_pool convention of
 * [gdn_chunkwise] gdn_extend_chunkwise, applied to one decode token).
 *
 *   state_pool     f32 [pool_size, Hv, Dv, Dk]   updated in place at the referenced slots only
 *   cache_indices  int64 [B]    distinct slots; duplicates give an undefined result
 *   q, k, v, g, beta, y, y_dtype, scale: as gdn_decode_step
 *   dev_status     device int32, zeroed by the caller; bit GDN_STATUS_BAD_CACHE_INDEX is set for a
 *                  slot outside [0, pool_size), whose batch row is then skipped (y not written)
 * Supported: as gdn_decode_step.
 */
gdn_status gdn_decode_step_pooled(float* state_pool, int pool_size, const int64_t* cache_indices,
                                  const void* q, const void* k, const void* v, const float* g,
                                  const void* beta, void* y, gdn_dtype y_dtype, int B, int Hk, int Hv,
                                  int Dk, int Dv, float scale, int32_t* dev_status,
                                  gdn_stream_t stream);

/*
 * comba_decode_step -- one Comba decode step for B sequences.  [comba spec] spec_md:
 *     S = exp(g) S;  u = beta (v - S^T p);  S_new = S + k u^T;  o = S_new^T (scale q).
 * The state is read with p and written with k.
 *
 *   state      f32  [B, H, K, V]  (V contiguous)          read
 *   state_new  f32  [B, H, K, V]                          written; may equal state (in place),
 *                                                         must not partially overlap it
 *   q, k, p    bf16 [B, H, K]
 *   v          bf16 [B, H, V]
 *   beta       bf16 [B, H]
 *   g          f32  [B, H]   log-decay (<= 0 in use; any finite value is accepted)
 *   o          [B, H, V] of o_dtype (GDN_BF16 or GDN_F32)
 *   scale      query scale ([comba spec]: K^-0.5 when the caller has no other value)
 * Supported: K in {64, 128} and V in {64, 128} (the shapes of the Comba spec's regime).
 */
gdn_status comba_decode_step(const float* state, float* state_new, const void* q, const void* k,
                             const void* v, const void* p, const void* beta, const float* g,
                             void* o, gdn_dtype o_dtype, int B, int H, int K, int V, float scale,
                             gdn_stream_t stream);

/*
 * comba_forward -- the Comba recurrence over T consecutive tokens of each of B sequences.
 * [comba spec] spec_md: the decode step is the comba-forward task's recurrence run for one token,
 * and running it T times reproduces that task.  Per (b, h) head and token t, the comba_decode_step
 * function on the state carried from token t - 1 (evaluated 8 tokens at a time in the equivalent
 * WY-regrouped form, so results match T single steps up to rounding order):
 *     S = exp(g_t) S;  u_j = beta_t (v_j - sum_i p_i S_ij);  S_ij += k_i u_j;
 *     o_t,j = sum_i (scale q_i) S_ij.
 *
 *   state      f32  [B, H, K, V]   V contiguous; the initial state, overwritten IN PLACE with the
 *                                  state after the last token (left as given when T = 0)
 *   q, k, p    bf16 [B, T, H, K]   k writes the state, p reads it
 *   v          bf16 [B, T, H, V]
 *   beta       bf16 [B, T, H]
 *   g          f32  [B, T, H]      log-decay (the gate is exp(g))
 *   o          [B, T, H, V] of o_dtype (GDN_BF16 round to nearest even, or GDN_F32); must not
 *              overlap state
 * Supported: K, V in {64, 128}.  The state is read once and written once per call; all arithmetic
 * is f32.
 */
gdn_status comba_forward(float* state, const void* q, const void* k, const void* v, const void* p,
                         const void* beta, const float* g, void* o, gdn_dtype o_dtype, int B, int T, int H,
                         int K, int V, float scale, gdn_stream_t stream);

/*
 * gdn_prefill_workspace_size -- bytes of device workspace gdn_prefill_chunked needs for these
 * sizes, with cap = ceil(T / 64) + num_seqs chunks and cap2 = floor(cap / 2):
 *   - a header padded to 1 KB: the first chunk of every sequence (8 bytes each, num_seqs + 1 of
 *     them, padded to 16 bytes), a 16-byte entry per chunk, and the schedule of the sequential
 *     kernel (16 bytes, 16 per task for num_seqs + 16 tasks, 16 per split for 8 splits, 16 per
 *     scratch chunk for cap2 of them);
 *   - one 66,560-byte record per (chunk, value head) (what a chunk contributes independently of
 *     the carried state: Tw, Tu and the output-scaled M split into bf16 high / low parts, the
 *     output-scaled q rows, and per-token scales);
 *   - the scratch of sequences split in two (a long sequence's second half runs next to its first
 *     half and is corrected afterwards): 3 x 65,536 bytes per split (at most 8) and value head,
 *     and 65,536 bytes per scratch chunk (cap2) and value head.
 * A workspace holding the header and the records but not the split scratch is also accepted;
 * then no sequence is split (same results up to rounding, slower when one sequence dominates).
 * Pure host function; returns 0 when num_seqs is 0 and for sizes gdn_prefill_chunked does not
 * support.
 */
size_t gdn_prefill_workspace_size(int num_seqs, int64_t T, int Hk, int Hv, int K, int V,
                                  int chunk_size);

/*
 * gdn_prefill_chunked -- varlen prefill of num_seqs sequences, chunkwise WY form.
 * [gdn_chunkwise] module doc, steps 1-3, and gdn_extend_chunkwise parameters.  Per sequence n
 * (tokens cu_seqlens[n] .. cu_seqlens[n+1]-1) and value head h (key head h / (Hv / Hk)):
 *     S <- state_pool[cache_indices[n], h];  per token t:
 *     log g_t = -exp(A_log[h]) softplus(a_t + dt_bias[h]) (softplus threshold 20);
 *     beta_t = sigmoid(b_t);  k^ = k / sqrt(|k|^2 + 1e-6);  q^ = scale q / sqrt(|q|^2 + 1e-6);
 *     S <- g_t S (I - beta_t k^ k^^T) + beta_t v_t k^^T;  out_t = S q^;
 *     state_pool[cache_indices[n], h] <- S.
 * computed chunk by chunk (64 tokens, chunks restart at each sequence start, the last one may be
 * short) with the WY representation; the inter-chunk carry is f32.  The chunked form gives the same
 * function for every chunk size up to rounding, so chunk_size selects nothing: the page's two
 * defaults, 64 and 128, are accepted and both run 64-token chunks.
 *
 *   q, k           bf16 [T, Hk, K]    not pre-normalised
 *   v              bf16 [T, Hv, V]
 *   a, b           bf16 [T, Hv]       raw gate inputs (before softplus / sigmoid)
 *   A_log, dt_bias f32  [Hv]
 *   state_pool     f32  [pool_size, Hv, V, K]  updated IN PLACE at the referenced slots only;
 *                                     other slots are not touched
 *   cache_indices  int64 [num_seqs]   distinct slots; duplicates give an undefined result
 *   cu_seqlens     int64 [num_seqs + 1]
 *   out            bf16 [T, Hv, V]    16-byte aligned; tokens of skipped sequences are not written
 *   workspace      device buffer of gdn_prefill_workspace_size(...) bytes (or at least its header
 *                  and records, see there; workspace_bytes tells which), 256-byte aligned,
 *                  overlapping neither out nor state_pool (NULL only when num_seqs is 0);
 *                  contents need not be initialised and are scratch after the call; calls that
 *                  share a workspace must not overlap on the GPU
 *   dev_status     device int32, zeroed by the caller; the kernels OR in GDN_STATUS_* bits for a
 *                  sequence they skip (slot out of range, malformed bounds)
 *   scale          query scale (K^-0.5 when the caller has no other value)
 * Supported: K = V = 128, chunk_size 64 or 128, Hv % Hk == 0.
 */
gdn_status gdn_prefill_chunked(const void* q, const void* k, const void* v, const void* a,
                               const void* b, const float* A_log, const float* dt_bias,
                               float* state_pool, int pool_size, const int64_t* cache_indices,
                               const int64_t* cu_seqlens, int num_seqs, int64_t T, int Hk, int Hv,
                               int K, int V, int chunk_size, float scale, void* out,
                               void* workspace, size_t workspace_bytes, int32_t* dev_status,
                               gdn_stream_t stream);

/*
 * gdn_prefill_chunked_f16 -- gdn_prefill_chunked with q, k, v, a, b and out in f16 instead of bf16
 * ([gdn_chunkwise] gdn_extend_chunkwise: q, k, v "bf16/fp16").  Same arguments, layouts, workspace
 * (gdn_prefill_workspace_size), checks and status bits; out is rounded to f16 (nearest even).
 * Inputs are widened exactly.  The products of raw k and v rows run on f16 operands; their
 * computed partners (the WY factors and the scaled Delta) are split into f16 high and low parts,
 * whose range is f16's: a key row of norm below |Delta| / 65504 (|Delta| the size of a value
 * correction) overflows them and gives non-finite outputs.  bf16 inputs have no such limit.
 */
gdn_status gdn_prefill_chunked_f16(const void* q, const void* k, const void* v, const void* a,
                                   const void* b, const float* A_log, const float* dt_bias,
                                   float* state_pool, int pool_size, const int64_t* cache_indices,
                                   const int64_t* cu_seqlens, int num_seqs, int64_t T, int Hk, int Hv,
                                   int K, int V, int chunk_size, float scale, void* out,
                                   void* workspace, size_t workspace_bytes, int32_t* dev_status,
                                   gdn_stream_t stream);

/*
 * comba_prefill_chunked -- varlen prefill of the Comba recurrence ([comba spec] spec_md: the decode
 * step is the comba-forward recurrence for one token; here over every token of num_seqs sequences),
 * computed chunk by chunk with the same WY representation as gdn_prefill_chunked ([gdn_chunkwise]
 * steps 1-3), the read key p taking k's place where the state is read (the in-chunk triangular
 * system and W) and k kept where it is written.  Per sequence n and head h:
 *     S <- state_pool[cache_indices[n], h]  (K x V, V contiguous);  per token t:
 *     S <- exp(g_t) S;  u = beta_t (v_t - S^T p_t);  S <- S + k_t u^T;  out_t = S^T (scale q_t);
 *     state_pool[cache_indices[n], h] <- S.
 *   q, k, p        bf16 [T, H, K]     used as given (the spec passes them L2-normalised)
 *   v              bf16 [T, H, V]
 *   beta           bf16 [T, H]        the value itself
 *   g              f32  [T, H]        log decay (the gate is exp(g))
 *   state_pool     f32  [pool_size, H, K, V]  updated IN PLACE at the referenced slots only
 *   out            bf16 [T, H, V]     16-byte aligned
 *   q, k, p, v     16-byte aligned; beta 2-byte, g 4-byte aligned
 * cache_indices, cu_seqlens, workspace (gdn_prefill_workspace_size(num_seqs, T, H, H, K, V,
 * chunk_size)), dev_status, chunk_size and the checks are those of gdn_prefill_chunked.
 * Supported: K = V = 128, chunk_size 64 or 128.
 */
gdn_status comba_prefill_chunked(const void* q, const void* k, const void* v, const void* p,
                                 const void* beta, const float* g, float* state_pool, int pool_size,
                                 const int64_t* cache_indices, const int64_t* cu_seqlens, int num_seqs,
                                 int64_t T, int H, int K, int V, int chunk_size, float scale, void* out,
                                 void* workspace, size_t workspace_bytes, int32_t* dev_status,
                                 gdn_stream_t stream);

/*
 * gdn_prefill_chunked_noalloc -- gdn_prefill_chunked for callers that cannot allocate device memory
 * themselves, for instance code running under a host framework whose allocator owns all device
 * memory, or in a place where calling cudaMalloc is not allowed.  No page has a counterpart: this
 * is a deployment variant, not a different computation.  Same arguments, layouts and results as
 * gdn_prefill_chunked, without the workspace arguments.
 *
 * The workspace is a 64 MiB array of the library's own device memory (a static device variable,
 * which every GPU that loads the library holds until the process exits).  The call allocates and
 * frees nothing:
 *   - Sizes whose header and records (gdn_prefill_workspace_size without the split scratch)
 *     exceed 64 MiB are rejected with GDN_ERR_UNSUPPORTED before anything runs (use
 *     gdn_prefill_chunked then).  About 1,000 (chunk, value head) records fit: for instance
 *     T = 3,000 tokens over a few sequences with Hv = 16.  Long sequences are split only when the
 *     whole gdn_prefill_workspace_size(...) fits.
 *   - The first call on a device looks up the array's device address (cudaGetSymbolAddress, with
 *     that device current) and keeps it; make that first call before any stream capture.  The
 *     address kept is the one in the device's primary context (the CUDA runtime's default), so
 *     every call must run in that context: a caller that makes its own driver-API context on the
 *     same device current (cuCtxCreate, cuCtxPushCurrent) must not use this entry point.
 *   - Every call on a device shares the one array.  Nothing in it has to start at zero: each call
 *     writes everything it reads.  Calls whose kernels overlap on the GPU (different streams, no
 *     ordering between them) race on the array and give undefined results; order them on one stream.
 */
gdn_status gdn_prefill_chunked_noalloc(const void* q, const void* k, const void* v, const void* a,
                                       const void* b, const float* A_log, const float* dt_bias,
                                       float* state_pool, int pool_size,
                                       const int64_t* cache_indices, const int64_t* cu_seqlens,
                                       int num_seqs, int64_t T, int Hk, int Hv, int K, int V,
                                       int chunk_size, float scale, void* out, int32_t* dev_status,
                                       gdn_stream_t stream);

/*
 * gdn_window_fused -- fused decode window over ntok tokens for N independent sequences.
 * [gdn.metal] header comment, per token:
 *     conv: s = h0 w0 + h1 w1 + h2 w2 + x_t w3 (history oldest first), SiLU(s); history shifts;
 *     q, k: x / sqrt(sum x^2 + eps) (the page's rsqrt(sum/128 + eps/128) / sqrt(128));
 *     gate = exp(softplus(alpha + dt) ssm_a) (softplus threshold 20);  beta = sigmoid(beta_raw);
 *     kv_j = sum_i S[i][j] k_i;  delta_j = (v_j - gate kv_j) beta;  S[i][j] = gate S[i][j] + k_i delta_j;
 *     o_j = (sum_i S[i][j] q_i) / sqrt(128);  y_j = o_j rsqrt(mean(o^2) + eps) gamma_j sigmoid(z_j).
 * Value head h reads key head h % h_k.  Head dim is 128; C = (2 h_k + h_v) * 128 channels.  The
 * window is evaluated as one WY-regrouped chunk (the same function up to rounding order); a commit
 * after token k gives bit for bit what a k-token window gives.
 *
 *   state     f32 [N, 128, h_v, 128]  (key row i, head h, value column j)  read; written in place
 *                                     only when committing
 *   hist      f32 [N, C, 3]   conv history, oldest first                    read
 *   hist_out  f32 [N, C, 3]   committed history; must not overlap hist      written only when
 *                                                                           committing
 *   qkv       f32 [N, ntok, C]  q of key head hk at hk*128, k at (h_k+hk)*128, v of head h at
 *                                (2 h_k + h)*128
 *   alpha, beta  f32 [N, ntok, h_v]
 *   z, y      f32 [N, ntok, h_v, 128]
 *   conv_w    f32 [C, 4];  dt, ssm_a  f32 [h_v];  gamma  f32 [128]   shared by all sequences
 *   commit    0: verify (nothing but y written); 1: commit state and history after the last token;
 *             0x100 | k (1 <= k <= ntok): commit after token k (y still computed for all tokens)
 *   eps       1e-6 on the page
 * Supported: 1 <= ntok <= 8, h_k >= 1, h_v >= 1.
 */
gdn_status gdn_window_fused(float* state, const float* hist, float* hist_out, const float* qkv,
                            const float* alpha, const float* beta, const float* z,
                            const float* conv_w, const float* dt, const float* ssm_a,
                            const float* gamma, float* y, int N, int h_k, int h_v, int ntok,
                            unsigned commit, float eps, gdn_stream_t stream);

/*
 * gdn_prefill_set_wait_limit -- bound every device-side wait of the prefill kernels
 * (gdn_prefill_chunked, _f16, _noalloc and comba_prefill_chunked: the chunk preparation and the
 * chunk recurrence) to `polls` polls of its mbarrier instead of the built-in limits (seconds of
 * waiting).  No page has a counterpart: this is the knob of the failure path.  A wait that runs out
 * sets GDN_STATUS_TIMEOUT in the call's dev_status and its CTA stops after one more bounded wait
 * for the copies and products it has in flight, so the call returns with that status and partial
 * results (the state of a CTA that gave up is not written back; outputs may be partly written) and
 * the device stays usable.  A limit small enough to run out on a healthy GPU (say 1) is for tests
 * of that path; a caller may also use a tighter limit than the default as a watchdog.  0 restores
 * the built-in limits.  Process-wide; it applies to calls launched after it returns.
 */
void gdn_prefill_set_wait_limit(uint32_t polls);

/*
 * The paged attention cache.  Keys and values of all sequences live in pages of page_size tokens:
 *   k_cache, v_cache   [num_pages, Hkv, page_size, D] of cache_dtype
 *   k_scale, v_scale   f32 [num_pages, Hkv, page_size]   cache_dtype GDN_E4M3 only (else NULL): a cached
 *                      element stands for value * scale of its (token, head)
 *   page_table         int64 [num_seqs, max_pages]   token t of sequence n is in page
 *                      page_table[n][t / page_size] at t % page_size; only the entries that a
 *                      sequence's length reaches are read
 * page_size is any positive number.  A page or slot outside the cache sets GDN_STATUS_BAD_CACHE_INDEX
 * and is not accessed.  dev_status is a device int32, zeroed by the caller; the kernels OR bits in.
 */

/*
 * attn_cache_write -- T tokens' keys and values into the cache.
 *   k, v       [T, Hkv, D] of dtype (GDN_BF16 or GDN_F16); token t begins k_stride (v_stride) elements
 *              after token t - 1 (a slice of a fused projection needs no copy); 16-byte aligned, strides
 *              multiples of 8
 *   slots      int64 [T]   where token t goes: page * page_size + offset; a negative slot leaves the token
 *              out; distinct (of two tokens with one slot parts of either may stay)
 *   cache_dtype  dtype (rows are copied), or GDN_E4M3: per (token, head) row the scale is the least power
 *              of two s >= 2^-100 with max |x| <= 448 s (1 for a row of zeros) and the stored value
 *              e4m3(x / s), to nearest even; but in rows at the top of dtype's range (s = 2^8 for binary16, 2^120
 *              for bf16) a value that would round to 256, and 256 s past the range, is 240.  x / s is exact, and
 *              value * s is a finite number of dtype.  Elements that are not finite are stored as NaN and do not
 *              count for the scale.
 * The sources must not overlap the cache.  Supported: D in {64, 128, 256}, Hkv <= 65535.
 */
gdn_status attn_cache_write(const void* k, const void* v, int64_t k_stride, int64_t v_stride, gdn_dtype dtype,
                            const int64_t* slots, int64_t T, void* k_cache, void* v_cache, float* k_scale,
                            float* v_scale, gdn_dtype cache_dtype, int64_t num_pages, int page_size, int Hkv,
                            int D, int32_t* dev_status, gdn_stream_t stream);

/*
 * attn_cache_read -- the cached tokens of num_seqs sequences as dense rows.
 *   cu_seqlens int64 [num_seqs + 1]   token t of sequence n is row cu_seqlens[n] + t
 *   k, v       [T, Hkv, D] of dtype, 16-byte aligned, T = cu_seqlens[num_seqs]; rows that no sequence
 *              covers, and rows whose page is outside the cache, are not written
 *   cache_dtype  dtype, or GDN_E4M3: value * scale in fp32, rounded to dtype (exact in bf16 for scales that
 *              attn_cache_write made)
 * Supported: D in {64, 128, 256}, Hkv <= 65535.
 */
gdn_status attn_cache_read(const void* k_cache, const void* v_cache, const float* k_scale, const float* v_scale,
                           gdn_dtype cache_dtype, int64_t num_pages, int page_size, const int64_t* page_table,
                           int max_pages, const int64_t* cu_seqlens, int num_seqs, int64_t T, int Hkv, int D,
                           void* k, void* v, gdn_dtype dtype, int32_t* dev_status, gdn_stream_t stream);

/*
 * attn_paged_workspace_size -- bytes of device workspace that attn_paged needs for heads of D features
 * (it depends on D alone); 0 for a D that it does not support.  Pure host function.
 */
size_t attn_paged_workspace_size(int D);

/*
 * attn_paged -- causal attention of new tokens over a paged cache that already holds their keys and
 * values.  Sequence n has L = kv_lens[n] cached tokens; its m = cu_seqlens[n+1] - cu_seqlens[n] queries
 * are the last m of them: query i stands at position L - m + i and sees keys 0 .. L - m + i.  Query head
 * h reads key head h / (Hq / Hkv):
 *     s_j = scale q.k_j;   out = sum_j e^{s_j} v_j / sum_j e^{s_j};   lse = ln sum_j e^{s_j}.
 * One token per sequence is a decode step; a few are a window of drafted tokens; m = L is a whole prompt.
 *
 *   q          [T, Hq, D] of dtype (GDN_BF16 or GDN_F16), token t q_stride elements after token t - 1;
 *              16-byte aligned, q_stride a multiple of 8
 *   kv_lens    int64 [num_seqs]
 *   cu_seqlens int64 [num_seqs + 1]
 *   max_q      the largest m, as far as the caller knows it: it chooses the kernel and changes no result
 *              beyond rounding
 *   out        [T, Hq, D] of dtype, 16-byte aligned
 *   lse        f32 [T, Hq], natural logarithm; may be NULL
 *   workspace  attn_paged_workspace_size(D) bytes, 16-byte aligned, contents need not be initialised;
 *              calls that share it must not overlap on the GPU
 * A query that sees no key (L < m - i) gets out = 0, lse = -infinity.  Memory of the cache past a
 * sequence's length is never used, whatever it holds.  Keys and values that some query of a sequence's
 * chunk sees must be finite: the products with them also run, with weight zero, for the chunk's earlier
 * queries.  Scales must be positive and finite, those of values at least 2^-100.  A sequence with malformed bounds sets
 * GDN_STATUS_BAD_SEQLENS and is skipped (its rows are not written); one with a page outside the cache sets
 * GDN_STATUS_BAD_CACHE_INDEX and its rows hold no meaningful value.
 * Products take 16-bit operands (dtype; binary16 for an 8-bit cache, which its values and the scaled
 * queries fit exactly), weights are rounded to that type for the second product; scores, sums and
 * outputs accumulate in f32.  binary16 weights (dtype GDN_F16, or an 8-bit cache, where they include the value's
 * scale) below 2^-32 of the row's largest add nothing to out; they count in lse.  Results do not depend on timing.
 * Supported: D in {64, 128, 256}, Hq % Hkv == 0, Hq / Hkv <= 128, cache_dtype dtype or GDN_E4M3,
 * max_pages * page_size < 2^31, T < 2^30; a length of more than 2^31 - 1024 is malformed.
 */
gdn_status attn_paged(const void* q, int64_t q_stride, gdn_dtype dtype, const void* k_cache, const void* v_cache,
                      const float* k_scale, const float* v_scale, gdn_dtype cache_dtype, int64_t num_pages,
                      int page_size, const int64_t* page_table, int max_pages, const int64_t* kv_lens,
                      const int64_t* cu_seqlens, int num_seqs, int64_t T, int64_t max_q, int Hq, int Hkv, int D,
                      float scale, void* out, float* lse, void* workspace, size_t workspace_bytes,
                      int32_t* dev_status, gdn_stream_t stream);

/*
 * attn_set_wait_limit -- bound every device-side wait of attn_paged's kernels to `polls` polls of its
 * barrier (to the next multiple of 16 in the kernel for many rows; at most the built-in limit) instead of
 * the built-in limit (seconds), as gdn_prefill_set_wait_limit does for the prefill: a
 * wait that runs out sets GDN_STATUS_TIMEOUT, its CTA lets the copies and products it has in flight end
 * (bounded) and stops, and the call's rows hold no meaningful value.  0 restores the built-in limit.
 * Process-wide; it applies to calls launched after it returns.
 */
void attn_set_wait_limit(uint32_t polls);

/*
 * draft_verify -- verification of drafted tokens by rejection sampling, from given random numbers.
 * Drafted token t of sequence n is accepted while u_accept * draft_p[x] < target_p[x] (x the token, rows
 * t).  At the first rejection r the next token is drawn from max(target_p[r] - draft_p[r], 0); with all T
 * accepted from target_p[T].  With P = floor(clamp(p, 0, 1) 2^36) entry by entry, Q likewise:
 *     w_i = max(P_i - Q_i, 0) (P_i where all of these are 0, or nothing was rejected);
 *     mark = floor(sum w * floor(u_sample 2^24) / 2^24);  the token is the least i with w_0 + .. + w_i > mark,
 * so results are a function of the inputs alone.  The count is what gdn_window_fused commits: a window over
 * the last sampled token and T drafts commits after its token accepted + 1 (0x100 | accepted + 1).
 *
 *   target_p   f32 [N, T + 1, V]     probabilities
 *   draft_p    f32 [N, T, V]
 *   drafts     int64 [N, T]
 *   num_drafts int64 [N] or NULL     drafts of each sequence where they are fewer than T (clamped to 0 .. T)
 *   u_accept   f32 [N, T]            uniform in [0, 1)
 *   u_sample   f32 [N]               uniform in [0, 1)
 *   accepted   int64 [N]
 *   tokens     int64 [N, T + 1]      the accepted drafts, the drawn token, then -1
 *   dev_status device int32, zeroed by the caller: GDN_STATUS_BAD_TOKEN where a draft is outside [0, V)
 *              (it counts as rejected), GDN_STATUS_BAD_PROBS where a row to draw from has no mass (token 0)
 * Supported: T >= 0, 1 <= V <= 2^20.
 */
gdn_status draft_verify(const float* target_p, const float* draft_p, const int64_t* drafts,
                        const int64_t* num_drafts, const float* u_accept, const float* u_sample, int N, int T,
                        int V, int64_t* accepted, int64_t* tokens, int32_t* dev_status, gdn_stream_t stream);

/* Static description of a status code. */
const char* gdn_status_string(gdn_status status);

/* Detail of the last failure on the calling thread ("" if none). */
const char* gdn_last_error(void);

#ifdef __cplusplus
}
#endif

#endif /* GDN_H */
