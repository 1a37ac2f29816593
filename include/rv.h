/*
 * rv.h - C ABI of the River-LLM token-level early-exit decode library
 * (librv.so, CUDA, sm_103a).
 *
 * The method: "River-LLM: Large Language Model Seamless Exit Based on KV
 * Share" (Shen, Zou).  Page summaries used as the definition:
 *   - paperlayer.ai summary, section 4 "KV-Shared Exit Layer": every exit
 *     layer is a plug-in copy of the backbone layer with the same index,
 *     4-bit weight-only quantized, addressing the backbone's KV cache.
 *   - same page, section 4 "Inference with Seamless Exit": exit layers run
 *     in series from a predefined entry layer; after an exit the remaining
 *     layers run as exit layers and the original LM head gives the logits;
 *     prefill uses one sequence-level exit, generation a token-level exit.
 *   - aitrends.kr article: s(l) = cos(h(l-1), h(l)) between the input and
 *     output of layer l; a token exits when s(l) is greater than tau; the
 *     exit layers are W4A16 copies of the backbone blocks.
 *
 * Conventions
 *   - Every call returns an int status (RV_OK or a negative RV_E* code) and
 *     records a message readable with rv_last_error() on the calling thread.
 *     No call throws, aborts the process or traps on the device.
 *   - The library owns all device memory behind the opaque rv_model handle:
 *     backbone weights, river copies, the KV cache, activations, scratch.
 *   - The caller owns every array passed in.  Pointers are HOST pointers
 *     unless the function name ends in _dev, in which case they are DEVICE
 *     pointers on the model's device and the call is asynchronous on the
 *     model's stream.
 *   - Layers are numbered 1..L.  An exit layer e in 1..L means layers 1..e
 *     ran in the backbone and e+1..L in the river; e = L means the token never
 *     left the backbone; e = 0 (forced mode only) means every layer ran in the
 *     river.
 *   - 16-bit types: act_dtype 0 = fp16, 1 = bf16.  Weights, the KV cache and
 *     every activation that enters a matrix product use it; the residual
 *     stream, accumulations, norms, softmax and s(l) are fp32.
 */
#ifndef RV_H
#define RV_H

#include <stddef.h>
#include <stdint.h>

#ifdef __cplusplus
extern "C" {
#endif

#define RV_OK 0
#define RV_EINVAL (-1)     /* bad argument (range, pointer, shape) */
#define RV_ENOMEM (-2)     /* device or pinned host allocation failed; nothing leaked */
#define RV_ECUDA (-3)      /* a CUDA runtime call failed */
#define RV_ECAPACITY (-4)  /* a row's KV cache is full (len == max_seq); nothing changed */
#define RV_ESTATE (-5)     /* call out of order, e.g. tau-rule decode before rv_quantize_river */
#define RV_ETIMEOUT (-6)   /* a bounded device wait gave up (persistent engine, tensor-core GEMM) */

/* Projection ids of a decoder layer (for rv_export_river). */
#define RV_PROJ_Q 0
#define RV_PROJ_K 1
#define RV_PROJ_V 2
#define RV_PROJ_O 3
#define RV_PROJ_GATE 4
#define RV_PROJ_UP 5
#define RV_PROJ_DOWN 6

/* What rv_debug_dump copies out (all host layouts, row-major). */
#define RV_DUMP_HIDDEN 0  /* float [L+1][B][d]: residual stream after layers 0..L of the last step */
#define RV_DUMP_S 1       /* float [L][B]: s(l) of the last step, NaN where not evaluated */
#define RV_DUMP_LOGITS 2  /* float [B][V]: logits of the last step */
#define RV_DUMP_KV 3      /* uint16 [L][2][max_batch][Hkv][max_seq][hd]: the whole cache */
#define RV_DUMP_LENS 4    /* int32 [max_batch]: cached positions per row */

typedef struct rv_model rv_model; /* opaque */

/* Decoder shape (Llama-style: RMSNorm, GQA with rotate-half RoPE, SwiGLU).
 * max_batch and max_seq size the KV cache once, at load. */
typedef struct rv_config {
  int n_layers, d_model, n_heads, n_kv_heads, head_dim, ffn, vocab;
  int tied_embed; /* 1: the LM head is the embedding matrix */
  int act_dtype;  /* 0 = fp16, 1 = bf16 */
  float rms_eps, rope_theta;
  int max_batch, max_seq;
} rv_config;

/* Last error message of the calling thread ("" if none). */
const char *rv_last_error(void);

/* Load a backbone.  weights holds 3 + 9*L host pointers to 16-bit arrays in
 * this order: embedding [V][d], final norm [d], LM head [V][d] (NULL when
 * tied_embed), then per layer: attention norm [d], W_q [H*hd][d],
 * W_k [Hkv*hd][d], W_v [Hkv*hd][d], W_o [d][H*hd], MLP norm [d],
 * W_gate [F][d], W_up [F][d], W_down [d][F].  The arrays are copied to the
 * device; the caller may free them afterwards.  stream is a cudaStream_t
 * (NULL: the library creates its own).  Allocates the one KV cache for
 * max_batch x max_seq positions, filled with the sentinel 0x7FFF (a NaN in
 * both 16-bit types).  Requires d_model, ffn and H*hd multiples of 8 and
 * head_dim in {64, 128}.  On failure nothing stays allocated. */
int rv_load_model(const rv_config *cfg, const void *const *weights, void *stream, rv_model **out);

/* Build the river: for every layer, copy the 7 projection matrices and
 * quantize them to int4 by round-to-nearest, asymmetric, per output row and
 * per group of group_size consecutive input columns, with an fp16 scale and
 * an fp16 (integer-valued) zero point; the exit layers share the backbone's
 * RMSNorm gains, RoPE and KV cache and allocate no KV memory.
 * entry_layer (1..L) is the first layer after which a token may exit by the
 * tau rule.  group_size: a multiple of 32.  Returns RV_EINVAL if a group's
 * scale overflows fp16.  May be called again (rebuilds the river). */
int rv_quantize_river(rv_model *m, int group_size, int entry_layer);

/* Copy one river matrix out in the canonical layout: q as uint32
 * [N][K/8] with element k of a row in bits 4*(k%8).. of word k/8, scales and
 * zeros as fp16 [N][ceil(K/group)].  layer in 1..L, proj an RV_PROJ_* id.
 * Any of the three pointers may be NULL. */
int rv_export_river(const rv_model *m, int layer, int proj, void *q_packed, void *scales, void *zeros);

/* Prefill rows 0..B-1 with tokens [B][T0] (row-major int32), starting each
 * row over at position 0, and return the first generated id per row.
 * Sequence-level exit: with fixed_exit_layer = -1 a row's exit layer is the
 * first l in [entry, L-1] at which s_t(l) > tau for every prompt token t
 * (else L); with fixed_exit_layer in 0..L it is that layer.  exit_layer[b]
 * receives it.  Cache slots at positions >= T0 keep their contents (use
 * rv_kv_reset first to restore the sentinel). */
int rv_prefill(rv_model *m, const int32_t *tokens, int B, int T0, float tau, int fixed_exit_layer,
               int32_t *next_ids, int32_t *exit_layer);

/* One decode step for rows 0..B-1: token b enters at position len_b, every
 * layer 1..L writes its K and V into slot (l, b, len_b) whichever path the
 * row takes, then len_b += 1.  Token-level exit: a row leaves the backbone
 * after the first layer l in [entry, L-1] with s(l) > tau and finishes in the
 * river.  forced_exit (NULL for the tau rule) gives each row's exit layer
 * 0..L instead.  next_ids[b] is the greedy id (lowest index on ties),
 * exit_layer[b] the row's exit layer.  RV_ECAPACITY if any row has
 * len_b == max_seq (nothing is changed). */
int rv_decode_step(rv_model *m, const int32_t *tokens, int B, float tau, const int32_t *forced_exit,
                   int32_t *next_ids, int32_t *exit_layer);

/* rv_decode_step with device pointers, asynchronous on the model's stream.
 * Arguments are checked on the host except token values and forced exit
 * values, which the device checks: an out-of-range value sets a device error
 * flag (reported by rv_sync_status) and is treated as token 0 / exit L. */
int rv_decode_step_dev(rv_model *m, const int32_t *d_tokens, int B, float tau, const int32_t *d_forced_exit,
                       int32_t *d_next_ids, int32_t *d_exit_layer);

/* Wait for the model's stream and report any device-side error flag. */
int rv_sync_status(rv_model *m);

/* Forget the cached positions of the given rows (NULL: all rows) and refill
 * their cache slots with the sentinel. */
int rv_kv_reset(rv_model *m, const int32_t *rows, int n_rows);

/* Keep per-step debug copies (hidden states per layer, s(l), logits) when
 * enable != 0.  Costs extra device writes; off by default. */
int rv_set_debug(rv_model *m, int enable);

/* Copy a debug buffer or the cache out (see RV_DUMP_*).  bytes must equal
 * the buffer's size for max_batch rows (hidden, s, logits use B = max_batch). */
int rv_debug_dump(rv_model *m, int what, void *dst, size_t bytes);

/* Options (rv_set_option).  RV_OPT_DECODE_ENGINE selects how a batch-1
 * decode step runs: RV_ENGINE_CHAIN (default) = a captured graph of one
 * kernel per GEMV / attention, chained by programmatic dependent launch;
 * RV_ENGINE_PERSISTENT = one cooperative launch of a persistent kernel with
 * every block resident and grid barriers between the phases of a layer.
 * Both compute the same step.  Returns RV_EINVAL for an unknown option or
 * value, RV_ESTATE if the persistent kernel cannot be made resident. */
#define RV_OPT_DECODE_ENGINE 0
#define RV_ENGINE_CHAIN 0
#define RV_ENGINE_PERSISTENT 1
/* RV_OPT_QUANTIZER selects how the next rv_quantize_river builds the river,
 * in the same packed format: RV_QUANT_RTN (default, integer fp16 zero) or
 * RV_QUANT_HQQ (the pages' quantizer, paperlayer.ai appendix A.1: the same
 * min/max scale, a float zero (stored as fp16) minimising the lp (p = 0.7)
 * norm of the error by half-quadratic splitting: beta 10, kappa 1.01, at
 * most 20 iterations, stopping when the mean absolute error stops falling;
 * deterministic, bit-identical to the oracle). */
#define RV_OPT_QUANTIZER 1
#define RV_QUANT_RTN 0
#define RV_QUANT_HQQ 1
/* RV_OPT_WAIT_LIMIT_US: the limit, in microseconds, of every bounded device
 * wait of the persistent kernel (grid barriers, weight-ring stages, route
 * hand-offs); 0 restores the default of two seconds.  A wait that runs out
 * sets an error flag; the kernel finishes its control flow without waiting,
 * lets its copies land, returns, and the step reports RV_ETIMEOUT without
 * advancing the cached positions.  A limit of a few microseconds makes
 * waits run out on purpose (a test of that path). */
#define RV_OPT_WAIT_LIMIT_US 2
/* RV_OPT_KV_CACHE: how the model keeps its K/V.  RV_KV_16BIT (default), or
 * 8 bits with one scale for each 64 positions and KV head, int8 or e4m3 (the
 * rv_kv8 cache below, block 64): about half the memory and half the bytes that
 * the decode attention reads.  Decode steps quantise their K/V as they are
 * written and attend over the 8-bit cache; a prefill attends over its own
 * 16-bit K/V and then quantises them.  A step has a kernel a layer more than on
 * the 16-bit cache, so at short contexts it is the slower one (batch 1 of the
 * 8B shape: below about 16K positions).  Setting it to another value forgets
 * every cached position (as rv_kv_reset does) and replaces the cache; the new
 * one is allocated before the old one is freed, and where that fails
 * (RV_ENOMEM) nothing changes.  The 8-bit caches run on the chain engine
 * (RV_ESTATE with the persistent one, either way round) and need rope_theta
 * above 1 or rv_set_rope's frequencies.  RV_DUMP_KV then gives the cache's
 * values rounded to act_dtype, and the sentinel at positions that are not
 * cached. */
#define RV_OPT_KV_CACHE 3
#define RV_KV_16BIT 0
#define RV_KV_INT8 1
#define RV_KV_E4M3 2
int rv_set_option(rv_model *m, int option, int value);

/* Test hook: make a device allocation of this library fail.  after >= 0:
 * the next `after` allocations (cudaMalloc) succeed and the one after them
 * fails as if the device were out of memory (once); after < 0 turns the hook
 * off.  Process-wide; returns RV_OK.  The failing call returns RV_ENOMEM and
 * frees what it had allocated. */
int rv_debug_fail_alloc(int after);

/* Kernel timing for roofline reports: launch one batch-1 GEMV kernel of the
 * decode step `iters` times back to back on the model's stream (outside the
 * step graph) and return its mean device time per launch in *ms_per_launch
 * (CUDA events) and its algorithmic HBM bytes per launch in *bytes (weights,
 * the activation vector read, the outputs written).
 * kind: RV_TIME_GATEUP (RMSNorm + gate/up + SwiGLU of `layer`), RV_TIME_O
 * (O projection + residual), RV_TIME_LMHEAD (final norm + LM head + argmax),
 * RV_TIME_ATTN (the decode attention of row 0 in `layer` at its current
 * position; bytes = the K/V it reads).  river selects the int4 copy
 * (gate/up, O).  Leaves the KV cache and the cached positions untouched;
 * the step's activation buffers are overwritten. */
#define RV_TIME_GATEUP 0
#define RV_TIME_O 1
#define RV_TIME_LMHEAD 2
#define RV_TIME_ATTN 3
int rv_time_kernel(rv_model *m, int kind, int layer, int river, int iters, float *ms_per_launch, double *bytes);

/* Launch plan of the decode attention (host arithmetic only, no device
 * work; the pages have no counterpart: the plan is how this library splits
 * the attention over a single token's K/V, the "Memory Efficiency" long
 * contexts of paperlayer.ai section 5 included).  For `batch` rows with
 * n_kv_heads KV heads each, on a GPU of n_sm SMs whose largest launchable
 * cluster is max_cluster (a power of two <= 16), the longest context being
 * `context` positions: returns 0 for the cluster plan (the splits of a
 * (row, KV head) form one thread-block cluster and merge through
 * distributed shared memory; *splits = the cluster size: the largest power
 * of two <= max_cluster with splits x n_kv_heads x batch <= 2 n_sm) when
 * each warp of a split has at most 4 tiles of 32 positions, or when the
 * rows alone fill the GPU (n_sm / (n_kv_heads x batch) < 2); else 1 for the
 * global-merge plan (*splits = min(n_sm / (n_kv_heads x batch),
 * max_splits, 128) blocks per (row, KV head), merged through global
 * memory).  The decode step keys its captured graph by this plan.
 * RV_EINVAL for a null splits, batch, n_kv_heads, n_sm or max_splits below
 * 1, a negative context, or max_cluster not a power of two in 1..16. */
int rv_decode_attention_plan(int batch, int n_kv_heads, int n_sm, int max_cluster, int max_splits, int context,
                             int *splits);

/* Greedy LM head without allocation: final RMSNorm (gain d_final_norm, eps
 * rms_eps) of the fp32 vector d_h [d_model], the LM-head GEMV against
 * d_lm_head [vocab][d_model] (16-bit, act_dtype 0 = fp16, 1 = bf16) and the
 * argmax (lowest index on ties) into d_next_id[0]; d_logits [vocab] (fp32)
 * receives the logits when not NULL.  All pointers are device pointers; the
 * call is asynchronous on `stream` (a cudaStream_t, NULL = default stream).
 * The pages have no counterpart: this entry point exists for callers that
 * must not allocate device memory (a runtime that owns the whole memory
 * budget, or code that cannot afford the implicit synchronization of
 * cudaMalloc/cudaFree).  It runs the decode step's LM-head kernel with its
 * cross-block scratch (per-block results for at most 1024 blocks, ~8 KB) in
 * an array compiled into the library, which every GPU that loads the library
 * holds until the process exits; it calls no allocator.  The first call on a
 * device looks the array's address up (cudaGetSymbolAddress), so make that
 * first call before any stream capture.  All calls share the one array:
 * calls whose executions overlap on the GPU (other streams, other threads)
 * race and must be serialized by the caller.  Returns RV_EINVAL, before
 * any GPU work, for vocab not a positive multiple of 4, d_model not a
 * positive multiple of 8, d_model above the maximum of 16384, vocab x
 * d_model above 2^32 - 1, or d_lm_head, d_final_norm or d_h not 16-byte
 * aligned (the kernel reads them with 16-byte loads). */
int rv_greedy_head_noalloc(const void *d_lm_head, const void *d_final_norm, const float *d_h, int vocab,
                           int d_model, int act_dtype, float rms_eps, int32_t *d_next_id, float *d_logits,
                           void *stream);

/* Backbone offloading (paperlayer.ai section 4, "Backbone Offloading": with
 * most tokens leaving the backbone after a few layers, only the first
 * backbone layers need to stay on the device next to the river).  Frees the
 * 16-bit matrices of backbone layers keep_layers+1..L on the device (their
 * RMSNorm gains stay: the river shares them) and caps every exit at
 * keep_layers: a row still in the backbone after layer keep_layers
 * continues in the river, in decode and in prefill.  Needs the river
 * (RV_ESTATE otherwise); keep_layers in 1..L (RV_EINVAL), not above an
 * earlier call's value (RV_ESTATE: freed layers cannot come back without
 * reloading the model); keep_layers = L changes nothing.  Afterwards forced
 * and fixed exits above keep_layers are RV_EINVAL and rv_param_bytes(m, 0)
 * counts only the resident backbone. */
int rv_offload_backbone(rv_model *m, int keep_layers);

/* ------------------------------------------------------------ operators
 * Stand-alone operators of long-context serving, on device memory that the
 * caller owns: rotary positions, an 8-bit K/V cache (written, read back) and
 * the attention that reads it.  The 8-bit model cache (RV_OPT_KV_CACHE) runs
 * the same kernels.  The pages have no counterpart: they leave the cache in
 * 16 bits and the positions unscaled; long contexts are where both cost
 * (paperlayer.ai section 5, "Memory Efficiency").
 *
 * Every pointer in these calls is a DEVICE pointer of the current device
 * unless it names a struct; the calls are asynchronous on `stream` (a
 * cudaStream_t of that device, NULL = default stream), allocate nothing,
 * keep nothing between calls and may be captured into a graph.  A captured
 * call holds the pointers and the struct values it was given; positions and
 * counts are read when it runs.  All arguments are checked on the host
 * before any launch (RV_EINVAL); positions and counts, which live on the
 * device, are checked there as each call says.
 *
 * A batch has B rows of up to T tokens.  d_pos[b] is the position of row b's
 * first token (NULL: 0), token t sits at d_pos[b] + t, and d_count[b] says
 * how many of the T tokens row b has (NULL: T for every row; values outside
 * 0..T are taken as the nearer end).  Tokens at or beyond the count are
 * neither read nor written: what their output rows held stays. */
#define RV_F16 0
#define RV_BF16 1
#define RV_F32 2

/* A tensor [B][T][heads][head_dim] of heads.  The head dimension is
 * contiguous; the strides are in elements, rows start on 16-byte boundaries
 * (data and every stride that is used), and an output's rows must not
 * overlap.  An output may be the input itself (same data and strides) where
 * a call says "in place"; any other overlap of the two is the caller's
 * mistake and not detected. */
typedef struct rv_heads {
  void *data;
  int dtype; /* RV_F16, RV_BF16 or RV_F32 */
  int heads;
  int64_t stride_b, stride_t, stride_h;
} rv_heads;

/* Rotary positions: element pair i of a head's first rotary_dim elements is
 * turned by the angle p * f(i) at position p and scaled by the attention
 * factor; the rest of the head is copied.  Pairs are (i, i + rotary_dim/2)
 * in the half layout and (2i, 2i + 1) in the interleaved one.  With
 * f0(i) = theta^(-2i/rotary_dim), frequencies for contexts longer than the
 * ones trained on:
 *   RV_ROPE_PLAIN   f = f0
 *   RV_ROPE_LINEAR  f = f0 / factor
 *   RV_ROPE_BASE    f0 with theta * factor^(r/(r-2)), r = rotary_dim (the
 *                   fastest pair keeps its frequency, the slowest is
 *                   divided by factor); rotary_dim > 2
 *   RV_ROPE_BANDS   f = k f0 + (1-k) f0/factor, k = clamp((original_max_position
 *                   f0/2pi - low_freq_factor) / (high_freq_factor -
 *                   low_freq_factor), 0, 1)
 *   RV_ROPE_RAMP    f = (1-u) f0 + u f0/factor, u = clamp((i - lo)/(hi - lo),
 *                   0, 1), lo = floor(c(beta_fast)) and hi = ceil(c(beta_slow))
 *                   clamped to [0, r-1] (hi = lo + 0.001 where they meet),
 *                   c(n) = r ln(original_max_position/(2 pi n))/(2 ln theta);
 *                   attention_factor 0 means 0.1 ln(factor) + 1 (1 if
 *                   factor <= 1) */
#define RV_ROPE_HALF 0
#define RV_ROPE_INTERLEAVED 1
#define RV_ROPE_PLAIN 0
#define RV_ROPE_LINEAR 1
#define RV_ROPE_BASE 2
#define RV_ROPE_BANDS 3
#define RV_ROPE_RAMP 4
typedef struct rv_rope_config {
  int head_dim, rotary_dim; /* multiples of 16, rotary_dim <= head_dim <= 256 */
  int layout, scaling;
  int original_max_position; /* BANDS, RAMP: > 0 */
  double theta;              /* > 1 */
  double factor;             /* > 0; every scaling but PLAIN */
  double low_freq_factor, high_freq_factor; /* BANDS: 0 < low < high */
  double beta_fast, beta_slow;              /* RAMP: fast > slow > 0 */
  double attention_factor; /* factor on the rotated part; 0: 1 (RAMP: see above) */
} rv_rope_config;

/* What rv_rope needs of a configuration, filled in by rv_rope_init (host
 * arithmetic, no device work) and kept by the caller.  turns[i] is pair i's
 * frequency in turns per position as a 64-bit binary fraction: position x
 * turns wraps exactly at whole turns, so far positions lose no precision. */
typedef struct rv_rope_plan {
  int head_dim, rotary_dim, layout;
  float attention_factor;
  uint64_t turns[128];
} rv_rope_plan;

int rv_rope_init(const rv_rope_config *cfg, rv_rope_plan *plan);

/* Rotate B x T tokens' query heads and key heads (k_in and k_out both NULL:
 * queries alone) in one launch.  q_in/q_out and k_in/k_out have the same
 * number of heads; in and out may be in place.  All four share one dtype, or
 * the inputs are RV_F32 and the outputs one 16-bit type.  inverse != 0 turns
 * the other way (and scales by the same attention factor): that is the
 * gradient of the rotation, dL/dx from dL/dy.  The arithmetic is fp32, each
 * output rounded once.  Any int32 position, negative ones included.  A token's
 * query and key heads hold at most 2^19 elements together. */
int rv_rope(const rv_rope_plan *plan, const rv_heads *q_in, const rv_heads *q_out, const rv_heads *k_in,
            const rv_heads *k_out, int B, int T, const int32_t *d_pos, const int32_t *d_count, int inverse,
            void *stream);

/* An 8-bit K/V cache of one layer, in memory the caller owns.  A block is
 * `block` consecutive positions of one row and one KV head; its K values
 * share one scale and its V values another:
 *   s = max(up8(amax / Q), 2^-100),  Q = 127 (RV_KV8_INT8), 448 (RV_KV8_E4M3),
 * amax the largest magnitude among the block's present values and up8 the
 * next number of 8 significant bits (so that x / s has no near ties: every
 * rounding is the exact one).  A code is x / s rounded to the nearest code,
 * ties to even, and stands for code * s.  A block with a NaN or an infinity
 * among its values has a NaN scale: it reads back as NaN, and so does the
 * attention of every query row that sees a position of it.
 * The scales are a function of the values alone, however they were appended:
 * the last 2 x block originals of each row and KV head stay in 16 bits in
 * the tail (slot = position mod 2 block), and an append that ends in an open
 * block quantises the block anew from originals.
 * Layouts, all contiguous, N = max_seq rounded up to a multiple of block:
 *   codes [max_batch][n_kv_heads][N][head_dim], one byte each
 *   scale [max_batch][n_kv_heads][N / block], fp32
 *   tail  [max_batch][n_kv_heads][2 block][head_dim], act_dtype
 * 16-byte aligned.  No initial contents are needed. */
#define RV_KV8_INT8 0
#define RV_KV8_E4M3 1
typedef struct rv_kv8 {
  int max_batch, n_kv_heads, head_dim, max_seq; /* <= 65535, <= 1024, 64 or 128 */
  int block;     /* 16, 32, 64 or 128 */
  int format;    /* RV_KV8_* */
  int act_dtype; /* RV_F16 or RV_BF16: the type of the originals */
  void *k_codes, *v_codes;
  float *k_scale, *v_scale;
  void *k_tail, *v_tail;
} rv_kv8;

/* Append B x T tokens' K and V (n_kv_heads heads each; act_dtype, or RV_F32
 * rounded to act_dtype first) at positions d_pos[b].. of rows 0..B-1.  The
 * positions before d_pos[b] must have been appended before.  A row may go
 * back and continue from there, what lay behind is forgotten: to any multiple
 * of `block` (0: it starts over), and elsewhere (drafted tokens refused) to at
 * most `block` positions below the highest end that the row has reached since
 * the first token of that block was last written.  Rows of count 0 are left
 * alone.  A row whose d_pos is negative
 * or at least max_seq is left alone, and tokens at max_seq and beyond are
 * dropped: either sets bit 6 (64) of *d_err (or NULL: not reported). */
int rv_kv8_append(const rv_kv8 *cache, const rv_heads *k, const rv_heads *v, int B, int T, const int32_t *d_pos,
                  const int32_t *d_count, int32_t *d_err, void *stream);

/* Read positions d_pos[b] .. d_pos[b] + count - 1 of rows 0..B-1 back into
 * k_out and v_out (either may be NULL): code * scale, exact in RV_F32, else
 * rounded to RV_F16 / RV_BF16 with the type's largest finite value as the
 * limit.  The positions must have been appended.  Positions outside
 * 0..max_seq-1 leave their output rows alone and set bit 6 of *d_err. */
int rv_kv8_read(const rv_kv8 *cache, const rv_heads *k_out, const rv_heads *v_out, int B, int T, const int32_t *d_pos,
                const int32_t *d_count, int32_t *d_err, void *stream);

/* Attention of T new tokens per row (1..16: decoding, or drafted tokens to
 * verify) over the cache.  Query token t of row b sees positions
 * 0 .. d_pos[b] + t (its own included: append first), at most max_seq of
 * them; out = softmax(scale * q k^T) v with query head h on KV head
 * h / (heads / n_kv_heads).  A token that sees nothing (d_pos[b] + t < 0)
 * gives zeros.  q is act_dtype (RV_F32: rounded to it first); out is
 * act_dtype or RV_F32.  d_lse (NULL or fp32 [B][T][heads], contiguous)
 * receives the natural log of the softmax denominators (-infinity where
 * nothing is seen), with which partial results over several caches can be
 * merged.  Scores, softmax and sums are fp32; the probabilities enter the
 * product with V as fp16 (fp16 caches and RV_F32 outputs: as two fp16 terms,
 * 22 bits).  Finite rows give finite results where |scale| x |q| stays below
 * 2^130 and |scale| x |q| x |k| below 2^119 (largest magnitudes of the row and
 * of the blocks it sees): beyond, scores pass fp32.  A query row with an
 * infinity or a NaN gives NaN where it sees anything.  How the work is cut
 * depends on the shapes and on the cache's max_seq, not on the rows' lengths:
 * a cache with room for up to 4096 positions takes 6 us for one row of 1024
 * positions and 8 KV heads, one with room for 131,072 takes 10.  workspace:
 * rv_kv8_attention_workspace bytes, 16-byte aligned, no contents needed or
 * kept (short contexts may not use it); calls that may run at the same time
 * (other streams, graphs replayed concurrently) need one each. */
int rv_kv8_attention(const rv_kv8 *cache, const rv_heads *q, const rv_heads *out, int B, int T, float scale,
                     const int32_t *d_pos, const int32_t *d_count, float *d_lse, void *workspace,
                     size_t workspace_bytes, void *stream);

/* Workspace bytes of rv_kv8_attention for up to B rows, T tokens and n_heads
 * query heads on the current device; 0 with rv_last_error() set if the
 * arguments are bad.  Enough for every smaller B and T. */
size_t rv_kv8_attention_workspace(const rv_kv8 *cache, int B, int T, int n_heads);

/* Several answers to one prompt: rows that begin with the same positions.
 *
 * Copy rows of a cache to rows of the same or another one: pair i makes row
 * d_to[i] of dst hold the first d_len[i] positions of row d_from[i] of src
 * (d_len NULL: as many as both caches have room for), so that it may be read
 * or continued there as the source could be: at d_len[i] if the source could go
 * back to that position (rv_kv8_append).  A prompt is forked to the rows that go
 * on from it, beams are put into a new order, finished rows are closed up.  All
 * pairs are copied at once, as if every source were read before any
 * destination is written: rows may change places in one call, and a source may
 * be named by any number of pairs.  Of several pairs with one destination the
 * last counts.  Codes, their blocks' scales (the open block's whole) and the
 * row's tail are copied; what the destination holds behind them stays.  Pairs
 * with a negative row are passed over; rows at or beyond the cache's max_batch
 * are too, and lengths outside 0 .. the smaller max_seq are taken as the
 * nearer end: a row or a length that is too large sets bit 6 (64) of *d_err (or
 * NULL: not reported).  Every wait inside is bounded: one that runs out sets bit
 * 4 (16), and the destinations, and in place the sources that are also
 * destinations, are then not to be used: some are written and others not.  src
 * and dst agree in n_kv_heads, head_dim, block, format and act_dtype; they are one
 * cache (all six pointers, max_batch and max_seq the same) or have no memory in
 * common (RV_EINVAL; two ranges of rows of the same arrays that do not meet are
 * two caches).  n is at most 1024. */
int rv_kv8_copy(const rv_kv8 *src, const rv_kv8 *dst, int n, const int32_t *d_from, const int32_t *d_to, const int32_t *d_len,
                int32_t *d_err, void *stream);

/* Attention of T new tokens per row over a prefix that rows share and over each
 * row's own cache: `fan` consecutive rows go with one row of `prefix` (row b
 * with row b / fan), whose K and V are read once for all of them.  Query token t
 * of row b sees the first d_prefix_len[b / fan] positions of the prefix row
 * (NULL: max_seq of them; values outside 0..max_seq are taken as the nearer end)
 * and positions 0 .. d_pos[b] + t of row b of `cache`, at most max_seq of them
 * (none where d_pos[b] + t < 0); what it sees nothing of gives zeros.  Own
 * positions count from the prefix's end: rotary positions are d_prefix_len + own
 * position.  prefix and cache agree in n_kv_heads, head_dim and act_dtype; their
 * formats, blocks and lengths may differ.  q, out, scale, d_count, d_lse and
 * precision are as in rv_kv8_attention; the product of a weight and its block's
 * V scale is rounded to fp16 (fp16 caches and RV_F32 outputs: two fp16 terms)
 * and held down to 2^-31 of the largest weight times the largest V scale of the
 * prefix.  Every wait inside is bounded: one that runs out sets bit 4 (16) of
 * *d_err (or NULL: not reported), and the outputs are then not to be used.
 * In time it is ahead of rv_kv8_attention on rows that hold copies of the prefix
 * where fan x prefix length is some 32,000 to 64,000 or more (one token, 8 KV
 * heads of 128: 64 rows from 512 to 1,024 positions on, 32 from 1,024, 16 from
 * 4,096, 8 from 8,192, 4 from 16,384 to 32,768), and behind it below: 4 rows behind 200
 * positions take 12 us, copies of them 5.5.  For two rows it is behind up to
 * 32,768 at least.  As there, the own part's plan follows the cache's max_seq, not
 * the contents: 128 rows of up to 300 own positions (8 KV heads of 64) take 56 us
 * with room for 1,024 and 73 with room for 4,096.
 * workspace: rv_kv8_attention_shared_workspace bytes, 16-byte aligned, no
 * contents needed or kept; calls that may run at the same time need one each. */
int rv_kv8_attention_shared(const rv_kv8 *prefix, const rv_kv8 *cache, const rv_heads *q, const rv_heads *out, int B, int T, int fan,
                            float scale, const int32_t *d_prefix_len, const int32_t *d_pos, const int32_t *d_count, float *d_lse,
                            int32_t *d_err, void *workspace, size_t workspace_bytes, void *stream);

/* Workspace bytes of rv_kv8_attention_shared for up to B rows, T tokens and
 * n_heads query heads on the current device; 0 with rv_last_error() set if the
 * arguments are bad.  Enough for every smaller B and T with the same fan. */
size_t rv_kv8_attention_shared_workspace(const rv_kv8 *prefix, const rv_kv8 *cache, int B, int T, int fan, int n_heads);

/* Draw each row's next token from its logits.  d_logits [B] rows of `vocab`
 * numbers of `dtype`, `stride` elements apart (any alignment that dtype has).
 * NaN and -infinity are absent: they are never drawn.  Per row (NULL: off):
 *   d_temperature  1 where NULL; 0, negative or NaN: the largest logit, the
 *                  lowest index of equal ones (d_u is not used)
 *   d_top_k        keep the first k in order of descending logits, equal ones
 *                  by index; 0 or negative: all
 *   d_top_p        of those, keep the ones before which less than top_p of
 *                  their weight lies in that order (the first at least); 1,
 *                  above or NaN: all
 *   d_min_p        keep those whose exp((x - max) / temperature), before it is
 *                  rounded to a weight, is at least min_p (1 at most: the equals
 *                  of the largest); 0, negative or NaN: all
 * The weight of logit x is w = round(2^40 exp((x - max) / temperature)), a whole
 * number: whatever weighs less than 2^-41 of the largest is never drawn, and the
 * result does not depend on the order of any sum.  d_ids[b] is the first token,
 * by index, up to which more than d_u[b] of the kept weight lies (d_u in [0, 1);
 * below or NaN: 0, above: just below 1), d_logprob[b] (or NULL) the natural log
 * of its part of the kept weight.  A row without any token gives -1 and
 * -infinity.  1 <= vocab <= 262144, B <= 65535.  Weights are computed to 2^-29 of
 * themselves; sums, cuts and the draw are exact on them. */
int rv_sample(const void *d_logits, int dtype, int64_t stride, int B, int vocab, const float *d_temperature, const int32_t *d_top_k,
              const float *d_top_p, const float *d_min_p, const float *d_u, int32_t *d_ids, float *d_logprob, void *stream);

/* Rotary frequencies of a loaded model for contexts longer than its own
 * (rv_rope_config above): cfg's head_dim must be the model's, rotary_dim the
 * whole head and the layout RV_ROPE_HALF (RV_EINVAL otherwise).  NULL: back to
 * the plain frequencies of rope_theta (RV_ESTATE where the model's cache has 8
 * bits and rope_theta is not above 1).  Forgets every cached position, whose
 * keys were turned by the old ones.  Prefill, decode steps and the persistent
 * engine all follow. */
int rv_set_rope(rv_model *m, const rv_rope_config *cfg);

/* Sizes, for callers that allocate dump buffers.  rv_param_bytes: which = 0,
 * the 16-bit parameters resident on the device (embedding, LM head, norms,
 * backbone layers 1..keep_layers); which = 1, the river (codes and
 * (scale, zero) words). */
size_t rv_kv_bytes(const rv_model *m); /* of RV_DUMP_KV */
size_t rv_kv_cache_bytes(const rv_model *m); /* of the cache on the device (differs for the 8-bit caches) */
size_t rv_param_bytes(const rv_model *m, int which);

/* Free everything the model owns. */
void rv_free_model(rv_model *m);

#ifdef __cplusplus
}
#endif
#endif
