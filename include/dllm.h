/*
 * dllm.h - C ABI of the GB300 (sm_103a) block-cached, confidence-threshold
 * masked-diffusion decoder.
 *
 * The method (Fast-dLLM, as described in the zhongzhuzhou.org reading notes,
 * sections 3-6, and the dian8dian summary): the answer of length gen_len is
 * split into blocks of B positions decoded left to right (Algorithm 1).  While
 * the current block still holds MASK, one denoise step runs a bidirectional
 * transformer forward over the recomputed rows only - the current block
 * (DualCache), the block and the suffix (PrefixCache) or every position (no
 * cache) - reading cached K/V for the other positions; it takes, for every
 * masked position of the block, the largest softmax probability c_i and the
 * argmax token y_i over the vocabulary, and commits every position with
 * c_i >= tau, or only the single most confident one if none qualifies
 * (Algorithm 2).  A committed token is never changed again.  At each block
 * boundary a full-sequence forward rewrites every cached K/V in place.
 *
 * Conventions
 *  - Every call returns a dllm_status (dllm_denoise_step returns a count, or a
 *    negative status).  On failure dllm_last_error() holds a message (per
 *    thread) and no state has changed unless the text says otherwise.
 *  - Host pointers are owned by the caller and only read/written during the
 *    call.  Device memory of models and states is owned by the library and
 *    freed by dllm_free_model / dllm_free_state.
 *  - A dllm_state is used by one host thread at a time.  Calls are
 *    synchronous with respect to the host outputs they return.
 *  - Token ids are int32 in [0, vocab); the MASK id is `vocab`.
 *  - The dllm_op_* calls take device pointers, run on the given CUDA stream
 *    (NULL = legacy default stream) and return after the launch (asynchronous).
 */
#ifndef DLLM_H
#define DLLM_H

#include <stdint.h>

#ifdef __cplusplus
extern "C" {
#endif

typedef enum dllm_status {
    DLLM_OK = 0,
    DLLM_EINVAL = 1,    /* bad argument; nothing was changed */
    DLLM_ENOMEM = 2,    /* device or host allocation failed */
    DLLM_ECUDA = 3,     /* a CUDA runtime/driver call failed */
    DLLM_EIO = 4,       /* weight file missing, short or malformed */
    DLLM_ESTATE = 5,    /* a step committed nothing while MASK remained, or the
                           call does not fit the state (e.g. wrong block) */
    DLLM_ETIMEOUT = 6,  /* a kernel gave up a bounded wait; outputs are invalid */
    DLLM_ECANCELLED = 7 /* dllm_run stopped because its run hook returned nonzero */
} dllm_status;

typedef enum dllm_cache_mode {
    DLLM_CACHE_NONE = 0,    /* every step recomputes all T positions */
    DLLM_CACHE_PREFIX = 1,  /* recompute the current block and the suffix */
    DLLM_CACHE_DUAL = 2     /* recompute only the current block */
} dllm_cache_mode;

typedef enum dllm_sel_policy {
    DLLM_SEL_THRESHOLD = 0, /* Algorithm 2: c >= tau, else the single best */
    DLLM_SEL_FIXED_K = 1,   /* the k most confident (min(k, remaining)) */
    DLLM_SEL_FACTOR = 2,    /* Algorithm 3 / eq. 13: largest n with (n+1)(1-c_(n)) < f */
    DLLM_SEL_BUDGET = 3,    /* eq. 9: largest prefix with sum eps + max eps < 1 */
    DLLM_SEL_SCHEDULE = 4   /* page 1's LLaDA remasking schedule: with k steps left in the
                               block, the n_keep = (MASK count) / k most confident (n_keep
                               may be 0); dllm_run counts k down from the given k per block */
} dllm_sel_policy;

/* Selection rule.  Ties in confidence go to the lowest position, ties in the
 * argmax to the lowest token id; every comparison is made in float32 on the
 * float32 confidence.  Only MASK positions of the current block are eligible. */
typedef struct dllm_select {
    int32_t policy;   /* dllm_sel_policy */
    float tau;        /* THRESHOLD: threshold (> 1 gives one token per step) */
    int32_t k;        /* FIXED_K: tokens per step, >= 1 */
    float factor;     /* FACTOR: f > 0 */
} dllm_select;

/* Model shape (LLaMA-style, non-causal, MHA with n_heads * head_dim = d_model,
 * rotate-half RoPE, RMSNorm, SwiGLU FFN, untied embedding [vocab+1][d] and
 * LM head [vocab][d]).  head_dim must be 64 or 128; d_model a multiple of 128. */
typedef struct dllm_config {
    int32_t n_layers, d_model, n_heads, head_dim, d_ffn, vocab;
    float rope_theta, norm_eps;
} dllm_config;

/* Logical weight tensors, row-major [out][in] bf16 (uint16 bit patterns). */
typedef enum dllm_tensor {
    DLLM_T_EMBED = 1,       /* [vocab+1][d]  (row `vocab` is MASK)   */
    DLLM_T_ATTN_NORM = 2,   /* [d]    per layer                        */
    DLLM_T_WQ = 3,          /* [d][d] per layer, out = head*head_dim+j */
    DLLM_T_WK = 4,
    DLLM_T_WV = 5,
    DLLM_T_WO = 6,          /* [d][d] per layer                        */
    DLLM_T_FFN_NORM = 7,    /* [d]    per layer                        */
    DLLM_T_WG = 8,          /* [d_ffn][d] per layer                    */
    DLLM_T_WU = 9,          /* [d_ffn][d] per layer                    */
    DLLM_T_WD = 10,         /* [d][d_ffn] per layer                    */
    DLLM_T_FINAL_NORM = 11, /* [d]                                     */
    DLLM_T_LM_HEAD = 12     /* [vocab][d]                              */
} dllm_tensor;

/* Timings and counts of one dllm_run / dllm_generate (eq. 15 of the notes:
 * T_fast ~ S * C_active + R + T_selection; selection runs inside the step). */
typedef struct dllm_stats {
    double wall_ms;       /* whole call, host clock                             */
    double refresh_ms;    /* R: prefill + refreshes (CUDA events), the fused
                             refresh-and-step forwards included                 */
    double step_ms;       /* the other denoise steps (CUDA events)               */
    int32_t steps;        /* S: denoise steps run, fused ones included           */
    int32_t refreshes;    /* full-sequence forwards (prefill included)           */
    int32_t blocks;
    int32_t max_steps_per_block;
    int64_t committed;    /* tokens committed over all sequences                 */
    double tau_bar;       /* committed / sum over sequences of active steps      */
    int64_t kernel_launches; /* kernels this call launched                       */
    int32_t fused_steps;  /* steps run as the forward of the refresh before them
                             (counted in steps and in refreshes; their time is in
                             refresh_ms): C_active = step_ms / (steps - fused)   */
    int32_t reserved;
} dllm_stats;

typedef struct dllm_model dllm_model;
typedef struct dllm_state dllm_state;

/* ------------------------------------------------------------------ model */

/* Allocate a model's device weights (uninitialised) on the current device.
 * Fill every tensor with dllm_model_set_tensor before use. */
dllm_status dllm_model_create(const dllm_config* cfg, dllm_model** out);

/* Copy one logical tensor (count bf16 values, row-major [out][in]) into the
 * model's device layout.  src is a host pointer (src_on_device = 0) or a
 * device pointer (1).  count must equal the tensor's element count. */
dllm_status dllm_model_set_tensor(dllm_model* m, int32_t tensor, int32_t layer,
                                  const uint16_t* src, int64_t count, int32_t src_on_device);

/* Read a weight file and upload it: the model-loading call the decoder's
 * interface starts from (a trained model's weights in the pages' setting;
 * here seeded random-init weights of the same shapes).  Format: 8-byte magic
 * "DLLMW001", int32 n_layers, d_model,
 * n_heads, head_dim, d_ffn, vocab, float32 rope_theta, norm_eps, then every
 * tensor's bf16 bits: embed; per layer attn_norm wq wk wv wo ffn_norm wg wu wd;
 * final_norm; lm_head) and upload it.  DLLM_EIO on a short/malformed file. */
dllm_status dllm_load(const char* path, dllm_model** out);

dllm_status dllm_model_config(const dllm_model* m, dllm_config* cfg);
void dllm_free_model(dllm_model* m);

/* ------------------------------------------------------------------ state */

/* Create the decoding state of b sequences: canvas x = prompt ++ MASK*gen_len
 * (Algorithm 1 of the Fast-dLLM reading notes, section 3, step 1: append
 * gen_len MASK positions to the prompt; the tutorial's sampler starts from the
 * same all-MASK answer), K/V cache [layer][K|V][b][head][T][head_dim] bf16 with
 * T = P + gen_len, activations and workspaces.  prompts: host [b][P] int32, or
 * NULL to leave the prompt part for dllm_state_set_prompts_device.
 * gen_len % block == 0 and 1 <= block <= 256 are required.  cuda_stream is a
 * cudaStream_t (NULL = create a private stream).  Nothing runs on the GPU. */
dllm_status dllm_state_create(dllm_model* m, const int32_t* prompts, int32_t b, int32_t P,
                              int32_t gen_len, int32_t block, void* cuda_stream,
                              dllm_state** out);

/* Reset the canvas to prompt ++ MASK (prompts: host [b][P], or NULL to keep
 * the current prompt part) and forget the cache contents and counters. */
dllm_status dllm_state_reset(dllm_state* s, const int32_t* prompts);

/* Copy prompts already on the device ([b][P] int32) into the canvas and reset
 * the answer part to MASK (stream-ordered, no host synchronisation). */
dllm_status dllm_state_set_prompts_device(dllm_state* s, const int32_t* prompts_dev);

void dllm_free_state(dllm_state* s);

/* Full-sequence forward over all T positions of the current canvas; writes
 * every layer's K and V for every position into the cache in place (Algorithm
 * 1, steps 2 and 11).  Commits nothing; skips the last layer's attention/FFN
 * and the LM head, which K/V do not need. */
dllm_status dllm_prefill_refresh(dllm_state* s);

/* One denoise step of block block_idx with the threshold rule (Algorithm 2)
 * and the given cache mode.  committed_per_seq: host [b] or NULL.  Returns the
 * total number of tokens committed (>= 0), or -status on error.  A sequence
 * whose block has no MASK left commits 0.  block_idx must be in
 * [0, gen_len/block).  The cached modes read whatever the cache holds: call
 * dllm_prefill_refresh first. */
int32_t dllm_denoise_step(dllm_state* s, int32_t block_idx, float tau, int32_t cache_mode,
                          int32_t* committed_per_seq);

/* Same with any selection rule. */
dllm_status dllm_denoise_step_ex(dllm_state* s, int32_t block_idx, const dllm_select* sel,
                                 int32_t cache_mode, int32_t* committed_per_seq);

/* Algorithm 1 on the state's canvas: prefill refresh (cached modes), then for
 * each block, denoise steps until it has no MASK, then a refresh before the
 * next block (cached modes).  Tokens stay on the device (read them with
 * dllm_read_state).  refresh_interval > 0 also refreshes after every
 * refresh_interval steps inside a block (0 = only at block boundaries).
 * A refresh and the step after it run as one full forward over all T rows:
 * it rewrites every layer's K/V from the canvas, as the refresh does, and its
 * block rows are the step's, which after a refresh reads exactly those K/V
 * (stats->fused_steps counts them).  Under the block-causal mask this covers
 * the prefill and a refresh interval's refreshes, and in DualCache runs each
 * block-boundary commit forward (block j's K/V from the final canvas) runs in
 * one launch with block j+1's first step, over both blocks' rows.  The run
 * hook still sees the refresh (or commit-forward) event, then the step event.
 * stats may be NULL. */
dllm_status dllm_run(dllm_state* s, const dllm_select* sel, int32_t cache_mode,
                     int32_t refresh_interval, dllm_stats* stats);

/* Observer of dllm_run (and of nothing else): called on the calling thread
 * after each event of the loop has completed on the GPU, with the event kind,
 * the block index j and the step's index inside the block (for a refresh: the
 * number of steps the block had taken).  Events: DLLM_EVENT_REFRESH after the
 * prefill and every refresh (block boundary, or the refresh interval inside a
 * block), DLLM_EVENT_STEP after every denoise step, DLLM_EVENT_COMMIT_FORWARD
 * after the forward over a finished block that replaces the block-boundary
 * refresh under the block-causal mask.  A refresh (or commit forward) that
 * runs in one forward with the step after it is reported right before that
 * step's event, once both are done: the canvas then already holds the step's
 * commits.  Inside the hook the state may be read (dllm_read_state,
 * dllm_read_hidden, dllm_read_kv) but not changed.  A nonzero return stops
 * the run: dllm_run returns DLLM_ECANCELLED, with the canvas as the last
 * completed forward left it.  Use: stream committed tokens to a caller, or
 * follow the loop's decisions step by step. */
typedef enum dllm_event { DLLM_EVENT_REFRESH = 0, DLLM_EVENT_STEP = 1, DLLM_EVENT_COMMIT_FORWARD = 2 } dllm_event;
typedef int32_t (*dllm_run_hook)(void* user, int32_t event, int32_t block_idx, int32_t step_in_block);

/* Install (or with hook NULL remove) the state's run hook; user is passed back
 * unchanged.  It stays installed until changed or the state is freed. */
dllm_status dllm_state_set_run_hook(dllm_state* s, dllm_run_hook hook, void* user);

/* End-to-end call: prompts (host [b][P]) in, answers (host [b][gen_len]) out.
 * Creates a state on a private stream, runs Algorithm 1 with the threshold
 * rule, copies the answer back and frees the state. */
dllm_status dllm_generate(dllm_model* m, const int32_t* prompts, int32_t b, int32_t P,
                          int32_t gen_len, int32_t block, float tau, int32_t cache_mode,
                          int32_t* out_tokens, dllm_stats* stats);

/* Copy state to the host: tokens [b][T] (the whole canvas; Algorithm 1 of the
 * Fast-dLLM reading notes, section 3, returns its answer part), and the last
 * step's conf [b][block] (float32 max-softmax c_i) and arg [b][block] (argmax
 * y_i), the candidates and confidences of Algorithm 2 (section 4, steps 1-2).
 * Any pointer may be NULL. */
dllm_status dllm_read_state(const dllm_state* s, int32_t* tokens, float* conf, int32_t* arg);

/* The last denoise step's residual stream after the last layer for the block
 * rows, host float32 [b][block][d_model]. */
dllm_status dllm_read_hidden(const dllm_state* s, float* h);

/* Copy the cached K and V of one layer as float32, host [b][n_heads][T][head_dim] each
 * (hi + lo in split precision). */
dllm_status dllm_read_kv(const dllm_state* s, int32_t layer, float* k, float* v);

/* Precision of the activations fed to the tensor cores.  DLLM_PREC_SPLIT
 * (default) carries every GEMM input as a pair of bf16 arrays hi + lo with
 * lo = bf16(x - hi) (about 16 mantissa bits; the weights are read once, the
 * MMA is twice as wide).  DLLM_PREC_BF16 rounds activations to bf16 (half the
 * tensor work: for the compute-bound batch regime).  In split precision the
 * K/V cache, q and the attention probabilities are hi/lo pairs as well (the
 * cache holds both halves: twice the K/V bytes); in bf16 precision they are
 * bf16.  Accumulation is float32 in both.  Change the precision only before a
 * refresh: the cache's low halves are written only in split precision. */
typedef enum dllm_precision { DLLM_PREC_SPLIT = 0, DLLM_PREC_BF16 = 1 } dllm_precision;
dllm_status dllm_state_set_precision(dllm_state* s, int32_t mode);

/* DualCache steps with at most 128 activation rows (b * block <= 128, block
 * <= 32) run by default as one persistent cooperative launch: one CTA per SM
 * walks through every phase of the step (embedding, each layer's projections
 * and attention, LM head, merge and selection), ordered by dataflow flags (a
 * consumer waits only for the row tiles or heads it reads, no grid-wide
 * barrier), and streams the next phase's weights while a phase finishes.
 * enable 0 selects one launch per kernel instead (same arithmetic except the
 * attention key split; tracing always uses it). */
dllm_status dllm_state_set_persistent(dllm_state* s, int32_t enable);

/* dllm_run's fused forwards (on by default): a refresh and the step after it
 * run as one forward, and under the block-causal mask a DualCache run's
 * commit forward shares a launch with the next block's first step (see
 * dllm_run).  enable 0 runs every refresh and commit forward on its own, then
 * the step, as Algorithm 1 lists them; the trajectory is the same up to the
 * kernels' rounding. */
dllm_status dllm_state_set_fused_refresh(dllm_state* s, int32_t enable);

/* Run-ahead in dllm_run (enable 1, the default): within a block, the next
 * DualCache step that runs as one persistent launch is enqueued before the
 * current step's commit counts are read back, so the GPU does not wait for
 * the host between steps (Algorithm 1's inner loop, section 3 of the
 * Fast-dLLM reading notes, decides whether the block still holds a MASK only
 * after each step).  When the current step commits the block's last MASK,
 * the step launched ahead finds none at its start and ends without writing
 * anything; it is counted in kernel_launches, not in steps.  Tokens, steps
 * and refreshes are the same as with enable 0.  Run-ahead is off while a
 * run hook, per-kernel timing, the step timeline or the trace is set, and
 * for PrefixCache and no-cache runs, refresh-interval steps and steps that
 * do not fit one persistent launch. */
dllm_status dllm_state_set_run_ahead(dllm_state* s, int32_t enable);

/* Attention mask.  DLLM_MASK_BIDIRECTIONAL (default): every position sees
 * every position, the Fast-dLLM setting, in which the cached prefix and
 * suffix go stale and a block-boundary refresh recomputes them.
 * DLLM_MASK_BLOCK_CAUSAL: a prompt position sees the prompt, a position of
 * answer block j the prompt and blocks 0..j (block diffusion, BD3-LM style,
 * which the tutorial's section on caches and the dian8dian summary name as
 * the exact-cache alternative).  Nothing then attends to a later block, the
 * cache never goes stale, PrefixCache and DualCache compute the same as no
 * cache, and dllm_run replaces each block-boundary refresh by one forward
 * over the finished block's rows that caches their K/V.  Set before
 * dllm_prefill_refresh.  DLLM_EINVAL for another value. */
typedef enum dllm_mask { DLLM_MASK_BIDIRECTIONAL = 0, DLLM_MASK_BLOCK_CAUSAL = 1 } dllm_mask;
dllm_status dllm_state_set_mask(dllm_state* s, int32_t mask);

/* Diagnostics of the persistent step: with enable 1 the next persistent steps
 * record, per CTA and phase, 10 %globaltimer nanosecond stamps (uint64
 * [ctas][phases][10]): 0 the CTA's workers finished the phase, 1 its TMA
 * producer issued the phase's first activation tile (entry [cta][0][1] is the
 * kernel start), 2 its MMA issuer finished the phase, 3 the producer issued
 * the phase's last tile, 4 the workers started the phase, 5 they got its
 * first accumulator, 6 they were through their first segment, 7 they started
 * their last stream-K fix-up as the last contributor, 8 they had summed its
 * partials, 9 they published their last unit (row tile) of the phase; for
 * attention phases 5-9 are: first item's inputs ready, first item done, its
 * keys done, its split partial stored and counted, last head published; 0
 * where an event did not occur.  dllm_read_step_timeline copies the last step's
 * record. */
dllm_status dllm_state_set_step_timeline(dllm_state* s, int32_t enable);
dllm_status dllm_read_step_timeline(const dllm_state* s, uint64_t* out, int64_t capacity, int32_t* ctas,
                                    int32_t* phases);

/* Record the residual stream after the embedding and after every layer on the
 * next steps (1) or stop (0).  dllm_read_trace copies the last step's record,
 * host float32 [n_layers+1][rows][d_model], rows = b * rows_per_seq as
 * returned.  Tracing adds copies between layers: not for timing. */
dllm_status dllm_state_set_trace(dllm_state* s, int32_t enable);
dllm_status dllm_read_trace(const dllm_state* s, float* out, int64_t capacity_floats,
                            int32_t* rows_per_seq, int32_t* first_pos);

/* Accumulate per-kernel-class device time of the next calls with CUDA events
 * (enable 1), or stop (0).  dllm_kernel_times returns, per class, the summed
 * milliseconds, launch counts and algorithmic bytes (weights, K/V and
 * activations each counted once).  Classes of a denoise step: 0 embed,
 * 1 qkv_gemm, 2 attention, 3 o_gemm, 4 gateup_gemm, 5 down_gemm,
 * 6 lm_head_gemm, 7 merge_select; a refresh's launches use 8 + the same index;
 * 14 is the persistent step kernel.  16 classes in all.  The events serialise the kernels: not for the headline
 * time. */
dllm_status dllm_state_set_kernel_timing(dllm_state* s, int32_t enable);
dllm_status dllm_kernel_times(const dllm_state* s, double* ms, int64_t* launches,
                              double* bytes, int32_t n_classes);

/* ------------------------------------------------------------------ kernels */

/* Y[N][M] (float32) = X[N][K] * W[M][K]^T on the tensor cores (tcgen05, TMA,
 * stream-K split with a deterministic fix-up).  W, X bf16 row-major, 16-byte
 * aligned, K % 8 == 0.  X_lo (nullable) is a second bf16 array added to X
 * (the hi/lo activation pair).  Uses a library-owned workspace allocated on
 * first use. */
dllm_status dllm_op_gemm(const uint16_t* W, const uint16_t* X, const uint16_t* X_lo, float* Y,
                         int32_t M, int32_t N, int32_t K, void* cuda_stream);

/* dllm_op_gemm with a per-CTA timeline for diagnostics: trace (device,
 * uint64 [grid][8], grid <= the SM count, returned in *grid_out) receives per
 * CTA {SM id, start, first operand tile landed, last MMA issued, epilogue done,
 * end} in %globaltimer nanoseconds (entries 6-7 unused).  trace may be NULL. */
dllm_status dllm_op_gemm_trace(const uint16_t* W, const uint16_t* X, const uint16_t* X_lo, float* Y,
                               int32_t M, int32_t N, int32_t K, uint64_t* trace, int32_t* grid_out,
                               void* cuda_stream);

/* Non-causal attention, eq. 3: for every sequence s, head h and query row i,
 * out[s*R+i][h*hd..] = softmax(q k^T / sqrt(hd)) v over the T keys of
 * k_cache/v_cache [b][H][T][hd].  q: [b*R][H][hd] bf16, out [b*R][H*hd] bf16.
 * hd in {64, 128}.  Splits the keys across CTAs and merges the partial
 * softmax states deterministically (library-owned workspace). */
dllm_status dllm_op_attention(const uint16_t* q, const uint16_t* k_cache, const uint16_t* v_cache,
                              uint16_t* out, int32_t b, int32_t H, int32_t hd, int32_t R,
                              int32_t T, void* cuda_stream);

/* The same attention (eq. 3 of the Fast-dLLM reading notes, section 2; same
 * arguments, layouts and output as dllm_op_attention) on the tensor cores:
 * one CTA per (128-query tile, key split, head, sequence) runs S = q K^T and
 * O = P V as tcgen05.mma with S and O in tensor memory.  The keys are split
 * (at most 8 ways, 64-key granularity) when the query tiles alone would fill
 * the GPU's SMs unevenly; the last split of a query tile to finish merges the
 * partial softmax states in split order (deterministic), in a library-owned
 * workspace grown on first use.  This is the kernel the library uses for 65
 * or more query rows per sequence (the refresh's full forward, PrefixCache
 * and no-cache steps); block queries use the key-split kernel.  q, k_cache,
 * v_cache and out must be 16-byte aligned.  Results agree with
 * dllm_op_attention to bf16 rounding of the probabilities and the output,
 * not bit for bit. */
dllm_status dllm_op_attention_tc(const uint16_t* q, const uint16_t* k_cache, const uint16_t* v_cache,
                                 uint16_t* out, int32_t b, int32_t H, int32_t hd, int32_t R,
                                 int32_t T, void* cuda_stream);

/* dllm_op_attention_tc with the number of key splits chosen by the caller:
 * splits = 0 takes the library's plan (as dllm_op_attention_tc), 1..8 cuts
 * the keys into that many ranges of equal 64-key multiples (fewer when T is
 * short: ranges past T are dropped).  Other values: DLLM_EINVAL. */
dllm_status dllm_op_attention_tc_ex(const uint16_t* q, const uint16_t* k_cache, const uint16_t* v_cache,
                                    uint16_t* out, int32_t b, int32_t H, int32_t hd, int32_t R,
                                    int32_t T, int32_t splits, void* cuda_stream);

/* dllm_op_attention with no allocation of any kind.  The pages have no
 * counterpart to this entry point: it computes the same attention as
 * dllm_op_attention, with the same arguments, layouts and output, and is
 * bit-identical to it for every shape it accepts.  What differs is where the
 * scratch lives.  dllm_op_attention grows a library-owned workspace with
 * cudaMalloc + cudaMemset the first time a shape needs more; this variant uses
 * a fixed scratch in static device storage of the library (key-split
 * partials: 1 Mi floats = 4 MiB; merge counters: 4096; every device that
 * loads the library holds it until the process exits) and never calls
 * cudaMalloc, cudaFree or an allocating library.  It serves callers that must
 * not allocate device memory at call time: a caller whose device memory is
 * fully reserved up front (weights and K/V pools sized to the card), or one
 * that issues work where an allocation, or the device-wide synchronisation a
 * cudaMalloc may imply, is not allowed.
 *  - Set-up: the first call on each device looks up the scratch's device
 *    address (cudaGetSymbolAddress with that device current) and the driver's
 *    tensor-map entry point; make that first call before any stream capture.
 *  - Limit: b*H*ceil(R/QT) merge works and, when the keys are split,
 *    works*splits*QT*(hd+2) floats (QT = 32 for R <= 32, else 64; splits as
 *    dllm_op_attention plans them for this GPU).  A call over the limit
 *    returns DLLM_EINVAL, launches nothing and names the limit in
 *    dllm_last_error(); use dllm_op_attention for it.  The 8B DualCache block
 *    (b=1, H=32, hd=128, R=32, T=768) fits.
 *  - Zero state: each call clears the merge counters it uses (a
 *    cudaMemsetAsync on the caller's stream) before its launch, so a call
 *    after one that gave up a bounded wait starts clean.
 *  - Errors: a launch that gives up a bounded wait sets the scratch's error
 *    word; dllm_op_check reports it (DLLM_ETIMEOUT) and clears it.
 *  - Concurrency: all calls on a device share the one scratch.  Calls ordered
 *    on one stream are safe; calls that may overlap (different streams, or
 *    different host threads without ordering) race on the scratch and give
 *    wrong results.
 *  - Asynchronous like dllm_op_attention: returns after the launch. */
dllm_status dllm_op_attention_noalloc(const uint16_t* q, const uint16_t* k_cache,
                                      const uint16_t* v_cache, uint16_t* out, int32_t b,
                                      int32_t H, int32_t hd, int32_t R, int32_t T,
                                      void* cuda_stream);

/* Synchronise cuda_stream, then report whether any kernel launched by the
 * dllm_op_* calls on the current device (the no-alloc attention included)
 * gave up a bounded wait since the last check: DLLM_ETIMEOUT with the wait's
 * site code in *site (nullable), else DLLM_OK with *site = 0.  Clears the
 * error words it read.  Outputs of a call that timed out are invalid.
 * Allocates nothing. */
dllm_status dllm_op_check(int32_t* site, void* cuda_stream);

/* Failure detection without a fault: one GPU thread waits, with the same
 * bounded dataflow wait the persistent step uses between its phases, until
 * the device int32 *flag reaches need or limit_us microseconds (1 ..
 * 2,000,000) have passed.  Synchronous; returns DLLM_OK if the flag was
 * reached and DLLM_ETIMEOUT if the wait gave up (through dllm_op_check, which
 * also clears the error word, so the next call starts clean).  With a flag
 * that nothing raises it exercises the give-up path: error word set, the
 * kernel returns, the context stays usable. */
dllm_status dllm_op_wait_probe(const int32_t* flag, int32_t need, int32_t limit_us, void* cuda_stream);

/* The selection/commit kernel alone: given conf [b][B] float32 and arg [b][B]
 * int32 (device), select on the MASK positions x[s][blk_start .. +B) of the
 * canvas x [b][T] (device int32), write the chosen arg ids into x and the
 * per-sequence counts into count [b] (device). */
dllm_status dllm_op_select_commit(const float* conf, const int32_t* arg, int32_t* x,
                                  int32_t b, int32_t T, int32_t blk_start, int32_t B,
                                  int32_t mask_id, const dllm_select* sel, int32_t* count,
                                  void* cuda_stream);

/* --------------------------------------------------------------- 8-bit forms
 *
 * A decode step streams two things: the weights and the K/V cache.  These
 * entry points are their 8-bit forms, from the projection to the attention
 * output:  dllm_op_quantise8 + dllm_op_gemm8 (projections), dllm_op_rope
 * (positions), dllm_op_kv8_store / _load (the cache), dllm_op_attention_kv8
 * (attention over it).  They allocate nothing, keep nothing between calls and
 * can be captured into a CUDA graph; calls on different streams do not
 * disturb one another as long as their outputs and workspaces differ.  Device
 * pointers belong to the current device, and so does the stream.  Outputs do not overlap inputs
 * unless the text says so.  The pages have no counterpart: they quantise nothing.
 *
 * Codes are e4m3 (sign, 4 exponent, 3 mantissa bits; largest value 448).  A
 * block of values shares the scale 2^(byte - 127), one byte: the smallest with
 * max|x| / scale <= 448, at least 2^-127; 1 for a block of zeros.  A code is
 * x / scale rounded to nearest, ties to even.  The division by a power of two
 * is exact, so codes do not depend on the arithmetic that forms them, and
 * since e4m3 is a floating type the power of two costs no precision.  A block
 * that holds a NaN or an infinity gets the byte 255 and codes 0: every value
 * of it reads back as NaN. */

typedef enum dllm_dtype { DLLM_F32 = 0, DLLM_BF16 = 1, DLLM_F16 = 2 } dllm_dtype;

typedef enum dllm_rope_layout {
    DLLM_ROPE_HALF = 0,        /* pair i is elements i and i + rot_dim/2 (rotate-half) */
    DLLM_ROPE_INTERLEAVED = 1  /* pair i is elements 2i and 2i + 1 */
} dllm_rope_layout;

/* Turning rate of pair i, radians a position, f_i = theta^(-2i/rot_dim), and
 * its forms for contexts `factor` times as long: */
typedef enum dllm_rope_scaling {
    DLLM_ROPE_UNSCALED = 0,
    DLLM_ROPE_LINEAR = 1,      /* f_i / factor (position interpolation) */
    DLLM_ROPE_BASE = 2,        /* theta * factor^(rot_dim / (rot_dim - 2)) in place of theta */
    DLLM_ROPE_BY_PARTS = 3     /* YaRN: f_i where the pair turns at least beta_fast times within orig_len
                                  positions, f_i / factor where fewer than beta_slow, a linear ramp over
                                  the pair index between: from floor to ceil of
                                  rot_dim ln(orig_len / (2 pi beta)) / (2 ln theta), kept within
                                  0..rot_dim - 1 (so the ramp may end past the last pair) */
} dllm_rope_scaling;

typedef struct dllm_rope {
    int32_t layout, rot_dim;   /* the first rot_dim elements of a head turn (even, 2..256), the rest is copied */
    int32_t scaling, reserved;
    double theta, factor;      /* >= 1; factor is unused when unscaled */
    double orig_len, beta_fast, beta_slow;   /* by parts only */
    double amplitude;          /* multiplies cosine and sine; 0: 1, or 0.1 ln(factor) + 1 by parts */
} dllm_rope;

/* Rotary positions: out = x with the pairs of every head turned by
 * positions[row] * f_i.  x, out: [rows][heads][hd] of dtype (dllm_dtype), hd
 * even, 2..1024, with strides in elements between rows and heads (0: dense);
 * a head's elements are contiguous; a fused [rows][q|k|v] buffer or a
 * head-major one is covered by strides.  out may be x with the same strides.
 * positions: device int32 [rows], any value.  A rate is computed in 64-bit
 * floating point and its angle reduced by whole turns in fixed point, so that an angle is
 * off by at most |position| * f_i * 2^-49 radians for theta to 1e8 (2^-28 at position 2^21); the products
 * are float32, rounded once.  The rates reach the device with the launch:
 * *rope may be reused at once. */
dllm_status dllm_op_rope(const void* x, void* out, const int32_t* positions, int32_t rows, int32_t heads, int32_t hd,
                         int64_t x_row_stride, int64_t x_head_stride, int64_t out_row_stride,
                         int64_t out_head_stride, int32_t dtype, const dllm_rope* rope, void* cuda_stream);

/* An 8-bit K/V cache in the caller's device memory: codes [b][H_kv][T][hd]
 * (16-byte aligned) and scale bytes [b][H_kv][T], one scale for each row of hd
 * (a token's head).  hd in {64, 128}, T at most 2^31 - 4096.  The codes 0x7f and 0xff (NaN in
 * e4m3) are never stored; what a caller's own cache makes of them is not defined.  The struct is
 * read during the call. */
typedef struct dllm_kv8 {
    uint8_t *k, *v, *k_scale, *v_scale;
    int32_t b, H_kv, T, hd;
} dllm_kv8;

/* Quantise rows of K and V into the cache.  k, v: [b*R][H_kv][hd] of dtype,
 * 16-byte aligned, rows k_row_stride / v_row_stride elements apart (0: dense;
 * else a multiple of 16 bytes).  Row i of sequence s goes to position
 * starts[s] + i for i < counts[s] (device int32 [b]; NULL starts: 0, NULL
 * counts: R).  Rows from counts[s] on are padding, and rows whose position lies outside
 * [0, T) have no slot: neither is written, every other slot stays as it was. */
dllm_status dllm_op_kv8_store(const dllm_kv8* cache, const void* k, const void* v, int64_t k_row_stride,
                              int64_t v_row_stride, int32_t dtype, int32_t R, const int32_t* starts,
                              const int32_t* counts, void* cuda_stream);

/* Read rows back: the inverse of dllm_op_kv8_store with the same arguments,
 * code * scale rounded to dtype (exact in float32 and bf16 down to their
 * subnormals; in f16 where it is in range).  Rows without a slot are left as
 * they were in k and v. */
dllm_status dllm_op_kv8_load(const dllm_kv8* cache, void* k, void* v, int64_t k_row_stride, int64_t v_row_stride,
                             int32_t dtype, int32_t R, const int32_t* starts, const int32_t* counts,
                             void* cuda_stream);

/* Attention over the 8-bit cache: for sequence s, row i, head h
 *   out[s*R+i][h] = sum_t softmax_t(scale * q . K[s][g][t]) V[s][g][t],
 * over t < limits[s*R+i], g = h / (H / H_kv) (grouped heads; H a multiple of
 * H_kv).  q, out: bf16 [b*R][H][hd], 16-byte aligned, rows q_row_stride /
 * out_row_stride elements apart (0: dense; else a multiple of 8).  limits:
 * device int32 [b][R], the number of keys the row sees (values over T count
 * as T); NULL: all T.  So lengths, causal, block-causal and padded batches are
 * limits, and R = 1 is single-token decoding.  A row with limit <= 0 gives
 * zeros.  What lies in the cache at or past every limit of its sequence is
 * never used, whatever its bytes; a key or value row with scale byte 255
 * turns the rows that see it into NaN and no others.  Scores, softmax
 * statistics and sums are float32; a probability enters the value product
 * with 8 significant bits (an error of 2^-8 of itself, or of 2^-21 of the
 * largest p * 2^ev of its row among 32 neighbouring keys where that is more).
 * scale: > 0, at most 1e30.  Scores are formed in float32 from the codes and their
 * scales apart: elements of q and of K, and scale times either, stay within 2^100.  workspace: device memory for the partial results of
 * split keys, 16-byte aligned, at least dllm_op_attention_kv8_workspace
 * bytes (0: may be NULL), contents irrelevant; calls that may run at the same
 * time need one each. */
dllm_status dllm_op_attention_kv8(const uint16_t* q, int64_t q_row_stride, const dllm_kv8* cache,
                                  const int32_t* limits, float scale, uint16_t* out, int64_t out_row_stride,
                                  int32_t H, int32_t R, void* workspace, int64_t workspace_bytes,
                                  void* cuda_stream);
dllm_status dllm_op_attention_kv8_workspace(int32_t b, int32_t H, int32_t H_kv, int32_t hd, int32_t R, int32_t T,
                                            int64_t* bytes);

/* Quantise rows in blocks of 128 along K (the last block of a row may be
 * shorter): x [rows][K] of dtype, rows row_stride elements apart (0: dense), to
 * codes [rows][K] (16-byte aligned) and scales [ceil(K/128)][rows].
 * K % 16 == 0.  Weights and activations take the same form. */
dllm_status dllm_op_quantise8(const void* x, int64_t row_stride, int32_t dtype, int32_t rows, int32_t K,
                              uint8_t* codes, uint8_t* scales, void* cuda_stream);

/* Y[N][M] = X[N][K] * W[M][K]^T of quantised operands: codes 16-byte aligned,
 * row-major; scales as dllm_op_quantise8 lays them out, W_scale
 * [ceil(K/128)][M], X_scale [ceil(K/128)][N].  K % 16 == 0.  Y is float32 or bf16
 * (y_dtype), 16-byte aligned, rounded once from a float32 sum.  A block with scale byte 255
 * makes its row of X (column of Y for W) NaN. */
dllm_status dllm_op_gemm8(const uint8_t* W, const uint8_t* W_scale, const uint8_t* X, const uint8_t* X_scale, void* Y,
                          int32_t y_dtype, int32_t M, int32_t N, int32_t K, void* cuda_stream);

/* ------------------------------------------------------------ paged decoding
 *
 * What a decode step over sequences of different lengths does around its
 * products, on a cache whose pages lie anywhere in a pool:
 * dllm_op_qk_norm_rope_paged (head norms, positions, the cache's new rows),
 * dllm_op_attention_paged (attention over the pages, and the weight that each
 * key received), dllm_op_kv_paged_evict (the heaviest keys to new pages) and
 * dllm_op_token_logprobs (what the logits say).  As the 8-bit forms they
 * allocate nothing, keep nothing between calls and can be captured into a CUDA
 * graph; calls on different streams do not disturb one another as long as
 * their outputs and workspaces differ.  Device pointers belong to the current
 * device, and so does the stream.  Outputs do not overlap inputs unless the
 * text says so.  The pages this library follows have no counterpart: their
 * cache is one canvas. */

/* A paged K/V cache in the caller's device memory.  A page holds page_size
 * positions of every cached head: k, v [pages][H_kv][page_size][hd] of dtype
 * (bf16 or f16), 16-byte aligned, hd in {64, 128}, page_size a power of two,
 * 16..256.  table: device int32 [b][max_pages]; position t of sequence s lies
 * on page table[s][t / page_size], slot t % page_size.  Entries past a
 * sequence's last page are never read.  An entry outside [0, pages) is no page:
 * nothing is written there, and its positions hold no key.  A sequence has at
 * most max_pages * page_size positions (at most 2^31 - 4096 in all).  Sequences
 * may share pages that are only read.  The struct is read during the call. */
typedef struct dllm_kv_paged {
    void *k, *v;
    const int32_t* table;
    int32_t b, H_kv, hd, dtype;
    int32_t pages, page_size, max_pages, reserved;
} dllm_kv_paged;

/* Head norms and rotary positions in one pass: for every row and head x of q
 * (H heads) and k (H_kv heads)
 *   y = x / sqrt(mean(x^2) + eps) * weight,  then y's pairs turned as in
 * dllm_op_rope; float32, rounded once (the angle's error as there).
 * q: [rows][H][hd], k: [rows][H_kv][hd] of dtype, outputs of out_dtype: dtype,
 * or bf16 / f16 from float32.  Rows are *_row_stride elements apart (0: dense;
 * else at least the row and a multiple of 16 bytes): one [rows][q|k|v] buffer
 * is covered.  Everything 16-byte aligned.  hd a multiple of 16, 16..256.
 * q_weight, k_weight: [hd] of dtype, NULL: ones; eps >= 0; eps < 0: no norm
 * (both weights NULL).  rope: NULL: nothing turns (positions may be NULL);
 * rot_dim a multiple of 16.  positions: device int32 [rows].  An output may be
 * its input with the same strides and type.  Squares are float32: elements
 * stay within 2^59, and with eps = 0 a head that is not all zeros has one of
 * 2^-50 at least. */
dllm_status dllm_op_qk_norm_rope(const void* q, int64_t q_row_stride, const void* k, int64_t k_row_stride, void* q_out,
                                 int64_t q_out_row_stride, void* k_out, int64_t k_out_row_stride,
                                 const int32_t* positions, int32_t rows, int32_t H, int32_t H_kv, int32_t hd,
                                 int32_t dtype, int32_t out_dtype, const void* q_weight, const void* k_weight,
                                 float eps, const dllm_rope* rope, void* cuda_stream);

/* The same with k, and v as it is, going to their places in the cache: q, k, v
 * [b*R] rows of H, H_kv and H_kv heads, of dtype (the cache's, or float32);
 * q_out of the cache's type.  Row i of sequence s goes to position
 * starts[s] + i for i < counts[s] (device int32 [b]; NULL starts: 0, NULL
 * counts: R).  positions: device int32 [b*R], what q and k turn by, or NULL:
 * starts[s] + i.  Rows from counts[s] on, and rows whose position in the cache
 * lies outside the table or on no page, take no part: their q_out and every
 * other slot stay as they were.  With rope NULL and eps < 0 it stores rows as
 * they are.  No two rows of a call may go to one slot. */
dllm_status dllm_op_qk_norm_rope_paged(const dllm_kv_paged* cache, const void* q, int64_t q_row_stride, const void* k,
                                       int64_t k_row_stride, const void* v, int64_t v_row_stride, void* q_out,
                                       int64_t q_out_row_stride, int32_t H, int32_t R, int32_t dtype,
                                       const int32_t* starts, const int32_t* counts, const int32_t* positions,
                                       const void* q_weight, const void* k_weight, float eps, const dllm_rope* rope,
                                       void* cuda_stream);

/* Attention over the pages: for sequence s, row i, head h
 *   out[s*R+i][h] = sum_t p_t V[s][g][t],  p = softmax_t(scale * q . K[s][g][t]),
 * over t < lens[s] (device int32 [b]; NULL, or more than the table holds: all
 * it holds), g = h / (H / H_kv) (grouped heads; H a multiple of H_kv).  R = 1
 * is single-token decoding; the R rows of a block see the same keys, each
 * other's among them once these are stored.  (Rows that see different keys are
 * sequences of their own, whose table rows name the same pages.)  A sequence of
 * lens <= 0 gives zeros.  What lies at or past lens[s], or on no page, is not
 * used, whatever its bytes.  q, out: of the cache's type, [b*R][H][hd], 16-byte
 * aligned, rows q_row_stride / out_row_stride elements apart (0: dense; else a
 * multiple of 8).  scale: > 0, at most 1e38.  Scores, statistics and sums are float32; a probability
 * enters the value product as the sum of two values of the cache's type: to
 * 2^-16 of it in bf16; in f16 to 2^-22 of it, or 2^-45 of the row's largest.
 * K, V and q are finite, and so are the scores.
 *   mass (nullable): device float32 [b][H_kv][mass_stride] (0: max_pages *
 * page_size); mass[s][g][t] += the sum of p_t over the R rows and the heads of
 * g, for t < lens[s]; the rest stays as it was, and weights of positions from
 * mass_stride on are not kept.  In a fixed order: the same inputs give the same
 * bits.
 *   workspace: device memory, 16-byte aligned, of at least
 * dllm_op_attention_paged_workspace bytes for the same shape on the current
 * device (T = max_pages * page_size, with_mass: whether mass is given; 0: may
 * be NULL), contents irrelevant; calls that may run at the same time need one
 * each. */
dllm_status dllm_op_attention_paged(const void* q, int64_t q_row_stride, const dllm_kv_paged* cache,
                                    const int32_t* lens, float scale, void* out, int64_t out_row_stride, int32_t H,
                                    int32_t R, float* mass, int64_t mass_stride, void* workspace,
                                    int64_t workspace_bytes, void* cuda_stream);
dllm_status dllm_op_attention_paged_workspace(int32_t b, int32_t H, int32_t H_kv, int32_t hd, int32_t R, int32_t T,
                                              int32_t with_mass, int64_t* bytes);

/* Eviction by accumulated weight: of the n = lens[s] positions of every
 * sequence s and cached head g, keep m = min(n, keep) and copy their K and V rows,
 * in the order of their positions, to positions 0..m-1 of dst.  All n are kept
 * when n <= keep; else the first `sinks`, the last `recent`, and of the others
 * the keep - sinks - recent of largest mass[s][g][t] (ties: the lowest
 * position; a NaN counts as less than every number).  src and dst: of the same b, H_kv, hd and
 * dtype, page sizes of their own; dst's pages are not among src's (they may lie
 * in the same pool), and its table holds at least keep positions.
 *   lens: device int32 [b]; NULL, or more than src's table holds: all it holds.
 *   mass: device float32 [b][H_kv][mass_stride] (0: max_pages * page_size of
 *   src); n is at most mass_stride.
 *   kept: device int32 [b][H_kv][keep], the positions kept, ascending, -1 from m on.
 *   new_lens: device int32 [b], m; not lens itself.
 *   mass_out (nullable): device float32 [b][H_kv][mass_out_stride] (0: keep),
 *   mass_out_stride >= keep: the weights of the kept, its other elements stay as they were.
 * A kept position that lies on no page gives a row of zeros.
 * keep >= 1, sinks, recent >= 0, sinks + recent <= keep. */
dllm_status dllm_op_kv_paged_evict(const dllm_kv_paged* src, const dllm_kv_paged* dst, const float* mass,
                                   int64_t mass_stride, const int32_t* lens, int32_t keep, int32_t sinks,
                                   int32_t recent, int32_t* kept, int32_t* new_lens, float* mass_out,
                                   int64_t mass_out_stride, void* cuda_stream);

/* What rows of logits say: with z = inv_temperature * logits[r] and
 * log p_i = z_i - log sum_j exp z_j,
 *   logprobs[r] = log p at targets[r] (NaN for a target outside [0, vocab)),
 *   entropy[r]  = -sum_i p_i log p_i (in nats),
 *   top_ids[r][0..top), top_logprobs[r][0..top): the largest logits, ties the
 *   lowest id first, and their log p.
 * logits: device [rows][vocab] of dtype, rows row_stride elements apart (0:
 * vocab; else >= vocab), aligned to their elements; rows and vocab at most
 * 2^31 - 4096.  targets: device int32
 * [rows], goes with logprobs; every output may be NULL, top_ids and
 * top_logprobs are given together when top > 0; top <= 64 and <= vocab.
 * inv_temperature: > 0, at most 1e38.  Sums are float32, taken apart from the largest
 * term, so that log p and entropy of a nearly certain row keep their relative
 * accuracy, in chains of at most 256 terms that are joined one by one: about
 * (300 + vocab / 2^14) 2^-24 of a sum where all roundings go one way.  A logit
 * of -inf is a token that cannot come: p = 0, and an alternative only after all
 * others.  A row with a NaN or +inf, or of nothing but -inf, has NaN for every
 * log p and entropy; a NaN is no alternative (id -1 where there are too few
 * others). */
dllm_status dllm_op_token_logprobs(const void* logits, int64_t row_stride, int32_t dtype, int32_t rows, int32_t vocab,
                                   float inv_temperature, const int32_t* targets, float* logprobs, float* entropy,
                                   int32_t top, int32_t* top_ids, float* top_logprobs, void* cuda_stream);

/* Cache staleness diagnostics for block block_idx of the current canvas (the
 * Fast-dLLM notes, section 14, Algorithm 4 steps 4-5: compare fresh and
 * cached representations and predictions at the positions about to be
 * committed; the notes' section 3 on what DualCache freezes).  Without
 * changing the canvas or the cache's prefix/suffix rows it runs a full
 * forward over all T positions of the current canvas into a scratch K/V
 * ("fresh") and the block forward twice, on the cache and on the fresh K/V,
 * and returns (host outputs):
 *   k_cos[l], v_cos[l]  float32 [n_layers]: the mean over sequences, heads
 *                       and every position outside the block of the cosine
 *                       between the cached and the fresh K (V) row;
 *   agree               the fraction of the block's MASK positions whose
 *                       argmax is the same from both;
 *   max_dconf           the largest |max-prob(cached) - max-prob(fresh)| there.
 * The block's own K/V rows in the cache are rewritten with the current
 * canvas's (as the next step would).  Allocates a second K/V of the cache's
 * size on first use.  DLLM_EINVAL for a bad block or NULL output. */
dllm_status dllm_staleness(dllm_state* s, int32_t block_idx, float* k_cos, float* v_cos, float* agree,
                           float* max_dconf);

/* ------------------------------------------------------------------ misc */

const char* dllm_last_error(void);
const char* dllm_status_string(int32_t status);
/* Library version as major*10000 + minor*100 + patch. */
int32_t dllm_version(void);

#ifdef __cplusplus
}
#endif
#endif /* DLLM_H */
