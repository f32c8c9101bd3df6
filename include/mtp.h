/*
 * mtp.h -- C ABI of libmtp: the Gemma-4-assistant Multi-Token-Prediction drafter step,
 * draft block and greedy verification on one NVIDIA GB300 (sm_103a).
 *
 * Conventions for every entry point
 *   - Pointers named "device" are CUDA device pointers (cudaMalloc / torch CUDA tensors)
 *     on the current device; the library borrows them and never frees them.
 *   - Matrices are row-major [out][in]; "model dtype" means bf16 (MTP_DTYPE_BF16) or fp32
 *     (MTP_DTYPE_F32) as fixed at init. Norm gains are always fp32.
 *   - Device pointers must be 16-byte aligned; row strides are multiples of 16 bytes.
 *   - `stream` is a cudaStream_t passed as void* (NULL = legacy default stream). Calls
 *     only enqueue work on it and return; nothing synchronises except mtp_init_weights,
 *     mtp_get_status and mtp_destroy.
 *   - Return value: MTP_OK or an MTP_ERR_* code; on error nothing was enqueued and
 *     mtp_last_error() describes the cause (per calling thread).
 *
 * Precision contract (both this library and its CPU oracle): stored tensors (weights,
 * shared K, embedding tables, the caller's hidden state, target logits) are bf16, or fp32
 * for fp32 models. Activations are fp32 and are never rounded to a narrower type: no
 * projection input, attention operand or intermediate vector is rounded to bf16, and the
 * post-projected hidden state carried to the next draft step stays fp32 (unrounded).
 * Top-k and argmax decide on fp32 values, ties going to the lower centroid index / lower
 * vocabulary id.
 */
#ifndef MTP_H_
#define MTP_H_

#include <stdint.h>

#if defined(__GNUC__)
#define MTP_API __attribute__((visibility("default")))
#else
#define MTP_API
#endif

#ifdef __cplusplus
extern "C" {
#endif

#define MTP_MAX_LAYERS 8

enum mtp_status {
  MTP_OK = 0,
  MTP_ERR_INVALID_ARG = 1,       /* NULL / out-of-range argument (missing hidden or KV included) */
  MTP_ERR_UNSUPPORTED_SHAPE = 2, /* shape outside what the kernels implement */
  MTP_ERR_BAD_ORDERING = 3,      /* vocab % n_centroids != 0 or ordering not a permutation */
  MTP_ERR_CUDA = 4,              /* a CUDA runtime call failed */
  MTP_ERR_TIMEOUT = 5            /* a device-side wait gave up (reported by mtp_get_status) */
};

enum mtp_dtype { MTP_DTYPE_BF16 = 0, MTP_DTYPE_F32 = 1 };

/* Value of the vocabulary entries outside the selected clusters in a materialised logits row
 * of the centroid head: -1e30f ("Gemma 4 Assistant tensor inventory", "Centroid / ordered
 * embeddings LM head", step 5: dense fill, then the sparse logits set at their ids), or the
 * smallest selected logit minus one ("Gemma 4 Assistant 使用指南", section 五, step 3 of
 * use_ordered_embeddings; named there as the MLX-style alternative). The argmax is the same
 * either way. */
enum mtp_logit_mask { MTP_MASK_NEG_1E30 = 0, MTP_MASK_MIN_MINUS_ONE = 1 };
enum mtp_layer_kind { MTP_LAYER_SLIDING = 0, MTP_LAYER_FULL = 1 };
/* Traversal of the sparse head (the candidate-row gather and GEMV, steps 3-4 of "Gemma 4
 * Assistant tensor inventory", "Centroid / ordered embeddings LM head"): per sequence (each
 * sequence reads the rows of its own top_k clusters), or cluster-major (each distinct
 * selected cluster is streamed once per step, with bulk copies, for every sequence that
 * selected it). Both give the same selected sets and the same logits up to fp32 summation
 * order. AUTO: per sequence (on GB300 the L2 already serves the rows that sequences share,
 * and the per-sequence gather was the faster of the two at every batch measured). */
enum mtp_sparse_head { MTP_HEAD_AUTO = 0, MTP_HEAD_PER_SEQUENCE = 1, MTP_HEAD_CLUSTER_MAJOR = 2 };

/* Drafter hyper-parameters.
 * Cited: "Gemma 4 Multi-Token Prediction (MTP) drafter", sections "Conversion" (metadata
 * keys backbone_hidden_size, num_centroids, centroid_intermediate_top_k,
 * use_ordered_embeddings) and "Tensor schema"; "Gemma 4 Assistant tensor inventory",
 * "HF config highlights" (layer_types, attention_k_eq_v, vocab_size, hidden_size). */
typedef struct mtp_config {
  int32_t backbone;        /* target hidden size bb (pre_projection input is 2*bb) */
  int32_t hidden;          /* assistant hidden size H */
  int32_t n_layers;        /* 1..MTP_MAX_LAYERS */
  int32_t n_head;          /* query heads */
  int32_t head_dim_swa;    /* head dim of sliding layers (and of the sliding shared K) */
  int32_t head_dim_full;   /* head dim of full layers (and of the full shared K) */
  int32_t n_kv_head;       /* shared KV heads; n_head % n_kv_head == 0 */
  int32_t ffn;             /* MLP intermediate size */
  int32_t vocab;           /* V */
  int32_t n_centroids;     /* C (ordered embeddings only) */
  int32_t top_k;           /* selected centroids (ordered embeddings only), <= 64 */
  int32_t window;          /* sliding window W (keys attended by sliding layers) */
  int32_t use_ordered_embeddings; /* 1: centroid head; 0: dense tied head */
  int32_t dtype;           /* enum mtp_dtype */
  int32_t max_batch;       /* largest B any later call will pass (sizes the workspace) */
  int32_t max_ctx;         /* largest shared-K length any later call will pass */
  uint8_t layer_type[MTP_MAX_LAYERS]; /* enum mtp_layer_kind per block */
  float rms_eps;           /* RMSNorm epsilon (1e-6) */
  float attn_scale;        /* softmax scale; 0 -> 1/sqrt(head_dim) */
  float rope_theta_swa;    /* RoPE base of sliding layers; 0 disables RoPE */
  float rope_theta_full;   /* RoPE base of full layers; 0 disables RoPE */
} mtp_config;

/* Per-block tensors ("Tensor schema": attn_q, attn_q_norm, attn_output, attn_norm,
 * post_attention_norm, ffn_norm, post_ffw_norm, ffn_gate/up/down, layer_output_scale).
 * There are no K/V projections: the drafter is Q-only and reads the target's K. */
typedef struct mtp_layer_weights {
  const void *q;      /* device [n_head*d][H], model dtype */
  const void *o;      /* device [H][n_head*d] */
  const void *gate;   /* device [ffn][H] */
  const void *up;     /* device [ffn][H] */
  const void *down;   /* device [H][ffn] */
  const float *q_norm;          /* device [d] */
  const float *attn_norm;       /* device [H] */
  const float *post_attn_norm;  /* device [H] */
  const float *ffn_norm;        /* device [H] */
  const float *post_ffn_norm;   /* device [H] */
  float layer_scalar;           /* host value: multiplies the residual after the block */
} mtp_layer_weights;

typedef struct mtp_weights {
  const void *pre_proj;     /* device [H][2*bb]  (input [target_hidden ; embed(token)]) */
  const void *post_proj;    /* device [bb][H] */
  const void *token_embd;   /* device [V][H]: tied LM head rows */
  const void *centroids;    /* device [C][H] (ordered embeddings only, else NULL) */
  const float *out_norm;    /* device [H] */
  const int32_t *token_ordering; /* device [V] viewed [C][V/C]: centroid c owns ids
                                    ordering[c*V/C .. (c+1)*V/C) (ordered only) */
  mtp_layer_weights layer[MTP_MAX_LAYERS];
} mtp_weights;

/* Shared K of one attention type: the target's last layer of that type
 * ("Gemma 4 Assistant 使用指南", section 二.4: shared_kv_states maps
 * "full_attention" / "sliding_attention" to (key, value)).
 * Element (b, t, kv_head, i) sits at k[b*stride_b + t*stride_t + kv_head*d + i].
 * v == NULL means V = K (attention_k_eq_v: "Gemma 4 Assistant tensor inventory",
 * "Notes for llama.cpp port" item 2); otherwise v has the same layout. ctx_len[b] >= 1 is the
 * number of valid keys of sequence b (right-padded storage; padding is never read); values
 * are clamped to [0, max_ctx] on the device, and a sequence with no keys attends nothing
 * (its attention output is 0). */
typedef struct mtp_kv {
  const void *k;           /* device, model dtype */
  const void *v;           /* device or NULL (V = K) */
  const int32_t *ctx_len;  /* device [B] */
  int64_t stride_b;        /* elements between sequences */
  int64_t stride_t;        /* elements between tokens (>= n_kv_head*d, multiple of 8) */
  int32_t max_ctx;         /* upper bound of ctx_len[*] (<= mtp_config.max_ctx) */
} mtp_kv;

typedef struct mtp_handle mtp_handle;

/* Validate the configuration and the weights, check token_ordering, allocate the
 * workspace for max_batch sequences, and return a handle.
 * The weight tensors must stay valid and unchanged while the handle lives: some paths read
 * them directly, others read device copies made here (token_embd in token_ordering order;
 * per-CTA weight images of the one-sequence grid path; for max_batch >= 2 in bf16, the
 * stacked [gate ; up] and [post_proj ; centroids] pairs of the tensor-core path).
 * config/weights: host structs (copied). target_embed: device [V][bb] model dtype, the
 * target's input embedding table that embed(last_token) reads ("Gemma 4 drafter
 * explained", "Target Activations": the input table is shared with the target).
 * Errors: INVALID_ARG (NULL pointer, bad field), UNSUPPORTED_SHAPE, BAD_ORDERING
 * (vocab % n_centroids != 0 -- "Gemma 4 Assistant tensor inventory", "GGUF / converter
 * layout" verification note -- or ordering not a permutation of 0..V-1), CUDA.
 * Synchronises the current device. */
MTP_API int mtp_init_weights(const mtp_config *config, const mtp_weights *weights,
                     const void *target_embed, mtp_handle **out);

/* Run a draft block: n_draft drafter steps for B independent sequences.
 * Step 1 consumes hidden[b] (the target's last hidden state) and last_token[b]; step i+1
 * consumes step i's greedy token and its post-projected hidden state, kept in fp32 without
 * rounding ("Gemma 4 Assistant 使用指南", section 二.3; "Gemma 4 drafter explained",
 * "Target Activations"). Each step: pre_projection of [hidden ; embed(token)], every block
 * (norm, Q projection, q_norm, RoPE at pos[b], attention over the shared K of the block's
 * type -- sliding blocks attend the last `window` keys, full blocks all ctx_len[b] keys --,
 * o projection, post-attention norm + residual, gated GELU-tanh MLP, post-FFN norm +
 * residual, layer_scalar), output_norm, post_projection, and the LM head (centroid head:
 * top_k centroids, gather of their token_ordering ids, sparse logits, argmax; or the
 * dense tied head + argmax).
 *   hidden      device [B][bb] model dtype
 *   last_token  device [B] int32 in [0, V)
 *   kv_sliding  host struct, required when any block is sliding (else may be NULL)
 *   kv_full     host struct, required when any block is full (else may be NULL)
 *   pos         device [B] int32: the constant position id of the block
 *   out_tokens  device [B][n_draft] int32
 *   out_hidden  device [B][n_draft][bb] fp32 post_projection output of every step, or NULL
 * Errors: INVALID_ARG (NULL hidden / token / needed KV, B outside [1, max_batch],
 * n_draft < 1, bad stride), UNSUPPORTED_SHAPE, CUDA. */
MTP_API int mtp_draft_block(mtp_handle *h, const void *hidden, const int32_t *last_token,
                    const mtp_kv *kv_sliding, const mtp_kv *kv_full, const int32_t *pos,
                    int32_t B, int32_t n_draft, int32_t *out_tokens, float *out_hidden,
                    void *stream);

/* LM head on given final-normed hidden states (testing / sampling entry point).
 * Centroid head ("Gemma 4 Assistant tensor inventory", "Centroid / ordered embeddings LM
 * head", steps 1-5): centroid logits, top_k centroids, gather of their ids, sparse logits,
 * and -- when out_logits != NULL -- the full row filled with -1e30f with the sparse logits
 * scattered at their ids (or the other mask of mtp_set_logit_mask). Dense head
 * (use_ordered_embeddings == 0): all V logits.
 *   y             device [B][H] fp32, used as given (never rounded to bf16)
 *   out_logits    device [B][V] fp32 or NULL
 *   out_token     device [B] int32 (argmax, lowest id on ties)
 *   out_centroids device [B][top_k] int32 selected centroids, best first (ties: lower
 *                 index first), or NULL; must be NULL for the dense head
 * Errors: INVALID_ARG, CUDA. */
MTP_API int mtp_centroid_head(mtp_handle *h, const float *y, int32_t B, float *out_logits,
                      int32_t *out_token, int32_t *out_centroids, void *stream);

/* Select the mask of the materialised rows of mtp_centroid_head on this handle (default
 * MTP_MASK_NEG_1E30). With MTP_MASK_MIN_MINUS_ONE, after the sparse logits are scattered,
 * every entry still holding the -1e30f fill becomes min over the sequence's candidate
 * logits minus 1 (fp32). A candidate logit equal to -1e30f exactly would be treated as
 * fill. Has no effect on the dense head or on mtp_draft_block (which materialises no row).
 * Errors: INVALID_ARG (NULL handle, unknown mode). */
MTP_API int mtp_set_logit_mask(mtp_handle *h, int32_t mode);

/* Select the sparse-head traversal (enum mtp_sparse_head) of mtp_draft_block's batched paths
 * (1 and 5; the persistent path 2 always gathers per sequence) and of mtp_centroid_head on
 * this handle; default MTP_HEAD_AUTO. Cluster-major reads the token_embd copy in
 * token_ordering order that init makes for every centroid head, and falls back to the
 * per-sequence gather where its shared-memory plan does not fit (about max_batch x hidden x 4
 * bytes of y plus a 4-stage ring of 32 KB must stay under 227 KB). It changes no output beyond
 * the fp32 summation order of a logit. No effect on the dense head or the single-sequence
 * paths. Errors: INVALID_ARG (NULL handle, unknown mode). */
MTP_API int mtp_set_sparse_head(mtp_handle *h, int32_t mode);

/* Greedy accept-prefix verification ("Gemma 4 drafter explained", "What is Speculative
 * Decoding?"): t_i = argmax of target row i (lowest id on ties); accept_len[b] = the
 * largest m with draft[b][i] == t_i for all i < m; out_tokens[b] = draft[b][0..m) followed
 * by t_m (the target's correction, or its extra token when m == n), then -1 padding.
 * Rows after the first disagreement never change the result. Rows are read in batches of up
 * to five (copied together into shared memory); batches after the one holding the first
 * disagreement are not read. accept_len[b] = -1 reports that a bounded device wait on those
 * copies gave up (not expected on a working GPU); that sequence's undecided rows stay -1.
 *   target_logits device [B][n+1][V] bf16
 *   draft         device [B][n] int32
 *   accept_len    device [B] int32
 *   out_tokens    device [B][n+1] int32
 * Errors: INVALID_ARG (NULL, B < 1, n < 0, V < 1, V % 8 != 0), CUDA. */
MTP_API int mtp_verify_greedy(const void *target_logits, const int32_t *draft, int32_t B, int32_t n,
                      int32_t V, int32_t *accept_len, int32_t *out_tokens, void *stream);

/* Sampled verification at temperature T (the pages give the accept-until-disagreement
 * structure, "Gemma 4 drafter explained", "What is Speculative Decoding?", and note that the
 * accept rate varies with temperature, "Gemma 4 Multi-Token Prediction (MTP) drafter",
 * "Status"; they give no stochastic rule). Speculative sampling with the drafter's proposal
 * a point mass on each drafted token: p_i = softmax(target row i / T); draft i is accepted
 * while u_accept[b][i] < p_i(draft[b][i]); at the first rejection the emitted token is the
 * inverse-CDF sample, over increasing ids, of p_i without the drafted token (renormalised)
 * at u_sample[b][i]; when all n drafts are accepted the extra token is the sample of p_n at
 * u_sample[b][n]. The emitted tokens are distributed as sampling from the target at T.
 * T = 0 is mtp_verify_greedy (the uniforms are not read). Decisions are taken in fp32; a
 * uniform within about 1e-6 (relative) of a decision boundary may fall either way.
 *   target_logits device [B][n+1][V] bf16
 *   draft         device [B][n] int32
 *   temperature   host float, finite, >= 0
 *   u_accept      device [B][n] fp32 uniforms in [0, 1) (may be NULL when n == 0)
 *   u_sample      device [B][n+1] fp32 uniforms in [0, 1)
 *   accept_len    device [B] int32
 *   out_tokens    device [B][n+1] int32 (-1 padded after the emitted token)
 * Rows after the first rejection are not read. Asynchronous on `stream`; caller-owned
 * buffers. Errors: INVALID_ARG (NULL, B < 1, n < 0, V < 1, V % 8 != 0, T < 0 or not
 * finite), CUDA. */
MTP_API int mtp_verify_sample(const void *target_logits, const int32_t *draft, int32_t B, int32_t n,
                              int32_t V, float temperature, const float *u_accept,
                              const float *u_sample, int32_t *accept_len, int32_t *out_tokens,
                              void *stream);

/* Log probabilities of given tokens, with the rows' entropies and most probable tokens, in one pass
 * over the logits (what a serving program answers with beside the tokens: rows of a prompt, or the
 * target's rows of a verified draft block with the emitted tokens). The pages have no counterpart.
 * With p = softmax(row / temperature): logprob = ln p[token], entropy = -sum_i p_i ln p_i (0 ln 0 = 0),
 * top_ids the top_k tokens of the largest logits in descending order (ties: lower id first) and
 * top_logprobs their ln p. fp32 arithmetic from the logits as they are. -inf is a logit of
 * probability 0, also among the top_k where fewer are above it; a log probability below fp32's range is -inf. A row without a softmax (a NaN, a
 * +inf, or nothing above -inf) gets NaN for its values and -1 for its ids; a token outside [0, V)
 * gets a logprob of NaN.
 *   logits       device [rows][V], dtype (enum mtp_dtype), row_stride elements apart (>= V; any
 *                alignment of the type)
 *   token        device [rows] int32 (may be NULL when logprob is)
 *   temperature  host float in [1e-30, 1e30]
 *   logprob, entropy  device [rows] fp32, or NULL
 *   top_ids, top_logprobs  device [rows][top_k] int32 and fp32 (may be NULL when top_k == 0)
 *   workspace    16-byte aligned, of mtp_token_logprobs_workspace bytes (0 where rows are many), not
 *                shared by calls that may overlap
 * rows <= 2^24, V <= 2^30, top_k <= MTP_MAX_TOP_K. Outputs are buffers of their own. May be captured into
 * CUDA graphs. Errors: INVALID_ARG, CUDA. */
#define MTP_MAX_TOP_K 32
MTP_API int mtp_token_logprobs(const void *logits, int32_t dtype, int64_t row_stride, const int32_t *token,
                               int32_t rows, int32_t V, float temperature, int32_t top_k, float *logprob,
                               float *entropy, int32_t *top_ids, float *top_logprobs, void *workspace,
                               int64_t workspace_bytes, void *stream);
MTP_API int mtp_token_logprobs_workspace(int32_t dtype, int32_t rows, int32_t V, int32_t top_k, int64_t *bytes);

/* Size of the static device scratch of mtp_centroid_head_noalloc (1 MiB). */
#define MTP_NOALLOC_SCRATCH_BYTES (1u << 20)

/* The centroid LM head of mtp_centroid_head for callers that cannot allocate device memory:
 * code running where cudaMalloc is unavailable or forbidden, such as inside a region being
 * captured into a CUDA graph, an allocator callback, or a runtime that owns every device
 * allocation and hands out only the caller's tensors. The pages have no counterpart; this is
 * a library convenience. It needs no handle (creating one allocates a workspace): the head's
 * tensors are passed directly, and its scratch lives in a fixed device array of
 * MTP_NOALLOC_SCRATCH_BYTES that every GPU loading the library holds until the process exits.
 * Results equal mtp_centroid_head's on the same tensors. token_ordering is not validated
 * here (mtp_init_weights checks it is a permutation; this entry has no handle): a candidate
 * whose id lies outside [0, vocab) is skipped, neither read nor written.
 *   y              device [B][hidden] fp32 final-normed hidden states
 *   centroids      device [n_centroids][hidden], dtype (MTP_DTYPE_BF16 or MTP_DTYPE_F32)
 *   token_ordering device [vocab] int32, a permutation viewed [n_centroids][vocab/n_centroids]
 *   token_embd     device [vocab][hidden], dtype
 *   out_logits     device [B][vocab] fp32 (-1e30 outside the selected clusters) or NULL
 *   out_token      device [B] int32;  out_centroids device [B][top_k] int32 or NULL
 * Scratch needed: 4*B*(n_centroids + top_k + hidden) + 8*B bytes, each part rounded up to 256;
 * larger requests fail with MTP_ERR_INVALID_ARG and a message giving both sizes. The first
 * call on a device looks up the array's device address (cudaGetSymbolAddress); make that
 * first call before any stream capture. Calls share the array and keep its last contents:
 * calls that overlap on the GPU (concurrent streams, several host threads) race. No
 * cudaMalloc, cudaFree or allocating library routine is called.
 * Errors: INVALID_ARG, BAD_ORDERING (vocab % n_centroids != 0), CUDA. */
MTP_API int mtp_centroid_head_noalloc(const float *y, const void *centroids, const int32_t *token_ordering,
                                      const void *token_embd, int32_t dtype, int32_t B, int32_t hidden,
                                      int32_t n_centroids, int32_t top_k, int32_t vocab, float *out_logits,
                                      int32_t *out_token, int32_t *out_centroids, void *stream);

/* Synchronise the device and return the handle's device-side status word: MTP_OK,
 * MTP_ERR_TIMEOUT when a bounded device wait of a previous call gave up, or
 * MTP_ERR_INVALID_ARG when a device-resident input was out of range (a last_token outside
 * [0, V): embedding row 0 was read instead). The word is cleared by this call. Also reports
 * a pending CUDA error as MTP_ERR_CUDA. */
MTP_API int mtp_get_status(mtp_handle *h);

/* Testing only: failure injection on the host side of a device wait. With
 * skip_arrival_cta >= 0, that CTA of the persistent draft-block kernel (path 2) does not
 * arrive at the first grid barrier of the next launches; every CTA's bounded wait then
 * gives up, the call's status word reads MTP_ERR_TIMEOUT (mtp_get_status), the kernel
 * returns early without a fault, and the handle stays usable. spin_limit_cycles > 0 replaces
 * the bound of the device waits of the phase and persistent paths (default about 2 s of
 * clock64 cycles). On the grid path (7), CTA skip_arrival_cta does not publish its slice of
 * the first all-reduce of the next launches; on the streamed cluster path (6), CTA
 * skip_arrival_cta of the cluster sends none of its rows in the launch's first exchange; on
 * the tensor-core path (5), CTA skip_arrival_cta of the first projection GEMM issues no copy
 * for its last k stage; in a paged draft block (paths 1 and 5), the first layer's tensor-core
 * attention looks up no page of sequence skip_arrival_cta. Each has the same timeout outcome, and
 * the bound applies to the waits of these paths too. (-1, 0) restores the defaults. No other path is affected.
 * Errors: INVALID_ARG (NULL handle, skip_arrival_cta < -1, spin_limit_cycles < 0). */
MTP_API int mtp_set_debug(mtp_handle *h, int32_t skip_arrival_cta, int64_t spin_limit_cycles);

/* Select the implementation of mtp_draft_block: 0 = automatic, 1 = one kernel per phase,
 * 2 = persistent whole-block kernel with grid barriers, 5 = one kernel per phase with every
 * projection (and the dense tied head) as a tcgen05 tensor-core GEMM (bf16, max_batch <= 64;
 * mtp_init_weights keeps the tensor maps and a staging buffer of 3 * roundup(max_batch, 32) *
 * max input width bf16), 6 = streamed-tile cluster kernel for one sequence (one 16-CTA
 * cluster; every projection on tensor cores from weight tiles packed once into one stream
 * per CTA (see below), about the size of all projection weights; vectors exchanged
 * register-to-peer in distributed shared memory; bf16 centroid-head shapes within its
 * limits, one KV head, V = K, 16-byte aligned hidden and K rows), 7 = grid kernel for one
 * sequence (every co-resident thread-block cluster of the GPU; each projection split over
 * all CTAs by rows or by input columns, the split weights and the attended K resident in
 * shared memory -- K of long contexts is read from global memory instead --, vectors
 * exchanged by all-gathers and all-reduces over distributed shared memory and epoch-tagged
 * global mailboxes; bf16 centroid-head shapes with hidden in {64, 128, 256, 512},
 * power-of-two head dims and vocab / n_centroids, whose per-CTA share fits shared memory,
 * V = K, 16-byte aligned K rows; mtp_init_weights packs the per-CTA weight images, about the
 * size of all projection weights). Paths 3 and 4 (earlier single-sequence kernels) no longer
 * exist and are rejected. Automatic picks 7 for B = 1 when available, else 6; 5 for B >= 2
 * when available; else 2 when co-resident, else 1. Results agree within the precision
 * contract.
 * The streamed cluster path's weight streams are built (device memory about the size of the
 * projection weights, packed once; the call synchronises) when path 6 is first selected, or
 * by mtp_init_weights when the grid path cannot serve the handle and path 6 is the automatic
 * one-sequence path.
 * Errors: INVALID_ARG (NULL handle, path outside {0, 1, 2, 5, 6, 7}), CUDA (building the
 * path-6 streams); a forced path the call cannot use makes mtp_draft_block return
 * UNSUPPORTED_SHAPE. */
MTP_API int mtp_set_path(mtp_handle *h, int32_t path);

/* ---------------------------------------------------------------- paged key cache
 *
 * Serving programs hold the target's K (and V) in pages of P tokens; the pages of the framework
 * describe the shared K only as one tensor per attention type, so these entry points are the
 * library's own. The key of sequence b at position t lies in physical page
 * block_table[b * table_stride + t / P] at offset t % P: element (page, t % P, kv_head, i) is
 * k[page * stride_page + (t % P) * stride_t + kv_head * stride_h + i], so token-major
 * ([n_pages][P][n_kv][d]) and head-major ([n_pages][n_kv][P][d]) caches, and K and V in one
 * allocation, are strides. A slot is page * P + offset.
 * Limits: dtype bf16 or fp32; head_dim <= 512, a multiple of 16 bytes; page_size a power of two
 * <= 256; n_pages * page_size and max_pages * page_size <= 2^30 (element offsets are 64-bit);
 * 16-byte aligned pointers; strides >= head_dim and multiples of 16 bytes. A block_table entry
 * outside [0, n_pages) is no page: its keys are left out (and never read). ctx_len is clamped to
 * [0, max_pages * page_size] on the device. Rows of a page at or past ctx_len are never used,
 * whatever they hold.
 * Except for the draft block at the end, these calls keep no state, need no handle, use the
 * current device and may be captured into CUDA graphs. Scratch is the caller's `workspace`
 * (16-byte aligned, not shared by calls that may overlap), sized by the *_workspace call with the
 * same arguments. */
typedef struct mtp_paged_kv {
  void *k;                    /* device, model dtype */
  void *v;                    /* device, the layout of k, or NULL (V = K) */
  const int32_t *block_table; /* device [B][table_stride] (not read by mtp_page_append) */
  const int32_t *ctx_len;     /* device [B]: valid keys (not read by mtp_page_append) */
  int8_t *codes;              /* device [n_pages][n_kv][head_dim] page summaries, or NULL */
  float *scales;              /* device [n_pages][n_kv], or NULL (with codes) */
  int64_t stride_page, stride_t, stride_h; /* elements */
  int64_t table_stride;       /* entries between sequences (>= max_pages) */
  int32_t n_pages;            /* physical pages */
  int32_t page_size;          /* P */
  int32_t max_pages;          /* logical pages of a sequence (columns of block_table used) */
  int32_t n_kv_head, head_dim;
  int32_t dtype;              /* enum mtp_dtype */
} mtp_paged_kv;

/* Block tables and slot maps from request lengths. Sequence b holds old_len[b] tokens in
 * ceil(old_len[b] / P) pages and shall hold new_len[b]:
 *   growers   (new > old) take ceil(new / P) - ceil(old / P) pages from the head of the ring of
 *             free pages, in batch order, appended to their block_table rows. A grower is granted
 *             while the sums of pages and of new tokens over the growers up to it fit ring_state's
 *             count and max_tokens; the first that does not fit and every later grower are denied
 *             and keep their length;
 *   shrinkers (new < old; 0 ends a sequence) return the pages behind ceil(new / P) to the ring's
 *             tail; these can be taken from the next call on;
 *   a new_len outside [0, max_pages * P] is denied.
 * Entries of block_table behind a sequence's pages are left as they were.
 *   old_len, new_len device [B] int32;  block_table device [B][table_stride], updated in place
 *   free_ring   device [n_pages] int32, updated in place: the free pages are
 *               free_ring[(head + i) % n_pages], i < count
 *   ring_state  device [2] int32: head, count
 *   len_out     device [B] int32: length after the call
 *   slot_map    device [max_tokens] int32: the slots of the new tokens, sequence after sequence;
 *               -1 behind the last (NULL only when max_tokens == 0); 16-byte aligned
 *   cu_new      device [B + 1] int32: sequence b's new tokens are [cu_new[b], cu_new[b + 1])
 *   state_out   device [2] int32: the ring's head and count after the call
 *   status      device [4] int32: new tokens, pages taken, pages returned, denied sequences
 * len_out and state_out must not be old_len / new_len and ring_state (the inputs stay readable,
 * so the call can be repeated). B <= 8192. Errors: INVALID_ARG, UNSUPPORTED_SHAPE, CUDA. */
MTP_API int mtp_page_plan(const int32_t *old_len, const int32_t *new_len, int32_t B, int32_t *block_table,
                          int64_t table_stride, int32_t max_pages, int32_t *free_ring, int32_t n_pages,
                          const int32_t *ring_state, int32_t page_size, int32_t max_tokens, int32_t *len_out,
                          int32_t *slot_map, int32_t *cu_new, int32_t *state_out, int32_t *status, void *stream);

/* Writes T rows into their slots: row t of k_new (and of v_new when the cache has a V) to slot
 * slot_map[t]; rows whose slot is outside [0, n_pages * P) are skipped. When the cache has
 * summaries, every page whose last slot is written gets its summary from all P rows it then
 * holds: per KV head m = the mean key in fp32, scale = fl32(max |m| * fl32(1 / 127)),
 * codes = rint(fl32(m / scale)); a mean that is not finite gives scale NaN and codes 0. The mean
 * of a bf16 dimension whose non-zero values lie within 2^24 of one another is exact, rounded once,
 * whatever the order of the rows and calls; otherwise it is off by at most 2^-24 of itself and
 * P^2 2^-48 of the dimension's largest value (and, from fp32 values below 2^-118, 2^-142). A slot
 * may occur once in slot_map; T <= 2^30.
 *   k_new, v_new device rows of [n_kv][head_dim], model dtype, row_stride_k / row_stride_v
 *                elements apart (>= n_kv * head_dim, multiples of 16 bytes), not in the cache
 *   slot_map     device [T] int32
 * Errors: INVALID_ARG, UNSUPPORTED_SHAPE, CUDA. */
MTP_API int mtp_page_append(const mtp_paged_kv *kv, const void *k_new, const void *v_new, int64_t row_stride_k,
                            int64_t row_stride_v, const int32_t *slot_map, int32_t T, void *stream);

/* Forks of sequences over shared pages (n samples of one prompt, the beams of a search). Fork i makes
 * sequence dst[i] a copy of the first length[i] tokens of sequence src[i]: the entries of the complete
 * pages are copied from block_table row src[i] to row dst[i] (from then on both sequences hold these
 * pages), and where length[i] % P != 0 a page is taken from the head of the ring of free pages, gets the
 * rows [0, length[i] % P) of src[i]'s page (k and v) and becomes the next entry. A sequence forked onto
 * itself (src[i] == dst[i]) is cut to length[i] with a partial page of its own. Forks are granted in
 * order while the pages taken fit ring_state's count; the first that does not fit and every later one
 * are denied, as are forks whose src or dst is outside [0, B) or length outside [0, ctx_len[src]],
 * those whose dst an earlier one has, and those whose src is the dst of another one. Denied sequences
 * stay as they are. Pages that dst held before are not returned: mtp_page_collect does that.
 * Sharing pages asks two things of a program: a sequence that holds shared pages returns pages with
 * mtp_page_collect, not as a shrinker of mtp_page_plan; and rows are appended behind complete pages or
 * into a partial page of the sequence's own, so after a cut inside a shared page the sequence is
 * forked onto itself first.
 *   kv           block_table is updated in place; k and v get the partial pages' rows
 *   src, dst, length  device [n] int32;  free_ring device [n_pages] int32;  ring_state device [2] int32
 *   len_out      device [B] int32: every sequence's length after the call
 *   state_out    device [2] int32: the ring's head and count after the call
 *   status       device [4] int32: forks granted, pages taken, pages shared, forks denied
 * len_out and state_out are buffers of their own, so that the call can be repeated. B, n <= 8192.
 * Errors: INVALID_ARG, UNSUPPORTED_SHAPE, CUDA. */
MTP_API int mtp_page_fork(const mtp_paged_kv *kv, int32_t B, const int32_t *src, const int32_t *dst,
                          const int32_t *length, int32_t n, const int32_t *free_ring, const int32_t *ring_state,
                          int32_t *len_out, int32_t *state_out, int32_t *status, void *stream);

/* The free pages of a cache from its block tables alone: pages that are an entry of no sequence's
 * first ceil(ctx_len / P) become the ring of free pages, in increasing order from its beginning (head
 * 0; entries of free_ring behind them are left as they were). With table_out the held pages are also
 * moved into the front of the pool: the held pages from the first `used` ones on, in increasing order,
 * take the free places in front, in increasing order, with their rows (k and v) and summaries;
 * table_out gets every sequence's entries under the new numbers (-1 for entries that are no page and
 * behind a sequence's pages), and the ring the pages used .. n_pages - 1. Their old contents stay, so
 * a call with a table_out of its own can be repeated; a program then reads the new table.
 *   free_ring  device [n_pages] int32
 *   table_out  device [B][table_out_stride] int32: NULL, block_table itself (of the same stride) or a
 *              buffer of its own
 *   state_out  device [2] int32: the ring's head and count
 *   status     device [4] int32: pages held (`used`), pages free, pages moved, entries of held
 *              positions that are no page
 * B <= 2^20. Errors: INVALID_ARG (workspace too small included), UNSUPPORTED_SHAPE, CUDA. */
MTP_API int mtp_page_collect(const mtp_paged_kv *kv, int32_t B, int32_t *free_ring, int32_t *table_out,
                             int64_t table_out_stride, int32_t *state_out, int32_t *status, void *workspace,
                             int64_t workspace_bytes, void *stream);
MTP_API int mtp_page_collect_workspace(const mtp_paged_kv *kv, int32_t compact, int64_t *bytes);

/* Attention of one new token per sequence over the paged cache, split over the cache's length
 * and joined: out[b][h] = sum_j p_j v_j, p = softmax(scale q[b][h] . k_j) over the attended
 * positions: [0, L), the last `window` of them when window > 0, and with `pages` only those in
 * the listed logical pages of the head's KV head (entries outside the sequence's pages are
 * skipped; a page listed twice counts twice). fp32 arithmetic; bf16 keys enter exactly. A
 * sequence with nothing to attend gets out 0 and lse -inf. What is not attended may hold anything.
 * Where an attended row or the query is not finite, or a score leaves the range of fp32, the
 * outputs that it reaches are NaN, infinite, or those without the keys of score -inf; a sequence
 * whose every attended key scores -inf gets NaN. So do the outputs concerned when a device wait
 * gives up after about 2 s (mtp_draft_block_paged reports that through mtp_get_status, too).
 * Query head h reads KV head h / (n_head / n_kv_head).
 *   q         device [B][n_head][head_dim] fp32
 *   pages     device [B][n_kv_head][n_list] int32 or NULL
 *   scale     softmax scale, 0 -> 1 / sqrt(head_dim)
 *   out       device [B][n_head][head_dim] fp32, not over q
 *   lse       device [B][n_head] fp32 log of the sum of exponentials, or NULL
 * Errors: INVALID_ARG (workspace too small included), UNSUPPORTED_SHAPE, CUDA. */
MTP_API int mtp_paged_attention(const mtp_paged_kv *kv, const float *q, int32_t B, int32_t n_head, int32_t window,
                                float scale, const int32_t *pages, int32_t n_list, float *out, float *lse,
                                void *workspace, int64_t workspace_bytes, void *stream);
MTP_API int mtp_paged_attention_workspace(const mtp_paged_kv *kv, int32_t B, int32_t n_head, int32_t n_list,
                                          int64_t *bytes);

/* Attention of a chunk of new tokens per sequence over the paged cache, which holds their keys
 * already: the last n_b = cu_new[b + 1] - cu_new[b] of the ctx_len[b] tokens of sequence b are the
 * rows cu_new[b] .. cu_new[b + 1] - 1 of q and out (mtp_page_plan's cu_new; slices of a prompt, or
 * the tokens of a draft block to verify). The row of position t attends the keys j <= t of its
 * sequence, with window > 0 those with j > t - window: out = sum_j p_j v_j, p = softmax(scale q . k_j).
 * q, out and the cache have the model dtype; an output is rounded to it once. fp32 models are computed
 * in fp32. For bf16 the products are exact, sums, maxima and exp-sums are fp32, and on tensor cores
 * (head_dim 128, 256 or 512, page_size >= 8) the probabilities enter the second product as bf16, off by
 * at most 2^-8 of themselves each; lse has their fp32 sum.
 * A row with nothing to attend (a sequence that holds fewer tokens than its new ones, pages that are
 * none) gets out 0 and lse -inf. What a row does not attend may hold anything and does not reach it;
 * where a row's query or an attended key or value is not finite, or a score leaves the range of
 * fp32, its outputs are NaN, infinite, or those without the keys of score -inf (a row whose every
 * attended key scores -inf gets NaN). A device wait that gives up after about 2 s leaves NaN.
 * cu_new must not decrease; its entries are clamped to [0, T] on the device. Rows of out and lse
 * outside [cu_new[0], cu_new[B]) are left as they were.
 *   q         device, token t and head h at q + t * q_stride + h * head_dim, 16-byte aligned
 *   q_stride  elements between tokens (n_head * head_dim to 2^38, a multiple of 16 bytes)
 *   cu_new    device [B + 1] int32
 *   T         rows of out and lse; T <= 2^24 and T * n_head <= 2^26
 *   out       device [T][n_head][head_dim], not over q
 *   lse       device [T][n_head] fp32 log of the sum of exponentials, or NULL
 * Errors: INVALID_ARG (workspace too small included), UNSUPPORTED_SHAPE, CUDA. */
MTP_API int mtp_paged_attention_chunk(const mtp_paged_kv *kv, const void *q, int64_t q_stride, const int32_t *cu_new,
                                      int32_t B, int32_t T, int32_t n_head, int32_t window, float scale, void *out,
                                      float *lse, void *workspace, int64_t workspace_bytes, void *stream);
MTP_API int mtp_paged_attention_chunk_workspace(const mtp_paged_kv *kv, int32_t B, int32_t T, int32_t n_head,
                                                int64_t *bytes);
/* For tests of the device waits of mtp_paged_attention_chunk, as mtp_set_debug is for a handle's: in the
 * calling host thread's later calls on tensor cores no page of sequence skip_sequence is looked up, so
 * that the waits for it run out, and spin_limit_cycles > 0 replaces their bound. The sequence's rows,
 * and those of others in the same CTAs, then get NaN; later calls are not affected. (-1, 0) restores the
 * defaults. Errors: INVALID_ARG (skip_sequence < -1, spin_limit_cycles < 0). */
MTP_API int mtp_set_chunk_debug(int32_t skip_sequence, int64_t spin_limit_cycles);

/* Pages a query attends, by a cheap score of each page: per query head the step
 * s = fl32(max |q| * fl32(1 / 127)) and codes c = rint(fl32(q / s)) (all 0 when q is not
 * finite), the page's score per KV head = max over its query heads of
 * fl32(fl32((c . codes) * s) * scale) with the integer dot product. A page of scale NaN scores
 * +inf (a page whose keys are not finite is read), a block_table entry that is no page -inf; the
 * first keep_first and the last keep_last pages of a sequence come before all others. sel[b][g]
 * lists the n_select pages of the highest scores (ties: lower page) in increasing order, -1 behind
 * them when the sequence has fewer. Only complete pages need a summary when keep_last >= 1.
 *   q    device [B][n_head][head_dim] fp32;  sel device [B][n_kv_head][n_select] int32
 * Errors: INVALID_ARG (keep_first < 0, keep_last < 1, n_select < keep_first + keep_last, no
 * summaries, workspace too small), UNSUPPORTED_SHAPE, CUDA. */
MTP_API int mtp_page_select(const mtp_paged_kv *kv, const float *q, int32_t B, int32_t n_head, int32_t n_select,
                            int32_t keep_first, int32_t keep_last, int32_t *sel, void *workspace,
                            int64_t workspace_bytes, void *stream);
MTP_API int mtp_page_select_workspace(const mtp_paged_kv *kv, int32_t B, int64_t *bytes);

/* mtp_draft_block over paged caches: the same drafter steps, with every block's attention read
 * through the block tables (sliding blocks attend the last `window` keys). With n_select > 0 the
 * full-attention blocks attend, per KV head, the n_select pages that mtp_page_select picks for the
 * block's queries (keep_first and keep_last always among them): fewer keys read per draft step at
 * the price of a lower accept rate; what is emitted after verification is the target's either way.
 * n_select == 0 attends every page. dtype, n_kv_head and head_dim of the caches are the drafter's;
 * max_pages * page_size may exceed mtp_config.max_ctx.
 * Runs on path 5 when the handle has it, else 1 (mtp_set_path 1 or 5 selects; other forced paths
 * are refused), replayed as a CUDA graph while the same arguments come again.
 *   workspace  device scratch of mtp_draft_block_paged_workspace bytes, 16-byte aligned
 * Errors: INVALID_ARG, UNSUPPORTED_SHAPE, CUDA. */
MTP_API int mtp_draft_block_paged(mtp_handle *h, const void *hidden, const int32_t *last_token,
                                  const mtp_paged_kv *kv_sliding, const mtp_paged_kv *kv_full, const int32_t *pos,
                                  int32_t B, int32_t n_draft, int32_t n_select, int32_t keep_first, int32_t keep_last,
                                  int32_t *out_tokens, float *out_hidden, void *workspace, int64_t workspace_bytes,
                                  void *stream);
MTP_API int mtp_draft_block_paged_workspace(mtp_handle *h, const mtp_paged_kv *kv_sliding, const mtp_paged_kv *kv_full,
                                            int32_t B, int32_t n_select, int64_t *bytes);

/* Free the workspace and the handle (synchronises). NULL is ignored. */
MTP_API void mtp_destroy(mtp_handle *h);

/* Text of the last error raised on the calling thread ("" when none). */
MTP_API const char *mtp_last_error(void);

#ifdef __cplusplus
}
#endif

#endif /* MTP_H_ */
