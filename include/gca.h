/*
 * gca.h -- C ABI of the Grouped Cross Attention (GCA) hot path on GB300.
 *
 * GCA is defined in "Efficient Length-Generalizable Attention via Causal
 * Retrieval for Long-Context Language Modeling" (Hu, Teng, Zhao, Wu, Tu;
 * ICML 2025, arXiv 2410.01651).  Each chunk of S tokens has one landmark
 * vector; the landmark of chunk c-1 scores earlier chunks, the top-k are
 * retrieved for chunk c, every token of chunk c attends separately to each
 * retrieved chunk (stage 1) and the per-chunk outputs are summed with the
 * softmaxed relevance scores as weights (stage 2).
 *
 * Conventions shared by every entry point
 *  - Tensor arguments are DEVICE pointers owned by the caller, except where
 *    an argument says "host".  The library allocates no memory and keeps no
 *    state except a per-device status word (see gca_get_status) and the
 *    fixed scratch array of gca_decode_retrieve_noalloc.
 *  - `stream` is a cudaStream_t (NULL = the legacy default stream).  All
 *    work is enqueued asynchronously on it.
 *  - The return value reports argument validation and launch errors.
 *    Errors detected on the device (a bounded wait that ran out, an index
 *    out of range) are recorded in the status word and returned by
 *    gca_get_status().  No call ever traps or aborts the GPU context.
 *  - Layouts are row-major, innermost dimension last.  Token tensors are
 *    [B, tokens, H, d]; the chunk c of a token tensor is tokens cS .. cS+S-1.
 *  - Pointers must be 16-byte aligned.
 *
 * Supported shapes (anything else returns GCA_ERR_UNSUPPORTED):
 *  - dtype GCA_BF16: d in {32, 64, 128}, S in {64, 128} (tensor-core path)
 *  - dtype GCA_F32 : d in {16, 32, 64}, S in {16, 32, 64} (fp32 FFMA path)
 *  - 1 <= topk <= 32, landmark dimension <= 8192, chunks per row <= 16384.
 *  - sliding-window entries: see gca_swa_params_t, gca_swa_sink_params_t and
 *    gca_paged_params_t.
 */
#ifndef GCA_H_
#define GCA_H_

#include <stddef.h>
#include <stdint.h>

#ifdef __cplusplus
extern "C" {
#endif

typedef enum {
    GCA_OK = 0,
    GCA_ERR_INVALID_ARG = 1,   /* null pointer, bad size, misaligned pointer */
    GCA_ERR_UNSUPPORTED = 2,   /* valid but outside the supported shapes     */
    GCA_ERR_WORKSPACE = 3,     /* workspace missing or too small             */
    GCA_ERR_CUDA = 4,          /* a CUDA runtime/driver call failed          */
    GCA_ERR_TIMEOUT = 5,       /* a bounded device-side wait ran out         */
    GCA_ERR_DEVICE_INDEX = 6   /* the device saw an index outside its range  */
} gca_status_t;

typedef enum { GCA_BF16 = 0, GCA_F32 = 1 } gca_dtype_t;

typedef struct {
    int B;                  /* batch rows                                         */
    int Lq;                 /* query tokens per row; a multiple of S (nQ = Lq/S)  */
    int S;                  /* tokens per chunk                                   */
    int H;                  /* heads                                              */
    int d;                  /* head dimension                                     */
    int topk;               /* retrieved chunks per query chunk                   */
    int n_pool_chunks;      /* K/V chunks per row (nP); nQ in training            */
    int landmark_dim;       /* D of the landmark vectors; 0 means H*d             */
    gca_dtype_t dtype;      /* element type of landmarks and all token tensors    */
    int softmax_off_by_one; /* 0: vanilla softmax; 1: denominator 1 + sum         */
    int include_self;       /* 0: candidates kappa < c-1; 1: kappa <= c-1         */
    float score_scale;      /* r = score_scale * l_{c-1}.l_kappa; 0 => 1/sqrt(D)  */
    float attn_scale;       /* logits scale inside a chunk; 0 => 1/sqrt(d)        */
} gca_params_t;

/*
 * gca_score_topk -- causal relevance scoring, top-k and weight softmax.
 * Defines: the rebuttal comment "Cmt 1" (Eq. 1 with one group:
 * r = l_t^T l_k / sqrt(d)); README "Model Architecture" (the landmark of the
 * previous chunk selects the chunks for the next one); rebuttal Q4 (Eq. 3,
 * softmax off by one).
 *   landmarks [B, nC, D] (nC = Lq / S), dtype = params->dtype.
 *   For query chunk c >= 1 with landmark chunk t = c-1, the candidates are
 *   kappa < t (or kappa <= t with include_self).  s = l_t . l_kappa is
 *   accumulated in fp32 (exact for integer landmarks with |s| < 2^24).
 *   Slots are ordered by s descending, then kappa ascending.
 *   idx    [B, nC, topk] int32: retrieved chunk, -1 for an empty slot.
 *   score  [B, nC, topk] fp32: r = score_scale * s (0 for an empty slot).
 *   weight [B, nC, topk] fp32: softmax or off-by-one softmax of the valid r
 *                              (0 for an empty slot).
 */
gca_status_t gca_score_topk(const gca_params_t* params, const void* landmarks,
                            int32_t* idx, float* score, float* weight, void* stream);

/*
 * gca_score_topk_noisy -- gca_score_topk with the training-time exploration
 * of section 3.2 (Gumbel noise is added to the relevance scores before the
 * top-k selection).  The noise is drawn by the caller.
 *   noise [B, nC, nC] fp32: noise[b][c][kappa] perturbs candidate kappa of
 *   query chunk c (entries for kappa outside the candidate set are unused).
 *   The selection key is fl32(fl32(s * score_scale) + noise), rounded step
 *   by step (no fused multiply-add); ties go to the lower chunk index.
 *   score and weight are computed from the clean scores of the selected
 *   chunks, exactly as in gca_score_topk.  Other arguments as gca_score_topk.
 */
gca_status_t gca_score_topk_noisy(const gca_params_t* params, const void* landmarks,
                                  const float* noise, int32_t* idx, float* score, float* weight,
                                  void* stream);

/*
 * gca_fwd -- GCA forward: per-chunk attention (stage 1) and weighted fusion
 * (stage 2).  Defines: README "Model Architecture" (two stages), Figure 1/2,
 * Eq. 2 (the batch form of Figure 2, rebuttal W2); App. B (the forward
 * returns O and the log-sum-exp).
 *   q [B, Lq, H, d]; k, v [B, n_pool_chunks * S, H, d].
 *   idx, weight [B, nQ, topk] as written by gca_score_topk (or by the caller;
 *   entries must be -1 or in [0, n_pool_chunks)).
 *   o   [B, Lq, H, d]: O_t = sum_j weight_j * softmax(attn_scale q_t K_j^T) V_j,
 *       0 for a chunk without a valid slot.  fp32 accumulation.
 *   lse [B, Lq, H, topk] fp32 or NULL: ln sum_s exp(attn_scale q_t.k_s) per
 *       slot, -inf for an empty slot.  Required later by gca_bwd.
 */
gca_status_t gca_fwd(const gca_params_t* params, const void* q, const void* k, const void* v,
                     const int32_t* idx, const float* weight, void* o, float* lse, void* stream);

/* Bytes of device workspace gca_bwd needs for these parameters. */
size_t gca_bwd_workspace_size(const gca_params_t* params);

/*
 * gca_bwd -- gradients of GCA into Q, K, V and the relevance scores.
 * Defines: App. B backward (gradients for Q, K, V and the weights);
 * section 3 and README "Model Architecture" (the retrieval scores receive
 * gradients from the next-token loss through the fusion weights).
 *   Inputs as gca_fwd, plus lse from gca_fwd and dout [B, Lq, H, d].
 *   dq [B, Lq, H, d]; dk, dv [B, n_pool_chunks * S, H, d] are fully
 *   overwritten (chunks that no query retrieved get 0).
 *   dscore [B, nQ, topk] fp32: dLoss/dr for valid slots, 0 for empty ones.
 *   The reduction over the queries that share a retrieved chunk is done in a
 *   fixed order without atomics, so results are bitwise reproducible.
 *   workspace: device buffer of at least gca_bwd_workspace_size() bytes,
 *   256-byte aligned, owned by the caller, contents need not be initialised.
 */
gca_status_t gca_bwd(const gca_params_t* params, const void* q, const void* k, const void* v,
                     const int32_t* idx, const float* weight, const float* lse, const void* dout,
                     void* dq, void* dk, void* dv, float* dscore, void* workspace,
                     size_t ws_bytes, void* stream);

/* Bytes of device workspace gca_landmark_bwd needs. */
size_t gca_landmark_bwd_workspace_size(const gca_params_t* params);

/*
 * gca_landmark_bwd -- gradient into the landmark vectors, closing the loop
 * from the relevance-score gradient (gca_bwd's dscore) to the retriever.
 * Defines: sections 1 and 3 (the retriever learns from the next-token loss
 * through the relevance scores) with r = score_scale * l_{c-1} . l_kappa.
 *   landmarks [B, nC, D], idx [B, nC, topk] (as used in the forward),
 *   dscore [B, nC, topk] fp32 -> dlandmarks [B, nC, D] (params->dtype),
 *   fully overwritten; fp32 accumulation in a fixed order, no atomics.
 *   The selection itself is not differentiated.
 *   workspace: >= gca_landmark_bwd_workspace_size() bytes, 256-byte aligned.
 */
gca_status_t gca_landmark_bwd(const gca_params_t* params, const void* landmarks,
                              const int32_t* idx, const float* dscore, void* dlandmarks,
                              void* workspace, size_t ws_bytes, void* stream);

/* Bytes of device workspace gca_decode_retrieve needs. */
size_t gca_decode_workspace_size(int n_landmarks, int D, int topk);

/*
 * gca_decode_retrieve -- decode-time retrieval: one query landmark against
 * every stored landmark, top-k, softmax.  Defines: section 3.2 and 4.3 /
 * Table 3 (retrieval runs once per chunk of generated tokens).
 *   landmarks [N, D], query_landmark [D], element type `dtype`.
 *   idx/score/weight [topk] as in gca_score_topk (score desc, index asc).
 *   workspace: >= gca_decode_workspace_size() bytes, 256-byte aligned.
 */
gca_status_t gca_decode_retrieve(const void* landmarks, const void* query_landmark, int N, int D,
                                 int topk, gca_dtype_t dtype, int softmax_off_by_one,
                                 float score_scale, int32_t* idx, float* score, float* weight,
                                 void* workspace, size_t ws_bytes, void* stream);

/*
 * gca_decode_retrieve_noalloc -- gca_decode_retrieve for callers that cannot
 * allocate device memory.  The paper has no counterpart: this is a usage
 * variant of the same decode retrieval, not a different operation.
 *   Some callers are handed only their input and output buffers and may not
 *   call cudaMalloc (or any allocating routine) themselves: plugin interfaces
 *   of inference engines, runtimes that plan every device byte at start-up,
 *   and latency-critical loops where an allocation's implicit device
 *   synchronisation is not acceptable.  This entry point needs no workspace
 *   argument: its scratch (a ticket counter, a score bound and the per-CTA
 *   candidate lists)
 *   lives in a file-scope device array of GCA_DECODE_STATIC_SCRATCH_BYTES
 *   bytes that every GPU loading the library holds until the process exits.
 *   Arguments, layouts and results are those of gca_decode_retrieve.
 *   Limits: the scratch holds 32768 (CTA, rank) candidates, i.e. any N with
 *   topk <= 16, or N <= 131072 with topk <= 32; larger requests return
 *   GCA_ERR_WORKSPACE and enqueue nothing.
 *   The first call on each device looks up the array's device address (with
 *   that device current); make that first call before any stream capture.
 *   All calls on a device share the one array, which keeps the previous
 *   call's contents (counter and bound are cleared on the stream before each
 *   launch): calls whose executions overlap on the GPU (other streams, other
 *   host threads) race on it and must be serialised by the caller.
 *   Calls no cudaMalloc, cudaFree or other allocating routine.
 */
#define GCA_DECODE_STATIC_SCRATCH_BYTES (256u + 262144u)
gca_status_t gca_decode_retrieve_noalloc(const void* landmarks, const void* query_landmark, int N,
                                         int D, int topk, gca_dtype_t dtype,
                                         int softmax_off_by_one, float score_scale, int32_t* idx,
                                         float* score, float* weight, void* stream);

/*
 * gca_gather_chunks -- bring the retrieved chunks of an offloaded K/V cache
 * into a compact device pool.  Defines: section 3.2 (past chunks can be
 * offloaded to CPU memory and reloaded when retrieved) and the rebuttal's
 * offload-cost estimate (answer to Q2 of reviewer 3).
 *   src_k, src_v: caches of n_src chunks of chunk_bytes each, in memory the
 *     device can address (device memory, or page-locked host memory, whose
 *     host pointer is device-valid under unified addressing); read-only.
 *   idx [topk] int32 (device): retrieved chunks, -1 for an empty slot.
 *   dst_k, dst_v [topk, chunk_bytes] (device): chunk idx[j] is copied to
 *     slot j; empty slots are zero-filled.
 *   dst_idx [topk] int32 (device): j for a filled slot, -1 for an empty one,
 *     i.e. the idx to pass to gca_fwd together with n_pool_chunks = topk.
 *   chunk_bytes must be a multiple of 16.  An index >= n_src is reported as
 *   GCA_ERR_DEVICE_INDEX and its slot zero-filled.
 */
gca_status_t gca_gather_chunks(const void* src_k, const void* src_v, int n_src,
                               size_t chunk_bytes, const int32_t* idx, int topk, void* dst_k,
                               void* dst_v, int32_t* dst_idx, void* stream);

/*
 * Sliding-window self-attention: the fixed-size window self-attention that a
 * DRT layer runs before its GCA module.  Defines: paper summary section 1
 * (DRT combines the top-k past chunks of GCA with fixed-size sliding-window
 * self-attention) and section 4.1.2 (a 512-token window; the GCA modules are
 * appended after the attention modules).  The norm and residual between the
 * two modules are not part of this library.
 *   Token t of a row attends to the keys max(0, t - window + 1) .. t:
 *   o_t = sum_s softmax_s(attn_scale q_t . k_s) v_s per head.
 */
typedef struct {
    int B, L, H, d;       /* q, k, v, o: [B, L, H, d], d contiguous                   */
    int window;           /* W >= 1 (512 in the paper's model)                          */
    gca_dtype_t dtype;    /* element type of q/k/v/o (GCA_BF16 with d = 64 supported)   */
    float attn_scale;     /* 0 => 1/sqrt(d)                                             */
} gca_swa_params_t;

/*
 * gca_swa_fwd -- sliding-window self-attention forward.
 *   q, k, v, o [B, L, H, d] device pointers (16-byte aligned; o fully written).
 *   lse [B, L, H] fp32 or NULL: ln sum_s exp(attn_scale q_t . k_s) over the
 *   window; needed later by gca_swa_bwd.  fp32 accumulation, bf16 output.
 *   Returns GCA_ERR_UNSUPPORTED for another dtype or head dimension.
 */
gca_status_t gca_swa_fwd(const gca_swa_params_t* params, const void* q, const void* k,
                         const void* v, void* o, float* lse, void* stream);

/* Bytes of device workspace gca_swa_bwd needs. */
size_t gca_swa_bwd_workspace_size(const gca_swa_params_t* params);

/*
 * gca_swa_bwd -- gradients of the sliding-window self-attention: for an
 * upstream gradient dout, with p_ts the forward's probabilities,
 * delta_t = dout_t . o_t and ds_ts = attn_scale p_ts (dout_t . v_s - delta_t):
 *   dq_t = sum_s ds_ts k_s,  dk_s = sum_t ds_ts q_t,  dv_s = sum_t p_ts dout_t.
 *   q, k, v, o, dout, dq, dk, dv [B, L, H, d]; lse [B, L, H] from gca_swa_fwd.
 *   dq, dk, dv are fully overwritten; fp32 accumulation in a fixed order,
 *   no atomics (bitwise reproducible).
 *   workspace: >= gca_swa_bwd_workspace_size() bytes, 256-byte aligned.
 */
gca_status_t gca_swa_bwd(const gca_swa_params_t* params, const void* q, const void* k,
                         const void* v, const void* o, const float* lse, const void* dout, void* dq,
                         void* dk, void* dv, void* workspace, size_t ws_bytes, void* stream);

/*
 * Windowed self-attention with sinks: the sliding-window self-attention above,
 * whose first `sinks` tokens stay visible to every later token.  Token t of a
 * row attends to the keys
 *   V(t) = { s <= t : s > t - window  or  s < sinks },
 *   o_t = sum_{s in V(t)} softmax_s(attn_scale q_t . k_s) v_s per head,
 * with H / Hkv consecutive query heads sharing a key head (query head h reads
 * key head h / (H / Hkv)).  sinks = 0 is the plain window; window >= L is full
 * causal attention.
 * Sizes: B * L * H below 2^31, and up to about 2.1e9 tiles of 128 (token, query
 * head) rows x 128 keys that some of them see (full causal attention over 1M
 * tokens with 16 query heads has 0.54e9), for the gradients about half as many;
 * larger calls return GCA_ERR_UNSUPPORTED.
 */
typedef struct {
    int B, L;             /* rows, tokens per row (any L >= 1)                              */
    int H, Hkv, d;        /* query heads, key heads (H a multiple, H / Hkv <= 128), 64 or 128 */
    int window;           /* W >= 1                                                         */
    int sinks;            /* first tokens that stay visible, >= 0                           */
    gca_dtype_t dtype;    /* GCA_BF16                                                       */
    float attn_scale;     /* 0 => 1/sqrt(d)                                                 */
    int q_stride;         /* elements between consecutive tokens of q; 0 => H*d             */
    int kv_stride;        /* the same of k and v; 0 => Hkv*d.  Both multiples of 8; rows of
                             one batch entry are L * stride elements apart, heads are dense
                             (a slice of a packed q/k/v projection has this form)           */
} gca_swa_sink_params_t;

/* Bytes of device workspace gca_swa_sink_fwd needs (0 for invalid parameters; 256 where the call leaves
   its workspace untouched). */
size_t gca_swa_sink_fwd_workspace_size(const gca_swa_sink_params_t* params);

/*
 * gca_swa_sink_fwd -- forward.
 *   q [B, L, H, d], k, v [B, L, Hkv, d] (token strides as in params);
 *   o [B, L, H, d] dense, fully written.
 *   lse [B, L, H] fp32 or NULL: ln sum_{s in V(t)} exp(attn_scale q_t . k_s);
 *   needed later by gca_swa_sink_bwd.  fp32 accumulation, bf16 output.
 *   workspace: >= gca_swa_sink_fwd_workspace_size() bytes, 256-byte aligned,
 *   contents need not be initialised; calls that may overlap need their own.
 *   K and V must be finite wherever some token of the row sees them.  A token
 *   whose q is not finite gets NaN, in o and lse, and leaves the others alone.
 */
gca_status_t gca_swa_sink_fwd(const gca_swa_sink_params_t* params, const void* q, const void* k,
                              const void* v, void* o, float* lse, void* workspace, size_t ws_bytes,
                              void* stream);

/* Bytes of device workspace gca_swa_sink_bwd needs (0 for invalid parameters). */
size_t gca_swa_sink_bwd_workspace_size(const gca_swa_sink_params_t* params);

/*
 * gca_swa_sink_bwd -- gradients: with p_ts the forward's probabilities,
 * delta_t = dout_t . o_t and ds_ts = attn_scale p_ts (dout_t . v_s - delta_t):
 *   dq_t = sum_s ds_ts k_s,  dk_s = sum_t ds_ts q_t,  dv_s = sum_t p_ts dout_t,
 *   dk and dv summed over the query heads of the key head as well.
 *   q, k, v as in the forward; o, lse from it; dout [B, L, H, d] dense; all of
 *   them finite (a token's NaN may reach the gradients of tokens near it).
 *   dq [B, L, H, d]; dk, dv [B, L, Hkv, d]: dense, fully overwritten; fp32
 *   accumulation in a fixed order, no atomics (bitwise reproducible).
 *   workspace: >= gca_swa_sink_bwd_workspace_size() bytes, 256-byte aligned.
 */
gca_status_t gca_swa_sink_bwd(const gca_swa_sink_params_t* params, const void* q, const void* k,
                              const void* v, const void* o, const float* lse, const void* dout,
                              void* dq, void* dk, void* dv, void* workspace, size_t ws_bytes,
                              void* stream);

/*
 * Paged K/V cache of the window self-attention, for generation: the keys and
 * values of B running sequences live in pages of `page` tokens,
 *   k_cache, v_cache [n_pages, page, Hkv, d],
 * and token s of sequence b is row s % page of page table[b][s / page].
 * A call serves a batch of sequences with any number of new tokens each
 * (none, one, a prompt chunk): the new tokens of sequence b are the rows
 * cu_q[b] .. cu_q[b+1]-1 of the token tensors, and their positions are the last
 * ones of its kv_len[b] tokens (the new ones included).  Rows behind
 * cu_q[B] are neither read nor written.
 *   table [B, table_width], cu_q [B + 1], kv_len [B]: int32, device.  They are
 *   read on the device only, so a captured call follows their contents.
 * A sequence whose entries contradict each other (cu_q decreasing or beyond
 * total_q, more than max_q new tokens, kv_len below 0 or beyond
 * table_width * page) is left out and GCA_ERR_DEVICE_INDEX recorded.  Behind a
 * sequence whose cu_q decreases others could claim its predecessors' rows:
 * gca_paged_attn leaves them all out, gca_paged_append writes a row that is
 * claimed twice for one of the two.
 * Sizes: B up to 65535, B * table_width below 2^31, table_width * page up to 2^29;
 * for gca_paged_attn total_q * H below 2^31, max_q (total_q where it is 0) up to
 * 2^30, and the key tiles of gca_swa_sink_params_t's limit, each sequence counted
 * at the table's whole width or its window.  Larger calls return
 * GCA_ERR_UNSUPPORTED.
 */
typedef struct {
    int B;                /* sequences, >= 1                                                */
    int total_q;          /* rows of the token tensors, >= 0 (0: nothing is enqueued)       */
    int max_q;            /* at least the new tokens of any one sequence; 0 => total_q      */
    int H, Hkv, d;        /* as in gca_swa_sink_params_t                                    */
    int page;             /* tokens per page: 16, 32, 64 or 128                             */
    int n_pages;          /* pages in the cache                                             */
    int table_width;      /* table entries per sequence                                     */
    int window;           /* 0: every earlier token is visible; else as above               */
    int sinks;            /* first tokens that stay visible behind a window                 */
    gca_dtype_t dtype;    /* GCA_BF16                                                       */
    float attn_scale;     /* 0 => 1/sqrt(d)                                                 */
    int q_stride;         /* elements between consecutive tokens of q; 0 => H*d             */
    int kv_stride;        /* the same of k_new and v_new; 0 => Hkv*d; multiples of 8        */
} gca_paged_params_t;

/*
 * gca_paged_append -- write new tokens into the cache.  Takes the attention's
 *   parameters, of which H may be 0.
 *   k_new, v_new [total_q, Hkv, d]; token i of sequence b goes to its position
 *   kv_len[b] - (cu_q[b+1] - cu_q[b]) + i.  Tokens at negative positions and
 *   tokens whose page is not in [0, n_pages) are not written (the latter records
 *   GCA_ERR_DEVICE_INDEX); no other row of the cache changes.  With a window,
 *   tokens that no later token can see (neither sinks nor among the last
 *   window + new tokens) are still written.  Where the table gives two tokens of
 *   the call one row of the cache, that row is left with parts of either.
 */
gca_status_t gca_paged_append(const gca_paged_params_t* params, const void* k_new,
                              const void* v_new, const int32_t* cu_q, const int32_t* kv_len,
                              const int32_t* table, void* k_cache, void* v_cache, void* stream);

/* Bytes of device workspace gca_paged_attn needs (0 for invalid parameters; 256 where the call leaves
   its workspace untouched). */
size_t gca_paged_attn_workspace_size(const gca_paged_params_t* params);

/*
 * gca_paged_attn -- attention of the new tokens over the cache, which already
 * holds their own keys and values (gca_paged_append first): gca_swa_sink_fwd's
 * formula at the tokens' positions.
 *   q [total_q, H, d] -> o [total_q, H, d] dense; lse [total_q, H] fp32 or NULL.
 *   A token at a negative position (kv_len below the number of new tokens)
 *   sees nothing: its output is 0 and its lse -inf.  A token that sees keys and
 *   whose q is not finite gets NaN in both.
 *   Only pages that hold a visible token are looked up, so the table entries of
 *   pages that left the window may be anything.  Such a page outside
 *   [0, n_pages) reads as zeros and records GCA_ERR_DEVICE_INDEX.  Cache rows that
 *   no new token sees (at or behind kv_len, or between the sinks and the window of a
 *   sequence's first new token) may hold anything, NaN included; the others must be
 *   finite.  Sequences may share pages, and a page may stand more than once in a row
 *   of the table.
 *   workspace: >= gca_paged_attn_workspace_size() bytes, 256-byte aligned,
 *   contents need not be initialised; calls that may overlap need their own.
 */
gca_status_t gca_paged_attn(const gca_paged_params_t* params, const void* q, const void* k_cache,
                            const void* v_cache, const int32_t* cu_q, const int32_t* kv_len,
                            const int32_t* table, void* o, float* lse, void* workspace,
                            size_t ws_bytes, void* stream);

/*
 * gca_get_status -- synchronise `stream`, then return and clear the device
 * status word of the current device (GCA_OK if no device-side error was
 * recorded since the last call).
 */
gca_status_t gca_get_status(void* stream);

/* Human-readable name of a status code (static storage). */
const char* gca_status_string(gca_status_t status);

/* Number of kernel launches the most recent successful call on this host
 * thread enqueued (for launch accounting in benchmarks). */
int gca_last_launch_count(void);

#ifdef __cplusplus
}
#endif

#endif /* GCA_H_ */
