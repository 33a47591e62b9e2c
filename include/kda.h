/*
 * kda.h -- C ABI of libkda, the Kimi Delta Attention (KDA) forward pass on B200 (sm_100a).
 *
 * The operator.  Per (sequence, head), with state S in R^{dk x dv}:
 *
 *     S_t = (I - beta_t k_t k_t^T) Diag(alpha_t) S_{t-1} + beta_t k_t v_t^T,    o_t = S_t^T q_t,
 *
 * alpha_t = exp(log_alpha_t) in (0,1)^{dk} (a channel-wise decay on the key axis), beta_t in (0,1)
 * a scalar per token and head.  Source: "Kimi Linear: 표현력과 효율을 높인 어텐션 아키텍처(2025)"
 * (GeekNews topic 31936), section "Kimi Delta Attention의 세밀한 메모리 제어" (Gated DeltaNet's
 * scalar forget gate refined to one rate per feature channel) building on section "선형 어텐션에서
 * Gated DeltaNet까지" (delta rule, scalar gate); and "From GPT-2 to Kimi K3, Explained", section
 * "Kimi Linear (KDA) -- 채널별 세밀한 게이팅" (alpha becomes Diag(alpha)).
 * Readings taken where the pages leave a step open: the delta read uses the decayed state
 * Diag(alpha_t) S_{t-1}; the output is read after the write; there is no query scale.
 *
 * Conventions for every entry point:
 *   - Every tensor pointer is caller-owned DEVICE memory (cudaMalloc / PyTorch), densely packed
 *     row-major in the layout given, 16-byte aligned.  The library keeps no pointer after a call
 *     returns and allocates no device memory.
 *   - `stream` is a cudaStream_t passed as void* (NULL = the legacy default stream).  Calls are
 *     asynchronous on that stream: a returned KDA_OK means "validated and launched".
 *   - Arguments are validated on the host before any launch; an invalid argument returns a status
 *     and launches nothing.  Problems only the device can see (the contents of cu_seqlens, a bounded
 *     wait that gave up) set sticky flags that kda_get_device_status reads.  Nothing traps or
 *     asserts on the device.
 *   - dtypes: q/k/v share `dtype_qkv`; log_alpha/beta share `dtype_gate`; o has `dtype_o`.
 *     The recurrent state is always fp32.
 */
#ifndef KDA_H_
#define KDA_H_

#include <stddef.h>
#include <stdint.h>

#if defined(__GNUC__)
#define KDA_API __attribute__((visibility("default")))
#else
#define KDA_API
#endif

#ifdef __cplusplus
extern "C" {
#endif

typedef enum {
    KDA_OK = 0,
    KDA_ERR_INVALID_ARG = 1,   /* null/misaligned pointer, bad size, workspace too small */
    KDA_ERR_UNSUPPORTED = 2,   /* valid but not implemented: dk, dv not in {64,128}, chunk != 64 */
    KDA_ERR_CUDA = 3,          /* a CUDA runtime call or launch failed */
    KDA_ERR_TIMEOUT = 4,       /* a bounded device wait gave up (see kda_get_device_status) */
    KDA_ERR_DEVICE_CHECK = 5   /* a device-side argument check failed (see kda_get_device_status) */
} kda_status;

typedef enum {
    KDA_BF16 = 0,
    KDA_FP32 = 1,
    KDA_E4M3 = 2   /* 8-bit floating point, 4 exponent and 3 mantissa bits: the latent cache only */
} kda_dtype;

/* Sticky device flags returned by kda_get_device_status (bitwise OR). */
#define KDA_DEVFLAG_CU_SEQLENS 0x1u   /* cu_seqlens[0] != 0, decreasing, or cu_seqlens[N] != T_total;
                                         the offending sequences were skipped */
#define KDA_DEVFLAG_DECAY_RANGE 0x2u  /* reserved (bit kept for ABI stability): no path raises it, since
                                         every path is exact for every decay in (0, 1) */
#define KDA_DEVFLAG_TIMEOUT 0x4u      /* a bounded inter-CTA wait gave up */
#define KDA_DEVFLAG_PAGE_TABLE 0x8u   /* a page number that is used lies outside 0 .. num_pages - 1; its tokens
                                         were taken as absent (kda_mla_*) */
#define KDA_DEVFLAG_SEQ_LENS 0x10u    /* a length or start is negative, longer than the page table reaches, or
                                         shorter than the new tokens; the sequence was skipped (kda_mla_*) */

/*
 * Workspace bytes kda_chunk_fwd needs for these sizes (0 is a valid answer).
 * T_total: packed tokens; N: sequences.  Pure host function, no CUDA call.
 */
KDA_API size_t kda_chunk_fwd_workspace_size(int64_t T_total, int N, int H, int dk, int dv, int chunk_size);

/*
 * Chunkwise-parallel KDA prefill over a packed batch of N variable-length sequences.
 *
 * Passage: "Kimi Linear: 표현력과 효율을 높인 어텐션 아키텍처(2025)", section "청크 단위 병렬
 * 알고리듬": fixed-length chunks, each starting from the previous chunk's final state; the WY
 * representation packs the chunk's rank-1 updates; the UT transform; the lower-triangular inverse
 * by forward substitution; chunk-level state recurrence plus intra-chunk parallel output with the
 * intra-chunk work arranged as matrix multiplies for the tensor cores.
 *
 *   q, k        [T_total, H, dk]  dtype_qkv        queries, keys (callers usually L2-normalise)
 *   v           [T_total, H, dv]  dtype_qkv        values
 *   log_alpha   [T_total, H, dk]  dtype_gate       natural log of the decay, <= 0
 *   beta        [T_total, H]      dtype_gate       write strength
 *   initial_state [N, H, dk, dv]  fp32 or NULL     NULL = zero initial state
 *   cu_seqlens  [N+1] int32 (device) or NULL       token offsets, cu_seqlens[0] = 0, non-decreasing,
 *                                                  cu_seqlens[N] = T_total.  NULL = N sequences of
 *                                                  T_total / N tokens each (T_total % N must be 0).
 *                                                  Contents are checked on the device only.
 *   T_total >= 0, N >= 1, H >= 1, dk, dv in {64, 128}, chunk_size == 64
 *   o           [T_total, H, dv]  dtype_o          output (may not alias an input)
 *   final_state [N, H, dk, dv]    fp32 or NULL     NULL = not written; may alias initial_state
 *   workspace   device scratch, 16-byte aligned, workspace_bytes >= kda_chunk_fwd_workspace_size(...);
 *               or NULL / 0 bytes.  Owned by the caller; its contents on entry do not matter and are
 *               garbage on exit.  A non-NULL workspace smaller than the size returns
 *               KDA_ERR_INVALID_ARG.
 *
 * Path: KDA_BF16 with dk = dv = 128 and a workspace runs on the tensor cores (tf32 products, fp32
 * accumulation and fp32 state): a chunk-local kernel over all chunks at once followed by a scan over
 * each sequence's chunks (about 2.5 KB of workspace per token and head).  Every other call -- fp32
 * q/k/v, dk or dv = 64, or no workspace -- runs the CUDA-core path (every product in fp32, no
 * workspace used), which is exact at fp32 tolerances but much slower on long sequences (B=1, H=32,
 * T=32768 bf16: about 14x the tensor-core path's time).
 * Both paths are exact up to rounding for every decay.  A chunk whose log-decay spans at most 80 nats
 * in every channel takes one anchor per channel (the fastest form); any other chunk splits its decay
 * factors at 16-row block boundaries so that none exceeds e^40, and channels that decay by more than
 * 80 nats within a block take exact per-element factors there (slower: such inputs cost up to a few
 * times the common case).
 */
KDA_API kda_status kda_chunk_fwd(const void* q, const void* k, const void* v,
                         const void* log_alpha, const void* beta,
                         const float* initial_state, const int32_t* cu_seqlens,
                         int64_t T_total, int N, int H, int dk, int dv, int chunk_size,
                         kda_dtype dtype_qkv, kda_dtype dtype_gate, kda_dtype dtype_o,
                         void* o, float* final_state,
                         void* workspace, size_t workspace_bytes, void* stream);

/* Bytes of the device array kda_chunk_fwd_static_scratch works in (32 MiB). */
#define KDA_STATIC_SCRATCH_BYTES (32u << 20)

/*
 * kda_chunk_fwd for callers that cannot allocate device memory: the same arguments without the
 * workspace, the same results (the same kernels run).  The pages have no counterpart to this entry
 * point; it only changes where the scratch lives.  It allocates nothing itself: its scratch is a
 * file-scope device array of KDA_STATIC_SCRATCH_BYTES, whose address is looked up once per device
 * on the first call made with that device current.
 *   - The array belongs to the library's device code, which CUDA loads onto a device lazily (by
 *     default): the first call on a device that uses the array (one that runs on the tensor cores,
 *     see the limit below) is when its 32 MiB get reserved there, and that call returns KDA_ERR_CUDA
 *     if the device has no room left.  One small such call made once at set-up settles this early.
 *   - Limit: a call that runs on the tensor cores (bf16 q/k/v, dk = dv = 128, T_total > 0) and whose
 *     kda_chunk_fwd_workspace_size(...) exceeds KDA_STATIC_SCRATCH_BYTES returns KDA_ERR_UNSUPPORTED
 *     before any CUDA call.  The size is one 160.5 KB chunk record per 64-token chunk slot and head
 *     (slots = T_total / 64 + N + 1) plus 128 KB per (sequence, head) and 4 bytes per sequence; e.g. 2
 *     sequences x 2048 tokens x 2 heads need 21.5 MiB.  Every other call (fp32 q/k/v, dk or dv = 64) reads no scratch
 *     and has no limit, whatever kda_chunk_fwd_workspace_size says for its sizes.
 *   - Nothing in the scratch has to start at zero: every part a call reads is written earlier in the
 *     same call.
 *   - Every call on a device shares the one array: two calls that can run at the same time (on
 *     different streams, or from host threads without ordering between them) race on it and corrupt
 *     each other's results.  Order such calls (one stream, or synchronise in between).
 * Other statuses and behaviour as kda_chunk_fwd.
 */
KDA_API kda_status kda_chunk_fwd_static_scratch(const void* q, const void* k, const void* v,
                         const void* log_alpha, const void* beta,
                         const float* initial_state, const int32_t* cu_seqlens,
                         int64_t T_total, int N, int H, int dk, int dv, int chunk_size,
                         kda_dtype dtype_qkv, kda_dtype dtype_gate, kda_dtype dtype_o,
                         void* o, float* final_state, void* stream);

/*
 * One recurrent decode step for B sequences (one new token each), state updated in place.
 *
 * Passage: "Kimi Linear: 표현력과 효율을 높인 어텐션 아키텍처(2025)", section "NoPE 적용과 평가
 * 결과" (decoding keeps a fixed-size recurrent state instead of a growing KV cache; time per output
 * token), with the step of section "Kimi Delta Attention의 세밀한 메모리 제어".
 *
 *   q, k        [B, H, dk]  dtype_qkv;  v [B, H, dv] dtype_qkv
 *   log_alpha   [B, H, dk]  dtype_gate; beta [B, H] dtype_gate
 *   state       [B, H, dk, dv] fp32, read and overwritten with the new state
 *   o           [B, H, dv]  dtype_o
 *   B >= 0 (0 launches nothing), H >= 1, dk, dv in {64, 128}
 */
KDA_API kda_status kda_decode_step(const void* q, const void* k, const void* v,
                           const void* log_alpha, const void* beta, float* state,
                           int B, int H, int dk, int dv,
                           kda_dtype dtype_qkv, kda_dtype dtype_gate, kda_dtype dtype_o,
                           void* o, void* stream);

/*
 * Gated DeltaNet: the same operator with one decay rate per token and head instead of one per key
 * channel, alpha_t = exp(log_alpha_t) a scalar in (0,1):
 *
 *     S_t = (I - beta_t k_t k_t^T) alpha_t S_{t-1} + beta_t k_t v_t^T,    o_t = S_t^T q_t.
 *
 * Passage: "Kimi Linear: 표현력과 효율을 높인 어텐션 아키텍처(2025)", section "선형 어텐션에서
 * Gated DeltaNet까지" (a scalar forget gate on the whole state, then the delta rule), and "From
 * GPT-2 to Kimi K3, Explained", section "Gated DeltaNet — 망각을 더하다" (alpha = 1 is the plain
 * delta rule, alpha = 0 clears the memory).  It is KDA with Diag(alpha_t) = alpha_t I, so these entry points run the same kernels
 * as kda_chunk_fwd / kda_decode_step, which read the gate once per token and head and broadcast it
 * over the dk channels.
 *
 * Arguments, workspace, paths, statuses and behaviour are those of kda_chunk_fwd (resp.
 * kda_decode_step) except:
 *   log_alpha   [T_total, H]  (resp. [B, H])  dtype_gate   natural log of the scalar decay, <= 0;
 *               aligned to its element size (it is not read by the tensor memory copier).
 * The workspace size is kda_chunk_fwd_workspace_size(...) of the same sizes.
 */
KDA_API kda_status kda_gdn_chunk_fwd(const void* q, const void* k, const void* v,
                         const void* log_alpha, const void* beta,
                         const float* initial_state, const int32_t* cu_seqlens,
                         int64_t T_total, int N, int H, int dk, int dv, int chunk_size,
                         kda_dtype dtype_qkv, kda_dtype dtype_gate, kda_dtype dtype_o,
                         void* o, float* final_state,
                         void* workspace, size_t workspace_bytes, void* stream);

KDA_API kda_status kda_gdn_decode_step(const void* q, const void* k, const void* v,
                           const void* log_alpha, const void* beta, float* state,
                           int B, int H, int dk, int dv,
                           kda_dtype dtype_qkv, kda_dtype dtype_gate, kda_dtype dtype_o,
                           void* o, void* stream);

/* Options of kda_chunk_fwd_ex / kda_decode_step_ex (bitwise OR). */
#define KDA_OPT_SCALAR_GATE 0x1u  /* log_alpha is [T_total, H] (resp. [B, H]): Gated DeltaNet, as
                                     kda_gdn_chunk_fwd / kda_gdn_decode_step */
#define KDA_OPT_L2NORM_QK 0x2u    /* q and k are raw: each (token, head) vector is divided by its
                                     Euclidean length inside the kernels (in fp32, from the dtype_qkv
                                     values; an all-zero vector stays zero) */
#define KDA_OPT_BETA_LOGITS 0x4u  /* beta holds logits x: the kernels use beta = 1 / (1 + e^{-x}) */
#define KDA_OPT_OUTPUT_NORM_GATE 0x8u  /* output epilogue: each (token, head) row of o becomes
                                          o / sqrt(mean_j o_j^2 + norm_eps) * norm_weight
                                          * sigmoid(out_gate) before it is stored */

/*
 * kda_chunk_fwd / kda_decode_step with the steps that come right before and right after the operator
 * in a KDA layer fused into its kernels.  Passage: "Kimi Linear: 표현력과 효율을 높인 어텐션
 * 아키텍처(2025)", section "Kimi Linear 모델 구성": queries and keys are L2-normalised (eigenvalue
 * stability) before the KDA update, the write strength beta lies in (0, 1), and before the output
 * projection every head's output goes through RMSNorm and a data-dependent output gate.  The
 * projections, short convolutions, the decay-gate function and the output gate's low-rank
 * projection need weights and are the caller's: the gate arrives as its pre-activation values.
 *   options     KDA_OPT_* bits; 0 gives exactly kda_chunk_fwd (resp. kda_decode_step).  Unknown bits
 *               return KDA_ERR_INVALID_ARG.
 *   out_gate    [T_total, H, dv] (resp. [B, H, dv]) dtype_qkv, the output gate's pre-activations;
 *   norm_weight [dv] fp32, the RMSNorm weight shared by the heads;
 *   norm_eps    >= 0, finite: all three read only with KDA_OPT_OUTPUT_NORM_GATE (then out_gate and
 *               norm_weight must be non-NULL when there are rows, aligned to their element size).
 *               On the bf16 dk = dv = 128 path with a workspace the epilogue runs inside the scan
 *               (the two CTAs of a head form a cluster and trade per-token sums of squares); on the
 *               other prefill paths it is a separate pass over o after the kernel, which with a bf16 o
 *               normalises the rounded values.  The decode step applies it in its kernel.
 * Every other argument, status and behaviour as kda_chunk_fwd (resp. kda_decode_step); with
 * KDA_OPT_SCALAR_GATE log_alpha is laid out and aligned as for kda_gdn_chunk_fwd.
 */
KDA_API kda_status kda_chunk_fwd_ex(const void* q, const void* k, const void* v,
                         const void* log_alpha, const void* beta,
                         const float* initial_state, const int32_t* cu_seqlens,
                         int64_t T_total, int N, int H, int dk, int dv, int chunk_size,
                         kda_dtype dtype_qkv, kda_dtype dtype_gate, kda_dtype dtype_o,
                         void* o, float* final_state,
                         void* workspace, size_t workspace_bytes, uint32_t options,
                         const void* out_gate, const float* norm_weight, float norm_eps, void* stream);

KDA_API kda_status kda_decode_step_ex(const void* q, const void* k, const void* v,
                           const void* log_alpha, const void* beta, float* state,
                           int B, int H, int dk, int dv,
                           kda_dtype dtype_qkv, kda_dtype dtype_gate, kda_dtype dtype_o,
                           void* o, uint32_t options, const void* out_gate, const float* norm_weight,
                           float norm_eps, void* stream);

/*
 * Latent attention, the other attention layer of the pages' stack.  Passage: "Kimi Linear: 표현력과
 * 효율을 높인 어텐션 아키텍처(2025)", sections "KDA와 MLA의 3:1 하이브리드" and "NoPE 적용과 평가 결과":
 * three KDA layers to one layer of multi-head latent attention (MLA), in which every token leaves one
 * latent vector c_j (shared by the heads, from which keys and values are expanded) and one positional
 * key p_j (shared by the heads; without positional encoding simply 64 further key channels).  For
 * decoding, the expansion is absorbed into the query and the layer becomes attention over the latents
 * themselves, with one key and value head (MQA).
 *
 *   expanded (kda_mla_prefill):  x_ij = scale (q_i^nope . k_j + q_i^pe . p_j),  o_i = sum_j softmax_j(x_ij) v_j
 *   absorbed (kda_mla_decode):   x_ij = scale (q_i^latent . c_j + q_i^pe . p_j), o_i = sum_j softmax_j(x_ij) c_j
 *
 * The projections (down to c and p; k and v from c; q^latent = W_k^T q^nope; values from o) need weights
 * and are the caller's.  Both forms can return lse_i = log sum_j e^{x_ij} (natural log).  A row that sees
 * no key gives o = 0 and lse = -infinity.
 *
 * The paged latent cache, shared by the entry points below:
 *   cache_latent [num_pages, page_size, d_latent]  dtype_cache (KDA_BF16 or KDA_E4M3)
 *   cache_pe     [num_pages, page_size, d_pe]      bf16
 *   cache_scale  [num_pages, page_size]            fp32, KDA_E4M3 only (NULL otherwise): a cached value is its
 *                                                  code times its token's scale, a power of two in
 *                                                  [2^-64, 2^120] (what kda_mla_cache_write stores)
 *   page_table   [B, max_pages] int32 (device)     token j of sequence b lies in page page_table[b][j / page_size]
 *                                                  at row j % page_size.  Entries past a sequence's length are
 *                                                  not read.
 *   page_size a power of two from 16 to 1024; num_pages * page_size, max_pages * page_size and the packed rows T,
 *   Tq, Tk at most 2^31 - 256; d_latent = 512, d_pe = 64 (other sizes: KDA_ERR_UNSUPPORTED).
 * cu_seqlens of these entry points: [B + 1] int32 (device) or NULL (equal lengths, T a multiple of B), as in
 * kda_chunk_fwd, but cu_seqlens[B] may be less than T: the rows behind it are not written, and may hold anything.
 * Outputs, cache_* of a write and the workspace may overlap neither inputs nor one another (KDA_ERR_INVALID_ARG).
 * What only the device can see (cu_seqlens, lengths, page numbers) raises KDA_DEVFLAG_CU_SEQLENS,
 * KDA_DEVFLAG_SEQ_LENS or KDA_DEVFLAG_PAGE_TABLE; nothing outside the given arrays is touched.  The rows of
 * a sequence skipped for its length (kda_mla_decode) or its cu_seqlens_k (kda_mla_prefill) get o = 0,
 * lse = -infinity; those of a sequence with bad cu_seqlens_q are left as they were.
 * An infinity or NaN in a key, value or cached token stays within its sequence, but there can reach rows that do
 * not see it (a weight of 0 times it is NaN).  What lies behind a sequence's last token may be anything.
 */

/*
 * Writes new tokens into the cache, quantising them on the way for KDA_E4M3.
 *   latent     [T, d_latent], pe [T, d_pe]  dtype_in (KDA_BF16 or KDA_FP32; rounded to nearest)
 *   cu_seqlens the new tokens of each sequence: n_b = cu_seqlens[b+1] - cu_seqlens[b]
 *   seq_lens   [B] int32 (device): lengths that already count the new tokens; those of sequence b become its
 *              positions seq_lens[b] - n_b .. seq_lens[b] - 1
 * KDA_E4M3: a token's scale is the smallest power of two s in [2^-64, 2^120] with max |latent| <= 448 s (NaN
 * ignored), its codes are latent / s rounded to nearest even (infinities become +-448, NaN stays NaN).
 * Where two sequences' new tokens fall on the same pool row (a page given to both), its values are unspecified.
 * T >= 0, B >= 1.
 */
KDA_API kda_status kda_mla_cache_write(const void* latent, const void* pe, const int32_t* cu_seqlens,
                         const int32_t* seq_lens, int64_t T, int B, int d_latent, int d_pe,
                         kda_dtype dtype_in, kda_dtype dtype_cache,
                         void* cache_latent, void* cache_pe, float* cache_scale,
                         const int32_t* page_table, int64_t num_pages, int page_size, int max_pages, void* stream);

/*
 * Reads cached tokens back into packed arrays (a chunked prefill expands its prefix from them).
 *   cu_seqlens how many tokens of each sequence, n_b, and where they go in the packed arrays
 *   starts     [B] int32 (device) or NULL (zeros): the positions read are starts[b] .. starts[b] + n_b - 1
 *   latent     [T, d_latent], pe [T, d_pe]  dtype_o (KDA_BF16 or KDA_FP32)
 * Values are code times scale, exact in both types, but for those of 2^128 and more, which become infinite: what
 * kda_mla_cache_write rounded to code 256 or more under the scale 2^120, from magnitudes of 3.30e38 on.
 * Rows of a skipped sequence and tokens of a bad page are left as they were.  T >= 0, B >= 1.
 */
KDA_API kda_status kda_mla_cache_read(const void* cache_latent, const void* cache_pe, const float* cache_scale,
                         const int32_t* page_table, const int32_t* cu_seqlens, const int32_t* starts,
                         int64_t T, int B, int d_latent, int d_pe, int64_t num_pages, int page_size, int max_pages,
                         kda_dtype dtype_cache, kda_dtype dtype_o, void* latent, void* pe, void* stream);

/* Workspace bytes kda_mla_decode wants for these sizes (0 is a valid answer).  Pure host function. */
KDA_API size_t kda_mla_decode_workspace_size(int B, int S, int H, int d_latent, int d_pe);

/*
 * Absorbed latent attention of S new tokens per sequence over the paged cache (they have been written to it).
 *   q_latent [B, S, H, d_latent], q_pe [B, S, H, d_pe]  dtype_q (KDA_BF16)
 *   seq_lens [B] int32 (device): cached tokens, the new ones included.  New token s of sequence b is token
 *            seq_lens[b] - S + s and sees itself and the tokens before it.  Length 0 is allowed.
 *   o        [B, S, H, d_latent] dtype_o (KDA_BF16 or KDA_FP32);  lse [B, S, H] fp32 or NULL
 *   workspace  device scratch, 16-byte aligned, of kda_mla_decode_workspace_size bytes, or NULL / 0 bytes: then
 *              no sequence is split over several SMs (slow for few long sequences).  Its contents on entry do not
 *              matter.  Calls that can run at the same time need a workspace each.
 *   B >= 0 (0 launches nothing), S >= 1, H >= 1, S * H <= 65535
 * Arithmetic: products of bf16 values with fp32 accumulation; softmax statistics and the output are held in
 * fp32; the weights enter the second product in bf16.  With KDA_E4M3 the codes are multiplied as they are and
 * queries and weights enter as two e4m3 parts each: a value is off by at most 2^-8 of itself, as in bf16, or by an
 * absolute amount where it is small: a query's channel by 2^-21 of its row's largest one, a weight times its
 * token's scale by an amount that, over all tokens of a row however many, adds up to at most 2^-6 of the row's
 * sum of (weight x scale) times the largest mean |code| of 512 neighbouring tokens.
 */
KDA_API kda_status kda_mla_decode(const void* q_latent, const void* q_pe, const void* cache_latent,
                         const void* cache_pe, const float* cache_scale, const int32_t* page_table,
                         const int32_t* seq_lens, int B, int S, int H, int d_latent, int d_pe,
                         int64_t num_pages, int page_size, int max_pages, float softmax_scale,
                         kda_dtype dtype_q, kda_dtype dtype_cache, kda_dtype dtype_o, void* o, float* lse,
                         void* workspace, size_t workspace_bytes, void* stream);

/*
 * Expanded latent attention over a packed batch.
 *   q    [Tq, H, d_nope + d_pe]  dtype_qkv (KDA_BF16)    per head: the part without position, then the positional part
 *   kv   [Tk, H, d_nope + dv]    dtype_qkv               per head: the key's expanded part, then the value
 *   k_pe [Tk, d_pe]              dtype_qkv               the positional key, shared by the heads
 *   cu_seqlens_q, cu_seqlens_k   the queries and the keys of each sequence.  cu_seqlens_k = NULL: equal key
 *                                lengths, Tk a multiple of B.
 *   causal   1: query i of a sequence with n_q queries and n_k keys sees keys j <= i + n_k - n_q (the last query
 *            sees the last key); 0: every query sees all n_k keys
 *   o    [Tq, H, dv] dtype_o (KDA_BF16 or KDA_FP32);  lse [Tq, H] fp32 or NULL
 *   d_nope = 128, d_pe = 64, dv = 128;  Tq, Tk >= 0, B >= 1, 1 <= H <= 65535
 * Arithmetic: products of bf16 values with fp32 accumulation; softmax statistics and the output are held in
 * fp32; the weights enter the second product in bf16.  No workspace.
 */
KDA_API kda_status kda_mla_prefill(const void* q, const void* kv, const void* k_pe, const int32_t* cu_seqlens_q,
                         const int32_t* cu_seqlens_k, int64_t Tq, int64_t Tk, int B, int H, int d_nope, int d_pe,
                         int dv, int causal, float softmax_scale, kda_dtype dtype_qkv, kda_dtype dtype_o,
                         void* o, float* lse, void* stream);

/*
 * Waits for `stream`, then reads and clears the sticky device flags (KDA_DEVFLAG_*) of the current
 * device into *flags (may be NULL).  Returns KDA_OK if no flag was set, KDA_ERR_TIMEOUT if the
 * timeout flag was set, KDA_ERR_DEVICE_CHECK for any other flag, KDA_ERR_CUDA on a CUDA error.
 */
KDA_API kda_status kda_get_device_status(void* stream, uint32_t* flags);

/* Static English text for a status code; never NULL. */
KDA_API const char* kda_status_string(kda_status status);

/* Library ABI version, (major << 16) | minor. */
KDA_API uint32_t kda_version(void);

#ifdef __cplusplus
}
#endif

#endif /* KDA_H_ */
