/*
 * gcs_attn.h -- C ABI of the GB300 (sm_103a) gated causal softmax attention library.
 *
 * Four calls make up the hot path:
 *   attn_fwd           prefill forward  (O, LSE)
 *   attn_bwd           prefill backward (dQ, dK, dV, d log_gate, d sink)
 *   attn_decode_paged  paged single-query / short-query decode over an fp8 e4m3 KV cache
 *   attn_prefill_paged paged chunked prefill (query chunks of any length) over the same cache
 *   attn_decode_paged_shared  paged decode of requests that share a prefix, which is read once
 * and these make what the four read (library calls with no counterpart in the pages):
 *   attn_qk_norm_rope_fwd, attn_qk_norm_rope_bwd   per-head norm and rotation of q and k
 *   attn_cache_append, attn_cache_append_rope      write of k, v and log gates into the paged cache
 *   attn_cache_gather                              read of the paged cache into packed tensors
 *   attn_cache_weights, attn_cache_select, attn_cache_compact   eviction: the weight that cached
 *                                                  tokens gather, the choice of those that stay, their move
 *
 * Sources for what each call computes (page title, section):
 *   [FLA] fla-org/flash-linear-attention issue #1322 "[Perf] Gluon attention backend with
 *         large head dimensions" -- Description: the causal attention contract (dense and
 *         packed variable-length inputs, MHA/GQA/MQA, unequal query/key and value head
 *         dims up to 512, logarithmic gates, sliding windows, sink bias, gradients);
 *         comment of Oct 3: the sink gradient is accumulated in fp32 from the backward
 *         probabilities, not from the rounded output; comment of Oct 5: dQ partials
 *         accumulate into a zero-initialised fp32 buffer and are converted afterwards.
 *   [AIT] ROCm/aiter PR #6660 (gfx1250 unified attention) -- commit messages and
 *         "Technical details": per-token fp32 K/V scales laid out [num_blocks,
 *         num_kv_heads, block_size]; K scales multiply QK columns; V scales multiply P
 *         columns after the row sum; slots past seq_len get scale 0; split-K over context
 *         segments with an LSE-weighted reduce in which an empty partial (M = -inf)
 *         weighs 0; per-token scales on a prefill shape are rejected.
 *
 * Conventions for every call:
 *   - All tensor pointers are DEVICE pointers owned by the caller (inputs, outputs and
 *     workspace).  The library never allocates, frees or synchronises.
 *   - Every call is asynchronous on the given stream.  Arguments are validated on the
 *     host first; on any error the call returns a nonzero gcs_status and launches
 *     nothing, so outputs are untouched.
 *   - Tensors are row-major with the last dimension contiguous and base addresses 16-byte
 *     aligned.  The [tokens, heads, head_dim] tensors of the prefill and paged calls (q, k,
 *     v, o, dout, the gradients, the paged q and out) take element strides (token, head)
 *     given as gcs_strides, and the paged caches take element strides (block, kv head, slot);
 *     all-zero strides mean contiguous.  Everything else (gates, sinks, LSE, scales, index
 *     arrays) is contiguous.
 *   - No output may share a byte with an input or with another output (the kernels read
 *     and write concurrently); such a call returns GCS_ERR_INVALID_ARG.  Inputs may share
 *     memory with each other.
 *   - bf16 = bfloat16 stored as uint16; fp8 = OCP e4m3 ("fn") stored as uint8.
 *   - Device-side contents (cu_seqlens monotone and ending at total_tokens, page-table
 *     entries in [0, num_blocks), seq_lens >= q_len) are preconditions; they are not
 *     checked on the host because reading them would synchronise.  gcs_set_device_checks
 *     makes every attention call check them on the device first (see "device-content
 *     checks"); the norm, rotation and cache calls always check what they index with.
 *   - Every wait inside a kernel is bounded (2 s).  A kernel that gives up records
 *     GCS_ERR_DEVICE_TIMEOUT in a per-device status word, releases its resources and
 *     returns; read it with gcs_get_device_status().
 *   - The library caches, per device, the device addresses of its own status word and of
 *     the scratch of attn_decode_paged_noalloc.  cudaDeviceReset unloads the library's
 *     device code and those addresses go stale: do not call the library on a device after
 *     cudaDeviceReset of that device in the same process.
 */
#ifndef GCS_ATTN_H_
#define GCS_ATTN_H_

#include <stddef.h>
#include <stdint.h>

#ifdef __cplusplus
extern "C" {
#endif

typedef struct CUstream_st* gcs_stream_t; /* same type as cudaStream_t; NULL = legacy default stream */

/* Element strides of a [tokens, heads, head_dim] tensor whose head_dim is contiguous: element
 * (t, h, d) sits at base[t * token + h * head + d].  {0, 0} means the contiguous layout
 * {heads * head_dim, head_dim}.  Otherwise the layout must be token-major without overlap,
 * head >= head_dim and token >= heads * head, with both multiples of 8 elements (16 bytes, the
 * granule of the tensor copies and vector stores); any other layout returns
 * GCS_ERR_UNSUPPORTED.  A slice of a fused projection, e.g. q, k and v as views of one
 * [tokens, (hq + 2 hkv) * d] buffer, is such a layout. */
typedef struct {
  int64_t token;
  int64_t head;
} gcs_strides;

typedef enum {
  GCS_OK = 0,
  GCS_ERR_INVALID_ARG = 1,   /* null pointer, bad size, misaligned base, inconsistent shape */
  GCS_ERR_UNSUPPORTED = 2,   /* a shape / dtype / layout this library does not implement   */
  GCS_ERR_WORKSPACE = 3,     /* workspace pointer NULL or smaller than the *_workspace size */
  GCS_ERR_CUDA = 4,          /* a CUDA launch or runtime call failed                       */
  GCS_ERR_DEVICE_TIMEOUT = 5 /* a kernel gave up on a bounded wait (device status word)    */
} gcs_status;

const char* gcs_status_str(int status);

/* ------------------------------------------------------------------ prefill
 * Causal softmax attention over packed sequences ([FLA] Description).
 * Sequence s occupies tokens cu_seqlens[s] .. cu_seqlens[s+1]-1 of the packed tensors;
 * dense [B, T] inputs are the special case cu_seqlens = {0, T, 2T, ..., B*T}.
 * Query head h reads kv head h / (hq / hkv) (MHA: hq == hkv; MQA: hkv == 1).
 * Score of query token i and key token j of the same sequence:
 *     s_ij = scale * (q_i . k_j) + G_i - G_j,   G = per-sequence inclusive cumsum of log_gate
 * visible iff j <= i and (window == 0 or i - j < window).  The per-head sink logit sigma_h
 * joins the softmax denominator only:  P_ij = e^{s_ij} / (sum_j e^{s_ij} + e^{sigma_h}).
 * Supported (dqk, dv): (64, 64), (128, 128), (256, 256), (256, 512), (512, 512).
 */
typedef struct {
  int num_seqs;               /* >= 1                                                    */
  const int32_t* cu_seqlens;  /* device int32 [num_seqs + 1]                            */
  int total_tokens;           /* host copy of cu_seqlens[num_seqs]; >= 1                */
  int max_seqlen;             /* host upper bound on any sequence length                */
  int hq, hkv;                /* query heads, kv heads; hq % hkv == 0                    */
  int dqk, dv;                /* head dims of q/k and of v                               */
  float scale;                /* softmax scale (usually 1/sqrt(dqk))                     */
  int window;                 /* 0 = none, else number of visible keys including self    */
  const void* q;              /* bf16 [total_tokens, hq, dqk]                            */
  const void* k;              /* bf16 [total_tokens, hkv, dqk]                           */
  const void* v;              /* bf16 [total_tokens, hkv, dv]                            */
  const float* log_gate;      /* fp32 [total_tokens, hq] per-token log forget gates, or NULL */
  const float* sink;          /* fp32 [hq] sink logits, or NULL                          */
  int deterministic;          /* attn_bwd: 1 = a separate query-stationary dQ pass, every
                                 gradient written once or summed in a fixed order; 0 = the
                                 faster route for the shape: a single pass with fp32
                                 reduce-adds of dQ and the dS row sums at head dim 128 and at
                                 dqk = 256, the separate dQ pass at 64 (the only route there)
                                 and at dqk = 512. */
  gcs_strides q_stride, k_stride, v_stride;  /* layouts of q, k, v ({0, 0} = contiguous)      */
  gcs_strides o_stride;       /* attn_fwd's output o and attn_bwd's input o                    */
  gcs_strides do_stride;      /* attn_bwd's dout                                               */
  gcs_strides dq_stride, dk_stride, dv_stride;  /* attn_bwd's outputs dq, dk, dv              */
} gcs_prefill_args;

/* Workspace bytes attn_fwd needs (0 when there is no gate). */
size_t attn_fwd_workspace(const gcs_prefill_args* a);

/* Forward.  o: bf16 [total_tokens, hq, dv] (layout a->o_stride); lse: fp32 [hq, total_tokens]
 * contiguous, natural-log logsumexp of each row's scores including the sink term (needed by
 * attn_bwd).  Outputs that share bytes with an input or with each other are rejected; two
 * strided tensors with the same token stride whose per-token byte ranges interleave without
 * meeting (e.g. heads of one fused buffer) do not share bytes. */
int attn_fwd(const gcs_prefill_args* a, void* o, float* lse, void* workspace, size_t workspace_bytes,
             gcs_stream_t stream);

/* Workspace bytes attn_bwd needs. */
size_t attn_bwd_workspace(const gcs_prefill_args* a);

/* Backward of L = sum(O * dO) ([FLA] Description, the gradient list; Oct 3 / Oct 5 comments).
 * o, lse: the forward's outputs (o in layout a->o_stride); dout: bf16 [total_tokens, hq, dv]
 * (a->do_stride).  Outputs: dq bf16 [total_tokens, hq, dqk] (a->dq_stride), dk bf16
 * [total_tokens, hkv, dqk] (a->dk_stride), dv bf16 [total_tokens, hkv, dv] (a->dv_stride),
 * dlog_gate fp32 [total_tokens, hq] contiguous (must be NULL iff
 * log_gate is NULL), dsink fp32 [hq] (must be NULL iff sink is NULL).
 * The sink gradient is -sum_i p_sink,i * sum_j P_ij (dO_i . v_j), accumulated in fp32.
 * With a->deterministic = 1 (and always at head dim 64, and at dqk = 512) dQ is accumulated per
 * query tile in a separate pass and every gradient is written once or summed in a fixed order,
 * so repeated calls give the same bits.  Otherwise (head dim 128, dqk = 256) dQ, d log_gate and
 * d sink come from fp32 reduce-adds into zero-initialised buffers (the [FLA] comment of Oct 5),
 * and their low bits may vary from run to run. */
int attn_bwd(const gcs_prefill_args* a, const void* o, const float* lse, const void* dout, void* dq, void* dk,
             void* dv, float* dlog_gate, float* dsink, void* workspace, size_t workspace_bytes,
             gcs_stream_t stream);

/* ------------------------------------------------------------------ paged decode
 * Decode / short-query attention over a paged KV cache ([AIT] commits 1-3, Technical
 * details): fp8 e4m3 with per-token fp32 scales (the default), fp8 e4m3 with one K and one
 * V scale for the whole cache (per-tensor, which the page leaves on its earlier code path),
 * or bf16 with no scales (the bf16-KV route of commit 3).  Request r has
 * q_len = cu_q[r+1] - cu_q[r] query rows (1..4) and seq_len = seq_lens[r] cached tokens (the
 * query tokens are the last q_len of them); query row t sits at position seq_len - q_len + t
 * and sees keys 0 .. seq_len - q_len + t.  Key j of request r lives in block
 * block_table[r][j / block_size],
 * slot j % block_size.  Dequantised key = e4m3(k) * k_scale[block][kv_head][slot], same for
 * values.  s_j = scale * k_scale_j * (q . k8_j); the row sum uses the unscaled e^{s_j - m};
 * the V scales multiply the probabilities after the row sum.  Slots at or past seq_len are
 * never used (scale 0, probability 0), whatever their bytes or scales hold (NaN allowed).
 * The context is split into segments of segment_len tokens; each (request, kv head,
 * segment) yields a partial (acc, M, L) and a combine kernel merges them with weights
 * e^{M_s - max M}; a partial with no visible key (M = -inf) weighs 0.
 * With per-tensor scales, k_scale and v_scale each point to one fp32 used for every token;
 * with a bf16 cache, k_cache / v_cache hold bf16 values and k_scale, v_scale must be NULL.
 * Decoding features (the [FLA] Description asks for the prefill features on the packed
 * single-query decode too), each optional: g_cache holds the cumulative log gates G of the
 * cached tokens, paged like the scales but per query head, fp32 [num_blocks, hq, block_size]
 * (natural-log units); the score becomes scale*q.k_j + G_i - G_j with G_i the entry at the query row's
 * own position.  window W > 0 keeps keys with position_i - j < W.  sink fp32 [hq] adds
 * e^sink_h to the softmax denominator (once, in the combine).
 * Supported: d == 128; hq / hkv == 16 or 8 (GQA groups of 16 or 8 query heads); block_size
 * 16 x 2^k tokens (16, 32, 64, 128, ..., 4096); 1 <= q_len <= 4; segment_len a positive multiple
 * of 16.
 * Operand precision of an fp8 cache: the tensor cores see f16.  q is rounded from bf16 to f16,
 * so no |q| may exceed 65504 (the f16 maximum); K and V codes convert to f16 exactly;
 * P * vscale is rounded to nearest f16 after a 2^5 pre-scale (P <= 2^3: a row's reference max
 * moves only when the row max grows by more than 2^3), so every V scale of a slot below
 * seq_len must stay below 255.  Outside these limits the output holds inf or NaN.
 * The host cannot read device values; checked mode (gcs_set_device_checks) checks both on the
 * device and records GCS_ERR_INVALID_ARG when one fails.
 */
enum { GCS_KV_FP8_E4M3 = 0, GCS_KV_BF16 = 1 };
enum { GCS_SCALE_PER_TOKEN = 0, GCS_SCALE_PER_TENSOR = 1 };
typedef struct {
  int num_reqs;                /* >= 1                                                   */
  const int32_t* cu_q;         /* device int32 [num_reqs + 1]                           */
  int total_q;                 /* host copy of cu_q[num_reqs]                           */
  int max_q_len;               /* host upper bound on q_len, 1..4                        */
  const int32_t* seq_lens;     /* device int32 [num_reqs], each >= its q_len             */
  int max_seq_len;             /* host upper bound on seq_lens                           */
  const int32_t* block_table;  /* device int32 [num_reqs, max_blocks_per_req]           */
  int max_blocks_per_req;      /* row stride of block_table                             */
  const void* k_cache;         /* fp8 e4m3 or bf16 [num_blocks, hkv, block_size, d]     */
  const void* v_cache;         /* same format as k_cache                                 */
  const float* k_scale;        /* fp32 [num_blocks, hkv, block_size], or [1], or NULL   */
  const float* v_scale;        /* same layout as k_scale                                 */
  int num_blocks, block_size;  /* cache blocks, tokens per block                        */
  int hq, hkv, d;              /* query heads, kv heads, head dim                       */
  float scale;                 /* softmax scale                                         */
  int segment_len;             /* split-K segment length in tokens                      */
  const void* q;               /* bf16 [total_q, hq, d]                                 */
  int kv_format;               /* GCS_KV_FP8_E4M3 or GCS_KV_BF16                         */
  int scale_mode;              /* GCS_SCALE_PER_TOKEN or GCS_SCALE_PER_TENSOR (fp8 only) */
  const float* g_cache;        /* fp32 [num_blocks, hq, block_size] cumulative log gates, or NULL */
  const float* sink;           /* fp32 [hq] sink logits, or NULL                          */
  int window;                  /* sliding window in keys, 0 = none                        */
  gcs_strides q_stride;        /* layout of q ({0, 0} = contiguous)                       */
  gcs_strides out_stride;      /* layout of out ({0, 0} = contiguous)                     */
  int64_t kv_stride_block, kv_stride_head, kv_stride_slot;
                               /* element strides of both caches (block, kv head, slot); all 0 =
                                  contiguous [num_blocks, hkv, block_size, d].  The d elements of
                                  a slot are contiguous; every stride is a multiple of 16 bytes;
                                  the slots and kv heads of a block nest without overlap (slot
                                  >= d and head >= block_size * slot, or head >= d and slot >=
                                  hkv * head: the [num_blocks, block_size, hkv, d] cache layout of
                                  vLLM-style engines) and block covers both.  Scales and gates
                                  stay contiguous [num_blocks, ..., block_size]. */
} gcs_decode_args;

/* Workspace bytes attn_decode_paged needs (split-K partials). */
size_t attn_decode_workspace(const gcs_decode_args* a);

/* out: bf16 [total_q, hq, d]. */
int attn_decode_paged(const gcs_decode_args* a, void* out, void* workspace, size_t workspace_bytes,
                      gcs_stream_t stream);

/* Allocation-free variant of attn_decode_paged (no counterpart in the pages: this is a
 * library convenience).  Some callers cannot allocate device memory for a workspace: a
 * host runtime with a fixed, pre-planned memory budget, a C program without a device
 * allocator of its own, or a latency-critical decode loop in which a cudaMalloc (which
 * may synchronise the device) is not acceptable.  This entry point takes the same
 * arguments minus the workspace and keeps the split-K partials in a fixed scratch array
 * compiled into the library (64 MiB, held on every GPU that loads the library until the
 * process exits).  It calls no allocator.
 *   - Sizes whose partials exceed the scratch (attn_decode_workspace(a) > 64 MiB) are
 *     rejected with GCS_ERR_WORKSPACE before anything is launched.
 *   - The first call on a device looks up the scratch's device address (with that device
 *     current); make that first call before any stream capture on that device.
 *   - All calls share the one scratch array and it keeps the previous call's contents;
 *     nothing needs clearing because every partial a call reads it first writes.  Calls
 *     that overlap on the GPU (e.g. on two concurrent streams) race on the scratch and
 *     give wrong results: serialise them.
 * out: bf16 [total_q, hq, d]; returns the same statuses as attn_decode_paged. */
int attn_decode_paged_noalloc(const gcs_decode_args* a, void* out, gcs_stream_t stream);

/* ------------------------------------------------------------------ paged chunked prefill
 * Attention of query chunks of any length over the same paged fp8 KV cache ([AIT] commit
 * messages: a batch that is not all-decode takes the 2d unified-attention route, one
 * program per (kv head, query block)).  Arguments and semantics are those of
 * attn_decode_paged (gcs_decode_args, the decoding features included), except:
 *   - q_len = cu_q[r+1] - cu_q[r] may be any value in 1 .. seq_lens[r]; max_q_len >= 1 is
 *     its host upper bound.  Query row t of request r still sits at position
 *     seq_len - q_len + t and sees keys 0 .. seq_len - q_len + t (and the window).
 *   - fp8 e4m3 with per-token or per-tensor scales; a bf16 cache is GCS_ERR_UNSUPPORTED.
 *     (The pages' 2d route rejects per-token scales; here they are applied as in decode.)
 *   - segment_len == 0 lets the library split the context: one segment per request when
 *     the query blocks alone give about two CTAs per SM (the kernel then writes out
 *     directly and needs no workspace), otherwise segments sized for that many CTAs whose
 *     split-K partials the decode combine merges.  A positive segment_len must be a
 *     multiple of 128 tokens.  attn_prefill_paged_workspace(a) gives the bytes needed
 *     (0 when nothing is split; the choice depends on the current device's SM count).
 *   - The tensor cores see Q rounded from bf16 to f16 (|q| < 65504), K and V as exact f16
 *     from e4m3, and P * vscale rounded to f16 (vscale < 255), with fp32 accumulation.
 * out: bf16 [total_q, hq, d].  Preconditions: q_len <= seq_len per request. */
size_t attn_prefill_paged_workspace(const gcs_decode_args* a);
int attn_prefill_paged(const gcs_decode_args* a, void* out, void* workspace, size_t workspace_bytes,
                       gcs_stream_t stream);

/* ------------------------------------------------------------------ paged decode behind shared prefixes
 * attn_decode_paged for requests that share the front of their contexts (a system prompt, one long
 * document): the same result, with the shared tokens read once for all of them.  Group g is
 * the requests cu_groups[g] .. cu_groups[g+1]-1; the tokens at positions below prefix_lens[g] are the
 * same for all of them and are read through the block table of the group's first request.  A
 * request's own table is read from there on (from the start of the cache block that holds position
 * prefix_lens[g]; the last, partly shared block may be each request's own copy): its entries before
 * that, and such a copy's slots before that position, are not looked at (by this call: the others,
 * the cache calls among them, know no groups and read every position through the request's own
 * table).  A query row may stand inside the prefix (prefix_lens[g] up to the seq_len).  A group may be
 * one request or none, a prefix 0.
 * Everything of attn_decode_paged is supported (formats, groups of 16 or 8 heads, block sizes,
 * strides, q_len 1..4, gates, window, sink), except: segment_len is that of the tokens behind the
 * prefixes, 0 lets the library choose; and no kernel events are recorded (they stay armed).
 * Preconditions on the device's arrays, beside those of attn_decode_paged: cu_groups[0] == 0,
 * cu_groups[num_groups] == num_reqs, sorted; prefix_lens[g] <= max_prefix_len and the seq_len of
 * every request of the group; seq_len - prefix_lens[g] <= max_suffix_len; at most
 * max_group_q query rows a group; the first request's table holds the prefix's blocks, whatever the
 * window.  Checked mode checks them; where one fails the call's kernels see an empty batch.
 * The prefix's values are finite, also those that a row does not see for its window or because it
 * stands in front of them: 128 tokens at a time they are multiplied by 0. */
typedef struct {
  int num_groups;              /* >= 1                                                    */
  const int32_t* cu_groups;    /* device int32 [num_groups + 1]                          */
  const int32_t* prefix_lens;  /* device int32 [num_groups]                              */
  int max_group_q;             /* host upper bound on the query rows of a group, 1 .. total_q */
  int max_prefix_len;          /* host upper bound on prefix_lens, 0 .. max_seq_len      */
  int max_suffix_len;          /* host upper bound on seq_len - prefix_len, 0 .. max_seq_len */
} gcs_prefix_args;

/* Workspace bytes (split-K partials of the prefixes and of what lies behind them; the choice of
 * segments depends on the current device's SM count). */
size_t attn_decode_paged_shared_workspace(const gcs_decode_args* a, const gcs_prefix_args* x);

/* out: bf16 [total_q, hq, d]. */
int attn_decode_paged_shared(const gcs_decode_args* a, const gcs_prefix_args* x, void* out, void* workspace,
                             size_t workspace_bytes, gcs_stream_t stream);

/* ------------------------------------------------------------------ norm and rotation of q and k
 * Between the projections and the attention calls: each query and key head goes through an
 * RMS norm over its d elements and a rotation by its token's position, in one pass:
 *     r = (mean(x^2) + eps)^(-1/2),   y = x * r * weight          (norm = 0: y = x)
 *     pairs (a, b) of y's first rotary_dim elements, i < m = rotary_dim / 2:
 *         interleaved = 0: (y_i, y_{i+m});   interleaved = 1: (y_{2i}, y_{2i+1})
 *         a' = a c - b s,  b' = b c + a s,   c = cos_sin[p][i], s = cos_sin[p][m + i], p = positions[t]
 *     elements from rotary_dim on are passed through.
 * All in fp32 with one rounding to bf16.  The table is the caller's (computed in 64 bits for far
 * positions, with whatever frequency scaling the model uses).
 * A token with a negative position is padding: its outputs are left as they were, and its
 * gradients are 0.  A position of max_pos or more is not read: the token is treated as padding
 * and GCS_ERR_INVALID_ARG is recorded in the device status word (in every mode; checked mode
 * adds nothing to these calls).
 * The sum of squares is held in fp32: it overflows from one element of about 1.8e19 on (128 of
 * 1.6e18), and such a row's outputs and gradients are 0 or NaN; with eps = 0 it also underflows, for
 * rows of elements below about 1e-19, whose outputs lose bits and become infinite or NaN.
 * Supported: d 64, 128, 256 or 512; rotary_dim a multiple of 16, <= d; q_out and k_out (dq and dk)
 * apart from q and k.
 */
typedef struct {
  int total_tokens;            /* rows of q and k, >= 1                                   */
  int hq, hkv, d;              /* hq % hkv == 0                                           */
  int rotary_dim;              /* 0 (exactly when cos_sin is NULL), or a multiple of 16   */
  int interleaved;             /* 0: halves, 1: neighbouring pairs                        */
  int norm;                    /* 1: RMS norm, 0: rotation only (weights must be NULL)    */
  float eps;                   /* >= 0                                                    */
  const void* q;               /* bf16 [total_tokens, hq, d]                              */
  const void* k;               /* bf16 [total_tokens, hkv, d]                             */
  const float* q_weight;       /* fp32 [d], 16-byte aligned, or NULL: ones                */
  const float* k_weight;       /* fp32 [d], 16-byte aligned, or NULL: ones                */
  const float* cos_sin;        /* fp32 [max_pos, rotary_dim], cosines then sines; or NULL */
  int max_pos;                 /* rows of cos_sin (>= 1 with cos_sin)                     */
  const int32_t* positions;    /* int32 [total_tokens]; NULL only without cos_sin, and in
                                  attn_cache_append_rope (there: the cached positions)    */
  gcs_strides q_stride, k_stride;          /* layouts of q and k                          */
  gcs_strides q_out_stride, k_out_stride;  /* of q_out and k_out (backward: dq_out, dk_out) */
  gcs_strides dq_stride, dk_stride;        /* backward: of dq and dk                      */
} gcs_qk_rope_args;

/* Forward.  q_out bf16 [total_tokens, hq, d] (q_out_stride), k_out bf16 [total_tokens, hkv, d]
 * (k_out_stride).  No workspace. */
int attn_qk_norm_rope_fwd(const gcs_qk_rope_args* a, void* q_out, void* k_out, gcs_stream_t stream);

/* Backward of L = sum(q_out * dq_out) + sum(k_out * dk_out): dq, dk (bf16) and, with the norm,
 * dq_weight and dk_weight (fp32 [d], summed over tokens and heads; each may be NULL when it is
 * not wanted, and must be NULL when its weight is NULL).  Reads the forward's q and k (with
 * norm = 0 they are not read).  Every gradient is summed in a fixed order, so repeated calls
 * give the same bits.  The workspace (256-byte aligned) holds the blocks' parts of the weights'
 * gradients; none is needed when neither is wanted.  Calls that may run at the same time (two
 * streams, two graphs) need one each. */
size_t attn_qk_norm_rope_bwd_workspace(const gcs_qk_rope_args* a);
int attn_qk_norm_rope_bwd(const gcs_qk_rope_args* a, const void* dq_out, const void* dk_out, void* dq, void* dk,
                          float* dq_weight, float* dk_weight, void* workspace, size_t workspace_bytes,
                          gcs_stream_t stream);

/* ------------------------------------------------------------------ write and read of the paged cache
 * The cache has the layout that attn_decode_paged and attn_prefill_paged read.  They attend over it
 * where they support its shape: d 128 with 8 or 16 query heads a kv head, and for
 * attn_prefill_paged an fp8 cache.  These calls take more (d 64, 256 and 512, any group, bf16 in
 * chunks): over such a cache the way on is attn_cache_gather and attn_fwd.  Packed row t belongs to
 * request r with cu_rows[r] <= t < cu_rows[r + 1]; with len = cu_rows[r + 1] - cu_rows[r] it is
 * cached position p = seq_lens[r] - len + t - cu_rows[r], like the paged calls' query rows: the
 * same cu_q, seq_lens and block_table serve an append and the attention call after it.  Rows
 * from cu_rows[num_reqs] on (a padded batch) are left out.
 *   fp8, per token:  scale = max|x| / 448 over the d elements of (token, kv head), written to
 *                    k_scale / v_scale; code = e4m3(x / scale), nearest even.  A row of zeros
 *                    has scale 0 and codes 0.  An infinity gives scale inf, a NaN scale NaN
 *                    (and the row reads back as NaN).
 *   fp8, per tensor: code = e4m3(x / scale) saturating at +-448, with the caller's scale (read;
 *                    codes 0 where it is not above 0).
 *   bf16:            the elements.
 *   gates:           g_cache at p = (g_cache at p - 1, or 0 before the first) + log_gate, in fp32,
 *                    running on through the request's rows.  (Each 64 positions add up the sums of
 *                    all before them: a part of the work grows with the square of a request's rows.)
 * Slots outside the rows' positions are not touched.
 * Preconditions: no two rows share a slot (blocks that are written belong to one request), and
 * cu_rows is sorted from 0.  A row whose position or block-table entry lies outside the cache
 * (0 <= p < max_blocks_per_req * block_size, entry in [0, num_blocks)) is left out, and
 * GCS_ERR_INVALID_ARG is recorded in the device status word: in every mode; checked mode adds nothing
 * to these calls.  So are the gates of a request with any position outside, and those that have no
 * cached gate inside to continue from.
 * Supported: d 64, 128, 256 or 512; any hq, hkv with hq % hkv == 0; block_size 16 x 2^k, 16..4096;
 * the cache strides of gcs_decode_args.  K and V may interleave within one buffer (block by block,
 * slot by slot or head by head) as long as no byte belongs to both. */
typedef struct {
  int num_reqs;                /* >= 1                                                    */
  const int32_t* cu_rows;      /* device int32 [num_reqs + 1]                            */
  int total_rows;              /* rows of the packed tensors, >= 1                        */
  int max_rows;                /* host upper bound on the rows of a request, >= 1 (it chooses
                                  how the gates are summed; nothing else depends on it)   */
  const int32_t* seq_lens;     /* device int32 [num_reqs]: cached tokens, these rows included */
  const int32_t* block_table;  /* device int32 [num_reqs, max_blocks_per_req]            */
  int max_blocks_per_req;
  void* k_cache;               /* fp8 e4m3 or bf16 [num_blocks, hkv, block_size, d]      */
  void* v_cache;               /* same format and strides                                 */
  float* k_scale;              /* fp32 [num_blocks, hkv, block_size], or [1], or NULL    */
  float* v_scale;
  int num_blocks, block_size;
  int hq, hkv, d;              /* hq: heads of the gates and of the rotated queries       */
  int kv_format, scale_mode;   /* as in gcs_decode_args                                   */
  float* g_cache;              /* fp32 [num_blocks, hq, block_size], or NULL              */
  int64_t kv_stride_block, kv_stride_head, kv_stride_slot;  /* as in gcs_decode_args      */
  gcs_strides k_stride, v_stride;  /* layouts of the packed k and v                       */
  const int32_t* first_lens;   /* attn_cache_compact: device int32 [num_reqs], or NULL: 0; the
                                  other calls do not look at it                           */
} gcs_cache_args;

/* Workspace bytes of the two append calls (256-byte aligned; 0 without g_cache and for short
 * appends).  Calls that may run at the same time (two streams, two graphs) need one each. */
size_t attn_cache_append_workspace(const gcs_cache_args* a);

/* Write k, v (bf16 [total_rows, hkv, d]) and, with g_cache, log_gate (fp32 [total_rows, hq]; NULL
 * exactly when g_cache is) into the cache. */
int attn_cache_append(const gcs_cache_args* a, const void* k, const void* v, const float* log_gate, void* workspace,
                      size_t workspace_bytes, gcs_stream_t stream);

/* attn_qk_norm_rope_fwd and attn_cache_append in one launch: r->q goes through norm and rotation
 * into q_out (r->q_out_stride), r->k straight into the cache (quantised from fp32, without the
 * rounding to bf16 in between), v as it is.  r's total_tokens, hq, hkv and d are those of a;
 * a->k_stride is not used.  r->positions NULL: the cached positions; otherwise a row with a
 * negative position is padding and left out of q_out and of the cache (not of the gates). */
int attn_cache_append_rope(const gcs_cache_args* a, const gcs_qk_rope_args* r, const void* v, const float* log_gate,
                           void* q_out, void* workspace, size_t workspace_bytes, gcs_stream_t stream);

/* Read the rows back: k, v bf16 [total_rows, hkv, d] (a->k_stride, a->v_stride), each value
 * bf16(code * scale); log_gate (with g_cache; NULL exactly when g_cache is) fp32 [total_rows, hq],
 * g_cache at p minus g_cache at p - 1 (or 0).  With cu_rows the cumulated seq_lens the whole cache is
 * read, as attn_fwd takes it; with fewer rows the last ones of each request.  A log gate whose
 * g_cache at p - 1 lies in a block outside the cache is left out (and recorded); blocks that hold
 * neither the rows nor the gate before the first are not looked at.  The caches, scales and g_cache
 * are only read.  No workspace. */
int attn_cache_gather(const gcs_cache_args* a, void* k, void* v, float* log_gate, gcs_stream_t stream);

/* ------------------------------------------------------------------ eviction from the paged cache
 * A cache that outgrows its memory keeps the tokens that the queries look at.  attn_cache_weights adds
 * up the attention weight of every cached token, attn_cache_select chooses the tokens that stay, and
 * attn_cache_compact moves them to the front of the request's pages; the blocks behind them are
 * free.  Each kv head keeps tokens of its own, as many as the others, in their order.  After it:
 *   - seq_lens of the next calls are kept_lens, and a token's position in the cache is no longer its
 *     place in the text: attn_cache_append_rope then takes the positions from the caller, and a
 *     window counts cached tokens.  Cumulative gates stay as they are: their differences
 *     are still the sums of the log gates between two tokens.
 *   - with gates, every kv head's last token has to stay (recent >= 1): the next append runs on from the
 *     gates of the cached position in front of it, and the log gates of tokens between that one and the
 *     end would be missing from all later tokens.  In checked mode attn_cache_compact with g_cache leaves
 *     out a request of which some kv head keeps tokens but not the last, and records it.
 *   - blocks whose tokens all stay where they are are not written.  Where requests share the blocks of a
 *     prefix, first_lens covers it in all three calls, and each request's budget (and max_keep) is at least
 *     first_lens + recent, or its seq_len: the choice takes the last tokens before the first ones, and
 *     with less they would go to the prefix's places.  attn_cache_compact leaves such a request out.
 * w_cache is fp32 [num_blocks, hkv, block_size], contiguous and 16-byte aligned, like the scales.
 * Like the cache calls, these check every index that they take from a device array, in every
 * mode (checked mode adds only what is said above): a request whose lengths do not fit (cu_q not
 * sorted within 0 .. total_q, q_len above max_q_len or seq_len, seq_len above max_seq_len or the table)
 * is left out, a key whose block-table entry is not in [0, num_blocks) is left out, and
 * GCS_ERR_INVALID_ARG is recorded in the device status word.
 *
 * Weights.  With the scores s of attn_decode_paged (scale, causal mask at the end of the context,
 * and gates, window and sink where given), for every cached token j of a request and every kv head:
 *     w_j = decay * w_j + sum_t sum_h exp(s_thj - lse_th)
 * over the request's query rows t and the kv head's query heads h, lse_th the row's sum of exponentials
 * with the sink.  The rows' own tokens (the last q_len positions) start from 0: no earlier call has
 * written them.  So do all with decay = 0 (w_cache is not read then).  Slots past seq_len are not
 * touched.  A request without query rows has its weights multiplied by decay.
 * first_lens: device int32 [num_reqs], or NULL (0): the weights of each request's first tokens are left as
 * they are (those below 0: none).  No block that is written may belong to another request: where
 * requests share the blocks of a prefix, first_lens covers it, here as in the choice.
 * a: the arguments of attn_decode_paged or attn_prefill_paged; v_cache, v_scale, segment_len
 * and out_stride are not looked at.  Any q_len in 0 .. seq_len, d 64, 128, 256 or 512, any hq and
 * hkv with hq % hkv == 0, fp8 or bf16 caches.  With an fp8 cache q is rounded to f16, as in the
 * attention calls (|q| <= 65504).
 * lse: fp32 [hq, total_q] natural log, as attn_fwd gives it, or NULL: summed here first, which reads
 * the keys once more; a row whose lse is -inf adds nothing, whatever its elements are.  decay: finite.
 * Every sum has a fixed order: repeated calls give the same bits.  The workspace (256-byte aligned)
 * holds the sums' parts (none with lse) and, for many rows, their constants and mostly a copy of the
 * queries; calls that may run at the same time need one each. */
size_t attn_cache_weights_workspace(const gcs_decode_args* a, int with_lse);
int attn_cache_weights(const gcs_decode_args* a, const float* lse, const int32_t* first_lens, float decay,
                       float* w_cache, void* workspace, size_t workspace_bytes, gcs_stream_t stream);

/* Choice.  Of the L = seq_lens[r] tokens of request r, n = min(budgets[r], L, max_keep) stay (0 if
 * that is negative): the last `recent` (the latest of them when n is smaller), then the first
 * first_lens[r] (the lowest positions), then those of the largest weight; of equal weights (0 and -0 are
 * equal) the lowest positions, and a NaN or a token whose block lies outside the cache weighs less
 * than anything.  kept int32 [num_reqs, hkv, max_keep]: their positions in
 * ascending order, -1 behind them; kept_lens int32 [num_reqs]: n (0 for a request that is left out).
 * No workspace. */
typedef struct {
  int num_reqs;                /* >= 1                                                    */
  const int32_t* seq_lens;     /* device int32 [num_reqs], each <= max_seq_len           */
  int max_seq_len;             /* host upper bound on seq_lens, within the table          */
  const int32_t* block_table;  /* device int32 [num_reqs, max_blocks_per_req]            */
  int max_blocks_per_req;
  int num_blocks, block_size;  /* block_size 16 x 2^k, 16..4096                           */
  int hkv;
  const float* w_cache;        /* fp32 [num_blocks, hkv, block_size]                     */
  const int32_t* budgets;      /* device int32 [num_reqs]: tokens that may stay          */
  const int32_t* first_lens;   /* device int32 [num_reqs], or NULL: 0                    */
  int recent;                  /* >= 0                                                    */
  int max_keep;                /* >= 1: row length of kept                                */
} gcs_select_args;
int attn_cache_select(const gcs_select_args* a, int32_t* kept, int32_t* kept_lens, gcs_stream_t stream);

/* Move.  For every request r, kv head and i < kept_lens[r], cached position i takes what position
 * kept[r][kv head][i] holds: K, V, per-token scales, with a->g_cache the gates of the kv head's
 * query heads, with w_cache the weights (NULL: left).  In place; every source is read before it is
 * overwritten.  Needs kept[i] >= i (ascending positions are): an entry below i or at or past
 * seq_lens[r] is left out and recorded, and so is a request with kept_lens outside 0 ..
 * min(seq_len, max_keep).  a->first_lens: the places of each request's first tokens are not written: a
 * request that would move others there (some kv head's kept does not begin with 0, 1, ..,
 * min(first_lens, kept_lens) - 1) is left out as a whole and recorded, and its cache is as it was; with
 * positions that do not ascend the entries for these places are.  Slots from kept_lens[r] on are left
 * as they were.
 * a: the cache, its index arrays and hq (with gates); a->seq_lens are the lengths before the
 * move; cu_rows, total_rows, max_rows, k_stride and v_stride are not looked at.  No block
 * that is written may belong to another request: where a prefix's blocks do, first_lens covers them.
 * No workspace. */
int attn_cache_compact(const gcs_cache_args* a, const int32_t* kept, const int32_t* kept_lens, int max_keep,
                       float* w_cache, gcs_stream_t stream);

/* ------------------------------------------------------------------ status
 * Per-device status word written by kernels that gave up on a bounded wait.
 * Copies the word for the current device into *status (synchronous) and, if clear != 0,
 * resets it to GCS_OK.  Returns GCS_OK or GCS_ERR_CUDA. */
int gcs_get_device_status(int* status, int clear);

/* Self-test of the bounded waits (a library diagnostic with no counterpart in the pages).
 * Launches one small kernel on the stream that waits, through the same bounded wait every
 * kernel uses, on a barrier phase that nothing completes.  After the 2 s wait limit it
 * records GCS_ERR_DEVICE_TIMEOUT in the current device's status word and exits; the context
 * stays usable.  Read (and clear) the word with gcs_get_device_status.
 * Returns GCS_OK once the kernel is launched, or GCS_ERR_CUDA. */
int gcs_selftest_bounded_wait(gcs_stream_t stream);

/* ------------------------------------------------------------------ device-content checks
 * A library diagnostic with no counterpart in the pages.  The preconditions checked:
 *   prefill: cu_seqlens[0] == 0, cu_seqlens[num_seqs] == total_tokens, and every length
 *            cu_seqlens[s+1] - cu_seqlens[s] in 0 .. max_seqlen;
 *   paged:   cu_q[0] == 0, cu_q[num_reqs] == total_q; for every request
 *            0 <= q_len <= max_q_len and q_len <= seq_len <= max_seq_len; and, for a request
 *            with q_len >= 1, every block_table entry in [0, num_blocks) from the 128-key tile
 *            that holds the earliest key one of its query rows sees (key 0 without a window)
 *            up to the page of its last cached token (the pages the paged calls can read; behind
 *            a shared prefix those from the block of its first own token on, and for the prefix
 *            those of the group's first request);
 *            with an fp8 cache, the f16 operand limits: every |q| <= 65504 and every V scale
 *            of those pages' slots below seq_len (or the per-tensor V scale) < 255.
 * A failed check records GCS_ERR_INVALID_ARG in the current device's status word (first
 * writer wins, like a timeout); read it with gcs_get_device_status.
 *
 * gcs_set_device_checks(1) turns on checked mode for every later call of this process (0
 * turns it off; other values return GCS_ERR_INVALID_ARG).  In checked mode each attention call
 * (attn_fwd, attn_bwd, attn_decode_paged, attn_prefill_paged, attn_decode_paged_shared) first
 * launches one single-CTA kernel (the last one two) on its stream that checks its arrays and writes a
 * copy of cu_seqlens (or cu_q) to the end of the call's workspace; the call's kernels read that
 * copy.  When a check fails the copy is all zeros, an empty batch: no kernel then reads through an
 * index taken from these arrays, so a broken array cannot send a kernel outside a buffer.
 * The outputs of such a call are unspecified.  The copy takes ((num_seqs or num_reqs) + 1)
 * x 4 bytes, rounded up to 256, more workspace: the *_workspace queries include it while
 * checked mode is on (query them after switching the mode), so attn_fwd and
 * attn_prefill_paged then need a workspace even where they otherwise take none;
 * attn_decode_paged_noalloc keeps it in its scratch.  gcs_get_device_checks returns the mode.
 *
 * gcs_check_prefill_inputs / gcs_check_paged_inputs run the same checks on their own (no
 * copy, nothing else launched) on the stream, after the host validation of attn_fwd (or
 * attn_bwd) and of attn_decode_paged or attn_prefill_paged, whose errors they return.
 * Return GCS_OK once the kernel is launched, or the host validation's error, or
 * GCS_ERR_CUDA. */
int gcs_set_device_checks(int enable);
int gcs_get_device_checks(void);
int gcs_check_prefill_inputs(const gcs_prefill_args* a, gcs_stream_t stream);
int gcs_check_paged_inputs(const gcs_decode_args* a, gcs_stream_t stream);

/* ------------------------------------------------------------------ instrumentation
 * Arms two caller-created CUDA events (cudaEvent_t, passed as void*) for the next attn_fwd,
 * attn_bwd, attn_decode_paged or attn_prefill_paged call made by this host thread (the norm,
 * rotation and cache calls leave them armed): `before`
 * is recorded on the call's stream immediately before its main attention kernels (the
 * prefill forward kernel; the backward's attention kernels -- dQ pass + dK/dV pass, or the
 * wide-head role kernels; the split-K decode kernel; the paged prefill kernel) and `after`
 * immediately after them, so
 * cudaEventElapsedTime(before, after) is their device time.  The events are
 * disarmed once used; passing NULL, NULL disarms them.  Returns GCS_OK. */
int gcs_set_kernel_events(void* before, void* after);

/* Library version string. */
const char* gcs_version(void);

#ifdef __cplusplus
}
#endif

#endif /* GCS_ATTN_H_ */
