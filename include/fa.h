/*
 * fa.h — C ABI of libfa_gb300.so: exact softmax attention, forward and backward,
 * on one NVIDIA GB300 (sm_103a).
 *
 * What it computes (the plain definition; the kernels reach it with an online
 * softmax that never materialises the S x S matrix):
 *
 *   O_i   = sum_j P_ij v_j,   P_ij = exp(scale * q_i.k_j - LSE_i) over the allowed keys j
 *   LSE_i = log( sum_j exp(scale * q_i.k_j) [+ exp(sink_h)] )
 *
 * following the "Flash Attention Tutorial" README (GitHub search results page for
 * "flash attention implementation notes"), sections 1-5 for the forward and
 * section 6 "Key derivations" for the backward (dV = P^T dO; D_i = dO_i.O_i;
 * dS_ij = P_ij (dO_i.v_j - D_i); dQ = scale dS K; dK = scale dS^T Q — the scale
 * is kept in dQ and dK, which that tutorial's listing omits).
 *
 * Masks are bottom-right aligned when s_q != s_kv (vllm-project/flash-attention
 * README, flash_attn_func and flash_attn_with_kvcache docstrings, changelog 2.1):
 * with off = s_kv - s_q of the sequence, query i keeps key j iff
 *   causal      : j <= i + off
 *   window_left  >= 0 : j >= i + off - window_left
 *   window_right >= 0 : j <= i + off + window_right      (inclusive; -1 = unbounded)
 * A causal call with a window keeps the intersection.  A row with no allowed key
 * gets O = 0 and LSE = -inf (LSE = sink_h when the head has a sink).
 *
 * Grouped-query heads: h_kv divides h_q and query head h reads key/value head
 * h / (h_q / h_kv) (same README, flash_attn_func docstring: 6 query heads on 2
 * key/value heads map 0,1,2 -> 0 and 3,4,5 -> 1).
 *
 * Sinks: one fp32 logit per query head joins every row's softmax denominator and
 * carries no value (dew-flash-attn PyPI page, the sinks paragraph).  The returned
 * LSE includes the sink; fa_bwd returns the sink gradient
 *   dsink_h = - sum_rows exp(sink_h - LSE_i) D_i.
 *
 * Packed batches (dew-flash-attn PyPI page, "Packed sequences"; fa4-jax PyPI page,
 * "Varlen semantics"): with cu_seqlens_q / cu_seqlens_k given, tensors are
 * [T, H, D], sequence b owns rows cu[b] .. cu[b+1]-1, masks apply per sequence,
 * attention never crosses sequences, zero-length sequences are legal, and the
 * LSE is laid out [h_q, T_q].  The offsets are read on the device and are not
 * checked unless FA_FLAG_VALIDATE_CU is set (tokens they do not cover get
 * unspecified outputs, as on the pages).  Passing the same array as cu_seqlens_q and
 * cu_seqlens_k (queries and keys packed alike, as in self-attention over a packed batch)
 * lets the d <= 128 kernels tile the packed token axis itself: a 128-row tile then holds
 * several short sequences, each row masked to its own sequence, so a batch of short
 * sequences costs about its tokens rather than a tile per sequence.  Two arrays with equal
 * contents give the same results, with tiles per sequence.
 *
 * Conventions common to every call:
 *  - Layouts: dense tensors are contiguous [B, S, H, D] (bf16 or fp16); packed ones [T, H, D].
 *    LSE is fp32 [B, h_q, s_q] (dense) or [h_q, T_q] (packed), natural log.
 *  - Ownership: every pointer is caller-owned device memory (except the params
 *    struct itself, read on the host during the call).  The library allocates no
 *    device memory; scratch lives in the caller's workspace, sized by the
 *    fa_*_workspace_size functions.  Base pointers of q, k, v, o, dout, dq, dk, dv
 *    and the workspace must be 16-byte aligned.
 *  - Streams: work is enqueued on `stream` (a cudaStream_t; NULL = legacy default
 *    stream) and the call returns without synchronising.
 *  - Errors: arguments are checked on the host before anything is launched; a
 *    violation returns a code and launches nothing.  No C++ exception crosses this
 *    ABI and no kernel traps: a kernel whose pipeline stalls gives up after a time
 *    limit (fa_params.wait_limit_ns) and records FA_ERR_TIMEOUT in the workspace status
 *    word, which fa_read_device_status reports.  Every kernel of a call reads the status
 *    word first and does nothing when it is set, so a failed offset check
 *    (FA_FLAG_VALIDATE_CU) or a timeout leaves the outputs of the rest of the call
 *    unwritten.
 *  - Supported: bf16 and fp16 (and e4m3 for the forward at d = 128, see below); head dim d in
 *    {64, 128, 192, 256} for the forward and the backward (FA_FLAG_DETERMINISTIC included);
 *    h_q / h_kv <= 128.  d = 192 is one of the head sizes the pages pad to (dew-flash-attn
 *    PyPI page, the FA3 head-dim padding to 64 / 128 / 192 / 256).
 *    Anything else returns FA_ERR_UNSUPPORTED.
 *  - Zero-initialise fa_params (memset or `= {0}`): every optional field then means
 *    "not used".
 *
 * Partly filled slots and paged caches:
 *  - seqused_q / seqused_k (fa4-jax PyPI page, "Varlen semantics": optional seqused_q /
 *    seqused_k limit each slot to its first seqused[b] tokens, the cache case where slots
 *    are larger than what is filled): sequence b uses only its first seqused_q[b] queries
 *    and seqused_k[b] keys of its slot (s_q / s_kv for dense tensors, the cu_seqlens
 *    difference for packed ones); the bottom-right alignment uses the used lengths, unused
 *    keys are invisible, and the outputs of unused query rows (O, LSE, dQ) and the dK, dV
 *    rows of unused keys are not written (unspecified).  Values are clamped to [0, slot].
 *    Forward and backward.
 *  - block_table (forward only; fa_bwd returns FA_ERR_UNSUPPORTED; vllm-project/flash-attention
 *    README, flash_attn_with_kvcache docstring ("Does not support backward pass"):
 *    a paged cache of shape (num_blocks, page_block_size, nheads_k, headdim) addressed
 *    through block_table (batch_size, max_num_blocks_per_seq) int32): dense q only; k and
 *    v are page pools [num_pages, page_size, h_kv, d] and key j of sequence b is row
 *    j % page_size of page block_table[b * max_blocks_per_seq + j / page_size].  s_kv is
 *    the logical cache length (at most max_blocks_per_seq * page_size); page_size must be
 *    a positive multiple of 128 (the page's builds ask for 256).  Table entries are read
 *    on the device and not checked.
 *  - block_table with cu_seqlens_q and without cu_seqlens_k (forward only, bf16 and fp16):
 *    packed queries over a paged cache, the form of a serving step, in which each sequence
 *    brings its new tokens (one, a few, a chunk of a prompt) and reads its whole cache, those
 *    tokens' keys included (fa_qk_norm_rope writes them there, fa_page_plan makes the table).
 *    q, o are [T_q, h_q, d] with T_q = s_q, the LSE is [h_q, T_q]; seqused_k is required and
 *    gives the keys of each sequence (clamped to [0, s_kv]), s_kv the longest cache that may
 *    occur.  page_size is a positive multiple of 16.  Offsets are kept within [0, T_q]; rows
 *    of q that no sequence covers (a padded batch) are left as they were.  What a page holds
 *    behind a sequence's used keys, NaN and infinities included, has no effect.  A table entry
 *    that is needed (some query sees a key of its page) and outside the pool is not followed and sets
 *    FA_ERR_DEVICE_CHECK in the status word (the outputs are then unspecified); one that no query needs, of a
 *    page freed behind a sliding window, may be anything.  FA_FLAG_VALIDATE_CU checks cu_seqlens_q (from 0, not decreasing, at most
 *    T_q) and seqused_k.  max_seqlen_q is used when given (the most query rows of a sequence;
 *    it picks the kernel's tile, and a wrong one costs time, not correctness: outputs stay within the
 *    types' roundings).  Results do not
 *    depend on how other work is scheduled: the same call gives the same bits.
 *
 *  - the same form over a cache in 8 bits (cache_dtype = FA_DTYPE_E4M3; dtype is the queries' and the
 *    output's, bf16 or fp16; every head dimension): k and v are pools of e4m3 bytes and the true keys and
 *    values are byte * scale, with one scale for scale_block rows of a page and a head: k_scale,
 *    v_scale [num_pages, page_size / scale_block, h_kv] (fp32, not negative).  scale_block is a positive multiple
 *    of 16 that divides page_size, the scales are finite.  fa_qk_norm_rope_append8 fills such a cache.  All else is
 *    as above; bytes of rows behind a sequence's used keys, and scales of blocks behind them, have no effect.  (A NaN among
 *    the bytes of a value that some query of a sequence sees may reach outputs of that sequence's other queries.)
 *    Two kernels share the work: one for sequences of few rows (8 to 32 of a key/value head's), which leaves the scales outside
 *    its products, and one for more, which takes keys and values times their scales in the queries' type: exactly where
 *    the scales are powers of two, as fa_qk_norm_rope_append8 makes them (fp16: wherever they lie, down to 2^-22 of the largest
 *    among the keys that a work item of up to 256 rows sees), else rounded once more, as a 16-bit cache would hold them.  max_seqlen_q
 *    decides which one takes short sequences, so a hint can change an output by such a rounding.
 *    fp16 outputs are kept within fp16's range (a value near its largest, appended, stands for the next e4m3 value).
 *
 * FP8 forward (vllm-project/flash-attention README, "FlashAttention-3 beta release":
 * "FP8 forward"): with dtype = FA_DTYPE_E4M3, q, k and v hold e4m3 bytes (1 byte per
 * element, same layouts) and the true inputs are q * q_descale[b * h_kv + g] (likewise k,
 * v) for batch b and key/value head g; a NULL descale means 1.  S = Q K^T and O = P V run
 * on the fp8 tensor cores with fp32 accumulation, P is rounded to e4m3 for the second
 * product, o is written as bf16 and lse (fp32) is that of the descaled problem.  d = 128
 * only, dense, packed (cu_seqlens; the descale index b is then the sequence) or with a
 * paged k / v cache; seqused_k, windows, causal and sinks are supported; anything else
 * returns FA_ERR_UNSUPPORTED, and fa_bwd rejects the type.  The workspace is the bf16 forward's for the same shape (v is transposed tile by
 * tile inside the kernel, not copied).
 */
#ifndef FA_GB300_H
#define FA_GB300_H

#include <stddef.h>
#include <stdint.h>

#ifdef __cplusplus
extern "C" {
#endif

struct CUstream_st; /* cudaStream_t is `struct CUstream_st *` */

typedef enum fa_status {
    FA_OK = 0,
    FA_ERR_INVALID_ARG = 1,  /* a null, misaligned or inconsistent argument */
    FA_ERR_UNSUPPORTED = 2,  /* a valid problem this build does not implement */
    FA_ERR_WORKSPACE = 3,    /* workspace smaller than fa_*_workspace_size */
    FA_ERR_CUDA = 4,         /* a CUDA runtime call or launch failed */
    FA_ERR_TIMEOUT = 5,      /* a kernel pipeline stalled and gave up (device status) */
    FA_ERR_DEVICE_CHECK = 6  /* a device-side argument check failed (device status) */
} fa_status;

/* Input element types.  bf16 and fp16 (dew-flash-attn PyPI page, usage: inputs in bf16
 * or fp16; fa4-jax PyPI page, restrictions: fp16/bf16) run every path of fa_fwd and fa_bwd
 * alike: o, dq, dk and dv have the inputs' type, accumulation and lse stay fp32.  e4m3 is
 * the FP8 forward above. */
#define FA_DTYPE_BF16 0
#define FA_DTYPE_E4M3 1
#define FA_DTYPE_F16 2

/* Flags */
#define FA_FLAG_VALIDATE_CU 1u  /* check cu_seqlens on the device; result in the status word */
#define FA_FLAG_NO_SPLIT 2u     /* forward: never split the key range across CTAs */
/* backward: bitwise-reproducible results.  dQ is summed over key blocks in a fixed order
 * (descending key block) instead of in arrival order; the workspace grows by 4 bytes per
 * (query tile, key/value head).  The deterministic backward option of the
 * vllm-project/flash-attention README (changelog 2.4).  A key block's CTA waits (bounded,
 * like every wait: FA_ERR_TIMEOUT) for the later blocks' contributions, which the launch
 * puts at lower CTA indices; slower than the default, markedly so without a causal mask.
 * The sink gradient is summed in a fixed order with or without the flag.  Every head
 * dimension (at d = 192 / 256 the key blocks are 64 keys). */
#define FA_FLAG_DETERMINISTIC 4u

typedef struct fa_params {
    int B;            /* batch (dense) or number of sequences (packed) */
    int s_q, s_kv;    /* sequence lengths (dense); total tokens T_q, T_k (packed) */
    int h_q, h_kv;    /* query heads, key/value heads (h_kv divides h_q) */
    int d;            /* head dimension */
    float softmax_scale;  /* <= 0 selects 1 / sqrt(d) */
    int causal;           /* nonzero: bottom-right aligned causal mask */
    int window_left, window_right;  /* -1 = unbounded side */
    const float *sinks;             /* device fp32 [h_q], or NULL */
    const int32_t *cu_seqlens_q;    /* device int32 [B+1], or NULL for dense tensors */
    const int32_t *cu_seqlens_k;    /* device int32 [B+1]; required iff cu_seqlens_q, absent with block_table */
    int max_seqlen_q, max_seqlen_k; /* optional hints (0 = unknown); never needed */
    unsigned flags;                 /* FA_FLAG_* */
    /* Partly filled slots and paged caches (see above).  Zero / NULL = not used. */
    const int32_t *seqused_k;       /* device int32 [B], or NULL */
    const int32_t *block_table;     /* device int32 [B * max_blocks_per_seq], or NULL */
    int page_size;                  /* keys per page (block_table only) */
    int max_blocks_per_seq;         /* row stride of block_table */
    int num_pages;                  /* pages in each of the k and v pools */
    /* Input element type (FA_DTYPE_*; 0 = bf16).  See the FP8 forward above and the types. */
    int dtype;
    const float *q_descale;         /* FA_DTYPE_E4M3 only: device fp32 [B * h_kv] or NULL (= 1) */
    const float *k_descale;
    const float *v_descale;
    const int32_t *seqused_q;       /* device int32 [B], or NULL (see partly filled slots) */
    /* Bound, in nanoseconds, on each wait of a kernel's pipeline (a stage of copies or
     * MMAs that should have landed); 0 selects 2 s.  A wait that runs past it makes the CTA
     * give up: it records FA_ERR_TIMEOUT in the status word, lets its own copies and MMAs
     * land, frees its tensor memory and returns, and the call's later kernels do nothing.
     * A limit below the kernels' own latencies (a few microseconds) turns every call in which something
     * is waited for into such a failure, which is how the failure path is exercised; outputs of a
     * failed call are unspecified. */
    unsigned long long wait_limit_ns;
    /* A cache in 8 bits (packed queries over a paged cache only; see above) */
    int cache_dtype;        /* 0: k and v have the queries' type; FA_DTYPE_E4M3 */
    int scale_block;        /* rows of a page that share a scale */
    const float *k_scale;   /* device fp32 [num_pages, page_size / scale_block, h_kv] */
    const float *v_scale;
} fa_params;

/* Bytes of workspace fa_fwd / fa_bwd need for these parameters (>= 256: the first
 * 256 bytes hold the device status word).  Returns 0 when the parameters are
 * invalid or unsupported.  The forward's plan (key splits, and the split of a last
 * partial wave of work at d = 192 / 256) follows the current device's SM count, so the
 * size is queried with the device that will run the call current. */
size_t fa_fwd_workspace_size(const fa_params *p);
size_t fa_bwd_workspace_size(const fa_params *p);

/* Forward.  q: [.., h_q, d]; k, v: [.., h_kv, d]; o: layout of q (written);
 * lse: fp32 (written; may be NULL when not wanted). */
fa_status fa_fwd(const fa_params *p, const void *q, const void *k, const void *v, void *o, float *lse,
                 void *workspace, size_t workspace_bytes, struct CUstream_st *stream);

/* Backward of L = sum(O * dout).  o and lse must be what fa_fwd returned for the
 * same inputs.  dq: layout of q; dk, dv: layout of k (all written, in the inputs' type).
 * dsinks: fp32 [h_q], written when p->sinks is given (must then be non-NULL). */
fa_status fa_bwd(const fa_params *p, const void *q, const void *k, const void *v, const void *o,
                 const float *lse, const void *dout, void *dq, void *dk, void *dv, float *dsinks,
                 void *workspace, size_t workspace_bytes, struct CUstream_st *stream);

/* Norm and position rotation of queries and keys (training and serving), ahead of fa_fwd.
 * For each token t and head, with x the head's d values and w its weight (q_weight or
 * k_weight, shared by the heads; NULL = ones):
 *   y = x * w / sqrt(mean(x^2) + eps),
 * then the pairs (a, b) of y's first rot_dim values turn by the token's angles:
 *   (a, b) -> (a cos - b sin, b cos + a sin).
 * The pairs are (j, j + rot_dim / 2), or with `interleaved` (2j, 2j + 1), j < rot_dim / 2, and use
 * cos[pos][j], sin[pos][j].  pos is positions[t], or t % seq_len without positions.  A token
 * at position -1 is padding and is skipped (its rows of the outputs are left as they were, or
 * with zero_skipped become 0; a cache is left alone either way); any other
 * position outside [0, max_pos) is skipped too and sets *status (when given) to
 * FA_ERR_DEVICE_CHECK.  Statistics and products are fp32, outputs are rounded once.
 * fa_qk_norm_rope writes q_out [T, h_q, d] and k_out [T, h_kv, d] (contiguous).  With k_cache,
 * v_cache (pools of num_slots rows [h_kv, d]), slots and v it also writes the key's row and a
 * copy of v's to row slots[t] of the pools (k_out may then be NULL); slot -1 is not stored, one
 * outside [-1, num_slots) is not stored either and sets *status.  Two tokens with one slot
 * leave a mix of their rows there (each 16 bytes one's or the other's).  q_out may be q and k_out may be k (contiguous); other overlaps are refused.
 * fa_qk_norm_rope_bwd takes the inputs and the gradients of q_out and k_out (contiguous) and
 * writes dq, dk (token strides dq_stride, dk_stride; dq may be q or dq_out and dk may be k or
 * dk_out, in the same layout; rows that share bytes in any other way are refused) and
 * dq_weight, dk_weight (fp32 [d], written whole, summed in a fixed order: the same bits from
 * call to call).  A skipped token adds nothing to them.  They and the workspace share no byte
 * with anything else of the call.
 * Several position axes (text, images, video: time, height, width): with axes = 2 to FA_ROPE_MAX_AXES
 * positions is [axes][T] (and must be given), and pair j turns by cos[pos][j], sin[pos][j] at its own
 * axis's position, pos = positions[pair_axis[j]][t].  The axes share the tables.  A token with -1 on
 * some axis is padding; one with another position outside [0, max_pos) on some axis sets *status.
 * Without the norm (no_norm; the weights must be NULL): y = x.  The gradient then reads neither q nor k,
 * which may be NULL, and has no weights' gradients (dq_weight and dk_weight must be NULL); the workspace is
 * given all the same.
 * A wait that passes wait_limit_ns ends the call's work early and sets *status to FA_ERR_TIMEOUT
 * (the outputs are then unspecified); without a status word the caller does not learn of it.
 * bf16 and fp16; d in {64, 128, 192, 256}; rot_dim a multiple of 16 up to d; strides multiples
 * of 8 elements, base pointers 16-byte aligned. */
#define FA_ROPE_MAX_AXES 4
#define FA_ROPE_MAX_PAIRS 128
typedef struct fa_rope_params {
    int T;                 /* tokens */
    int h_q, h_kv, d;
    int rot_dim;           /* leading values of a head that are rotated (0 = none) */
    int interleaved;       /* pairs (2j, 2j+1) instead of (j, j + rot_dim/2) */
    int seq_len;           /* without positions: token t is at position t % seq_len */
    int max_pos;           /* rows of cos and sin */
    float eps;
    int dtype;             /* FA_DTYPE_BF16 or FA_DTYPE_F16 */
    int weight_f32;        /* the weights are fp32 (0: the tensors' type) */
    long long q_stride, k_stride, v_stride;   /* elements from token to token of q, k, v */
    long long dq_stride, dk_stride;           /* gradient only: of dq, dk */
    const int32_t *positions;                 /* device int32 [T], or NULL */
    const float *cos, *sin;                   /* device fp32 [max_pos, rot_dim/2] */
    const void *q_weight, *k_weight;          /* device [d], or NULL (ones) */
    const int32_t *slots;                     /* device int32 [T]: cache rows, or NULL */
    long long num_slots;                      /* num_pages * page_size */
    int32_t *status;                          /* device int32, set on a bad position or slot or a timeout, never cleared; or NULL */
    int zero_skipped;                         /* q_out, k_out (dq, dk) of skipped tokens become 0 */
    unsigned long long wait_limit_ns;         /* bound on each wait of the kernels; 0 = 2 s */
    int axes;              /* position axes; 0 or 1: one */
    int no_norm;           /* y = x turned */
    unsigned char pair_axis[FA_ROPE_MAX_PAIRS];  /* with several axes: the axis of pair j < rot_dim / 2 */
} fa_rope_params;

fa_status fa_qk_norm_rope(const fa_rope_params *p, const void *q, const void *k, const void *v, void *q_out, void *k_out,
                          void *k_cache, void *v_cache, struct CUstream_st *stream);

/* Norm and rotation with append to a cache in 8 bits: queries and keys as in fa_qk_norm_rope, the keys
 * and a copy of v to pools of e4m3 bytes k_cache, v_cache [num_pages, page_size, h_kv, d] with a
 * scale for each block of scale_block rows of a page and each head, k_scale, v_scale
 * [num_pages, page_size / scale_block, h_kv]: a byte stands for its e4m3 value times its block's scale.
 * The new tokens of sequence b are rows cu_seqlens_q[b] .. cu_seqlens_q[b+1] - 1 and the last of its
 * seqused_k[b] keys (as fa_page_plan leaves them and fa_fwd takes them); key j is row j % page_size of
 * page block_table[b * max_blocks_per_seq + j / page_size].  Offsets are kept within [0, T] and may begin at any row (rows ahead
 * of the first one, as those behind the last, belong to no sequence); where they decrease, *status is set and tokens
 * of the sequences concerned may not be stored.  For each block that gets new rows
 *   s = max(old scale, smallest power of two with (largest finite |x| of its new rows) <= 448 s),
 * (at least 2^-126; the old scale counts as 0 where the block's first row is a new one and where it is no
 * positive finite number), new rows become e4m3(x / s), rounded once from fp32 (infinities: the largest
 * value, NaN: NaN; with an old scale that is no power of two x / s is itself off by up to 2^-23 of it), the block's
 * rows ahead of them are rescaled where s has grown (e4m3(byte * old / s)), rows behind them are left as they were.  A block that gets new rows must be the
 * writing sequence's alone.  positions must be given (they drive the rotation; the table and the
 * lengths say where a token goes); slots must be NULL, zero_skipped and q_out are as in fa_qk_norm_rope, q_out may be q
 * (contiguous).  A token that fa_qk_norm_rope would skip is not stored; nor is one of no sequence, and one whose
 * place is negative or behind the table or whose page is outside the pool, which sets *status.  A block of which a call
 * stores nothing is left alone, its scale too: where a sequence's first tokens in a block are all skipped, set the
 * scale to 0 before the next ones are appended, or what an earlier owner of the page left there counts as old.
 * page_size a positive multiple of 16, scale_block a positive multiple of 16 that divides it. */
typedef struct fa_cache8_params {
    int B;                        /* sequences */
    int page_size, max_blocks_per_seq, num_pages;
    int scale_block;              /* rows of a page that share a scale */
    const int32_t *cu_seqlens_q;  /* device int32 [B + 1] */
    const int32_t *seqused_k;     /* device int32 [B] */
    const int32_t *block_table;   /* device int32 [B * max_blocks_per_seq] */
} fa_cache8_params;

fa_status fa_qk_norm_rope_append8(const fa_rope_params *p, const fa_cache8_params *cache, const void *q, const void *k, const void *v,
                                  void *q_out, void *k_cache, void *v_cache, float *k_scale, float *v_scale,
                                  struct CUstream_st *stream);
size_t fa_qk_norm_rope_bwd_workspace_size(const fa_rope_params *p);
fa_status fa_qk_norm_rope_bwd(const fa_rope_params *p, const void *q, const void *k, const void *dq_out, const void *dk_out,
                              void *dq, void *dk, float *dq_weight, float *dk_weight, void *workspace, size_t workspace_bytes,
                              struct CUstream_st *stream);

/* Page plan of a serving step, from the requests' lengths: request b has cached[b] tokens in
 * its pages and brings fresh[b] new ones.  Takes the pages they need from free_pages (device
 * int32 [n_free]) from index *free_head on (NULL: 0), in the order of the requests, and writes
 *   block_table   the new pages' entries of each row (others are left as they were)
 *   cu_seqlens_q  [B + 1], seqused_k [B] = cached + fresh (not the arrays cached or fresh)
 *   positions, slots   [T]: place in its sequence and cache row (page * page_size + offset) of
 *                 each new token, packed request by request; -1 behind the last one
 *   free_head_out [1] = *free_head + pages taken (not the same word as free_head)
 * what fa_qk_norm_rope and fa_fwd take.  Pages past the end of the list or outside
 * [0, num_pages), table entries outside it, negative lengths (taken as 0), requests beyond
 * max_blocks_per_seq pages and more than T new tokens set *status (when given) to
 * FA_ERR_DEVICE_CHECK; the tokens concerned get slot -1 (and lengths are cut to what fits). */
typedef struct fa_page_plan_params {
    int B, T;                /* requests; rows of the packed batch (at least the new tokens) */
    int page_size, max_blocks_per_seq, num_pages;
    int n_free;              /* entries of free_pages */
} fa_page_plan_params;

fa_status fa_page_plan(const fa_page_plan_params *p, const int32_t *cached, const int32_t *fresh, const int32_t *free_pages,
                       const int32_t *free_head, int32_t *block_table, int32_t *cu_seqlens_q, int32_t *seqused_k,
                       int32_t *positions, int32_t *slots, int32_t *free_head_out, int32_t *status, struct CUstream_st *stream);

/* Synchronises `stream` and returns the status word the kernels of the last call
 * on this workspace left (FA_OK, FA_ERR_TIMEOUT or FA_ERR_DEVICE_CHECK), or
 * FA_ERR_CUDA if the stream itself reports an error. */
fa_status fa_read_device_status(const void *workspace, struct CUstream_st *stream);

/* Static text for a status code. */
const char *fa_status_string(fa_status s);

/* Per-kernel timing: when enabled, every launch the library makes is bracketed by
 * CUDA events on its stream.  fa_profile_read synchronises on the last launch of
 * the named kernel ("fwd", "decode", "combine", "bwd_pre", "bwd_main", "bwd_post",
 * "paged_prep", "paged_few", "paged_merge", "norm_rope", "norm_rope_bwd", "page_plan",
 * "append8")
 * and writes its duration in milliseconds; returns FA_ERR_INVALID_ARG for an
 * unknown name or a kernel not launched since profiling was enabled. */
fa_status fa_profile_enable(int on);
fa_status fa_profile_read(const char *kernel, float *ms);

/* Forward without a caller workspace, for callers that cannot allocate device memory
 * (a host framework that owns every allocation, or a loop that must not enter the CUDA
 * allocator).  No passage on the pages has a counterpart: it is fa_fwd run on a scratch
 * array of FA_NOALLOC_SCRATCH_BYTES (64 MiB) compiled into the library, which every GPU
 * that loads the library holds until the process exits.  Arguments, layouts and results
 * are those of fa_fwd.  Allocates nothing.  Returns FA_ERR_WORKSPACE, launching nothing,
 * when the problem needs more scratch than the array holds (fa_fwd_workspace_size(p)
 * larger than FA_NOALLOC_SCRATCH_BYTES); FA_ERR_CUDA if the array's address cannot be
 * had.  The first call on each device looks the array's address up (and again after the
 * device's context was destroyed and made anew, e.g. by cudaDeviceReset), so make the
 * first call, and the first after such a reset, before any stream capture.  All calls share the array and it keeps the last call's contents:
 * each call resets what must start at zero, but calls that overlap on the GPU race on
 * it, so serialise them (one stream, or events between streams).  The kernels' status
 * word also lives in the array and is not readable through this ABI. */
#define FA_NOALLOC_SCRATCH_BYTES ((size_t)64 << 20)
fa_status fa_fwd_noalloc(const fa_params *p, const void *q, const void *k, const void *v, void *o, float *lse,
                         struct CUstream_st *stream);

/* Library version string. */
const char *fa_version(void);

#ifdef __cplusplus
}
#endif

#endif /* FA_GB300_H */
