/*
 * msa.h -- C ABI of libmsa.so: MiniMax Sparse Attention (MSA) training on one GB300 (sm_103a).
 *
 * The method (Flash-MSA blog, "About MSA"; MSA forum summary, "Architecture: two-stage
 * block-sparse attention"): causal GQA attention in which one proxy (index) query head per GQA
 * group, scored against one shared proxy key head, picks for every query the top-k 128-token key
 * blocks -- the query's own (local) block always among them -- and the main attention runs
 * exactly, with softmax, over the picked blocks only.  The proxy is trained by a KL loss towards
 * the group's mean main-attention distribution over the same tokens (blog, "KL Divergence Loss").
 *
 * Conventions shared by every entry point
 *   Tensors are dense, row-major, on the current CUDA device, caller-owned:
 *     q, o, dout, dq    [B, S, Hq,  128]  bf16
 *     k, v, dk, dv      [B, S, Hkv, 128]  bf16
 *     qp, dqp           [B, S, Hp,  128]  bf16   (proxy queries, one head per selection row)
 *     kp, dkp           [B, S, 1,   128]  bf16   (one proxy key head shared by every proxy head)
 *     lse               [B, Hq, S]        fp32   natural-log sum of exp of the scaled scores
 *     block_idx         [B, Hp, S, top_k] int32  selected key blocks per (b, proxy head, token),
 *                                                ascending, padded with -1 when fewer than
 *                                                top_k blocks are visible
 *   Head mapping (blog, "Context parallelism" point 1: an MSA group is the query heads assigned
 *   to one proxy head; "Note about scheduler requiring proxy heads >= KV heads": more KV heads
 *   than proxy heads inverts that mapping; the top-k sweep footnote runs 4 proxy heads over 2 KV
 *   heads): query head h reads KV head h / (Hq / Hkv) and takes the selection of proxy head
 *   h / (Hq / Hp).  Hq must be a multiple of Hkv and of Hp, and one
 *   of Hp, Hkv a multiple of the other.  The KL teacher of proxy head p is the mean main
 *   softmax of its Hq / Hp query heads.  Key j is visible to token t iff j <= t.
 *   Every pointer must be 16-byte aligned (seq_len, positions and inv_freq: 4-byte).  Supported: head dim 128, block 128 (blog / package
 *   caveat 1), S % 128 == 0, 1 <= top_k <= 64, and Hq / max(Hp, Hkv) -- the query heads that
 *   share both one KV head and one selection row -- in {1, 2, 4, 8, 16} for the forward ops and
 *   {4, 8, 16} for the backward ops (the warmup forward, which has no selection: Hq / Hkv).
 *   Other shapes return MSA_ERR_UNSUPPORTED.
 *   `workspace` is caller-owned device memory of at least msa_workspace_size() bytes for the
 *   same op and shape; the library allocates no device memory.  The first 256 bytes hold a device status
 *   word (see msa_device_status) and the work-item counters of the persistent kernels (reset on
 *   the stream before each launch).  Calls sharing one workspace must not overlap on the GPU.
 *   `stream` is a cudaStream_t (NULL = legacy default stream); all work is asynchronous and
 *   ordered on it.  The backward ops run two independent memory-bound steps (zeroing of their
 *   accumulators with the row data D; the bf16 conversion of dQ, dK, dV) on a side stream that the
 *   library creates once per host thread and device, forked from `stream` with an event and
 *   joined back into it before the call returns: the call's work still completes in `stream`'s
 *   order, and a CUDA graph capture of the call stays closed.
 *   Return value: an msa_status code.  Argument errors are detected on the host before any
 *   launch; MSA_ERR_CUDA reports a launch or runtime error (msa_last_error() gives the text).
 *   No entry point synchronises the device except msa_device_status.
 */
#ifndef MSA_H_
#define MSA_H_

#include <stddef.h>
#include <stdint.h>

#if defined(__GNUC__)
#define MSA_API __attribute__((visibility("default")))
#else
#define MSA_API
#endif

#ifdef __cplusplus
extern "C" {
#endif

typedef struct msa_shape {
  int32_t B;      /* batch */
  int32_t S;      /* sequence length, multiple of 128 */
  int32_t Hq;     /* main query heads */
  int32_t Hkv;    /* main key/value heads (GQA groups) */
  int32_t Hp;     /* proxy query heads (see the head mapping above) */
  int32_t D;      /* head dim, must be 128 */
  int32_t top_k;  /* selected blocks per query, local block included (ignored by warmup ops) */
  float scale;    /* softmax scale of both attentions, usually 128^-0.5 */
} msa_shape_t;

enum msa_status {
  MSA_OK = 0,
  MSA_ERR_INVALID_ARG = 1, /* null / misaligned pointer, non-positive size */
  MSA_ERR_UNSUPPORTED = 2, /* D != 128, S % 128 != 0, head counts, group size or top_k */
  MSA_ERR_WORKSPACE = 3,   /* workspace too small */
  MSA_ERR_CUDA = 4         /* CUDA launch / runtime error */
};

enum msa_op {
  MSA_OP_FORWARD = 0,
  MSA_OP_BACKWARD = 1,
  MSA_OP_WARMUP_FORWARD = 2,
  MSA_OP_WARMUP_BACKWARD = 3,
  MSA_OP_DECODE = 4,
  MSA_OP_WINDOW_FORWARD = 5, /* msa_window_workspace_size */
  MSA_OP_WINDOW_BACKWARD = 6,
  MSA_OP_WINDOW_DECODE = 7,
  MSA_OP_NORM_ROPE_BACKWARD = 8, /* msa_norm_rope_workspace_size */
  MSA_OP_NORM_ROPE_APPEND = 9,
  MSA_OP_DECODE_Q4 = 10,       /* msa_workspace_size */
  MSA_OP_WINDOW_DECODE_Q4 = 11, /* msa_window_workspace_size */
  MSA_OP_PACKED_FORWARD = 12,   /* msa_packed_workspace_size */
  MSA_OP_PACKED_BACKWARD = 13
};

/* Bits of the device status word. */
#define MSA_DEVICE_BAD_INDEX 1u /* a given block index was out of range or not ascending */
#define MSA_DEVICE_BAD_ITEMS 2u /* internal work list overflow (a library bug) */
#define MSA_DEVICE_TIMEOUT 4u   /* a bounded device-side wait gave up */
#define MSA_DEVICE_INTERNAL 8u  /* a kernel's internal layout check failed (a library bug) */
/* With MSA_DEVICE_TIMEOUT set, the 32-bit word at byte offset 64 of the workspace may name the
 * first wait that gave up (a nonzero place number of the kernel that set it); diagnostic only. */

/* Bytes of workspace `op` needs for `shape` (0 if the shape is unsupported). */
MSA_API size_t msa_workspace_size(const msa_shape_t* shape, int op);

/*
 * Sparse forward (blog, "Forward": proxy attention, then sparse main attention; package usage
 * `flash_msa_func`).
 *   1. unless indices_given: proxy scores Qp.Kp^T per group, causal max-pool per 128-key block,
 *      the local block forced in, top-k with ties going to the lower block index
 *      (blog "Proxy attention") -> block_idx (written);
 *   2. exact softmax attention of every query head over the key blocks of its group in
 *      block_idx (blog "Main attention"; forum summary "Architecture") -> o, lse.
 * indices_given != 0: block_idx is an input (for instance the cached indices of an earlier
 * call); invalid entries are skipped and flagged with MSA_DEVICE_BAD_INDEX.
 * Workspace: the per-(token, head, slot) partial outputs of step 2 are produced and merged in
 * passes over consecutive sequence chunks.  msa_workspace_size sizes them for passes of at most
 * 8 GiB of partials; a larger workspace_bytes gives fewer passes, a smaller one more (down to one
 * chunk per pass; below that MSA_ERR_WORKSPACE).  The results do not depend on the passes.
 */
MSA_API int msa_forward(const msa_shape_t* shape, const void* q, const void* k, const void* v,
                const void* qp, const void* kp, int32_t* block_idx, int indices_given, void* o,
                float* lse, void* workspace, size_t workspace_bytes, void* stream);

/*
 * Sparse backward (blog, "Backward" and "KL Divergence Loss").  From the cached block_idx it
 * inverts the block map, recomputes the proxy normaliser over the selected tokens, and in one
 * fused pass per (key block, group) recomputes the main and proxy probabilities and emits
 *   dq, dk, dv  of  sum(o * dout)                     (teacher detached: no KL term here)
 *   dqp, dkp    of  kl_grad * L_KL,  L_KL = mean over (b, t, proxy head) of
 *               KL(teacher || student), teacher = mean over the proxy head's Hq / Hp query
 *               heads of the main softmax (stop-gradient),
 *               student = softmax(scale * qp . kp) over the same tokens; the score gradient is
 *               kl_grad / (B*S*Hp) * (p_student - p_teacher)  (blog, "KL Divergence Loss").
 * o and lse are the outputs of msa_forward for the same inputs.  kl_grad is the incoming
 * gradient of the (zero) KL placeholder the forward returns (package usage note), usually 1.
 * Workspace: the teacher rows (one fp16 row of 128 keys per list entry) live for one pass of
 * consecutive sequence chunks at a time (attn_bwd writes them, the proxy gradients read them);
 * msa_workspace_size sizes a pass for at most 8 GiB of them, a larger workspace_bytes gives fewer
 * passes and a smaller one more (down to one chunk per pass; below that MSA_ERR_WORKSPACE).
 * kl_grad_dev: NULL, or a device pointer to one float that is used instead of kl_grad, read by
 * the kernel (an autograd backward can pass the placeholder's incoming gradient tensor without a
 * host synchronisation).
 * kl_out: NULL, or a device pointer to one float that receives the KL value L_KL itself (not
 * scaled by kl_grad).  The gradients never need it (blog, "KL Divergence Loss": the proxy
 * gradient is p_student - p_teacher), so it is computed only on request -- for logging every n
 * steps -- from the teacher and student probabilities the proxy-gradient pass already holds, at
 * the cost of one logarithm per selected (token, key) pair (package caveat 2: the reference
 * package does not return it at all).
 */
MSA_API int msa_backward(const msa_shape_t* shape, const void* q, const void* k, const void* v,
                 const void* qp, const void* kp, const void* o, const float* lse,
                 const void* dout, const int32_t* block_idx, float kl_grad,
                 const float* kl_grad_dev, void* dq, void* dk, void* dv, void* dqp, void* dkp,
                 float* kl_out, void* workspace, size_t workspace_bytes, void* stream);

/*
 * Warmup forward (blog, "Warmup kernels"): dense causal GQA attention, no proxy pass.
 * Writes o and lse.  top_k is ignored.
 */
MSA_API int msa_warmup_forward(const msa_shape_t* shape, const void* q, const void* k, const void* v,
                       void* o, float* lse, void* workspace, size_t workspace_bytes,
                       void* stream);

/*
 * Warmup backward (blog, "Warmup kernels"): the proxy normaliser over the full causal prefix,
 * then the fused main + proxy backward with every visible key in the key set.  Same outputs
 * (kl_grad_dev and kl_out included) and KL definition as msa_backward.  top_k is ignored.
 * Workspace: the teacher rows live for one pass of consecutive dense lists at a time (a pass may
 * end inside a sequence chunk), so the workspace does not grow with the square of S beyond them:
 * msa_workspace_size sizes a pass for at most 8 GiB of teacher rows, a larger workspace_bytes
 * gives fewer passes and a smaller one more (down to one list -- at most one chunk of tokens --
 * per pass; below that MSA_ERR_WORKSPACE).  The results do not depend on the passes beyond the
 * order of the fp32 gradient reductions.
 */
MSA_API int msa_warmup_backward(const msa_shape_t* shape, const void* q, const void* k, const void* v,
                        const void* qp, const void* kp, const void* o, const float* lse,
                        const void* dout, float kl_grad, const float* kl_grad_dev, void* dq,
                        void* dk, void* dv, void* dqp, void* dkp, float* kl_out, void* workspace,
                        size_t workspace_bytes, void* stream);

/*
 * Decode step of MSA inference (forum summary, "GPU kernel co-design", deployment setting
 * B = 128, k = 16; the prefill is msa_forward).  One new token per sequence b, at position
 * t_b = seq_len[b] - 1 of its caches, whose K, V and proxy key rows must already hold it:
 *   q         [B, Hq, 128]  bf16   the new tokens' queries
 *   qp        [B, Hp, 128]  bf16   their proxy queries
 *   k_cache, v_cache [B, S, Hkv, 128] bf16, kp_cache [B, S, 128] bf16: caches of capacity S
 *             (shape->S, a multiple of 128); rows after t_b are never read
 *   seq_len   [B] int32 device array, 1 <= seq_len[b] <= S (other values: the row is skipped and
 *             MSA_DEVICE_BAD_INDEX set)
 * Writes block_idx [B, Hp, top_k] (the selection of the new token: the local block t_b / 128 and
 * the best top_k - 1 earlier blocks by raw proxy score, ties to the lower block, ascending, -1
 * padded), o [B, Hq, 128] bf16 and lse [B, Hq] fp32 -- the same values as row t_b of msa_forward
 * on the whole sequence.  Head mapping and limits as for msa_forward, with Hp <= 32.  Workspace:
 * msa_workspace_size(shape, MSA_OP_DECODE).
 */
MSA_API int msa_decode(const msa_shape_t* shape, const void* q, const void* qp,
                       const void* k_cache, const void* v_cache, const void* kp_cache,
                       const int32_t* seq_len, int32_t* block_idx, void* o, float* lse,
                       void* workspace, size_t workspace_bytes, void* stream);

/*
 * Causal GQA attention over a sliding window and the first tokens (sinks): the local layers that
 * stand between sparse ones.  Query t sees key j iff j <= t and (t - j < window or j < sinks); a
 * window of S or more is dense causal attention.  Layouts as above: q, o, dout, dq [B, S, Hq, 128],
 * k, v, dk, dv [B, S, Hkv, 128], lse [B, Hq, S].  Supported: head dim 128, any 1 <= S <= 2^23,
 * Hq / Hkv in {1, 2, 4, 8, 16}, window >= 1, sinks >= 0.  Whatever a K or V row holds, also an
 * infinity or NaN (the uninitialised padding behind a ragged prompt), the forward and the decode step
 * keep it from the queries that do not see it; a query that sees one that is not finite has an
 * undefined row.  The backward's inputs must be finite: every key is seen by a query, its own, whose
 * gradients would reach all the keys that it sees.
 * P and dS enter their products as bf16, as in the sparse ops, everything else is fp32: relative errors
 * are 2.1e-3 for o and 2.4e-3 for dq and dk, where rounding the exact result to bf16 once gives 1.7e-3.
 * The decode step of groups of up to eight heads keeps P's rounding errors too (1.7e-3).
 */
typedef struct msa_window_shape {
  int32_t B;       /* batch */
  int32_t S;       /* sequence length; decode: capacity of the caches */
  int32_t Hq;      /* query heads */
  int32_t Hkv;     /* key/value heads */
  int32_t D;       /* head dim, must be 128 */
  int32_t window;  /* keys a query sees, itself included */
  int32_t sinks;   /* first keys that stay visible */
  float scale;     /* softmax scale, usually 128^-0.5 */
} msa_window_shape_t;

/* Bytes of workspace a window op needs (0 if the shape is unsupported). */
MSA_API size_t msa_window_workspace_size(const msa_window_shape_t* shape, int op);

/*
 * The longest that a wait inside a window op's kernels may last, in milliseconds (0 if the shape is
 * unsupported).  A wait that runs out ends its block, sets MSA_DEVICE_TIMEOUT and leaves outputs that
 * are not valid; the limit grows with the window, whose whole walk the warps that store a row sit out.
 */
MSA_API unsigned msa_window_wait_limit_ms(const msa_window_shape_t* shape, int op);

/* Writes o and lse. */
MSA_API int msa_window_forward(const msa_window_shape_t* shape, const void* q, const void* k,
                       const void* v, void* o, float* lse, void* workspace, size_t workspace_bytes,
                       void* stream);

/* Gradients of sum(o * dout); o and lse are the outputs of msa_window_forward for the same inputs.
 * The same inputs give the same bits every time (no atomic sums). */
MSA_API int msa_window_backward(const msa_window_shape_t* shape, const void* q, const void* k,
                        const void* v, const void* o, const float* lse, const void* dout, void* dq,
                        void* dk, void* dv, void* workspace, size_t workspace_bytes, void* stream);

/*
 * Decode step: one new token per sequence at position t_b = seq_len[b] - 1 of its caches, which
 * already hold it.  q, o [B, Hq, 128] bf16, lse [B, Hq] fp32, k_cache, v_cache [B, S, Hkv, 128],
 * seq_len [B] int32 on the device, 1 <= seq_len[b] <= S (other values: the sequence's rows of o and
 * lse are left as they were and MSA_DEVICE_BAD_INDEX is set).  Cache rows the token does not see --
 * behind it, before its window, whatever they hold -- do not reach the result.
 */
MSA_API int msa_window_decode(const msa_window_shape_t* shape, const void* q, const void* k_cache,
                      const void* v_cache, const int32_t* seq_len, void* o, float* lse,
                      void* workspace, size_t workspace_bytes, void* stream);

/*
 * Causal GQA attention over packed sequences: the tokens of sequences of different lengths -- prompts of one
 * batch, documents of one training step -- lie one behind the other in q, o, dout, dq [rows, Hq, 128] and k, v, dk, dv
 * [rows, Hkv, 128], lse [Hq, rows].  Token t of a sequence sees its tokens j <= t with t - j < window (a window of
 * rows or more: all of them).  Rows behind the last sequence reach no other row; they are 0 in o and
 * the gradients and -inf in lse.
 * Hq / Hkv in {1, 2, 4, 8, 16}, rows <= 2^23, rows Hq < 2^31, sequences of length 0 among the others.
 *
 * msa_packed_plan makes the tables that a forward and a backward (of any number of layers) work by, on `stream`, from
 * lengths on the host, which are not read after the call and travel as kernel arguments: no copy, no wait, and a
 * captured plan keeps its lengths.  `plan` gets the host's part, `table` (device, msa_packed_table_bytes) the other; both
 * belong to the device and lengths that they were made for.  The plan is ready in the order of its stream.
 * NaN or infinities in one sequence's V reach no other sequence's o; the backward's inputs must be finite.
 * Precision as in the window ops; a gradient has the same bits every time.
 */
typedef struct msa_packed_shape {
  int32_t rows;   /* of the tensors, at least the sum of the lengths */
  int32_t Hq;     /* query heads */
  int32_t Hkv;    /* key/value heads */
  int32_t D;      /* head dim, must be 128 */
  int32_t window; /* keys a query sees, itself included */
} msa_packed_shape_t;
typedef struct msa_packed_plan {
  int32_t rows, tokens, Hq, Hkv, window; /* tokens: of all sequences */
  int32_t fwd_tiles, fwd_units, dq_units, chunk, items, slots, joins; /* how the work is cut */
} msa_packed_plan_t;

/* Bytes of a plan's table (0 if the shape or a length is not supported). */
MSA_API size_t msa_packed_table_bytes(const msa_packed_shape_t* shape, const int32_t* lengths, int32_t nseq);
MSA_API int msa_packed_plan(const msa_packed_shape_t* shape, const int32_t* lengths, int32_t nseq,
                    msa_packed_plan_t* plan, void* table, size_t table_bytes, void* stream);
/* Bytes of workspace of MSA_OP_PACKED_FORWARD or MSA_OP_PACKED_BACKWARD (0: another op, or not a plan). */
MSA_API size_t msa_packed_workspace_size(const msa_packed_plan_t* plan, int op);
/* Writes o and lse. */
MSA_API int msa_packed_forward(const msa_packed_plan_t* plan, const void* table, size_t table_bytes, const void* q,
                       const void* k, const void* v, float scale, void* o, float* lse, void* workspace,
                       size_t workspace_bytes, void* stream);
/* Gradients of sum(o * dout); o and lse are the outputs of msa_packed_forward for the same inputs. */
MSA_API int msa_packed_backward(const msa_packed_plan_t* plan, const void* table, size_t table_bytes, const void* q,
                        const void* k, const void* v, const void* o, const float* lse, const void* dout, float scale,
                        void* dq, void* dk, void* dv, void* workspace, size_t workspace_bytes, void* stream);

/*
 * RMS norm of every head's row and the position rotation in one pass, for the inputs of the
 * attention ops: q, k and the proxy heads, usually as slices of one packed projection.
 * A call takes up to 8 parts.  A part is `heads` consecutive heads (128 elements apart) of every
 * token; its tensors are bf16 [B, N, heads, 128] with batch and token strides in elements
 * (multiples of 8) and 16-byte aligned bases.  Per row x (all in fp32, rounded once):
 *     r = (mean(x^2) + eps)^-1/2,  u = weight x r   (weight NULL: u = x)
 *     y = u with its first `rotary` elements turned in pairs (i, i + rotary/2) -- interleaved:
 *         (2 i, 2 i + 1) -- by the angle position * inv_freq[i]   (without MSA_ROPE_ROTATE: y = u)
 * rotary: a multiple of 16, 0 .. 128.  inv_freq: rotary / 2 floats on the device.  positions: int32
 * [B, N] on the device, any value, or NULL for 0 .. N - 1.  Angles are exact to fp32 at every position
 * (for inv_freq up to 2^40 either side of zero).
 * The outputs of a call (y; backward: dx, dweight) may overlap neither each other nor an input, only
 * that dx may be the same rows as x or dy of its own part, and y, where it is not a cache, those of x.
 */
enum msa_rope_flags {
  MSA_ROPE_ROTATE = 1, /* rotate this part */
  MSA_ROPE_CACHE = 2,  /* append only: y is a cache, its token index the token's position */
  MSA_ROPE_CACHE_Q4 = 8 /* append only: y is a cache in 4 bits (below; its strides are not used) */
};
typedef struct msa_rope_part {
  const void* x;
  int64_t x_batch, x_token;
  void* y; /* forward, append: output; backward: dy, read only */
  int64_t y_batch, y_token;
  void* dx; /* backward only */
  int64_t dx_batch, dx_token;
  const float* weight; /* [128] fp32, NULL: not normed */
  float* dweight;      /* backward: [128] fp32, NULL: not wanted */
  int32_t heads;
  int32_t flags;
} msa_rope_part_t;
typedef struct msa_rope_shape {
  int32_t B;           /* batch */
  int32_t N;           /* tokens per sequence in x */
  int32_t D;           /* head dim, must be 128 */
  int32_t rotary;      /* rotated elements of a row */
  int32_t interleaved; /* pairs (2 i, 2 i + 1) */
  int32_t capacity;    /* append: tokens a cache holds */
  float eps;           /* >= 0 */
} msa_rope_shape_t;

MSA_API int msa_norm_rope_forward(const msa_rope_shape_t* shape, const msa_rope_part_t* parts,
                          int nparts, const int32_t* positions, const float* inv_freq,
                          void* stream);

/*
 * Serving form: the N tokens of x are the last N of sequences of length seq_len[b] (device int32;
 * N <= seq_len[b] <= capacity), so token i is at position seq_len[b] - N + i.  Parts with
 * MSA_ROPE_CACHE go to that row of their cache (y: [B, capacity, heads, 128] with the part's
 * strides), other rows of which are left as they were; other parts as in msa_norm_rope_forward.  A
 * sequence whose length is out of range is skipped and MSA_DEVICE_BAD_INDEX set.  Then msa_decode
 * or msa_window_decode run on the same caches and seq_len (N = 1).
 */
MSA_API int msa_norm_rope_append(const msa_rope_shape_t* shape, const msa_rope_part_t* parts,
                         int nparts, const int32_t* seq_len, const float* inv_freq,
                         void* workspace, size_t workspace_bytes, void* stream);

/* dx of every part, and dweight summed over its rows, from x and dy (in `y`).  The same inputs give
 * the same bits every time. */
MSA_API int msa_norm_rope_backward(const msa_rope_shape_t* shape, const msa_rope_part_t* parts,
                           int nparts, const int32_t* positions, const float* inv_freq,
                           void* workspace, size_t workspace_bytes, void* stream);

/*
 * The same three with positions of several axes -- time, height and width of images and video:
 * positions: int32 [axes->count][B][N] on the device, pair i turns by positions[axes->of_pair[i]] *
 * inv_freq[i].  axes NULL: one axis.  In the append they stand beside seq_len, which then says only which row
 * of a cache a token goes to (a text token's position behind an image is not its cache row).
 */
typedef struct msa_rope_axes {
  int32_t count;       /* 1 .. 4 */
  uint8_t of_pair[64]; /* axis of each of the rotary / 2 pairs */
} msa_rope_axes_t;
MSA_API int msa_norm_rope_axes_forward(const msa_rope_shape_t* shape, const msa_rope_part_t* parts,
                          int nparts, const int32_t* positions, const float* inv_freq,
                          const msa_rope_axes_t* axes, void* stream);
MSA_API int msa_norm_rope_axes_append(const msa_rope_shape_t* shape, const msa_rope_part_t* parts,
                          int nparts, const int32_t* seq_len, const int32_t* positions,
                          const float* inv_freq, const msa_rope_axes_t* axes, void* workspace,
                          size_t workspace_bytes, void* stream);
MSA_API int msa_norm_rope_axes_backward(const msa_rope_shape_t* shape, const msa_rope_part_t* parts,
                          int nparts, const int32_t* positions, const float* inv_freq,
                          const msa_rope_axes_t* axes, void* workspace, size_t workspace_bytes,
                          void* stream);

/*
 * Caches in 4 bits.  A row x of 128 values (a key, after norm and rotation, or a value) is kept as
 *     x[i] ~ 2^e s[i / 16] c[i],
 * c four bits (sign, two exponent bits, one of mantissa: 0, 1/2, 1, 3/2, 2, 3, 4, 6 and their negatives), s eight
 * (sign, four exponent bits, three of mantissa), e one byte:
 *     a = max |x| / 6,  e = floor(log2 a) - 7, at least -100 and at most 90
 *     s[g] = 2^-e max |x[16 g .. 16 g + 15]| / 6,  c[i] = 2^-e x[i] / s[i / 16],
 * each rounded to nearest, ties to even (c: at most 6; s: at most 448, so that kept values end at 2688 2^90; s = 0:
 * c = 0).  x is first rounded to bf16.  Every kept value is exact in bf16.  A row with an infinity or NaN is NaN throughout.
 * A cache is [B][heads][capacity / 128] blocks of 9344 bytes, 16-byte aligned, capacity a multiple of 128.  A block
 * is 128 rows of one head: [128][64] bytes of codes (low nibble first), [128][8] of scales, [128] of e + 127: 73
 * bytes a row, where bf16 takes 256.  Zero bytes, as in a new cache, are rows of zeros.
 * msa_norm_rope_append writes them (parts with MSA_ROPE_CACHE_Q4), new tokens as well as whole prompts.
 */
/* Bytes of such a cache (0: a size that is not positive, or a capacity that is no multiple of 128). */
MSA_API size_t msa_q4_cache_bytes(int32_t B, int32_t heads, int32_t capacity);

/* The values that rows first .. first + count - 1 of every sequence and head stand for: out [B, count, heads, 128]
 * bf16.  The rows have to lie in the cache. */
MSA_API int msa_q4_read(const void* cache, int32_t B, int32_t heads, int32_t capacity, int32_t first,
                        int32_t count, void* out, void* stream);

/*
 * msa_window_decode and msa_decode over K and V caches in 4 bits (kp_cache stays bf16, so the selection is that
 * of msa_decode).  Arguments, limits, status bits and the rows that are left as they were are those of the two;
 * S is the capacity.  The caches' values are used as they are kept; the softmax weights, V's powers of two in them, are
 * rounded to 11 bits for their product, those below 2^-20 of the largest to 2^-31 of it; elements of q below 2^-31 of their
 * head's largest to 2^-39 of that; everything else is fp32.  Workspace: MSA_OP_WINDOW_DECODE_Q4, MSA_OP_DECODE_Q4.
 */
MSA_API int msa_window_decode_q4(const msa_window_shape_t* shape, const void* q, const void* k_cache,
                      const void* v_cache, const int32_t* seq_len, void* o, float* lse,
                      void* workspace, size_t workspace_bytes, void* stream);
MSA_API int msa_decode_q4(const msa_shape_t* shape, const void* q, const void* qp,
                       const void* k_cache, const void* v_cache, const void* kp_cache,
                       const int32_t* seq_len, int32_t* block_idx, void* o, float* lse,
                       void* workspace, size_t workspace_bytes, void* stream);

/* Bytes of workspace MSA_OP_NORM_ROPE_BACKWARD or MSA_OP_NORM_ROPE_APPEND needs for nparts parts (0:
 * another op, or nparts out of range). */
MSA_API size_t msa_norm_rope_workspace_size(int nparts, int op);

/*
 * Reads (and clears) the device status word of `workspace` after the work queued on `stream`
 * finishes; this synchronises `stream`.  *flags receives MSA_DEVICE_* bits (0 = clean).
 */
MSA_API int msa_device_status(void* workspace, unsigned* flags, void* stream);

/*
 * Measurement aids (not part of the method).  msa_profile_begin() makes every later call record
 * a CUDA event pair around each kernel it launches, on the launch stream.  msa_profile_end()
 * waits for those events, writes one line per kernel name -- "<name> <launches> <total_ms>\n" --
 * into buf (NUL-terminated, truncated to len) and stops recording.  msa_launch_count() returns
 * the number of kernels this library has launched since it was loaded.
 */
MSA_API int msa_profile_begin(void);
MSA_API int msa_profile_end(char* buf, size_t len);
MSA_API long long msa_launch_count(void);

/*
 * Allocation-free variant of msa_forward (the method's pages have no counterpart; this is an
 * integration aid).  Some callers cannot allocate device memory where they call the forward --
 * for example a C layer embedded in a framework whose allocator it cannot reach, or code running
 * while a sequence of launches is being recorded for replay, where allocating is not allowed.
 * This entry point needs no workspace: it uses a fixed scratch array of 64 MiB (67108864 bytes)
 * that lives in device memory for as long as the library is loaded, one per GPU that loads it.  Arguments and results are those of msa_forward; inputs and outputs are still
 * the caller's.  Shapes whose forward workspace exceeds the array are rejected with
 * MSA_ERR_WORKSPACE before any launch.  The first call on a device looks up the array's device
 * address (cudaGetSymbolAddress), so make that first call before any stream capture.  Every call
 * on a device shares the one array and it keeps the last call's contents: the call re-initialises
 * what must start at zero itself, but calls that overlap on the GPU (different streams without
 * ordering) race on it and must be serialised by the caller.
 */
MSA_API int msa_forward_noalloc(const msa_shape_t* shape, const void* q, const void* k,
                                const void* v, const void* qp, const void* kp, int32_t* block_idx,
                                int indices_given, void* o, float* lse, void* stream);

/*
 * Device status word of the fixed scratch array that msa_forward_noalloc uses on the current
 * device: same bits and behaviour as msa_device_status (reads and clears the word once the work
 * queued on `stream` has finished; synchronises `stream`).  Callers of msa_forward_noalloc have no
 * workspace pointer to pass to msa_device_status, so this is how they learn that given block
 * indices were skipped as invalid (MSA_DEVICE_BAD_INDEX) or that a bounded wait gave up.  Every
 * call of msa_forward_noalloc on a device clears the word before it launches, so read it after
 * each call whose result matters.
 */
MSA_API int msa_forward_noalloc_status(unsigned* flags, void* stream);

/*
 * Failure-detection self-test (not part of the method).  Launches one block on `stream` whose
 * thread waits on a shared-memory mbarrier that nothing arrives at, through the same bounded wait
 * every kernel of the library uses; after limit_us microseconds (1 .. 1000000) the wait gives up
 * and sets MSA_DEVICE_TIMEOUT in the status word of `workspace` (any workspace of this library, or
 * 256 zeroed, 16-byte aligned device bytes).  Read it with msa_device_status.  Returns
 * MSA_ERR_INVALID_ARG for a null or misaligned workspace or a limit out of range.
 */
MSA_API int msa_selftest_wait_timeout(void* workspace, unsigned limit_us, void* stream);

/* Static text for a status code. */
MSA_API const char* msa_status_string(int status);

/* Detail of the last error on the calling thread ("" if none). */
MSA_API const char* msa_last_error(void);

#ifdef __cplusplus
}
#endif

#endif /* MSA_H_ */
