/*
 * qmv.h -- C ABI of libqmv.so: the decode-step matrix-vector product of a
 * GGUF block-quantized weight matrix (Q8_0, Q4_0, Q4_K, Q5_K, Q6_K) with f32
 * activations, dequantized on the fly, on one NVIDIA B200 (sm_100a).
 *
 * Sources (page title, section):
 *   BebeLM：纯Rust实现的端侧大模型推理引擎
 *     §量化格式支持 -- Q4_K: 256 weights per superblock in 144 bytes; Q6_K for
 *       sensitive tensors; dequantization happens at run time and activations
 *       stay f32.
 *     §核心算子 (MoE前馈网络) -- sigmoid router, top-k = 4 of 32 experts, the
 *       expert bias takes part in the selection only, weights normalised.
 *     §性能表现 -- decode is bound by memory bandwidth.
 *   FlareLLM：纯Rust打造的浏览器端LLM推理引擎
 *     §推理层面的深度优化 -- fused QKV and gate/up matvecs (43% fewer matvec
 *       calls per layer); n-gram speculative decoding (several tokens checked
 *       in one pass over the weights); zero-allocation forward pass.
 *     §计算路径的智能选择, §量化技术的全面支持 -- Q8_0, Q4_0 and the K-quants.
 *     §生态对比与定位 -- standard GGUF files.
 *
 * Block layouts (GGUF, little-endian, fp16 = IEEE binary16):
 *   Q8_0  32 weights / 34 B : d | q[32] int8                 w = d*q
 *   Q4_K 256 weights / 144 B: d | dmin | scales[12] | qs[128]
 *                             w = d*sc_j*q - dmin*m_j, j = sub-block of 32
 *   Q6_K 256 weights / 210 B: ql[128] | qh[64] | scales[16] int8 | d
 *                             w = d*scales[i/16]*(q - 32), q = 6 bits
 *   Q4_0  32 weights / 18 B : d | qs[16]; byte j holds weight j (low nibble)
 *                             and weight j+16 (high nibble);  w = d*(q - 8)
 *   Q5_K 256 weights / 176 B: d | dmin | scales[12] (as Q4_K) | qh[32] | qs[128]
 *                             (as Q4_K); the fifth bit of weight 64c + l is
 *                             bit 2c of qh[l], of weight 64c + 32 + l bit 2c+1;
 *                             w = d*sc_j*q - dmin*m_j
 * A matrix is rows x cols weights stored densely row-major: row r starts at
 * byte r * (cols / block_weights) * block_bytes; no padding.
 *
 * Conventions shared by every entry point:
 *   - Every array pointer is a DEVICE pointer owned by the caller (for
 *     example torch.empty(..., device="cuda").data_ptr()); the library keeps
 *     no reference after the call returns.
 *   - `stream` is a cudaStream_t (NULL = the legacy default stream).  Work is
 *     enqueued asynchronously on it; outputs are complete in stream order.
 *   - The library allocates no memory during any call; intermediates (the
 *     SwiGLU activations of moe_ffn) live in caller-provided buffers.
 *   - Outputs are fully overwritten, never accumulated into.
 *   - Argument errors are detected on the host and returned before anything
 *     is enqueued; outputs are then left untouched.  No call aborts.
 *   - Alignment: W (every expert base and expert stride) 16 B, x 16 B,
 *     y / out 4 B.
 *   - The arithmetic is f32: dequantized weights are exact f32 values, dot
 *     products accumulate in f32 (order unspecified, deterministic for a
 *     given shape).  There is no CPU fallback and no other backend.
 *   - Thread safety: calls may be made from several host threads.  Global
 *     state: a per-device properties cache, the programmatic-dependent-launch
 *     switch (qmv_set_pdl), and per device the sticky error word read by
 *     qmv_check(), qmv_argmax's workspace and the scratch array of
 *     moe_ffn_static.
 */
#ifndef QMV_H
#define QMV_H

#include <stddef.h>
#include <stdint.h>

#ifdef __cplusplus
extern "C" {
#endif

/* Same type as cudaStream_t, without including the CUDA headers. */
typedef struct CUstream_st *qmv_stream_t;

typedef enum { QMV_Q8_0 = 0, QMV_Q4_K = 1, QMV_Q6_K = 2, QMV_Q4_0 = 3, QMV_Q5_K = 4 } qmv_fmt;

typedef enum {
    QMV_OK = 0,
    QMV_ERR_NULL = -1,    /* a required pointer is NULL                         */
    QMV_ERR_FMT = -2,     /* fmt is not one of qmv_fmt                           */
    QMV_ERR_SHAPE = -3,   /* rows < 1, cols < 1, cols % block_weights != 0, or a
                             size above the limits below                        */
    QMV_ERR_ALIGN = -4,   /* a pointer or stride breaks the alignment rules      */
    QMV_ERR_NTOK = -5,    /* n_tok outside [1, QMV_MAX_NTOK]                     */
    QMV_ERR_NSEL = -6,    /* n_sel / top_k outside [1, min(n_expert, 8)], or
                             n_expert outside [1, QMV_MAX_EXPERTS]              */
    QMV_ERR_CUDA = -7,    /* a CUDA call or a kernel launch failed               */
    QMV_ERR_DEVICE = -8,  /* no usable CUDA device, or a device-side error was
                             recorded (see qmv_check)                            */
    QMV_ERR_WS = -9,      /* the workspace is smaller than the call needs        */
} qmv_status;

#define QMV_MAX_NTOK 8
#define QMV_MAX_SEL 8
#define QMV_MAX_EXPERTS 1024
#define QMV_MAX_ROWS 2147483647LL   /* rows of one matrix                       */
#define QMV_MAX_COLS 1048576LL      /* weights per row                          */

/* Device error bits reported by qmv_check(). */
#define QMV_DEVERR_EXPERT_ID 1      /* an expert id was outside [0, n_expert); that
                                       expert's contribution was dropped        */
#define QMV_DEVERR_TIMEOUT 2        /* a pipeline wait gave up (bounded wait)   */
#define QMV_DEVERR_DRAIN 4          /* after a timeout, a CTA also gave up waiting for
                                       its own copies in flight and exited: they may
                                       still land in shared memory reused by later
                                       kernels, so later results on this device are
                                       suspect (recreate the context to be sure)   */
#define QMV_DEVERR_PAGE_ID 8        /* a block table named a page outside [0, n_pages);
                                       its slots were left out (see kv_append ...) */
#define QMV_DEVERR_SEQ_LEN 16       /* a sequence length was negative or beyond its
                                       block table; it was clamped                 */

/* y[rows] = W x.  x: f32 [cols]; y: f32 [rows].
 * One launch covers a whole fused projection: pass the row-concatenation of
 * Q, K and V (or of gate and up) as W (FlareLLM page, §推理层面的深度优化).
 * Returns QMV_OK or a qmv_status error. */
int qmv_f32(int fmt, const void *W_blocks, int64_t rows, int64_t cols,
            const float *x, float *y, qmv_stream_t stream);

/* One matvec of a grouped launch (see qmv_multi). */
typedef struct {
    const void *W_blocks;   /* device, 16-byte aligned, rows x cols weights    */
    int64_t rows;
    int64_t cols;
    const float *x;         /* device f32 [n_tok][cols], 16-byte aligned       */
    float *y;               /* device f32 [n_tok][rows], 4-byte aligned        */
} qmv_task;

#define QMV_MAX_TASKS 4096

/* Several independent matvecs of one format and token count in as few
 * launches as possible: y_t = W_t x_t for every task t (same layouts as
 * qmv_batched).  The tasks run concurrently and in no defined order, so no
 * task may write memory another task of the call reads; the call as a whole
 * is ordered in `stream` like any other.  Each task's rows are split into
 * CTAs of roughly equal byte counts sized to the whole batch, so the CTAs of
 * all tasks stream together and the launch-to-launch latency of a chain of
 * small matvecs disappears.  `tasks` is a host array of n_tasks entries
 * (1 <= n_tasks <= QMV_MAX_TASKS), read during the call only. */
int qmv_multi(int fmt, int n_tok, const qmv_task *tasks, int n_tasks, qmv_stream_t stream);

/* One-token matvecs of one format executed IN ORDER, the way a decode step
 * runs its projections layer after layer (BebeLM：纯Rust实现的端侧大模型推理引擎,
 * §核心算子 and §性能表现: every layer's matvecs each decode step): task t+1
 * starts only after every row of task t is written, so a task's x may be the
 * y of any earlier task of the same call (tasks' n_tok is 1: x f32 [cols],
 * y f32 [rows]).  Each task is one streaming-kernel launch, ordered by
 * programmatic dependent launch (a kernel reads its x only after the previous
 * one has finished), and each launch, once its own weight copies are issued,
 * starts moving the next task's weights into L2, so the next launch reads them
 * from there while HBM already streams the one after.  The call keeps no
 * state between calls: calls on different streams may overlap.  A task shape
 * that the streaming kernel does not take turns the whole call into one
 * qmv_f32 call per task, in order.  `tasks` is a host array of
 * n_tasks entries (1 <= n_tasks <= QMV_MAX_TASKS), read during the call only.
 * Errors as qmv_multi. */
int qmv_chain(int fmt, const qmv_task *tasks, int n_tasks, qmv_stream_t stream);

/* Multi-token variant for speculative verification (FlareLLM page,
 * §推理层面的深度优化: n-gram speculative decoding): every weight is read once
 * and applied to n_tok activation vectors.
 * x: f32 [n_tok][cols] (token-major); y: f32 [n_tok][rows]; 1 <= n_tok <= 8. */
int qmv_batched(int fmt, const void *W_blocks, int64_t rows, int64_t cols,
                const float *x, float *y, int n_tok, qmv_stream_t stream);

/* MoE router on the device, no host round trip (BebeLM page, §核心算子):
 *   s_e = sigmoid(logits[e]),  b_e = s_e + bias[e]   (f32)
 *   ids_out[k] = the top_k experts by b, in descending b (ties to the lower
 *                index);  g_out[k] = s_{ids[k]} / sum_j s_{ids[j]}.
 * logits, bias: f32 [n_expert]; ids_out: int32 [top_k]; g_out: f32 [top_k].
 * 1 <= top_k <= min(n_expert, 8), n_expert <= QMV_MAX_EXPERTS. */
int moe_route(const float *logits, const float *bias, int n_expert, int top_k,
              int32_t *ids_out, float *g_out, qmv_stream_t stream);

/* Expert-indexed grouped matvec.  Expert e's matrix (rows x cols, format fmt)
 * starts at expert_blocks + e * expert_stride_bytes; the n_sel expert ids are
 * read on the device from expert_ids (int32 [n_sel]), so the call can follow
 * moe_route without a host synchronisation.
 * x_k = x + k * x_stride (x_stride in floats; 0 = one shared x [cols]).
 *   gate_w == NULL: y[k][r] = (W_{ids[k]} x_k)[r]           y: f32 [n_sel][rows]
 *   gate_w != NULL: y[r] = sum_k gate_w[k] * (W_{ids[k]} x_k)[r]  y: f32 [rows]
 *                   (gate_w: device f32 [n_sel]; summed in k order)
 * An id outside [0, n_expert) contributes zero and sets QMV_DEVERR_EXPERT_ID.
 * 1 <= n_sel <= min(n_expert, 8).  expert_stride_bytes must be a multiple of
 * 16 and at least the matrix size. */
int moe_qmv(int fmt, const void *expert_blocks, int64_t expert_stride_bytes, int n_expert,
            const int32_t *expert_ids, int n_sel, int64_t rows, int64_t cols,
            const float *x, int64_t x_stride, const float *gate_w, float *y,
            qmv_stream_t stream);

/* One MoE SwiGLU FFN step for the n_sel routed experts (BebeLM page, §核心算子):
 *   h_k = silu(G_{ids[k]} x) * (U_{ids[k]} x)        -> h_scratch f32 [n_sel][inter]
 *   y   = sum_k g[k] * D_{ids[k]} h_k                 -> y f32 [hidden]
 * G and U of expert e: [inter x hidden] in fmt_gu at gate_blocks / up_blocks
 * + e * gu_stride_bytes; D of expert e: [hidden x inter] in fmt_down at
 * down_blocks + e * down_stride_bytes.  x: f32 [hidden]; g: f32 [n_sel]
 * (e.g. from moe_route).  silu(z) = z / (1 + exp(-z)).  Two launches, no host
 * synchronisation; h_scratch is caller-owned scratch and is overwritten. */
int moe_ffn(int fmt_gu, const void *gate_blocks, const void *up_blocks,
            int64_t gu_stride_bytes, int fmt_down, const void *down_blocks,
            int64_t down_stride_bytes, int n_expert, const int32_t *expert_ids,
            const float *g, int n_sel, int64_t hidden, int64_t inter,
            const float *x, float *h_scratch, float *y, qmv_stream_t stream);

/* The MoE FFN step with its router, in one launch where the shapes allow
 * (BebeLM page, §核心算子, MoE前馈网络): moe_route on (logits, bias, n_expert,
 * top_k) -- ids_out, g_out as moe_route writes them, the same values -- then
 * moe_ffn with those ids and weights (n_sel = top_k): h_scratch
 * f32 [top_k][inter] holds the SwiGLU activations, y f32 [hidden] the result.
 * When both matrices have one format, expert rows are at most 2048 columns,
 * n_expert <= 256 and the rows are 16-byte multiples in pairs, one
 * cooperative launch does it all: every CTA routes on its own, streams the
 * routed gate/up rows and then the routed down rows through one pipeline, and
 * the CTAs meet once, at a grid barrier, between the two products (h complete).
 * Otherwise moe_route and moe_ffn run in turn.  `workspace`:
 * QMV_MOE_WS_BYTES of caller-owned device memory (8-byte aligned) that must be
 * zero before the first call and that every completed call leaves zero again
 * (the barrier's counters); calls that may overlap on the GPU need workspaces
 * of their own.  Errors as moe_route and moe_ffn. */
#define QMV_MOE_WS_BYTES 16
int moe_ffn_routed(const float *logits, const float *bias, int n_expert, int top_k,
                   int fmt_gu, const void *gate_blocks, const void *up_blocks,
                   int64_t gu_stride_bytes, int fmt_down, const void *down_blocks,
                   int64_t down_stride_bytes, int64_t hidden, int64_t inter, const float *x,
                   int32_t *ids_out, float *g_out, float *h_scratch, float *y, void *workspace,
                   qmv_stream_t stream);

/* moe_ffn without a caller-provided scratch buffer, for callers that cannot
 * allocate device memory: code running while a stream is being captured into
 * a CUDA graph (where cudaMalloc is not allowed), plugins and callbacks that
 * are handed only their input and output buffers, and real-time paths that
 * must not take an allocator's latency or locks.  (The pages have no
 * counterpart; this is a usage variant of the same MoE step.)
 * The SwiGLU activations go to a file-scope device array of
 * QMV_STATIC_H_FLOATS floats (512 KiB) that every GPU which loads the library
 * holds until the process exits; n_sel * inter above that is rejected with
 * QMV_ERR_SHAPE.  Nothing is allocated by the call.  The first call on a
 * device looks up the array's device address (a host call, no allocation):
 * make that first call before capturing a stream.  All calls share the one
 * array, which keeps the last call's contents (every call overwrites the part
 * it uses before reading it), so calls that can overlap on the GPU -- on two
 * streams of one device, say -- race and must be serialised by the caller.
 * Arguments and results are those of moe_ffn. */
#define QMV_STATIC_H_FLOATS (8 * 16384)
int moe_ffn_static(int fmt_gu, const void *gate_blocks, const void *up_blocks,
                   int64_t gu_stride_bytes, int fmt_down, const void *down_blocks,
                   int64_t down_stride_bytes, int n_expert, const int32_t *expert_ids,
                   const float *g, int n_sel, int64_t hidden, int64_t inter,
                   const float *x, float *y, qmv_stream_t stream);

/* Greedy next-token choice on the device (FlareLLM page, §推理层面的深度优化:
 * greedy decoding of the vocabulary projection): y = W x as qmv_batched (the
 * logits are kept in the caller's y, f32 [n_tok][rows]), and
 * idx_out[t] = the row of the largest y[t][row] -- IEEE > on f32, ties to
 * the lower row, NaN values skipped, -1 if every value of the token is NaN.
 * idx_out: device int32 [n_tok], 4-byte aligned.  rows <= INT32_MAX.
 * With one token on the shapes the one-token streaming kernel takes (rows of
 * at most 2048 columns) the choice is fused into the projection: every CTA
 * folds the best of its rows into a 64-bit key while it writes them, and the
 * last CTA writes idx -- one launch.  Otherwise a second launch scans y.
 * Either way the choice is deterministic (an order-independent atomic max
 * over keys: the value's order-preserving bits high, the complemented row
 * low).
 * The keys and arrival counters live in `workspace`, QMV_ARGMAX_WS_BYTES of
 * caller-owned device memory (8-byte aligned) that must be zero before the
 * first call and that every completed call leaves zero again; calls that may
 * overlap on the GPU need workspaces of their own.  Errors as qmv_batched,
 * QMV_ERR_NULL for a NULL workspace. */
#define QMV_ARGMAX_WS_BYTES 128
int qmv_argmax_ws(int fmt, const void *W_blocks, int64_t rows, int64_t cols,
                  const float *x, float *y, int n_tok, int32_t *idx_out, void *workspace,
                  qmv_stream_t stream);

/* qmv_argmax_ws with the library's own workspace on the current device: do
 * not run two qmv_argmax calls on one device at the same time (use
 * qmv_argmax_ws with separate workspaces for that). */
int qmv_argmax(int fmt, const void *W_blocks, int64_t rows, int64_t cols,
               const float *x, float *y, int n_tok, int32_t *idx_out, qmv_stream_t stream);

/* ------------------------------------------------- the key-value cache --
 * Between the fused QKV projection and the O projection a decode step writes
 * the new tokens' keys and values into a cache (kv_append), attends over it
 * (attn_decode) and, where a sequence outgrows its budget, prunes it
 * (kv_evict).  (Sources: BebeLM page, §独特的层设计 -- grouped-query attention
 * layers, 32 query and 8 kv heads; FlareLLM page, §推理层面的深度优化 -- several
 * tokens checked in one pass; the engines' KV caches.)
 *
 * The cache is a pool of pages.  A page holds page_size slots, a slot one
 * token's key and value of every kv head.  A sequence's slots 0, 1, 2, ... lie
 * in the pages that its row of the block table names, page_size slots each.
 * Value i of kv head h of the slot at place o of page p is element
 *     p * page_stride + h * head_stride + o * slot_stride + i
 * of `k` (and of `v`), strides in values, so [page][head][slot][value] and
 * [page][slot][head][value] pools are both usable, and so are pools with gaps.
 *   QMV_KV_F16, QMV_KV_BF16: 16-bit floats; head_dim a multiple of 16, 16 to
 *                 256; strides multiples of 8.
 *   QMV_KV_Q8_0:  int8 quants in k / v, in blocks of 32 with an IEEE binary16
 *                 scale each, value = scale * quant (the Q8_0 arithmetic; the
 *                 scales lie apart so that quants keep 16-byte alignment): the
 *                 scale of element e is element e / 32 of k_scale / v_scale.
 *                 head_dim 64, 128, 192 or 256; strides multiples of 64.
 * k, v: 16-byte aligned; scales: 4-byte aligned (NULL for the 16-bit types).
 *
 * Block tables are int32 [n_seq][table_stride] on the device; a sequence may
 * use its first max_pages entries.  kv_len is int32 [n_seq] on the device.  So
 * lengths and tables may change between replays of a captured graph.  An entry
 * that a call reads must lie in [0, n_pages): slots of one that does not are
 * left out (not read, not written, not attended) and QMV_DEVERR_PAGE_ID is
 * recorded.  Entries whose slots a call does not touch are never read as pages
 * (pages behind a sliding window may have been freed).  A length below 0 or above
 * max_pages * page_size records QMV_DEVERR_SEQ_LEN; attn_decode and kv_evict
 * clamp it, kv_append leaves the tokens out whose slots lie outside.
 * Sequences may share pages that no call writes.
 */
typedef enum { QMV_KV_F16 = 0, QMV_KV_BF16 = 1, QMV_KV_Q8_0 = 2 } qmv_kv_type;

typedef struct {
    int32_t type;           /* qmv_kv_type                                      */
    int32_t n_kv_head;      /* 1 .. 1024                                        */
    int32_t head_dim;
    int32_t page_size;      /* slots per page, >= 1                             */
    int64_t n_pages;        /* pages of the pool, 1 .. 2^31 - 1                 */
    int64_t page_stride, head_stride, slot_stride;
    void *k, *v;            /* device                                           */
    void *k_scale, *v_scale;
} qmv_kv_cache;

#define QMV_MAX_SEQ 1024            /* sequences of one call                    */
#define QMV_ROPE_HALVES 0           /* pairs (i, i + rope_dim / 2)              */
#define QMV_ROPE_PAIRS 1            /* pairs (2i, 2i + 1)                       */

/* The new tokens into the cache, with their rotary embedding:
 *   angle = pos * inv_freq[i], i < rope_dim / 2;  a' = a cos - b sin,
 *   b' = a sin + b cos for every pair (a, b) of the first rope_dim values of
 *   every q and k head (angles, sine and cosine in 64 bits, so that far
 *   positions keep their phase; the sums with 48 bits of either, rounded once
 *   to f32, then to the cache's type)
 *   Q8_0 blocks: scale = f16(min(amax / 127, 65504)), quant = value / scale
 *   rounded to even and clamped to +-127, 0 where the scale is 0; a block
 *   with a NaN gets the scale NaN and quants 0, an infinity counts as the
 *   largest value that the block can hold
 *   f16: values beyond its range become infinities, and NaN stays NaN in it
 *   and in bf16; attn_decode does not take either in a slot that it sees
 * Token t (0 <= t < n_tok) of sequence s goes to slot kv_len[s] - n_tok + t
 * (kv_len counts the new tokens already) at position pos[s * n_tok + t], or at
 * its slot number where pos is NULL.  A token whose slot is negative (a padded
 * batch) or lies beyond the block table, or whose page is bad, is not stored; its
 * rotated q is written all the same.
 * q, k, v: f32, token s * n_tok + t at + (s * n_tok + t) * stride floats, its heads
 * one after another: rows of a fused QKV product are read as they lie (q = y,
 * k = y + n_head * head_dim, all three strides the row length).  q_out: f32,
 * same layout with q_out_stride; q == q_out with equal strides rotates in place;
 * they may not overlap otherwise.  q and q_out may both be NULL.
 * inv_freq: device f32 [rope_dim / 2], 0 <= rope_dim <= head_dim, even; with
 * rope_dim 0 it may be NULL and values are stored as they are.
 * All float pointers 4-byte aligned.  Two tokens of one call may not name the
 * same slot of the same page. */
typedef struct {
    qmv_kv_cache cache;
    const float *q, *k, *v;
    float *q_out;
    int64_t q_stride, k_stride, v_stride, q_out_stride;
    int32_t n_head, n_seq, n_tok;               /* n_head 1 .. 8192; n_tok 1 .. 8 */
    int32_t rope_dim, rope_style;
    int32_t max_pages;
    int64_t table_stride;
    const int32_t *block_table, *kv_len, *pos;
    const float *inv_freq;
} qmv_append;

int kv_append(const qmv_append *a, qmv_stream_t stream);

/* Attention of each sequence's newest n_tok tokens over its cache.  Query t of
 * sequence s sits at slot p = kv_len[s] - n_tok + t and sees slot j when
 *   j <= p  and  (window == 0  or  j > p - window  or  j < n_sink):
 * causal, with a sliding window of `window` slots (the query's own counted)
 * and the first n_sink slots visible throughout.  For query head h, which
 * reads kv head h / (n_head / n_kv_head):
 *   s_j = scale * q . k_j,   out = sum_j softmax(s)_j v_j   over the visible j.
 * A query that sees nothing (p < 0, or bad pages only) yields zeros, and so
 * does one whose every score is -infinity.  Values in
 * slots that a query does not see never reach its result, NaN and infinities
 * included; the visible values and q have to be finite.
 * score != NULL: the weights are accumulated per slot and kv head for kv_evict,
 *   score[s][h][j] += sum over the group's query heads and the n_tok queries of
 *   softmax(s)_j,  f32, entry (s * n_kv_head + h) * score_stride + j;
 * the entries of the newest n_tok slots are set, not added to, so a new slot
 * needs no clearing; entries of slots that no query sees stay as they are.
 * A row of `score` has score_slots entries, 0 standing for score_stride; the
 * others of its score_stride are not touched (rows of a wider tensor).  A length
 * above that number is clamped like one beyond the block table.
 * q, out: f32, apart from each other, 16- and 4-byte aligned, token s * n_tok + t at + (s * n_tok + t) *
 * stride floats (q_stride a multiple of 4), heads one after another; n_head a
 * multiple of n_kv_head, 1 <= n_head / n_kv_head * n_tok <= 1024.  The longest
 * lengths, in steps of 64 slots, over all sequences and heads stay below 2^30.
 * Sums, maxima and products are f32; q and the weights reach the tensor cores
 * as sums of two f16 parts (f16 and Q8_0 caches) or three bf16 parts (24 bits).
 * What two parts leave of q's values is at most 2^-23 of the row's largest one;
 * of a weight at most 2^-23 of it or 2^-45 of the query's largest one, whichever
 * is more.  For Q8_0 it is a weight's product with a block's scale that is split:
 * at most 2^-23 of it or 2^-39 of the largest product among the query's 32
 * neighbouring slots.  (All for rows of q whose largest value is 2^-100 or more;
 * scores have to stay within f32's range.)  Weighted sums are divided by
 * the weights' sum at the end: values above 2^100 may overflow on the way.
 * The work of all sequences and heads is cut into equal shares, one per CTA;
 * sequences that several CTAs share are joined by the last one to finish, in a fixed
 * order: results do not vary from run to run.
 * workspace: attn_ws_bytes() of caller-owned device memory, 256-byte aligned,
 * zero before the first call; every completed call leaves its counters zero
 * again.  It may serve calls of other shapes it is large enough for; calls that may overlap on
 * the GPU need workspaces of their own.  max_pages bounds the
 * lengths that a captured graph may later see. */
typedef struct {
    qmv_kv_cache cache;
    const float *q;
    float *out, *score;
    int64_t q_stride, out_stride, score_stride;
    int32_t n_head, n_seq, n_tok, max_pages;
    int64_t table_stride;
    const int32_t *block_table, *kv_len;
    float scale;
    int32_t window, n_sink;
    void *workspace;
    size_t workspace_bytes;
    int64_t score_slots;        /* <= score_stride; 0: score_stride             */
} qmv_attn;

int attn_decode(const qmv_attn *a, qmv_stream_t stream);

/* Workspace bytes of attn_decode for these sizes (with_score: score != NULL);
 * 0 when the sizes are outside its limits.  Needs no device.  With scores it
 * grows with the block table: about 4 * n_seq * n_head * n_tok * max_pages *
 * page_size bytes, 4.3 GB for 32 sequences of 32 heads and 8 tokens over 131072
 * slots. */
size_t attn_ws_bytes(const qmv_kv_cache *cache, int n_head, int n_seq, int n_tok, int max_pages,
                     int with_score);

/* A smaller cache for each sequence, kv head by kv head: of the kv_len[s]
 * slots, the first keep_first, the last keep_last and, of the slots between,
 * the ones with the highest score (ties: the lower slot; NaN counts as lowest),
 * `budget` slots in all; all of them when kv_len[s] <= budget.  The kept slots
 * are copied in their old order to slots 0, 1, ... of the pages that dst_table
 * names, in the same pool.  The copy is never in place, because pages may be shared
 * between sequences: no destination page may be a source page of the call or
 * appear twice.  Then
 *   kept[s][h][i]      = the old slot of new slot i   int32 [n_seq][n_kv_head][budget]
 *   score_out[s][h][i] = its score                    f32, as score, with score_out_stride
 *   len_out[s]         = min(kv_len[s], budget)       int32 [n_seq]
 * Entries and slots behind the new length are left as they were.  score_out may not
 * overlap score, nor len_out kv_len.  A row of `score` has score_slots
 * entries (0: score_stride of them), and a length above that number is clamped
 * like one beyond the block table.  Slots of bad source pages
 * take part in the choice but their values are not copied; bad destination
 * pages are not written. */
typedef struct {
    qmv_kv_cache cache;
    const float *score;
    float *score_out;
    int64_t score_stride, score_out_stride;     /* >= 1, >= budget              */
    int32_t n_seq, max_pages, dst_max_pages;
    int32_t keep_first, keep_last, budget;      /* keep_first + keep_last <= budget,
                                                   1 <= budget <= dst_max_pages * page_size */
    int64_t table_stride, dst_table_stride;
    const int32_t *block_table, *kv_len, *dst_table;
    int32_t *kept, *len_out;
    int64_t score_slots;                        /* <= score_stride; 0: score_stride */
} qmv_evict;

int kv_evict(const qmv_evict *a, qmv_stream_t stream);

/* Penalties, biases and a grammar mask on logits, and the greedy choice, beside
 * qmv_argmax (which chooses from the plain product).  For row r and token v,
 * with c = how often v occurs in hist[r][0 .. hist_len[r]) and the row's
 * params[r] = { repetition, frequency, presence }, in f32, each step rounded:
 *   z = logits[r][v];
 *   if c > 0:  z = z > 0 ? z / repetition : z * repetition;
 *              z = z - (frequency * c + presence);
 *   z = z + bias      (bias_vals[r][i] of the last i < bias_len[r] with
 *                      bias_ids[r][i] == v; no entry: nothing is added);
 *   z = -infinity where bit v % 32 of mask[r][v / 32] is 0.
 * out[r][v] = z (out may be logits, with the same stride, or NULL) and
 * idx_out[r] = the lowest v among the largest z of the tokens that the mask
 * lets through, NaN and -infinity left out, -1 when none is left.
 * Ids outside [0, vocab) in hist and bias_ids are skipped.  hist, bias_* and
 * mask may be NULL (nothing to apply); hist needs hist_len and params; the
 * strides are in elements, hist_len and bias_len are device int32 [n_rows] and are clamped to
 * [0, stride].  logits, out, bias_vals, params: f32, 4-byte aligned.
 * workspace: logits_ws_bytes(n_rows) device bytes, 8-byte aligned, zero before
 * the first call and left zero by every completed call; calls that may overlap
 * need their own. */
typedef struct {
    const float *logits;
    float *out;
    int64_t logits_stride, out_stride;
    int32_t n_rows;                             /* 1 .. 65535                   */
    int32_t vocab;                              /* 1 .. 2^31 - 1                */
    const int32_t *hist, *hist_len;
    int64_t hist_stride;
    const float *params;                        /* [n_rows][3]                  */
    const int32_t *bias_ids, *bias_len;
    const float *bias_vals;
    int64_t bias_stride;
    const uint32_t *mask;
    int64_t mask_stride;                        /* words                        */
    int32_t *idx_out;                           /* [n_rows]                     */
    void *workspace;
    size_t workspace_bytes;
} qmv_logits;

int logits_argmax(const qmv_logits *a, qmv_stream_t stream);
size_t logits_ws_bytes(int n_rows);

/* Dequantize the whole matrix to f32: out[rows][cols].  The values are
 * bit-exact f32 evaluations of the block formulas above (every product in
 * them is exact in f32; Q4_K and Q5_K round once, in the subtraction). */
int qmv_dequant(int fmt, const void *W_blocks, int64_t rows, int64_t cols,
                float *out, qmv_stream_t stream);

/* Synchronises `stream`, then reads and clears the sticky device error word
 * of the current device.  Returns QMV_OK, QMV_ERR_CUDA if the synchronisation
 * failed, or QMV_ERR_DEVICE if an error bit was set (the bits are stored in
 * *dev_err_out when it is not NULL). */
int qmv_check(qmv_stream_t stream, int *dev_err_out);

/* Static, never-NULL description of a qmv_status value. */
const char *qmv_strerror(int status);

/* Description of the CUDA error behind the last QMV_ERR_CUDA returned on the
 * calling host thread ("no error" if there was none). */
const char *qmv_last_cuda_error(void);

/* Bytes and weights per block of a format; 0 for an unknown format. */
size_t qmv_block_bytes(int fmt);
int qmv_block_weights(int fmt);

/* Programmatic dependent launch for the matvec launches (process-wide, off by
 * default).  When enabled, a matvec launch may start -- and begin streaming
 * its weight blocks into shared memory -- while the previous kernel in the
 * stream is still running; it waits for that kernel to finish before it reads
 * x, expert ids or gate weights and before it writes any output.  This hides
 * the launch gap between back-to-back matvecs of a decode step.  Enable it
 * only when no kernel still in flight on the stream writes the weight blocks
 * (true for inference weights loaded once).  qmv_get_pdl returns the setting. */
void qmv_set_pdl(int enable);
int qmv_get_pdl(void);

/* Test hook: which kernel served the calling host thread's most recent
 * matvec call (qmv_f32, qmv_batched, qmv_multi, qmv_chain, moe_qmv, moe_ffn,
 * qmv_argmax), so tests can show that each kernel path is exercised.
 * QMV_KERNEL_NONE before the first such call on the thread. */
#define QMV_KERNEL_NONE 0
#define QMV_KERNEL_WARP_RING 1      /* one to four tokens, per-warp copy rings   */
#define QMV_KERNEL_GENERAL 2        /* general pipeline (groups, grouped launches) */
#define QMV_KERNEL_TENSOR_CORE 3    /* three to eight tokens, mma.sync          */
#define QMV_KERNEL_STREAM 4         /* one token, producer warp + whole-row stages */
int qmv_debug_last_kernel(void);

/* Test hook for host-side failure handling: the next `count` launches made by
 * this library fail with QMV_ERR_CUDA without reaching the GPU. */
void qmv_debug_fail_next_launches(int count);

/* Test hook for the device-side failure path: while bytes > 0, the
 * streaming, warp-ring and tensor-core launches (qmv_f32 / qmv_batched on the
 * shapes that take them, qmv_chain) expect `bytes` more per copied tile than
 * they copy, so every stage wait runs into its bound (about a second), records
 * QMV_DEVERR_TIMEOUT (and, where a kernel then also gives up waiting for its
 * own copies, QMV_DEVERR_DRAIN) for qmv_check, and the kernel still finishes;
 * results are then undefined.  0 (the default) turns it off.  Not for
 * production. */
void qmv_debug_short_copies(int bytes);

#ifdef __cplusplus
}
#endif
#endif /* QMV_H */
