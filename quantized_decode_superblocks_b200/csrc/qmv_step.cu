// qmv_step.cu -- the decode step's operators around the weight products
// (kv_append, attn_decode, kv_evict, logits_argmax of include/qmv.h): argument
// checks, workspace layout and launches.
#include <algorithm>
#include <climits>

#include "../../include/qmv.h"
#include "qmv_attn.cuh"
#include "qmv_attn_launch.h"
#include "qmv_host.h"
#include "qmv_kv.cuh"
#include "qmv_launch.cuh"
#include "qmv_logits.cuh"

namespace {

using namespace qmv;

static_assert(KV_F16 == QMV_KV_F16 && KV_BF16 == QMV_KV_BF16 && KV_Q8_0 == QMV_KV_Q8_0, "cache types");
static_assert(ATT_MAX_SEQ == QMV_MAX_SEQ, "sequences of a call");

constexpr int MAX_HEADS = 8192, MAX_KV_HEADS = 1024, MAX_GROUP_ROWS = 1024;

bool aligned(const void *p, uintptr_t a) { return (reinterpret_cast<uintptr_t>(p) % a) == 0; }
int64_t ceil_div(int64_t a, int64_t b) { return (a + b - 1) / b; }
size_t up256(size_t n) { return (n + 255) / 256 * 256; }
// true when a stride of b-element rows can be multiplied by n rows in 64 bits
bool stride_ok(int64_t v, int64_t least) { return v >= least && v <= (int64_t)1 << 40; }
// Rows of `score`: their entries (0: as many as the stride) may not reach into the next row.
bool score_ok(int64_t stride, int64_t slots) { return stride_ok(stride, 1) && slots >= 0 && slots <= stride; }
int64_t score_width(int64_t stride, int64_t slots) { return slots ? slots : stride; }

int check_cache(const qmv_kv_cache &c)
{
    if (c.type != QMV_KV_F16 && c.type != QMV_KV_BF16 && c.type != QMV_KV_Q8_0) return QMV_ERR_FMT;
    const bool q8 = c.type == QMV_KV_Q8_0;
    if (!c.k || !c.v || (q8 && (!c.k_scale || !c.v_scale))) return QMV_ERR_NULL;
    const int unit = q8 ? 64 : 16;
    if (c.head_dim < unit || c.head_dim > 256 || c.head_dim % unit) return QMV_ERR_SHAPE;
    if (c.n_kv_head < 1 || c.n_kv_head > MAX_KV_HEADS || c.page_size < 1) return QMV_ERR_SHAPE;
    if (c.n_pages < 1 || c.n_pages > INT_MAX) return QMV_ERR_SHAPE;
    // a slot's heads and a page's slots may lie in either order, but rows of
    // head_dim values may not overlap
    if (!stride_ok(c.page_stride, c.head_dim) || !stride_ok(c.head_stride, c.n_kv_head > 1 ? c.head_dim : 0) ||
        !stride_ok(c.slot_stride, c.page_size > 1 ? c.head_dim : 0)) return QMV_ERR_SHAPE;
    const int64_t sa = q8 ? 64 : 8;
    if (c.page_stride % sa || c.head_stride % sa || c.slot_stride % sa) return QMV_ERR_ALIGN;
    if (!aligned(c.k, 16) || !aligned(c.v, 16)) return QMV_ERR_ALIGN;
    if (q8 && (!aligned(c.k_scale, 4) || !aligned(c.v_scale, 4))) return QMV_ERR_ALIGN;
    return QMV_OK;
}

// The block table's shape; on success the slots that a sequence can have.
int check_table(const qmv_kv_cache &c, int n_seq, int max_pages, int64_t stride, int64_t *slots)
{
    if (n_seq < 1 || n_seq > QMV_MAX_SEQ || max_pages < 1 || !stride_ok(stride, max_pages)) return QMV_ERR_SHAPE;
    *slots = (int64_t)max_pages * c.page_size;
    // slot numbers, with a tile's rounding, are 32-bit
    if (*slots > INT_MAX - 64) return QMV_ERR_SHAPE;
    return QMV_OK;
}

int page_shift(int page_size)
{
    if (page_size & (page_size - 1)) return -1;
    int s = 0;
    while ((1 << s) < page_size) ++s;
    return s;
}

struct AttnWs {
    size_t ml, o, raw, stats, bytes;
    int64_t raw_stride, raw_rows;
    int64_t steps;           // of the longest lengths, at most
};

// Workspace: counters | parts' (m, l) | parts' outputs | raw scores | rows' (m, l)
int attn_ws(int head_dim, int n_kv, int n_head, int n_seq, int n_tok, int64_t slots, bool score, AttnWs &w)
{
    if (n_tok < 1 || n_tok > QMV_MAX_NTOK) return QMV_ERR_NTOK;
    if (n_head < 1 || n_head > MAX_HEADS || n_head % n_kv) return QMV_ERR_SHAPE;
    const int rows = n_head / n_kv * n_tok;
    if (rows > MAX_GROUP_ROWS) return QMV_ERR_SHAPE;
    const int mb = attn_mb(rows);
    w.steps = ceil_div(rows, 8 * mb) * n_seq * n_kv * (slots / (ATT_MIN_TILE * ATT_MIN_NW) + 2);
    if (w.steps > INT_MAX / 2) return QMV_ERR_SHAPE;       // step numbers are 32-bit, and whole shares may pad them by an eighth
    const size_t parts = (size_t)2 * ATT_MAX_CTAS * 8 * mb;
    w.raw_stride = ceil_div(slots, ATT_MAX_TILE) * ATT_MAX_TILE;
    w.raw_rows = ceil_div(rows, 2) * 2;
    w.ml = up256(ATT_MAX_CTAS * sizeof(unsigned));
    w.o = w.ml + up256(parts * 2 * sizeof(float));
    w.raw = w.o + up256(parts * head_dim * sizeof(float));
    const size_t all_rows = (size_t)n_seq * n_kv * w.raw_rows;
    w.stats = w.raw + (score ? up256(all_rows * w.raw_stride * sizeof(float)) : 0);
    w.bytes = w.stats + (score ? up256(all_rows * 2 * sizeof(float)) : 0);
    return QMV_OK;
}

// Whether an output of `bytes` bytes at `out` shares memory with an input.
bool overlap(const void *out, int64_t out_bytes, const void *in, int64_t in_bytes)
{
    const uintptr_t a = reinterpret_cast<uintptr_t>(out), b = reinterpret_cast<uintptr_t>(in);
    return a < b ? b - a < (uintptr_t)out_bytes : a - b < (uintptr_t)in_bytes;
}

int finish(cudaError_t e) { return e == cudaSuccess ? QMV_OK : host_cuda_fail(e); }

}  // namespace

extern "C" {

size_t attn_ws_bytes(const qmv_kv_cache *cache, int n_head, int n_seq, int n_tok, int max_pages, int with_score)
{
    if (!cache || check_cache(*cache) != QMV_OK) return 0;
    int64_t slots = 0;
    AttnWs w;
    if (check_table(*cache, n_seq, max_pages, max_pages, &slots) != QMV_OK ||
        attn_ws(cache->head_dim, cache->n_kv_head, n_head, n_seq, n_tok, slots, with_score != 0, w) != QMV_OK) return 0;
    return w.bytes;
}

int attn_decode(const qmv_attn *a, qmv_stream_t stream)
{
    if (!a) return QMV_ERR_NULL;
    const qmv_kv_cache &c = a->cache;
    int rc = check_cache(c);
    if (rc) return rc;
    if (!a->q || !a->out || !a->block_table || !a->kv_len || !a->workspace) return QMV_ERR_NULL;
    int64_t slots = 0;
    AttnWs w;
    if (a->n_tok < 1 || a->n_tok > QMV_MAX_NTOK) return QMV_ERR_NTOK;
    if ((rc = check_table(c, a->n_seq, a->max_pages, a->table_stride, &slots))) return rc;
    if ((rc = attn_ws(c.head_dim, c.n_kv_head, a->n_head, a->n_seq, a->n_tok, slots, a->score != nullptr, w))) return rc;
    const int64_t width = (int64_t)a->n_head * c.head_dim;
    if (!stride_ok(a->q_stride, width) || !stride_ok(a->out_stride, width) || (a->score && !score_ok(a->score_stride, a->score_slots))) return QMV_ERR_SHAPE;
    if (a->window < 0 || a->n_sink < 0 || !(a->scale - a->scale == 0.f)) return QMV_ERR_SHAPE;
    if (!aligned(a->q, 16) || a->q_stride % 4 || !aligned(a->out, 4) || !aligned(a->score, 4) || !aligned(a->block_table, 4) ||
        !aligned(a->kv_len, 4) || !aligned(a->workspace, 256)) return QMV_ERR_ALIGN;
    if (a->out == a->q) return QMV_ERR_SHAPE;
    if (a->workspace_bytes < w.bytes) return QMV_ERR_WS;
    if (host_injected_failure()) return QMV_ERR_CUDA;
    HostDev di;
    if ((rc = host_dev(di))) return rc;

    AttnParams p = {};
    p.k = static_cast<const uint8_t *>(c.k);
    p.v = static_cast<const uint8_t *>(c.v);
    p.ks = static_cast<const uint8_t *>(c.k_scale);
    p.vs = static_cast<const uint8_t *>(c.v_scale);
    p.page_stride = c.page_stride;
    p.head_stride = c.head_stride;
    p.slot_stride = c.slot_stride;
    p.q = a->q;
    p.out = a->out;
    p.score = a->score;
    p.q_stride = a->q_stride;
    p.out_stride = a->out_stride;
    p.score_stride = a->score_stride;
    p.table = a->block_table;
    p.kv_len = a->kv_len;
    p.table_stride = a->table_stride;
    p.n_pages = c.n_pages;
    p.n_seq = a->n_seq;
    p.n_tok = a->n_tok;
    p.n_kv = c.n_kv_head;
    p.group = a->n_head / c.n_kv_head;
    p.rows = p.group * p.n_tok;
    p.inv_group = 1.f / (float)p.group;
    p.dim = c.head_dim;
    p.page_size = c.page_size;
    p.page_shift = page_shift(c.page_size);
    p.max_len = (int)(a->score ? std::min(slots, score_width(a->score_stride, a->score_slots)) : slots);
    p.mb = attn_mb(p.rows);
    p.n_rb = (int)ceil_div(p.rows, 8 * p.mb);
    p.window = a->window >= slots ? 0 : a->window;      // every slot is within a window that long
    p.n_sink = a->n_sink;
    p.scale_log2 = a->scale * 1.4426950408889634f;
    p.l_shift = c.type == QMV_KV_F16 ? ATT_F16_SHIFT : 0.f;
    uint8_t *ws = static_cast<uint8_t *>(a->workspace);
    p.counters = reinterpret_cast<unsigned *>(ws);
    p.part_ml = reinterpret_cast<float *>(ws + w.ml);
    p.part_o = reinterpret_cast<float *>(ws + w.o);
    p.raw = reinterpret_cast<float *>(ws + w.raw);
    p.stats = reinterpret_cast<float *>(ws + w.stats);
    p.raw_stride = w.raw_stride;
    p.raw_rows = (int)w.raw_rows;
    p.err = di.err;

    const cudaStream_t st = reinterpret_cast<cudaStream_t>(stream);
    cudaError_t e = c.type == QMV_KV_F16    ? launch_attn_f16(p, di.sm_count, w.steps, st)
                    : c.type == QMV_KV_BF16 ? launch_attn_bf16(p, di.sm_count, w.steps, st)
                                            : launch_attn_q8_0(p, di.sm_count, w.steps, st);
    if (e != cudaSuccess || !p.score) return finish(e);
    // launched while the first kernel runs (it waits for its end itself)
    static SmemCfg configured;
    // by the longest lengths, but no more than a few waves: the table may be far longer than the sequences
    const int64_t heads = (int64_t)p.n_kv * p.n_seq;
    const unsigned gx = (unsigned)std::min<int64_t>(ceil_div(p.max_len, ATT_SCORE_SLOTS), ceil_div(16 * di.sm_count, heads));
    return finish(launch_with(attn_score_kernel, configured, p, dim3(gx, (unsigned)p.n_kv, (unsigned)p.n_seq), 0, st, true, false, ATT_SCORE_THREADS));
}

int kv_append(const qmv_append *a, qmv_stream_t stream)
{
    if (!a) return QMV_ERR_NULL;
    const qmv_kv_cache &c = a->cache;
    int rc = check_cache(c);
    if (rc) return rc;
    if (!a->k || !a->v || !a->block_table || !a->kv_len || !a->q != !a->q_out) return QMV_ERR_NULL;
    if (a->rope_dim > 0 && !a->inv_freq) return QMV_ERR_NULL;
    if (a->n_tok < 1 || a->n_tok > QMV_MAX_NTOK) return QMV_ERR_NTOK;
    int64_t slots = 0;
    if ((rc = check_table(c, a->n_seq, a->max_pages, a->table_stride, &slots))) return rc;
    if (a->rope_dim < 0 || a->rope_dim > c.head_dim || a->rope_dim % 2) return QMV_ERR_SHAPE;
    if (a->rope_style != QMV_ROPE_HALVES && a->rope_style != QMV_ROPE_PAIRS) return QMV_ERR_SHAPE;
    const int64_t width = (int64_t)c.n_kv_head * c.head_dim, q_width = (int64_t)a->n_head * c.head_dim;
    if (!stride_ok(a->k_stride, width) || !stride_ok(a->v_stride, width)) return QMV_ERR_SHAPE;
    if (a->q && a->q == a->q_out && a->q_stride != a->q_out_stride) return QMV_ERR_SHAPE;
    if (a->q && (a->n_head < 1 || a->n_head > MAX_HEADS || !stride_ok(a->q_stride, q_width) || !stride_ok(a->q_out_stride, q_width))) return QMV_ERR_SHAPE;
    for (const void *x : {(const void *)a->q, (const void *)a->k, (const void *)a->v, (const void *)a->q_out, (const void *)a->block_table,
                          (const void *)a->kv_len, (const void *)a->pos, (const void *)a->inv_freq})
        if (!aligned(x, 4)) return QMV_ERR_ALIGN;
    if (host_injected_failure()) return QMV_ERR_CUDA;
    HostDev di;
    if ((rc = host_dev(di))) return rc;

    AppendParams p = {};
    p.k = static_cast<uint8_t *>(c.k);
    p.v = static_cast<uint8_t *>(c.v);
    p.ks = static_cast<uint8_t *>(c.k_scale);
    p.vs = static_cast<uint8_t *>(c.v_scale);
    p.page_stride = c.page_stride;
    p.head_stride = c.head_stride;
    p.slot_stride = c.slot_stride;
    p.n_pages = c.n_pages;
    p.q_in = a->q;
    p.k_in = a->k;
    p.v_in = a->v;
    p.q_out = a->q_out;
    p.q_stride = a->q_stride;
    p.k_stride = a->k_stride;
    p.v_stride = a->v_stride;
    p.q_out_stride = a->q_out_stride;
    p.type = c.type;
    p.n_head = a->n_head;
    p.n_kv = c.n_kv_head;
    p.dim = c.head_dim;
    p.n_tok = a->n_tok;
    p.rope_dim = a->rope_dim;
    p.rope_pairs = a->rope_style == QMV_ROPE_PAIRS;
    p.page_size = c.page_size;
    p.page_shift = page_shift(c.page_size);
    p.max_len = (int)slots;
    p.table = a->block_table;
    p.kv_len = a->kv_len;
    p.pos = a->pos;
    p.table_stride = a->table_stride;
    p.inv_freq = a->inv_freq;
    p.err = di.err;
    const int tokens = a->n_seq * a->n_tok;
    const int heads = (a->q ? a->n_head : 0) + 2 * c.n_kv_head;
    const int gy = (int)std::min<int64_t>(ceil_div(heads, APP_THREADS / 32), std::max(1, APP_CTAS * di.sm_count / tokens));
    const dim3 grid((unsigned)a->n_tok, (unsigned)a->n_seq, (unsigned)gy);
    const cudaStream_t st = reinterpret_cast<cudaStream_t>(stream);
    if (c.head_dim <= 64) kv_append_kernel<2><<<grid, APP_THREADS, 0, st>>>(p);
    else if (c.head_dim <= 128) kv_append_kernel<4><<<grid, APP_THREADS, 0, st>>>(p);
    else kv_append_kernel<8><<<grid, APP_THREADS, 0, st>>>(p);
    return finish(cudaGetLastError());
}

int kv_evict(const qmv_evict *a, qmv_stream_t stream)
{
    if (!a) return QMV_ERR_NULL;
    const qmv_kv_cache &c = a->cache;
    int rc = check_cache(c);
    if (rc) return rc;
    if (!a->score || !a->score_out || !a->block_table || !a->kv_len || !a->dst_table || !a->kept || !a->len_out) return QMV_ERR_NULL;
    int64_t slots = 0, dst_slots = 0;
    if ((rc = check_table(c, a->n_seq, a->max_pages, a->table_stride, &slots))) return rc;
    if ((rc = check_table(c, a->n_seq, a->dst_max_pages, a->dst_table_stride, &dst_slots))) return rc;
    if (a->keep_first < 0 || a->keep_last < 0 || a->budget < 1 || (int64_t)a->keep_first + a->keep_last > a->budget ||
        a->budget > dst_slots) return QMV_ERR_SHAPE;
    if (!score_ok(a->score_stride, a->score_slots) || !stride_ok(a->score_out_stride, a->budget)) return QMV_ERR_SHAPE;
    const int64_t max_len = std::min(slots, score_width(a->score_stride, a->score_slots));
    for (const void *x : {(const void *)a->score, (const void *)a->score_out, (const void *)a->block_table, (const void *)a->kv_len,
                          (const void *)a->dst_table, (const void *)a->kept, (const void *)a->len_out})
        if (!aligned(x, 4)) return QMV_ERR_ALIGN;
    const int64_t rows = (int64_t)a->n_seq * c.n_kv_head;
    if (overlap(a->score_out, ((rows - 1) * a->score_out_stride + a->budget) * 4, a->score, ((rows - 1) * a->score_stride + max_len) * 4) ||
        overlap(a->len_out, (int64_t)a->n_seq * 4, a->kv_len, (int64_t)a->n_seq * 4)) return QMV_ERR_SHAPE;
    const int per = EV_COPY_THREADS / 32 * EV_SLOTS;                                          // slots of a CTA of the copy
    const int64_t gx = ceil_div(std::min<int64_t>(a->budget, max_len), per) * c.n_kv_head;
    if (gx > INT_MAX) return QMV_ERR_SHAPE;
    if (host_injected_failure()) return QMV_ERR_CUDA;
    HostDev di;
    if ((rc = host_dev(di))) return rc;

    EvictParams p = {};
    p.k = static_cast<uint8_t *>(c.k);
    p.v = static_cast<uint8_t *>(c.v);
    p.ks = static_cast<uint8_t *>(c.k_scale);
    p.vs = static_cast<uint8_t *>(c.v_scale);
    p.page_stride = c.page_stride;
    p.head_stride = c.head_stride;
    p.slot_stride = c.slot_stride;
    p.n_pages = c.n_pages;
    p.score = a->score;
    p.score_out = a->score_out;
    p.score_stride = a->score_stride;
    p.score_out_stride = a->score_out_stride;
    p.table_stride = a->table_stride;
    p.dst_table_stride = a->dst_table_stride;
    p.table = a->block_table;
    p.kv_len = a->kv_len;
    p.dst_table = a->dst_table;
    p.kept = a->kept;
    p.len_out = a->len_out;
    p.n_kv = c.n_kv_head;
    p.page_size = c.page_size;
    p.page_shift = page_shift(c.page_size);
    p.max_len = (int)max_len;
    p.keep_first = a->keep_first;
    p.keep_last = a->keep_last;
    p.budget = a->budget;
    p.eb = c.type == QMV_KV_Q8_0 ? 1 : 2;
    p.row_bytes = c.head_dim * p.eb;
    p.scale_words = c.type == QMV_KV_Q8_0 ? c.head_dim / 64 : 0;
    p.err = di.err;
    const cudaStream_t st = reinterpret_cast<cudaStream_t>(stream);
    static SmemCfg configured_choice[2], configured;
    const bool many = evict_cluster(p.max_len, a->n_seq * c.n_kv_head, di.sm_count);
    const dim3 grid((unsigned)(c.n_kv_head * (many ? EV_CL : 1)), (unsigned)a->n_seq);
    const size_t smem = (size_t)std::min(many ? (int)ceil_div(p.max_len, EV_CL * EV_THREADS) * EV_THREADS : p.max_len, EV_KEYS) * sizeof(uint32_t);
    const cudaError_t e = many ? launch_with(kv_evict_cluster_kernel, configured_choice[1], p, grid, smem, st, false, false, EV_THREADS)
                               : launch_with(kv_evict_kernel, configured_choice[0], p, grid, smem, st, false, false, EV_THREADS);
    if (e != cudaSuccess) return finish(e);
    // launched while the choice runs (it waits for its end itself)
    return finish(launch_with(kv_evict_copy_kernel, configured, p, dim3((unsigned)gx, (unsigned)a->n_seq), (size_t)per * 2 * p.row_bytes, st, true, false, EV_COPY_THREADS));
}

size_t logits_ws_bytes(int n_rows)
{
    if (n_rows < 1 || n_rows > 65535) return 0;
    return (size_t)n_rows * 16;
}

int logits_argmax(const qmv_logits *a, qmv_stream_t stream)
{
    if (!a || !a->logits || !a->idx_out || !a->workspace) return QMV_ERR_NULL;
    if (a->hist && (!a->hist_len || !a->params)) return QMV_ERR_NULL;
    if (a->bias_ids && (!a->bias_len || !a->bias_vals)) return QMV_ERR_NULL;
    if (a->n_rows < 1 || a->n_rows > 65535 || a->vocab < 1) return QMV_ERR_SHAPE;
    if (!stride_ok(a->logits_stride, a->vocab) || (a->out && !stride_ok(a->out_stride, a->vocab))) return QMV_ERR_SHAPE;
    if (a->out == a->logits && a->out_stride != a->logits_stride) return QMV_ERR_SHAPE;
    if ((a->hist && !stride_ok(a->hist_stride, 0)) || (a->mask && !stride_ok(a->mask_stride, ceil_div(a->vocab, 32)))) return QMV_ERR_SHAPE;
    if (a->bias_ids && (!stride_ok(a->bias_stride, 0) || a->bias_stride > INT_MAX)) return QMV_ERR_SHAPE;
    for (const void *x : {(const void *)a->logits, (const void *)a->out, (const void *)a->hist, (const void *)a->hist_len, (const void *)a->params,
                          (const void *)a->bias_ids, (const void *)a->bias_len, (const void *)a->bias_vals, (const void *)a->mask, (const void *)a->idx_out})
        if (!aligned(x, 4)) return QMV_ERR_ALIGN;
    if (!aligned(a->workspace, 8)) return QMV_ERR_ALIGN;
    if (a->workspace_bytes < logits_ws_bytes(a->n_rows)) return QMV_ERR_WS;
    if (host_injected_failure()) return QMV_ERR_CUDA;
    HostDev di;
    const int rc = host_dev(di);
    if (rc) return rc;

    LogitsParams p = {};
    p.logits = a->logits;
    p.out = a->out;
    p.logits_stride = a->logits_stride;
    p.out_stride = a->out_stride;
    p.hist_stride = a->hist_stride;
    p.bias_stride = a->bias_stride;
    p.mask_stride = a->mask_stride;
    p.vocab = a->vocab;
    p.hist = a->hist;
    p.hist_len = a->hist_len;
    p.bias_ids = a->bias_ids;
    p.bias_len = a->bias_len;
    p.params = a->params;
    p.bias_vals = a->bias_vals;
    p.mask = a->mask;
    p.idx = a->idx_out;
    p.keys = static_cast<unsigned long long *>(a->workspace);
    p.done = reinterpret_cast<unsigned *>(p.keys + a->n_rows);
    const bool wide = (p.hist && p.hist_stride > 65535) || (p.bias_ids && p.bias_stride >= 65535);
    p.slice = logits_slice(a->n_rows, a->vocab, di.sm_count, wide);
    const dim3 grid((unsigned)ceil_div(a->vocab, p.slice), (unsigned)a->n_rows);
    static SmemCfg configured[2];
    const size_t smem = logits_smem(p.slice, wide);
    const cudaStream_t st = reinterpret_cast<cudaStream_t>(stream);
    return finish(wide ? launch_with(logits_argmax_kernel<true>, configured[1], p, grid, smem, st, false, false, LG_THREADS)
                       : launch_with(logits_argmax_kernel<false>, configured[0], p, grid, smem, st, false, false, LG_THREADS));
}

}  // extern "C"
