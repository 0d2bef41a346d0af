// qmv_kv.cuh -- the new tokens into the paged cache (kv_append) and a smaller
// cache for each sequence (kv_evict); both declared in include/qmv.h.
#pragma once

#include <cooperative_groups.h>
#include <cuda_bf16.h>

#include "qmv_attn.cuh"

namespace qmv {

// -------------------------------------------------------------- append --
// One CTA per (token, share of the heads): the token's cosines and sines once
// in 64 bits, then one warp per head.  A few KB per token:
// bound by launch and memory latency, not by bandwidth.
constexpr int APP_THREADS = 256;

struct AppendParams {
    uint8_t *k, *v, *ks, *vs;
    int64_t page_stride, head_stride, slot_stride, n_pages;
    const float *q_in, *k_in, *v_in;
    float *q_out;
    int64_t q_stride, k_stride, v_stride, q_out_stride;
    int32_t type, n_head, n_kv, dim, n_tok, rope_dim, rope_pairs;
    int32_t page_size, max_len;
    const int32_t *table, *kv_len, *pos;
    int64_t table_stride;
    const float *inv_freq;
    int *err;
};

static __global__ void __launch_bounds__(APP_THREADS) kv_append_kernel(const __grid_constant__ AppendParams p)
{
    __shared__ double s_cos[128], s_sin[128];
    __shared__ long long s_at;                     // the slot's first element, -1: nothing to store
    const int tok = blockIdx.x, s = tok / p.n_tok, t = tok % p.n_tok;
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    const int raw = __ldg(p.kv_len + s), len = min(max(raw, 0), p.max_len), slot = len - p.n_tok + t;
    if (threadIdx.x == 0) {
        long long at = -1;
        if (slot >= 0) {
            const int page = __ldg(p.table + (int64_t)s * p.table_stride + slot / p.page_size);
            if (page >= 0 && page < p.n_pages) at = page * p.page_stride + (slot % p.page_size) * p.slot_stride;
            else atomicOr(p.err, 8 /* QMV_DEVERR_PAGE_ID */);
        }
        if (raw != len) atomicOr(p.err, 16 /* QMV_DEVERR_SEQ_LEN */);
        s_at = at;
    }
    const double pos = p.pos ? __ldg(p.pos + tok) : slot;
    for (int i = threadIdx.x; i < p.rope_dim / 2; i += APP_THREADS) sincos(pos * (double)__ldg(p.inv_freq + i), s_sin + i, s_cos + i);
    __syncthreads();
    const long long at = s_at;
    const int nb = (p.dim + 31) / 32, nq = p.q_out ? p.n_head : 0, heads = nq + 2 * p.n_kv;
    const int half = p.rope_dim / 2;
    for (int head = blockIdx.y * (APP_THREADS / 32) + warp; head < heads; head += gridDim.y * (APP_THREADS / 32)) {
        const bool is_q = head < nq, is_k = !is_q && head < nq + p.n_kv;
        const int h = is_q ? head : is_k ? head - nq : head - nq - p.n_kv;
        const float *x = is_q ? p.q_in + tok * p.q_stride : is_k ? p.k_in + tok * p.k_stride : p.v_in + tok * p.v_stride;
        x += (int64_t)h * p.dim;
        float y[8], z[8];                          // this lane's values and their partners
#pragma unroll
        for (int b = 0; b < 8; ++b) {
            const int d = b * 32 + lane;
            y[b] = b < nb && d < p.dim ? x[d] : 0.f;
            z[b] = !is_q && !is_k ? 0.f : d < p.rope_dim ? x[p.rope_pairs ? d ^ 1 : d < half ? d + half : d - half] : 0.f;
        }
        __syncwarp();                              // q may be rotated in place: all is read before anything is written
#pragma unroll
        for (int b = 0; b < 8; ++b) {
            if (b >= nb) break;
            const int d = b * 32 + lane;
            const bool in = d < p.dim;
            float w = y[b];
            if ((is_q || is_k) && d < p.rope_dim) {
                const int i = p.rope_pairs ? d >> 1 : d < half ? d : d - half;
                const bool second = p.rope_pairs ? d & 1 : d >= half;
                const double own = y[b], other = z[b];
                w = (float)(second ? other * s_sin[i] + own * s_cos[i] : own * s_cos[i] - other * s_sin[i]);
            }
            if (is_q) {
                if (in) p.q_out[tok * p.q_out_stride + (int64_t)h * p.dim + d] = w;
                continue;
            }
            if (at < 0) continue;
            const long long e = at + h * p.head_stride + d;
            uint8_t *pool = is_k ? p.k : p.v;
            if (p.type == KV_F16) {
                if (in) reinterpret_cast<__half *>(pool)[e] = __float2half_rn(w);
            } else if (p.type == KV_BF16) {
                if (in) reinterpret_cast<__nv_bfloat16 *>(pool)[e] = __float2bfloat16_rn(w);
            } else {
                float mx = fabsf(w);
                for (int o = 16; o; o >>= 1) mx = fmaxf(mx, __shfl_xor_sync(0xFFFFFFFFu, mx, o));
                const __half dh = __float2half_rn(fminf(__fdiv_rn(mx, 127.f), 65504.f));
                const float df = __half2float(dh);
                const float qv = df > 0.f ? fminf(fmaxf(rintf(__fdiv_rn(w, df)), -127.f), 127.f) : 0.f;
                reinterpret_cast<int8_t *>(pool)[e] = (int8_t)(int)qv;
                if (lane == 0) reinterpret_cast<__half *>(is_k ? p.ks : p.vs)[e / 32] = dh;
            }
        }
    }
}

// -------------------------------------------------------------- evict --
// A cluster of EV_CL CTAs per (sequence, kv head); CTA r looks after the r-th
// part of the slots.  The slots between the kept ends are ranked by a radix
// select over order-preserving 32-bit keys (four 8-bit digits, highest first):
// each CTA counts its own slots' digits, and all add up the cluster's counts
// over distributed shared memory, so that the key of the last slot to keep, and how
// many slots with exactly that key are kept (the lowest ones), are known to
// all after four rounds.  Then each CTA writes its kept slots in order, at
// the place that the counts of the CTAs before it give, and the cluster copies
// the kept slots' values, an equal share per CTA.
constexpr int EV_CL = 8, EV_THREADS = 512;

struct EvictParams {
    uint8_t *k, *v, *ks, *vs;
    int64_t page_stride, head_stride, slot_stride, n_pages;
    const float *score;
    float *score_out;
    int64_t score_stride, score_out_stride, table_stride, dst_table_stride;
    const int32_t *table, *kv_len, *dst_table;
    int32_t *kept, *len_out;
    int32_t n_kv, page_size, max_len, keep_first, keep_last, budget;
    int32_t row_bytes, scale_words, eb;       // of one slot and head; scale_words: 4-byte words of its scales
    int *err;
};

// Larger for a larger score; -0 equals +0; NaN is lowest.
__device__ __forceinline__ uint32_t evict_key(float x)
{
    if (x != x) return 0u;
    const uint32_t u = x == 0.f ? 0u : __float_as_uint(x);
    return (u & 0x80000000u) ? ~u : (u | 0x80000000u);
}

static __global__ void __cluster_dims__(EV_CL, 1, 1) __launch_bounds__(EV_THREADS) kv_evict_kernel(const __grid_constant__ EvictParams p)
{
    namespace cg = cooperative_groups;
    cg::cluster_group cl = cg::this_cluster();
    __shared__ int s_hist[4][256];
    __shared__ int s_cnt[2];                  // this CTA's slots above, and at, the last key
    __shared__ int s_sum[256];
    __shared__ int s_sel[2];
    __shared__ int s_warp[EV_THREADS / 32][2];
    const int rank = (int)cl.block_rank(), h = blockIdx.y, s = blockIdx.z;
    const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
    const int raw = __ldg(p.kv_len + s), n = min(max(raw, 0), p.max_len), m = min(n, p.budget);
    if (raw != n && tid == 0) atomicOr(p.err, 16 /* QMV_DEVERR_SEQ_LEN */);
    const int64_t sh = (int64_t)s * p.n_kv + h;
    const float *score = p.score + sh * p.score_stride;
    float *score_out = p.score_out + sh * p.score_out_stride;
    int32_t *kept = p.kept + sh * p.budget;
    const int part = (int)(((int64_t)n + EV_CL * EV_THREADS - 1) / (EV_CL * EV_THREADS)) * EV_THREADS;
    const int a = (int)min((int64_t)n, (int64_t)rank * part), b = (int)min((int64_t)n, (int64_t)a + part);
    const int mid0 = min(p.keep_first, n), mid1 = max(mid0, n - p.keep_last);     // ranked slots
    const bool all = n <= p.budget;
    const int need = p.budget - p.keep_first - p.keep_last;                       // of them (not all)

    uint32_t prefix = 0;
    int want = need;                                                              // still to take within the prefix
    if (!all) {
        for (int i = tid; i < 4 * 256; i += EV_THREADS) (&s_hist[0][0])[i] = 0;
        __syncthreads();
        const int c0 = max(a, mid0), c1 = min(b, mid1);
        for (int pass = 0; pass < 4; ++pass) {
            const int sft = 24 - 8 * pass;
            for (int j = c0 + tid; j < c1; j += EV_THREADS) {
                const uint32_t key = evict_key(__ldg(score + j));
                if (pass == 0 || (key >> (sft + 8)) == prefix) atomicAdd(&s_hist[pass][(key >> sft) & 255u], 1);
            }
            cl.sync();
            if (tid < 256) {
                int c = 0;
                for (int r = 0; r < EV_CL; ++r) c += cl.map_shared_rank(&s_hist[0][0], r)[pass * 256 + tid];
                s_sum[tid] = c;
            }
            __syncthreads();
            if (warp == 0) {
                // lane i has digits 255 - 8 i and the seven below: from the top down
                int own = 0;
                for (int d = 0; d < 8; ++d) own += s_sum[255 - 8 * lane - d];
                int up = own;
                for (int o = 1; o < 32; o <<= 1) {
                    const int y = __shfl_up_sync(0xFFFFFFFFu, up, o);
                    if (lane >= o) up += y;
                }
                int before = up - own;                                            // slots of larger digits
                if (before < want && up >= want) {
                    for (int d = 0; d < 8; ++d) {
                        const int dig = 255 - 8 * lane - d, c = s_sum[dig];
                        if (before + c >= want) {
                            s_sel[0] = dig;
                            s_sel[1] = want - before;
                            break;
                        }
                        before += c;
                    }
                }
                if (want == 0 && lane == 0) {                                     // nothing between the ends is kept
                    s_sel[0] = 255;
                    s_sel[1] = 0;
                }
            }
            __syncthreads();
            prefix = (prefix << 8) | (uint32_t)s_sel[0];
            want = s_sel[1];
            __syncthreads();
        }
    }
    // ---- how many slots this CTA keeps, and its place among the cluster's
    auto is_end = [&](int j) { return all || j < mid0 || j >= mid1; };
    int above = 0, at = 0;
    for (int j = a + tid; j < b; j += EV_THREADS) {
        const uint32_t key = all ? 0u : evict_key(__ldg(score + j));
        above += is_end(j) || (need > 0 && key > prefix);
        at += !is_end(j) && key == prefix;
    }
    for (int o = 16; o; o >>= 1) {
        above += __shfl_xor_sync(0xFFFFFFFFu, above, o);
        at += __shfl_xor_sync(0xFFFFFFFFu, at, o);
    }
    if (lane == 0) {
        s_warp[warp][0] = above;
        s_warp[warp][1] = at;
    }
    __syncthreads();
    if (tid < 2) {
        int c = 0;
        for (int w = 0; w < EV_THREADS / 32; ++w) c += s_warp[w][tid];
        s_cnt[tid] = c;
    }
    cl.sync();
    int pre_above = 0, pre_at = 0;
    for (int r = 0; r < rank; ++r) {
        const int *c = cl.map_shared_rank(s_cnt, r);
        pre_above += c[0];
        pre_at += c[1];
    }
    // ---- the kept slots in order
    for (int j0 = a; j0 < b; j0 += EV_THREADS) {
        const int j = j0 + tid;
        float sc = 0.f;
        bool up = false, eq = false;
        if (j < b) {
            sc = __ldg(score + j);
            const uint32_t key = evict_key(sc);
            up = is_end(j) || (need > 0 && key > prefix);
            eq = !is_end(j) && key == prefix;
        }
        const uint32_t mu = __ballot_sync(0xFFFFFFFFu, up), me = __ballot_sync(0xFFFFFFFFu, eq);
        __syncthreads();
        if (lane == 0) {
            s_warp[warp][0] = __popc(mu);
            s_warp[warp][1] = __popc(me);
        }
        __syncthreads();
        int bu = pre_above, be = pre_at;
        for (int w = 0; w < EV_THREADS / 32; ++w) {
            if (w < warp) {
                bu += s_warp[w][0];
                be += s_warp[w][1];
            }
            pre_above += s_warp[w][0];
            pre_at += s_warp[w][1];
        }
        const uint32_t below = (1u << lane) - 1u;
        bu += __popc(mu & below);
        be += __popc(me & below);
        if (up || (eq && be < want)) {
            const int i = bu + min(be, want);
            kept[i] = j;
            score_out[i] = sc;
        }
    }
    if (rank == 0 && h == 0 && tid == 0) p.len_out[s] = m;
    cl.sync();                                                                    // the list is complete
    // ---- copy: 16-byte pieces of k and v, 4-byte words of the scales
    const int32_t *src = p.table + (int64_t)s * p.table_stride, *dst = p.dst_table + (int64_t)s * p.dst_table_stride;
    const int i0 = (int)((int64_t)m * rank / EV_CL), i1 = (int)((int64_t)m * (rank + 1) / EV_CL);
    const int pieces = p.row_bytes / 16;
    for (int i = i0 + warp; i < i1; i += EV_THREADS / 32) {
        const int j = __ldcg(kept + i);
        const int ps = __ldg(src + j / p.page_size), pd = __ldg(dst + i / p.page_size);
        const bool ok = ps >= 0 && ps < p.n_pages && pd >= 0 && pd < p.n_pages;
        if (!ok) {
            if (lane == 0) atomicOr(p.err, 8 /* QMV_DEVERR_PAGE_ID */);
            continue;
        }
        const int64_t es = ps * p.page_stride + h * p.head_stride + (j % p.page_size) * p.slot_stride;
        const int64_t ed = pd * p.page_stride + h * p.head_stride + (i % p.page_size) * p.slot_stride;
        for (int c = lane; c < 2 * pieces; c += 32) {
            uint8_t *pool = c < pieces ? p.k : p.v;
            const int64_t o = (c < pieces ? c : c - pieces) * 16;
            *reinterpret_cast<uint4 *>(pool + ed * p.eb + o) = __ldcg(reinterpret_cast<const uint4 *>(pool + es * p.eb + o));
        }
        for (int c = lane; c < 2 * p.scale_words; c += 32) {
            uint8_t *pool = c < p.scale_words ? p.ks : p.vs;
            const int64_t o = (c < p.scale_words ? c : c - p.scale_words) * 4;
            *reinterpret_cast<uint32_t *>(pool + ed / 16 + o) = __ldcg(reinterpret_cast<const uint32_t *>(pool + es / 16 + o));
        }
    }
}

}  // namespace qmv
