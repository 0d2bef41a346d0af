// qmv_logits.cuh -- penalties for repeated tokens, biases and a grammar mask on
// logits, with the greedy choice (logits_argmax in include/qmv.h).
//
// A CTA takes a slice of one row's vocabulary.  It counts the row's history
// and notes the last bias entry per token of its slice in shared memory
// (integer atomics: their order does not matter), then runs over its logits
// once; the first of them are loaded before the history is read.  Every CTA
// reads the row's whole history and biases, so slices are long (up to
// LG_MAX_SLICE tokens, 64 KB of counts and entries, three CTAs a SM) where there
// are many rows, and short where a few rows have to reach all SMs.
// The best allowed (value, token) goes into the row's 64-bit key as in
// qmv_argmax; the row's last CTA writes idx_out and zeroes the workspace.
#pragma once

#include "qmv_device.cuh"

namespace qmv {

constexpr int LG_THREADS = 512, LG_FLY = 8;     // threads; logits that one has in flight
constexpr int LG_MIN_SLICE = 1024, LG_MAX_SLICE = 8192;

// Tokens of a slice: about three CTAs a SM.
static inline int logits_slice(int n_rows, int vocab, int sms)
{
    const int64_t each = ((int64_t)n_rows * vocab + 3 * sms - 1) / (3 * sms);
    int s = LG_MIN_SLICE;
    while (s < each && s < LG_MAX_SLICE) s *= 2;
    return s;
}

struct LogitsParams {
    const float *logits;
    float *out;
    int64_t logits_stride, out_stride, hist_stride, bias_stride, mask_stride;
    int32_t vocab, slice;
    const int32_t *hist, *hist_len, *bias_ids, *bias_len;
    const float *params, *bias_vals;
    const uint32_t *mask;
    int32_t *idx;
    unsigned long long *keys;
    unsigned *done;
};

static __global__ void __launch_bounds__(LG_THREADS, 3) logits_argmax_kernel(const __grid_constant__ LogitsParams p)
{
    extern __shared__ __align__(16) int2 s_tok[];                         // [slice] per token: count in the history, last bias entry + 1
    __shared__ float s_v[LG_THREADS / 32];
    __shared__ int s_i[LG_THREADS / 32];
    const bool pushed = p.hist || p.bias_ids;
    const int row = blockIdx.y, v0 = blockIdx.x * p.slice, nv = min(p.slice, p.vocab - v0);
    const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
    // a thread's tokens are v0 + tid, + LG_THREADS, ...: a warp's lie in one word of the mask
    const float *z0 = p.logits + (int64_t)row * p.logits_stride + v0 + tid;
    const uint32_t *mask = p.mask ? p.mask + (int64_t)row * p.mask_stride + (v0 >> 5) + warp : nullptr;
    float z[LG_FLY];
    uint32_t mw[LG_FLY];
    auto load = [&](int i0) {
        if (i0 + LG_FLY * LG_THREADS <= nv) {
#pragma unroll
            for (int u = 0; u < LG_FLY; ++u) z[u] = __ldcs(z0 + i0 + u * LG_THREADS);
#pragma unroll
            for (int u = 0; u < LG_FLY; ++u) mw[u] = mask ? __ldg(mask + (i0 >> 5) + u * (LG_THREADS / 32)) : 0xFFFFFFFFu;
        } else {
#pragma unroll
            for (int u = 0; u < LG_FLY; ++u) {
                const bool in = i0 + u * LG_THREADS + tid < nv;
                z[u] = in ? __ldcs(z0 + i0 + u * LG_THREADS) : 0.f;
                mw[u] = mask && in ? __ldg(mask + (i0 >> 5) + u * (LG_THREADS / 32)) : 0xFFFFFFFFu;
            }
        }
    };
    load(0);
    if (pushed)
        for (int i = tid; i < p.slice / 2; i += LG_THREADS) reinterpret_cast<int4 *>(s_tok)[i] = make_int4(0, 0, 0, 0);
    __syncthreads();
    // history and biases: LG_FLY entries a thread in flight
    auto scan = [&](const int32_t *ids, int64_t n, auto &&note) {
        for (int64_t i0 = 0; i0 < n; i0 += LG_FLY * LG_THREADS) {
            int id[LG_FLY];
#pragma unroll
            for (int u = 0; u < LG_FLY; ++u) {
                const int64_t i = i0 + u * LG_THREADS + tid;
                id[u] = i < n ? __ldg(ids + i) : -1;
            }
#pragma unroll
            for (int u = 0; u < LG_FLY; ++u) {
                const unsigned o = (unsigned)id[u] - (unsigned)v0;
                if (o < (unsigned)nv && id[u] >= 0) note((int)o, (int)(i0 + u * LG_THREADS + tid));
            }
        }
    };
    float rep = 1.f, freq = 0.f, pres = 0.f;
    if (p.hist) {
        rep = __ldg(p.params + 3 * (int64_t)row);
        freq = __ldg(p.params + 3 * (int64_t)row + 1);
        pres = __ldg(p.params + 3 * (int64_t)row + 2);
        scan(p.hist + (int64_t)row * p.hist_stride, min((int64_t)max(0, __ldg(p.hist_len + row)), p.hist_stride),
             [&](int o, int) { atomicAdd(&s_tok[o].x, 1); });
    }
    const float *bias = p.bias_vals + (int64_t)row * p.bias_stride;
    if (p.bias_ids)
        scan(p.bias_ids + (int64_t)row * p.bias_stride, min((int64_t)max(0, __ldg(p.bias_len + row)), p.bias_stride),
             [&](int o, int i) { atomicMax(&s_tok[o].y, i + 1); });
    __syncthreads();
    float *out = p.out ? p.out + (int64_t)row * p.out_stride + v0 + tid : nullptr;
    float bv = -INFINITY;
    int bi = -1;
    auto push = [&](float y, int2 t) {                                    // few tokens: not inlined into each of the unrolled steps
        if (t.x > 0) {
            y = y > 0.f ? __fdiv_rn(y, rep) : __fmul_rn(y, rep);
            y = __fsub_rn(y, __fadd_rn(__fmul_rn(freq, (float)t.x), pres));
        }
        return t.y > 0 ? __fadd_rn(y, __ldg(bias + t.y - 1)) : y;
    };
    for (int i0 = 0; i0 < nv; i0 += LG_FLY * LG_THREADS) {
        if (i0) load(i0);
        if (pushed) {
            int2 t[LG_FLY];
#pragma unroll
            for (int u = 0; u < LG_FLY; ++u) t[u] = i0 + u * LG_THREADS < p.slice ? s_tok[i0 + u * LG_THREADS + tid] : make_int2(0, 0);
#pragma unroll
            for (int u = 0; u < LG_FLY; ++u)
                if (t[u].x | t[u].y) z[u] = push(z[u], t[u]);
        }
#pragma unroll
        for (int u = 0; u < LG_FLY; ++u) {
            const int i = i0 + u * LG_THREADS;
            if (i + tid >= nv) break;
            const float y = (mw[u] >> lane) & 1u ? z[u] : -INFINITY;
            if (out) __stcs(out + i, y);
            if (y > bv) {                                                 // the first of equals; neither NaN nor -infinity
                bv = y;
                bi = v0 + tid + i;
            }
        }
    }
    for (int o = 16; o; o >>= 1) argmax_merge(bv, bi, __shfl_xor_sync(0xFFFFFFFFu, bv, o), __shfl_xor_sync(0xFFFFFFFFu, bi, o));
    if (lane == 0) {
        s_v[warp] = bv;
        s_i[warp] = bi;
    }
    __syncthreads();
    if (warp == 0) {
        bv = s_v[lane & (LG_THREADS / 32 - 1)];
        bi = s_i[lane & (LG_THREADS / 32 - 1)];
        for (int o = LG_THREADS / 64; o; o >>= 1) argmax_merge(bv, bi, __shfl_xor_sync(0xFFFFFFFFu, bv, o), __shfl_xor_sync(0xFFFFFFFFu, bi, o));
    }
    if (tid == 0) {
        if (bi >= 0) atomicMax(p.keys + row, argmax_key(bv, bi));
        __threadfence();
        if (atomicAdd(p.done + row, 1u) == gridDim.x - 1u) {              // the row's last CTA
            __threadfence();
            const unsigned long long k = atomicExch(p.keys + row, 0ull);
            atomicExch(p.done + row, 0u);
            p.idx[row] = k ? (int32_t)(0xFFFFFFFFu - (uint32_t)(k & 0xFFFFFFFFull)) : -1;
        }
    }
}

}  // namespace qmv
