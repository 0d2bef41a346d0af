// qmv_logits.cuh -- penalties for repeated tokens, biases and a grammar mask on
// logits, with the greedy choice (logits_argmax in include/qmv.h).
//
// A CTA takes a slice of a row's vocabulary and sets all its logits on the way
// into shared memory (cp.async, 16 bytes each).  Meanwhile it counts the row's
// history and notes the last bias entry per token of the slice in shared memory
// (integer atomics: their order does not matter).  Then it runs over the logits
// once, with the mask alone.  The tokens that occur in the history or the
// biases are few and are done over afterwards from a list (the thread that finds
// a token's word empty adds it), so that the division of one token does not hold
// up those beside it.  A token's count and entry share 32 bits where 16 hold
// either, else 64 (WIDE).  Every CTA reads the row's whole history, so slices are
// long where there are many rows, and short where a few rows have to reach all SMs.
// The best allowed (value, token) goes into the row's 64-bit key as in
// qmv_argmax; the row's last CTA writes idx_out and zeroes the workspace.
// Bound by the logits' way in and out: 128 rows of 151937, 2000 of history,
// 46 us against 24 us of bytes, 32 us of them without history, biases and mask.
// (Slices of 4096 tokens on 256 threads: 45 us, but 8 rows of 128000 with 4096 of
// history 9.6 instead of 8.8 us; of 16384: 70 us, too few CTAs to overlap their
// phases.  With the logits loaded into registers chunk by chunk: 54 to 65 us.)
#pragma once

#include "qmv_attn.cuh"

namespace qmv {

constexpr int LG_THREADS = 512, LG_IDS = 4;     // threads; ids of the history that one has in flight
constexpr int LG_MIN_SLICE = 1024, LG_MAX_SLICE = 8192;         // half of it WIDE

// Tokens of a slice: three on a SM while a few rows have to reach all of them.
static inline int logits_slice(int n_rows, int vocab, int sms, bool wide)
{
    const int64_t each = ((int64_t)n_rows * vocab + 3 * sms - 1) / (3 * sms);
    int s = LG_MIN_SLICE;
    while (s < each && s < (wide ? LG_MAX_SLICE / 2 : LG_MAX_SLICE)) s *= 2;
    return s;
}
// Shared memory of a slice: logits | words | bits of the tokens with either | mask | list of the tokens (a quarter)
static inline size_t logits_smem(int slice, bool wide) { return (size_t)slice * (wide ? 12 : 8) + slice / 4 + slice / 4 * 2; }

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

template <bool WIDE>
static __global__ void __launch_bounds__(LG_THREADS) logits_argmax_kernel(const __grid_constant__ LogitsParams p)
{
    extern __shared__ __align__(16) float s_z[];                          // from token `head` on
    uint32_t *s_tok = reinterpret_cast<uint32_t *>(s_z + p.slice);        // per token: count in the history, last bias entry + 1 (the upper half of the word)
    uint32_t *s_bits = s_tok + p.slice * (WIDE ? 2 : 1), *s_mask = s_bits + p.slice / 32;
    uint16_t *s_list = reinterpret_cast<uint16_t *>(s_mask + p.slice / 32);
    __shared__ int s_n;                                                   // tokens with either
    __shared__ uint2 s_best[LG_THREADS / 32];
    const int row = blockIdx.y, v0 = blockIdx.x * p.slice, nv = min(p.slice, p.vocab - v0);
    const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
    const int n_hist = p.hist ? (int)min((int64_t)max(0, __ldg(p.hist_len + row)), p.hist_stride) : 0;
    const int n_bias = p.bias_ids ? (int)min((int64_t)max(0, __ldg(p.bias_len + row)), p.bias_stride) : 0;
    const bool pushed = n_hist > 0 || n_bias > 0;
    const float *logits = p.logits + (int64_t)row * p.logits_stride + v0;
    const uint32_t *mask = p.mask ? p.mask + (int64_t)row * p.mask_stride + (v0 >> 5) : nullptr;
    float *out = p.out ? p.out + (int64_t)row * p.out_stride + v0 : nullptr;

    // The logits from the first 16-byte boundary on (token `head`) go in groups
    // of 4.  Up to 6 tokens lie outside the groups.
    const int head = min(nv, (int)((0u - (uint32_t)(reinterpret_cast<uintptr_t>(logits) >> 2)) & 3u)), n_groups = (nv - head) / 4;
    for (int g = tid; g < n_groups; g += LG_THREADS) cp_async16(smem_addr(s_z + 4 * g), logits + head + 4 * g, 16);
    if (mask)
        for (int i = tid; i < (nv + 31) / 32; i += LG_THREADS) cp_async4(smem_addr(s_mask + i), mask + i, 4);
    cp_commit();
    const bool has_odd = tid < nv - 4 * n_groups;
    const int odd = tid < head ? tid : 4 * n_groups + tid;
    float odd_z = 0.f;
    if (has_odd) odd_z = logits[odd];

    const int32_t *h_ids = p.hist + (int64_t)row * p.hist_stride, *b_ids = p.bias_ids + (int64_t)row * p.bias_stride;
    float rep = 1.f, freq = 0.f, pres = 0.f;
    if (pushed) {
        // the first ids are on their way while the words are cleared
        int id[LG_IDS];
        auto fetch = [&](int64_t i0) {
#pragma unroll
            for (int u = 0; u < LG_IDS; ++u) id[u] = i0 + u * LG_THREADS + tid < n_hist ? __ldg(h_ids + i0 + u * LG_THREADS + tid) : -1;
        };
        fetch(0);
        const int b_first = tid < n_bias ? __ldg(b_ids + tid) : -1;
        for (int i = tid; i < p.slice / (WIDE ? 2 : 4) + p.slice / 128; i += LG_THREADS) reinterpret_cast<int4 *>(s_tok)[i] = make_int4(0, 0, 0, 0);
        if (tid == 0) s_n = 0;
        __syncthreads();
        auto in_slice = [&](int x) { return x >= 0 && (unsigned)x - (unsigned)v0 < (unsigned)nv; };
        auto add = [&](int o) {
            atomicOr(s_bits + (o >> 5), 1u << (o & 31));
            const int i = atomicAdd(&s_n, 1);
            if (i < p.slice / 4) s_list[i] = (uint16_t)o;
        };
        if (p.bias_ids) {                                                 // before the counts, which are added to the words
            for (int64_t i = tid; i < n_bias; i += LG_THREADS) {
                const int x = i == tid ? b_first : __ldg(b_ids + i), o = (int)((unsigned)x - (unsigned)v0);
                if (in_slice(x) && (WIDE ? atomicMax(s_tok + 2 * o + 1, (uint32_t)i + 1u) : atomicMax(s_tok + o, ((uint32_t)i + 1u) << 16)) == 0u) add(o);
            }
            __syncthreads();
        }
        if (p.hist) {
            rep = __ldg(p.params + 3 * (int64_t)row);
            freq = __ldg(p.params + 3 * (int64_t)row + 1);
            pres = __ldg(p.params + 3 * (int64_t)row + 2);
            for (int64_t i0 = 0; i0 < n_hist; i0 += LG_IDS * LG_THREADS) {
                if (i0) fetch(i0);
#pragma unroll
                for (int u = 0; u < LG_IDS; ++u) {
                    const int o = (int)((unsigned)id[u] - (unsigned)v0);
                    if (in_slice(id[u]) && atomicAdd(s_tok + (WIDE ? 2 * o : o), 1u) == 0u && (!WIDE || s_tok[2 * o + 1] == 0u)) add(o);
                }
            }
        }
        __syncthreads();
    }

    float bv = -INFINITY;
    int bi = -1;
    cp_wait<0>();
    __syncthreads();
    const bool wide_out = (reinterpret_cast<uintptr_t>(out + head) & 15u) == 0;
#pragma unroll 2
    for (int g = tid; g < n_groups; g += LG_THREADS) {
        const int o = head + 4 * g;
        const float4 z = *reinterpret_cast<const float4 *>(s_z + 4 * g);
        float y[4] = {z.x, z.y, z.z, z.w};
        if (mask) {
            const uint32_t m = __funnelshift_r(s_mask[o >> 5], s_mask[(o + 3) >> 5], o & 31);
#pragma unroll
            for (int i = 0; i < 4; ++i) y[i] = (m >> i) & 1u ? y[i] : -INFINITY;
        }
        if (out) {
            if (wide_out) {
                __stcs(reinterpret_cast<float4 *>(out + o), make_float4(y[0], y[1], y[2], y[3]));
            } else {
#pragma unroll
                for (int i = 0; i < 4; ++i) __stcs(out + o + i, y[i]);
            }
        }
        // the best of the tokens without a list entry: looked at closely only where one may be it
        if (fmaxf(fmaxf(y[0], y[1]), fmaxf(y[2], y[3])) > bv) {                           // NaN is passed over
            const uint32_t later = pushed ? __funnelshift_r(s_bits[o >> 5], s_bits[(o + 3) >> 5], o & 31) : 0u;
#pragma unroll
            for (int i = 0; i < 4; ++i)
                if (y[i] > bv && !((later >> i) & 1u)) {                                  // the first of equals
                    bv = y[i];
                    bi = v0 + o + i;
                }
        }
    }
    if (has_odd) {
        const float y = !mask || (s_mask[odd >> 5] >> (odd & 31) & 1u) ? odd_z : -INFINITY;
        if (out) out[odd] = y;
        if (y > -INFINITY && !(pushed && (s_bits[odd >> 5] >> (odd & 31) & 1u))) argmax_merge(bv, bi, y, v0 + odd);
    }
    if (pushed) {
        __syncthreads();                                                  // what comes now is stored over what the run stored
        const float *bias = p.bias_vals + (int64_t)row * p.bias_stride;
        auto push = [&](int o) {
            const uint32_t n = WIDE ? s_tok[2 * o] : s_tok[o] & 0xFFFFu, e = WIDE ? s_tok[2 * o + 1] : s_tok[o] >> 16;
            float y = o >= head && o < head + 4 * n_groups ? s_z[o - head] : logits[o];
            if (n) {
                y = y > 0.f ? __fdiv_rn(y, rep) : __fmul_rn(y, rep);
                y = __fsub_rn(y, __fadd_rn(__fmul_rn(freq, (float)n), pres));
            }
            if (e) y = __fadd_rn(y, __ldg(bias + e - 1));
            if (mask && !(s_mask[o >> 5] >> (o & 31) & 1u)) y = -INFINITY;
            if (out) out[o] = y;
            if (y > -INFINITY) argmax_merge(bv, bi, y, v0 + o);
        };
        if (s_n <= p.slice / 4) {
            for (int i = tid; i < s_n; i += LG_THREADS) push(s_list[i]);
        } else {
            for (int o = tid; o < nv; o += LG_THREADS)
                if (s_bits[o >> 5] >> (o & 31) & 1u) push(o);
        }
    }
    // the CTA's best: the largest value's bits in order, of equals the lowest token
    auto best = [&](uint32_t &hi, uint32_t &lo) {
        const uint32_t m = __reduce_max_sync(0xFFFFFFFFu, hi);
        lo = __reduce_max_sync(0xFFFFFFFFu, hi == m ? lo : 0u);
        hi = m;
    };
    const unsigned long long key = bi >= 0 ? argmax_key(bv, bi) : 0ull;
    uint32_t hi = (uint32_t)(key >> 32), lo = (uint32_t)key;
    best(hi, lo);
    if (lane == 0) s_best[warp] = make_uint2(hi, lo);
    __syncthreads();
    if (warp) return;
    const uint2 w = lane < LG_THREADS / 32 ? s_best[lane] : make_uint2(0u, 0u);
    hi = w.x;
    lo = w.y;
    best(hi, lo);
    if (lane == 0) {
        if (lo) atomicMax(p.keys + row, (unsigned long long)hi << 32 | lo);
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
