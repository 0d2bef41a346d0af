// qmv_logits.cuh -- penalties for repeated tokens, biases and a grammar mask on
// logits, with the greedy choice (logits_argmax in include/qmv.h).
//
// A CTA takes a slice of one row's vocabulary.  It counts the row's history
// and notes the last bias entry per token of its slice in shared memory
// (integer atomics: their order does not matter), then runs over its logits
// once.  The best allowed (value, token) goes into the row's 64-bit key as in
// qmv_argmax; the row's last CTA writes idx_out and zeroes the workspace.
#pragma once

#include "qmv_device.cuh"

namespace qmv {

constexpr int LG_THREADS = 256, LG_SLICE = 2048;

struct LogitsParams {
    const float *logits;
    float *out;
    int64_t logits_stride, out_stride, hist_stride, bias_stride, mask_stride;
    int32_t vocab;
    const int32_t *hist, *hist_len, *bias_ids, *bias_len;
    const float *params, *bias_vals;
    const uint32_t *mask;
    int32_t *idx;
    unsigned long long *keys;
    unsigned *done;
};

static __global__ void __launch_bounds__(LG_THREADS) logits_argmax_kernel(const __grid_constant__ LogitsParams p)
{
    __shared__ int s_count[LG_SLICE], s_bias[LG_SLICE];
    __shared__ float s_v[LG_THREADS / 32];
    __shared__ int s_i[LG_THREADS / 32];
    const int row = blockIdx.y, v0 = blockIdx.x * LG_SLICE, nv = min(LG_SLICE, p.vocab - v0);
    const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
    for (int i = tid; i < LG_SLICE; i += LG_THREADS) {
        s_count[i] = 0;
        s_bias[i] = -1;
    }
    __syncthreads();
    float rep = 1.f, freq = 0.f, pres = 0.f;
    if (p.hist) {
        rep = __ldg(p.params + 3 * (int64_t)row);
        freq = __ldg(p.params + 3 * (int64_t)row + 1);
        pres = __ldg(p.params + 3 * (int64_t)row + 2);
        const int64_t n = min((int64_t)max(0, __ldg(p.hist_len + row)), p.hist_stride);
        const int32_t *h = p.hist + (int64_t)row * p.hist_stride;
        for (int64_t i = tid; i < n; i += LG_THREADS) {
            const unsigned o = (unsigned)__ldg(h + i) - (unsigned)v0;
            if (o < (unsigned)nv) atomicAdd(s_count + o, 1);
        }
    }
    const float *bias = p.bias_vals + (int64_t)row * p.bias_stride;
    if (p.bias_ids) {
        const int64_t n = min((int64_t)max(0, __ldg(p.bias_len + row)), p.bias_stride);
        const int32_t *id = p.bias_ids + (int64_t)row * p.bias_stride;
        for (int64_t i = tid; i < n; i += LG_THREADS) {
            const unsigned o = (unsigned)__ldg(id + i) - (unsigned)v0;
            if (o < (unsigned)nv) atomicMax(s_bias + o, (int)i);
        }
    }
    __syncthreads();
    const float *z0 = p.logits + (int64_t)row * p.logits_stride + v0;
    float *out = p.out ? p.out + (int64_t)row * p.out_stride + v0 : nullptr;
    float bv = 0.f;
    int bi = -1;
    for (int i = tid; i < nv; i += LG_THREADS) {
        float z = z0[i];
        const int c = s_count[i], b = s_bias[i];
        if (c > 0) {
            z = z > 0.f ? __fdiv_rn(z, rep) : __fmul_rn(z, rep);
            z = __fsub_rn(z, __fadd_rn(__fmul_rn(freq, (float)c), pres));
        }
        if (b >= 0) z = __fadd_rn(z, __ldg(bias + b));
        if (p.mask && !((__ldg(p.mask + (int64_t)row * p.mask_stride + ((v0 + i) >> 5)) >> ((v0 + i) & 31)) & 1u)) z = -INFINITY;
        if (out) out[i] = z;
        if (z > -INFINITY) argmax_merge(bv, bi, z, v0 + i);               // neither NaN nor -infinity
    }
    for (int o = 16; o; o >>= 1) argmax_merge(bv, bi, __shfl_xor_sync(0xFFFFFFFFu, bv, o), __shfl_xor_sync(0xFFFFFFFFu, bi, o));
    if (lane == 0) {
        s_v[warp] = bv;
        s_i[warp] = bi;
    }
    __syncthreads();
    if (tid == 0) {
        for (int w = 1; w < LG_THREADS / 32; ++w) argmax_merge(bv, bi, s_v[w], s_i[w]);
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
