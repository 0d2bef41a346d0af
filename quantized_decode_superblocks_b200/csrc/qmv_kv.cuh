// qmv_kv.cuh -- the new tokens into the paged cache (kv_append) and a smaller
// cache for each sequence (kv_evict); both declared in include/qmv.h.
#pragma once

#include <cooperative_groups.h>
#include <cuda_bf16.h>

#include "qmv_attn.cuh"

namespace qmv {

template <class Params>
__device__ __forceinline__ int page_of(int slot, const Params &p) { return p.page_shift >= 0 ? slot >> p.page_shift : slot / p.page_size; }

// -------------------------------------------------------------- append --
// One CTA per (token, share of the heads): the token's cosines and sines once
// in 64 bits, then one warp per head, whose first head is loaded meanwhile.  A
// few KB per token: one token of 32/8 heads of 64 takes 2.4 us, launch and memory
// latency; 64 x 4 tokens of 32/8 heads of 128, bf16, 5.2 us (1.8 us of bytes), the
// instructions of a head.
constexpr int APP_THREADS = 128, APP_CTAS = 4;     // CTAs on a SM

// Cosine and sine of pos * f, each as two floats (48 bits).  The angle is brought within one turn by k turns
// taken away in two parts (Cody and Waite), exact to 2^-53 of a turn for any
// 31-bit position, so that the library's function never takes its long path.
__device__ __forceinline__ float4 rope_turn(double pos, float f)
{
    const double a = pos * (double)f, k = rint(a * 0.15915494309189535);
    double sn, c;
    sincos(fma(-k, 2.4492935982947064e-16, fma(-k, 6.283185307179586, a)), &sn, &c);
    const float ch = (float)c, sh = (float)sn;
    return make_float4(ch, (float)(c - ch), sh, (float)(sn - sh));
}

// a c + b s, rounded once: the products' and the sum's roundings are caught in f32.  Infinities, also those of
// a sum beyond f32's range, are final: what they leave is a NaN (infinity minus infinity), which the minimum
// passes over for a number that changes neither them nor a NaN.
__device__ __forceinline__ float rope_sum(float a, float b, float4 t)
{
    const float p = a * t.x, q = b * t.z, r = p + q, v = r - p;
    const float left = fmaf(a, t.y, fmaf(a, t.x, -p)) + fmaf(b, t.w, fmaf(b, t.z, -q));
    return r + fminf(((p - (r - v)) + (q - v)) + left, 3.402823466e38f);
}

struct AppendParams {
    uint8_t *k, *v, *ks, *vs;
    int64_t page_stride, head_stride, slot_stride, n_pages;
    const float *q_in, *k_in, *v_in;
    float *q_out;
    int64_t q_stride, k_stride, v_stride, q_out_stride;
    int32_t type, n_head, n_kv, dim, n_tok, rope_dim, rope_pairs;
    int32_t page_size, page_shift, max_len;          // page_shift < 0: not a power of two
    const int32_t *table, *kv_len, *pos;
    int64_t table_stride;
    const float *inv_freq;
    int *err;
};

// NB: values of a head per lane, 32 apart.  A lane's partners and turns are the
// same for every head and stay in registers.
template <int NB>
static __global__ void __launch_bounds__(APP_THREADS, APP_CTAS) kv_append_kernel(const __grid_constant__ AppendParams p)
{
    __shared__ float4 s_turn[16 * NB];             // cosine and sine, each as a float and what it leaves
    __shared__ long long s_at;                     // the slot's first element, -1: nothing to store
    const int t = blockIdx.x, s = blockIdx.y, tok = s * p.n_tok + t;
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    const int raw = __ldg(p.kv_len + s);
    const long long slot = (long long)raw - p.n_tok + t;     // of the length as given: a clamped one would move the tokens onto slots in use
    if (threadIdx.x == 0) {
        long long at = -1;
        if (slot >= 0 && slot < p.max_len) {
            const int j = (int)slot, i = page_of(j, p), page = __ldg(p.table + (int64_t)s * p.table_stride + i);
            if (page >= 0 && page < p.n_pages) at = page * p.page_stride + (j - i * p.page_size) * p.slot_stride;
            else atomicOr(p.err, 8 /* QMV_DEVERR_PAGE_ID */);
        }
        if (raw < 0 || raw > p.max_len) atomicOr(p.err, 16 /* QMV_DEVERR_SEQ_LEN */);
        s_at = at;
    }
    const int nq = p.q_out ? p.n_head : 0, heads = nq + 2 * p.n_kv;
    const int half = p.rope_dim / 2, step = gridDim.z * (APP_THREADS / 32);
    auto second = [&](int d) { return p.rope_pairs ? d & 1 : d >= half; };          // of its pair
    int head = blockIdx.z * (APP_THREADS / 32) + warp, partner[NB];
#pragma unroll
    for (int b = 0; b < NB; ++b) {
        const int d = b * 32 + lane;
        partner[b] = d >= p.rope_dim ? -1 : p.rope_pairs ? d ^ 1 : d < half ? d + half : d - half;
    }
    float y[NB], z[NB];                            // this lane's values and their partners
    auto load = [&]() {
        if (head >= heads) return;
        const float *x = head < nq ? p.q_in + tok * p.q_stride + (int64_t)head * p.dim
                         : head < nq + p.n_kv ? p.k_in + tok * p.k_stride + (int64_t)(head - nq) * p.dim
                                              : p.v_in + tok * p.v_stride + (int64_t)(head - nq - p.n_kv) * p.dim;
#pragma unroll
        for (int b = 0; b < NB; ++b) y[b] = b * 32 + lane < p.dim ? x[b * 32 + lane] : 0.f;
        if (head < nq + p.n_kv) {
#pragma unroll
            for (int b = 0; b < NB; ++b) z[b] = partner[b] >= 0 ? x[partner[b]] : 0.f;
        }
    };
    load();
    const double pos = p.pos ? (double)__ldg(p.pos + tok) : (double)slot;
    for (int i = threadIdx.x; i < half; i += APP_THREADS) s_turn[i] = rope_turn(pos, __ldg(p.inv_freq + i));
    __syncthreads();
    const long long at = s_at;
    float4 turn[NB];
#pragma unroll
    for (int b = 0; b < NB; ++b) {
        const int d = b * 32 + lane;
        if (partner[b] < 0) continue;
        turn[b] = s_turn[p.rope_pairs ? d >> 1 : d < half ? d : d - half];
        if (!second(d)) {                          // a cos - b sin
            turn[b].z = -turn[b].z;
            turn[b].w = -turn[b].w;
        }
    }
    for (; head < heads; head += step, load()) {
        __syncwarp();                              // q may be rotated in place: all is read before anything is written
        if (head < nq + p.n_kv) {
#pragma unroll
            for (int b = 0; b < NB; ++b)
                if (partner[b] >= 0) y[b] = rope_sum(y[b], z[b], turn[b]);
        }
        if (head < nq) {
            float *o = p.q_out + tok * p.q_out_stride + (int64_t)head * p.dim;
#pragma unroll
            for (int b = 0; b < NB; ++b)
                if (b * 32 + lane < p.dim) o[b * 32 + lane] = y[b];
            continue;
        }
        if (at < 0) continue;
        const bool is_k = head < nq + p.n_kv;
        const int h = is_k ? head - nq : head - nq - p.n_kv;
        const long long e0 = at + h * p.head_stride + lane;
        uint8_t *pool = is_k ? p.k : p.v;
#pragma unroll
        for (int b = 0; b < NB; ++b) {
            const bool in = b * 32 + lane < p.dim;
            const long long e = e0 + b * 32;
            if (p.type == KV_F16) {
                if (in) reinterpret_cast<__half *>(pool)[e] = __float2half_rn(y[b]);
            } else if (p.type == KV_BF16) {
                if (in) reinterpret_cast<__nv_bfloat16 *>(pool)[e] = __float2bfloat16_rn(y[b]);
            } else if (b * 32 < p.dim) {
                const float w = y[b];
                float mx = fabsf(w);
                for (int o = 16; o; o >>= 1) mx = fmaxf(mx, __shfl_xor_sync(0xFFFFFFFFu, mx, o));
                // a NaN, which the maximum passes over, makes the scale one: the block reads as NaN
                const bool bad = __any_sync(0xFFFFFFFFu, w != w);
                const __half dh = __float2half_rn(bad ? __int_as_float(0x7FFFFFFF) : fminf(__fdiv_rn(mx, 127.f), 65504.f));
                const float df = __half2float(dh);
                const float qv = df > 0.f ? fminf(fmaxf(rintf(__fdiv_rn(w, df)), -127.f), 127.f) : 0.f;
                reinterpret_cast<int8_t *>(pool)[e] = (int8_t)(int)qv;
                if (lane == 0) reinterpret_cast<__half *>(is_k ? p.ks : p.vs)[e / 32] = dh;
            }
        }
    }
}

// -------------------------------------------------------------- evict --
// Two kernels: the choice, bound by latency, and the copy, bound by bandwidth;
// apart, so that the copy has every SM to itself and is spread evenly.
//
// Choice: a CTA per (sequence, kv head).  The slots between the kept ends are
// ranked by a radix select over order-preserving 32-bit keys (digits of 11, 11
// and 10 bits, highest first), which gives the key of the last slot to keep and
// how many slots with exactly that key are kept (the lowest ones).  A round that
// leaves no slot undecided is the last one: scores that all differ need two.
// Then each warp writes the kept slots of its part in order, at the place that
// the counts of the warps before it give: one cache of 4352 slots 5 us, 16 of
// up to 16384 slots 11 us, bound by the instructions of one SM per head.
// Long caches of few heads: a cluster of EV_CL CTAs per head, each for a part of
// the slots.  A CTA adds up the cluster's counts of its share of the digits over
// distributed shared memory, and only the shares' sums and the chosen digit go
// to all (every CTA reading all counts took 5 us a round).  One cache, 8 heads,
// choice and copy: 10000 slots 19 us instead of 15 us, 20000 slots 20
// instead of 21 us, 131072 slots 35 instead of 164 us.
//
// Copy: a warp per EV_SLOTS kept slots of a (sequence, head), the heads of the
// same slots next to each other; 16 x 8 heads x 4096 slots of 512 bytes, in and
// out, 87 us, 6.2 TB/s.  (With 32 slots a warp, k and v by the same lane: 95 us.  By
// 16-byte loads and stores through registers 104 to 130 us, depending on how
// many a lane has in flight.)
constexpr int EV_THREADS = 1024, EV_BINS = 2048;
constexpr int EV_KEYS = 40960;                // keys that shared memory holds; those of later slots are made anew in every round
constexpr int EV_CL = 8;                      // CTAs of a head, long caches
constexpr int EV_COPY_THREADS = 128, EV_SLOTS = 16;     // slots: of a warp of the copy

// Whether several CTAs choose for each head.
static inline bool evict_cluster(int max_len, int heads, int sms) { return max_len > 16384 && heads * EV_CL <= sms; }

struct EvictParams {
    uint8_t *k, *v, *ks, *vs;
    int64_t page_stride, head_stride, slot_stride, n_pages;
    const float *score;
    float *score_out;
    int64_t score_stride, score_out_stride, table_stride, dst_table_stride;
    const int32_t *table, *kv_len, *dst_table;
    int32_t *kept, *len_out;
    int32_t n_kv, page_size, page_shift, max_len, keep_first, keep_last, budget;
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

// CL: CTAs of a (sequence, head), a cluster where more than one; CTA `rank` looks after the rank-th part of the slots.
template <int CL>
__device__ __forceinline__ void evict_choose(const EvictParams &p)
{
    namespace cg = cooperative_groups;
    constexpr int NW = EV_THREADS / 32, PER = EV_BINS / EV_THREADS, FLY = 8;      // FLY: loads of a thread in flight
    static_assert(NW == 32 && PER == 2, "one warp reads the warps' counts; a thread has two digits");
    __shared__ __align__(16) int s_hist[EV_BINS];
    __shared__ int s_sel[3];
    __shared__ int s_up[NW], s_eq[NW];
    __shared__ int s_all[CL], s_cnt[2];                                           // slots of every CTA's digits; this one's kept, and at the last key
    const int rank = blockIdx.x % CL, h = blockIdx.x / CL, s = blockIdx.y;
    asm volatile("griddepcontrol.launch_dependents;" ::: "memory");              // the copy, which waits for this kernel's end
    const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
    const int raw = __ldg(p.kv_len + s), n = min(max(raw, 0), p.max_len), m = min(n, p.budget);
    if (raw != n && tid == 0) atomicOr(p.err, 16 /* QMV_DEVERR_SEQ_LEN */);
    const int chunk = (int)(((int64_t)n + CL * EV_THREADS - 1) / (CL * EV_THREADS)) * 32;            // slots of a warp
    const int a = (int)min((int64_t)n, (int64_t)rank * chunk * NW), b = (int)min((int64_t)n, (int64_t)a + (int64_t)chunk * NW);
    const int64_t sh = (int64_t)s * p.n_kv + h;
    const float *score = p.score + sh * p.score_stride;
    float *score_out = p.score_out + sh * p.score_out_stride;
    int32_t *kept = p.kept + sh * p.budget;
    const int mid0 = min(p.keep_first, n), mid1 = max(mid0, n - p.keep_last);     // ranked slots
    const bool all = n <= p.budget;

    extern __shared__ __align__(16) uint32_t s_key[];                             // [min(slots, EV_KEYS)] of this CTA's, the largest for the kept ends
    auto key_at = [&](int j, float x) { return j < mid0 || j >= mid1 ? 0xFFFFFFFFu : evict_key(x); };
    auto key_of = [&](int j) { return j - a < EV_KEYS ? s_key[j - a] : key_at(j, __ldg(score + j)); };
    uint32_t prefix = 0xFFFFFFFFu;            // no ranked key is that large
    int shift = 0, want = p.budget - p.keep_first - p.keep_last;                  // still to take within the prefix
    bool ties = false;                                                            // only some of the slots with the last key are kept
    if (!all) {
        reinterpret_cast<int2 *>(s_hist)[tid] = make_int2(0, 0);
        __syncthreads();
        for (int64_t j0 = a + tid; j0 < b; j0 += FLY * EV_THREADS) {              // keys, and the counts of their first digit
            float x[FLY];
#pragma unroll
            for (int u = 0; u < FLY; ++u) x[u] = j0 + u * EV_THREADS < b ? __ldg(score + j0 + u * EV_THREADS) : 0.f;
#pragma unroll
            for (int u = 0; u < FLY; ++u) {
                const int64_t j = j0 + u * EV_THREADS;
                if (j < b) {
                    const uint32_t key = key_at((int)j, x[u]);
                    if (j - a < EV_KEYS) s_key[j - a] = key;
                    if (key != 0xFFFFFFFFu) atomicAdd(s_hist + (key >> 21), 1);
                }
            }
        }
        auto sum_before = [&](int own) {                                          // over the threads before this one
            int up = own;
            for (int o = 1; o < 32; o <<= 1) {
                const int y = __shfl_up_sync(0xFFFFFFFFu, up, o);
                if (lane >= o) up += y;
            }
            if (lane == 31) s_up[warp] = up;
            __syncthreads();
            return __reduce_add_sync(0xFFFFFFFFu, lane < warp ? s_up[lane] : 0) + up - own;
        };
        for (int pass = 0; pass < 3 && want > 0; ++pass) {
            const int above = shift;                                              // the digits that are decided lie above this bit
            shift = pass == 0 ? 21 : pass == 1 ? 10 : 0;
            if (pass) {
                const uint32_t digits = pass == 1 ? 2047u : 1023u;
                reinterpret_cast<int2 *>(s_hist)[tid] = make_int2(0, 0);
                __syncthreads();
#pragma unroll 4
                for (int64_t j = max(mid0, a) + tid; j < min(mid1, b); j += EV_THREADS) {
                    const uint32_t key = key_of((int)j);
                    if ((key >> above) == prefix) atomicAdd(s_hist + ((key >> shift) & digits), 1);
                }
            }
            if constexpr (CL == 1) {
                __syncthreads();
                // this thread's two digits, from the top down
                const int lo = EV_BINS - PER * (tid + 1);
                const int2 c = *reinterpret_cast<const int2 *>(s_hist + lo);
                const int before = sum_before(c.x + c.y);                         // slots of larger digits
                if (before < want && before + c.x + c.y >= want) {
                    const bool first = before + c.y >= want;
                    s_sel[0] = lo + (first ? 1 : 0);
                    s_sel[1] = want - before - (first ? 0 : c.y);
                    s_sel[2] = first ? c.y : c.x;
                }
                __syncthreads();
            } else {
                // each CTA adds up the cluster's counts of an equal share of the digits and tells
                // the others their sum; the one whose share the last key's digit lies in tells the digit
                constexpr int SHARE = EV_BINS / CL;
                static_assert(SHARE <= EV_THREADS, "a thread has one digit at most");
                cg::cluster_group cl = cg::this_cluster();
                cl.sync();
                const int digit = EV_BINS - 1 - rank * SHARE - tid;               // from the top down
                int c = 0;
                if (tid < SHARE) {
#pragma unroll
                    for (int r = 0; r < CL; ++r) c += cl.map_shared_rank(s_hist, r)[digit];
                }
                int before = sum_before(c);
                if (tid == SHARE - 1) {
#pragma unroll
                    for (int r = 0; r < CL; ++r) cl.map_shared_rank(s_all, r)[rank] = before + c;
                }
                cl.sync();
                for (int r = 0; r < rank; ++r) before += s_all[r];
                if (tid < SHARE && before < want && before + c >= want) {
#pragma unroll
                    for (int r = 0; r < CL; ++r) {
                        int *sel = cl.map_shared_rank(s_sel, r);
                        sel[0] = digit;
                        sel[1] = want - before;
                        sel[2] = c;
                    }
                }
                cl.sync();
            }
            prefix = pass == 0 ? (uint32_t)s_sel[0] : (prefix << (above - shift)) | (uint32_t)s_sel[0];
            want = s_sel[1];
            ties = s_sel[2] != want;
            if (!ties) break;                                                     // all of that digit are kept
        }
    }
    __syncthreads();
    // ---- how many slots each warp keeps, and its place.  Without ties what is
    // kept are the keys from the last one up.
    const uint32_t least = all ? 0u : prefix << shift;
    const int w0 = (int)min((int64_t)b, a + (int64_t)warp * chunk), w1 = (int)min((int64_t)b, (int64_t)w0 + chunk);
    int n_up = 0, n_eq = 0;
    if (all) {
        n_up = lane == 0 ? w1 - w0 : 0;
    } else if (!ties) {
#pragma unroll 4
        for (int j = w0 + lane; j < w1; j += 32) n_up += key_of(j) >= least;
    } else {
        for (int j = w0 + lane; j < w1; j += 32) {
            const uint32_t key = key_of(j);
            n_up += key > least;                                                  // ties are decided by all 32 bits
            n_eq += key == least;
        }
    }
    n_up = __reduce_add_sync(0xFFFFFFFFu, n_up);
    n_eq = __reduce_add_sync(0xFFFFFFFFu, n_eq);
    if (lane == 0) {
        s_up[warp] = n_up;
        s_eq[warp] = n_eq;
    }
    __syncthreads();
    int bu = __reduce_add_sync(0xFFFFFFFFu, lane < warp ? s_up[lane] : 0);        // kept, and at the last key, before this warp
    int be = __reduce_add_sync(0xFFFFFFFFu, lane < warp ? s_eq[lane] : 0);
    if constexpr (CL > 1) {
        cg::cluster_group cl = cg::this_cluster();
        if (tid == EV_THREADS - 1) {
            s_cnt[0] = bu + n_up;
            s_cnt[1] = be + n_eq;
        }
        cl.sync();
        for (int r = 0; r < rank; ++r) {
            const int *c = cl.map_shared_rank(s_cnt, r);
            bu += c[0];
            be += c[1];
        }
        cl.sync();                                                                // no CTA leaves while its counts are read
    }
    // ---- the kept slots in order
    const uint32_t below = (1u << lane) - 1u;
    if (!ties) {
#pragma unroll 4
        for (int j = w0 + lane; j - lane < w1; j += 32) {
            const bool up = j < w1 && (all || key_of(j) >= least);
            const uint32_t mu = __ballot_sync(0xFFFFFFFFu, up);
            if (up) {
                const int i = bu + __popc(mu & below);
                kept[i] = j;
                score_out[i] = __ldg(score + j);
            }
            bu += __popc(mu);
        }
    } else {
        for (int j = w0 + lane; j - lane < w1; j += 32) {
            const uint32_t key = j < w1 ? key_of(j) : 0u;
            const bool up = j < w1 && key > least, eq = j < w1 && key == least;
            const uint32_t mu = __ballot_sync(0xFFFFFFFFu, up), me = __ballot_sync(0xFFFFFFFFu, eq);
            const int e = be + __popc(me & below);
            if (up || (eq && e < want)) {
                const int i = bu + __popc(mu & below) + min(e, want);
                kept[i] = j;
                score_out[i] = __ldg(score + j);
            }
            bu += __popc(mu);
            be += __popc(me);
        }
    }
    if (h == 0 && rank == 0 && tid == 0) p.len_out[s] = m;
}

static __global__ void __launch_bounds__(EV_THREADS) kv_evict_kernel(const __grid_constant__ EvictParams p) { evict_choose<1>(p); }
static __global__ void __cluster_dims__(EV_CL, 1, 1) __launch_bounds__(EV_THREADS) kv_evict_cluster_kernel(const __grid_constant__ EvictParams p)
{
    evict_choose<EV_CL>(p);
}

// A lane per row of k or v, which goes through shared memory by bulk copies; its
// scales (too short for one) go through registers.
static __global__ void __launch_bounds__(EV_COPY_THREADS) kv_evict_copy_kernel(const __grid_constant__ EvictParams p)
{
    extern __shared__ __align__(128) uint8_t s_rows[];                            // [warps][k, v][slots]
    __shared__ __align__(8) uint64_t s_bar[EV_COPY_THREADS / 32];
    const int h = blockIdx.x % p.n_kv, s = blockIdx.y, lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
    const int m = min(min(max(__ldg(p.kv_len + s), 0), p.max_len), p.budget);
    const int i = (blockIdx.x / p.n_kv * (EV_COPY_THREADS / 32) + warp) * EV_SLOTS + lane % EV_SLOTS;
    static_assert(2 * EV_SLOTS == 32, "a lane per row of k or v");
    const bool in = i < m;
    const int di = page_of(i, p), pd = in ? __ldg(p.dst_table + (int64_t)s * p.dst_table_stride + di) : -1;
    const uint32_t bar = smem_addr(s_bar + warp);
    if (lane == 0) {
        mbar_init(bar, 1);
        fence_mbar_init();
    }
    asm volatile("griddepcontrol.wait;" ::: "memory");                            // kv_evict_kernel is done
    int64_t es = 0, ed = 0;
    bool ok = false;
    if (in) {
        const int j = __ldcg(p.kept + ((int64_t)s * p.n_kv + h) * p.budget + i);
        const int si = page_of(j, p), ps = __ldg(p.table + (int64_t)s * p.table_stride + si);
        ok = ps >= 0 && ps < p.n_pages && pd >= 0 && pd < p.n_pages;
        if (!ok) atomicOr(p.err, 8 /* QMV_DEVERR_PAGE_ID */);
        es = ps * p.page_stride + h * p.head_stride + (j - si * p.page_size) * p.slot_stride;
        ed = pd * p.page_stride + h * p.head_stride + (i - di * p.page_size) * p.slot_stride;
    }
    const uint32_t n_ok = (uint32_t)__popc(__ballot_sync(0xFFFFFFFFu, ok)), rb = (uint32_t)p.row_bytes;
    if (n_ok == 0) return;
    const uint32_t row = smem_addr(s_rows) + (uint32_t)(warp * 2 * EV_SLOTS + lane) * rb;
    uint8_t *pool = lane < EV_SLOTS ? p.k : p.v, *scales = lane < EV_SLOTS ? p.ks : p.vs;
    if (lane == 0) mbar_arrive_expect_tx(bar, n_ok * rb);
    __syncwarp();
    if (ok) {
        bulk_g2s(row, pool + es * p.eb, rb, bar);
        for (int c = 0; c < p.scale_words; ++c)
            reinterpret_cast<uint32_t *>(scales + ed / 16)[c] = __ldg(reinterpret_cast<const uint32_t *>(scales + es / 16) + c);
    }
    if (!mbar_wait_bounded(bar, 0)) {
        atomicOr(p.err, mbar_wait_bounded(bar, 0) ? 2 : 2 | 4 /* QMV_DEVERR_TIMEOUT, QMV_DEVERR_DRAIN */);
        return;
    }
    if (ok) {
        bulk_s2g(pool + ed * p.eb, row, rb);
        bulk_s2g_drain();
    }
}

}  // namespace qmv
