// qmv_attn.cuh -- attention of a sequence's newest tokens over a paged
// key-value cache (attn_decode in include/qmv.h).
//
// For every kv head the rows are the n_tok queries of its group's query heads.
// One pass over the cache keeps, per row, the running maximum m of
// s = scale * log2(e) * q.k, the sum l of 2^(s - m) and the unnormalised
// output o (the online softmax): a new maximum scales l and o by 2^(old - new).
// Two parts (m, l, o) of one row join as m = max, l and o scaled by 2^(m_i - m)
// and added; out = o / l.
//
// Work split.  The cache is cut into tiles of 16 slots of one kv head.  The
// tiles of all sequences, heads and row blocks are numbered through, and CTA c
// takes the c-th equal range of them, so that ragged batches and single long
// sequences load every SM alike; the lengths are only known on the device, so
// every CTA finds its own range from a prefix sum over them.  A (sequence, row
// block, head) that lies in several ranges leaves its parts in the workspace,
// and the last of its CTAs to arrive (a counter) joins them in CTA order.
//
// In a CTA, warp w streams every 8th tile through a ring of its own
// (cp.async, NST stages) and multiplies on the tensor cores (m16n8k16, f32
// accumulation).  The 16 rows of a product are 8 query rows twice: the upper
// half holds the leading part of the f32 operand, the lower half the rest,
//   f16 cache:   q * 2^e (per row, so that the largest value is below 2^13) and
//                2^15 * p as two f16 parts: 22 bits, absolute error 2^-23 of
//                the row's largest value;
//   bf16 and Q8_0 cache (int8 is exact in both): p (and q for bf16) as three
//                bf16 parts, 24 bits; the third part is a product of its own.
// so one thread holds both halves of its scores and of its outputs and adds
// them without a shuffle, and p of one product is the A operand of the next.
// With more than 8 rows, mt warps form a group that shares its mt tiles: each
// loads one and multiplies all of them with its own 8 rows.
//
// Slots that no query of the call sees are not loaded (their shared memory is
// zeroed by the copy).  A slot that only some of several queries see is kept out of
// the others' results by zeroing its V operand per query, not by a zero
// weight, since 0 * NaN is NaN.
#pragma once

#include <cuda_bf16.h>

#include "qmv_device.cuh"
#include "qmv_launch.cuh"

namespace qmv {

enum { KV_F16 = 0, KV_BF16 = 1, KV_Q8_0 = 2 };

constexpr int ATT_NW = 8;                    // warps of a CTA (at most; see AttnGeom)
constexpr int ATT_TILE = 16;                 // slots of a tile

// 8-row blocks that one CTA takes: up to 4, 2 where q's fragments lie in shared memory
__host__ __device__ constexpr int attn_max_mt(int dim) { return dim <= 128 ? 4 : 2; }
constexpr int ATT_MAX_SEQ = 1024;
constexpr int ATT_MAX_CTAS = 320;            // bound for the workspace's parts

struct AttnParams {
    const uint8_t *k, *v, *ks, *vs;
    int64_t page_stride, head_stride, slot_stride;       // values
    const float *q;
    float *out;
    float *score;                                        // NULL: not accumulated
    int64_t q_stride, out_stride, score_stride;
    const int32_t *table, *kv_len;
    int64_t table_stride, n_pages;
    int32_t n_seq, n_tok, n_kv, group, rows, dim;        // rows = n_tok * group
    int32_t page_size, page_shift, max_len;              // page_shift < 0: not a power of two
    int32_t mt, n_rb;                                    // 8-row blocks of a CTA, row blocks of a head
    int32_t window, n_sink, min_tiles;
    float scale_log2, l_shift;                           // l counts 2^l_shift times the weights
    unsigned *counters;                                  // [ATT_MAX_CTAS], zero between calls
    float *part_ml, *part_o;                             // [2 * CTAs][8 mt][2], [..][dim]
    float *raw, *stats;                                  // scores s and (m, l) of every row, for `score`
    int64_t raw_stride;
    int *err;
};

// Which slots of a sequence the call's queries see, as tiles.
struct AttnSeq {
    int len, first;        // length; slot of the first query (may be negative)
    int lo, sinks;         // slots >= lo, and slots < sinks, are seen by some query
    int sink_tiles, base;  // tiles 0 .. sink_tiles - 1 start at slot 0, the others at slot base
    int n_tiles;           // at least 1, so that every row gets written

    __device__ __forceinline__ void set(int n, const AttnParams &p)
    {
        len = n;
        first = n - p.n_tok;
        lo = sinks = sink_tiles = base = 0;
        if (p.window > 0) {
            lo = max(0, max(first, 0) - p.window + 1);
            sinks = min(p.n_sink, lo);
            sink_tiles = (sinks + ATT_TILE - 1) / ATT_TILE;
            base = lo / ATT_TILE * ATT_TILE;
            if (sinks > 0 && sink_tiles * ATT_TILE >= base) sink_tiles = base = 0;   // the parts meet
        }
        n_tiles = max(1, sink_tiles + (len - base + ATT_TILE - 1) / ATT_TILE);
    }
    __device__ __forceinline__ int slot0(int tile) const
    {
        return tile < sink_tiles ? tile * ATT_TILE : base + (tile - sink_tiles) * ATT_TILE;
    }
    __device__ __forceinline__ bool seen(int j) const { return j < len && (j >= lo || j < sinks); }
};

__device__ __forceinline__ int attn_len(const AttnParams &p, int s)
{
    const int n = __ldg(p.kv_len + s);
    return min(max(n, 0), p.max_len);
}

__device__ __forceinline__ bool attn_sees(const AttnParams &p, int at, int j)
{
    return j <= at && (p.window == 0 || j > at - p.window || j < p.n_sink);
}

__device__ __forceinline__ void cp_async16(uint32_t dst, const void *src, uint32_t bytes)
{
    asm volatile("cp.async.cg.shared.global [%0], [%1], 16, %2;" :: "r"(dst), "l"(src), "r"(bytes) : "memory");
}
__device__ __forceinline__ void cp_async4(uint32_t dst, const void *src, uint32_t bytes)
{
    asm volatile("cp.async.ca.shared.global [%0], [%1], 4, %2;" :: "r"(dst), "l"(src), "r"(bytes) : "memory");
}
__device__ __forceinline__ void cp_commit() { asm volatile("cp.async.commit_group;" ::: "memory"); }
template <int N> __device__ __forceinline__ void cp_wait() { asm volatile("cp.async.wait_group %0;" :: "n"(N) : "memory"); }

__device__ __forceinline__ void ldsm4(uint32_t (&r)[4], uint32_t a)
{
    asm volatile("ldmatrix.sync.aligned.m8n8.x4.shared.b16 {%0, %1, %2, %3}, [%4];"
                 : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3]) : "r"(a) : "memory");
}
__device__ __forceinline__ void ldsm4t(uint32_t (&r)[4], uint32_t a)
{
    asm volatile("ldmatrix.sync.aligned.m8n8.x4.trans.shared.b16 {%0, %1, %2, %3}, [%4];"
                 : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3]) : "r"(a) : "memory");
}
__device__ __forceinline__ void mma_f16(float (&c)[4], uint32_t a0, uint32_t a1, uint32_t a2, uint32_t a3, uint32_t b0, uint32_t b1)
{
    asm volatile("mma.sync.aligned.m16n8k16.row.col.f32.f16.f16.f32 {%0, %1, %2, %3}, {%4, %5, %6, %7}, {%8, %9}, {%0, %1, %2, %3};"
                 : "+f"(c[0]), "+f"(c[1]), "+f"(c[2]), "+f"(c[3])
                 : "r"(a0), "r"(a1), "r"(a2), "r"(a3), "r"(b0), "r"(b1));
}
__device__ __forceinline__ void mma_bf16(float (&c)[4], uint32_t a0, uint32_t a1, uint32_t a2, uint32_t a3, uint32_t b0, uint32_t b1)
{
    asm volatile("mma.sync.aligned.m16n8k16.row.col.f32.bf16.bf16.f32 {%0, %1, %2, %3}, {%4, %5, %6, %7}, {%8, %9}, {%0, %1, %2, %3};"
                 : "+f"(c[0]), "+f"(c[1]), "+f"(c[2]), "+f"(c[3])
                 : "r"(a0), "r"(a1), "r"(a2), "r"(a3), "r"(b0), "r"(b1));
}

// (x, y) as two f16 parts / three bf16 parts, packed pairwise.
__device__ __forceinline__ void split_f16(float x, float y, uint32_t &hi, uint32_t &lo)
{
    const __half2 h = __floats2half2_rn(x, y);
    const float2 f = __half22float2(h);
    const __half2 l = __floats2half2_rn(x - f.x, y - f.y);
    hi = *reinterpret_cast<const uint32_t *>(&h);
    lo = *reinterpret_cast<const uint32_t *>(&l);
}
__device__ __forceinline__ void split_bf16(float x, float y, uint32_t &hi, uint32_t &mid, uint32_t &lo)
{
    const __nv_bfloat162 h = __floats2bfloat162_rn(x, y);
    const float2 f = __bfloat1622float2(h);
    const float rx = x - f.x, ry = y - f.y;
    const __nv_bfloat162 m = __floats2bfloat162_rn(rx, ry);
    const float2 g = __bfloat1622float2(m);
    const __nv_bfloat162 l = __floats2bfloat162_rn(rx - g.x, ry - g.y);
    hi = *reinterpret_cast<const uint32_t *>(&h);
    mid = *reinterpret_cast<const uint32_t *>(&m);
    lo = *reinterpret_cast<const uint32_t *>(&l);
}

// Four int8 of a word as two pairs of exact f16: the byte, its sign bit
// flipped, under the exponent of 1024 is 1024 + 128 + value.
__device__ __forceinline__ void i8_to_f16(uint32_t w, uint32_t &p01, uint32_t &p23)
{
    w ^= 0x80808080u;
    const __half2 off = __halves2half2(__ushort_as_half(0x6480), __ushort_as_half(0x6480));   // 1152
    uint32_t a = __byte_perm(w, 0x64646464u, 0x4140), b = __byte_perm(w, 0x64646464u, 0x4342);
    const __half2 x = __hsub2(*reinterpret_cast<__half2 *>(&a), off), y = __hsub2(*reinterpret_cast<__half2 *>(&b), off);
    p01 = *reinterpret_cast<const uint32_t *>(&x);
    p23 = *reinterpret_cast<const uint32_t *>(&y);
}

// Bytes (0, 2) and (1, 3) of a word as pairs of exact bf16: the low seven bits
// under the exponent of 128, less 128 for a clear and 256 for a set sign bit.
__device__ __forceinline__ void i8_to_bf16(uint32_t w, uint32_t &p02, uint32_t &p13)
{
    const uint32_t a = __byte_perm(w, 0x43434343u, 0x4240), b = __byte_perm(w, 0x43434343u, 0x4341);
    const uint32_t am = a & 0xFF7FFF7Fu, as = a & 0xFF80FF80u, bm = b & 0xFF7FFF7Fu, bs = b & 0xFF80FF80u;
    const __nv_bfloat162 x = __hsub2(*reinterpret_cast<const __nv_bfloat162 *>(&am), *reinterpret_cast<const __nv_bfloat162 *>(&as));
    const __nv_bfloat162 y = __hsub2(*reinterpret_cast<const __nv_bfloat162 *>(&bm), *reinterpret_cast<const __nv_bfloat162 *>(&bs));
    p02 = *reinterpret_cast<const uint32_t *>(&x);
    p13 = *reinterpret_cast<const uint32_t *>(&y);
}

// Shared-memory geometry of one instance.
template <int TYPE, int DP>
struct AttnGeom {
    static constexpr int EB = TYPE == KV_Q8_0 ? 1 : 2;           // bytes of a value
    static constexpr int PITCH = DP * EB;                        // bytes of a slot's k (or v)
    static constexpr int NCHUNK = PITCH / 16;
    static constexpr int KV_BYTES = ATT_TILE * PITCH;            // a tile's k (or v)
    static constexpr int SC_PITCH = DP / 32 * 2;                 // a slot's scales
    static constexpr int SC_BYTES = TYPE == KV_Q8_0 ? ATT_TILE * SC_PITCH : 0;
    static constexpr int STAGE = 2 * (KV_BYTES + SC_BYTES);      // one warp's stage: k | v | k scales | v scales
    // Warps and stages: 130 to 200 KB of ring per SM.
    static constexpr int NW = STAGE > 12 * 1024 ? 4 : ATT_NW;
    static constexpr int THREADS = NW * 32;
    static constexpr int NST = STAGE >= 8 * 1024 ? 3 : STAGE >= 4 * 1024 ? 4 : 6;
    static constexpr int RING = NW * NST * STAGE;
    static constexpr int MAX_MT = attn_max_mt(DP);
    static constexpr bool QREG = DP <= 128;                      // q's operand fragments in registers
    static constexpr int NPART = TYPE == KV_BF16 ? 3 : 2;        // words of q per k-step and k half
    static constexpr int QS_WORDS = 2 * NPART;                   // per lane and k-step
    static constexpr int Q_BYTES = QREG ? 0 : MAX_MT * (DP / 16) * 32 * QS_WORDS * 4;
    static constexpr int OPITCH = DP + 8;                        // floats: the 8 rows of a store in different banks
    static_assert(NW * 8 * OPITCH * 4 <= RING, "the warps' outputs are joined in the ring");
    static_assert(ATT_MAX_CTAS * 8 * MAX_MT * 4 <= RING, "the parts' factors lie in the ring");
    static constexpr int SMEM = RING + Q_BYTES;
    static_assert(SMEM + 6 * 1024 <= 227 * 1024, "one CTA's shared memory");
    // 16-byte chunk c of row r, so that 8 rows' chunks fall in different banks
    static __device__ __forceinline__ uint32_t at(int r, int c)
    {
        const int x = NCHUNK >= 8 ? (r & 7) : ((r >> 1) & 3);
        return (uint32_t)(r * PITCH + ((c ^ x) << 4));
    }
};

template <int TYPE, int DP>
__global__ void __launch_bounds__(AttnGeom<TYPE, DP>::THREADS, 1) attn_decode_kernel(const __grid_constant__ AttnParams p)
{
    using G = AttnGeom<TYPE, DP>;
    constexpr int NW = G::NW, NT = G::THREADS;
    extern __shared__ __align__(128) uint8_t smem[];
    __shared__ int s_pref[ATT_MAX_SEQ + 1];                      // tiles of one head before each sequence
    __shared__ int s_warp[NW];
    __shared__ float s_m[NW][8], s_l[NW][8];
    __shared__ float s_mr[8 * G::MAX_MT], s_lr[8 * G::MAX_MT];
    __shared__ uint32_t s_mask[NW][G::NST];                       // per warp and stage: slots to use
    __shared__ int s_last;
    const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
    const int g = lane >> 2, c4 = lane & 3;
    const int mt = p.mt, kg = warp / mt, mi = warp % mt;         // key group, row block in it
    const uint32_t ring0 = smem_addr(smem);
    const int units = p.n_rb * p.n_kv;

    // ---- where this CTA's tiles lie: prefix sum of the sequences' tiles
    {
        int run = 0;
        for (int s0 = 0; s0 < p.n_seq; s0 += NT) {
            const int s = s0 + tid;
            int n = 0;
            if (s < p.n_seq) {
                const int raw = __ldg(p.kv_len + s);
                if ((raw < 0 || raw > p.max_len) && blockIdx.x == 0) atomicOr(p.err, 16 /* QMV_DEVERR_SEQ_LEN */);
                AttnSeq q;
                q.set(attn_len(p, s), p);
                n = q.n_tiles;
            }
            int x = n;
            for (int o = 1; o < 32; o <<= 1) {
                const int y = __shfl_up_sync(0xFFFFFFFFu, x, o);
                if (lane >= o) x += y;
            }
            if (lane == 31) s_warp[warp] = x;
            __syncthreads();
            int before = run, all = run;
            for (int w = 0; w < NW; ++w) {
                if (w < warp) before += s_warp[w];
                all += s_warp[w];
            }
            if (s < p.n_seq) s_pref[s] = before + x - n;
            run = all;
            __syncthreads();
        }
        if (tid == 0) s_pref[p.n_seq] = run;
    }
    if (p.dim < DP) {      // columns behind head_dim are never copied: zero once
        for (int i = tid; i < G::RING / 16; i += NT) reinterpret_cast<uint4 *>(smem)[i] = make_uint4(0, 0, 0, 0);
    }
    __syncthreads();
    const int64_t total = (int64_t)s_pref[p.n_seq] * units;
    int64_t share = (total + gridDim.x - 1) / gridDim.x;
    share = max((int64_t)p.min_tiles, (share + NW - 1) / NW * NW);
    const int64_t x0 = share * blockIdx.x, x1 = min(total, x0 + share);

    const int nchunk = p.dim * G::EB / 16;
    const int rows_cta = 8 * mt;
    const uint32_t my_ring = ring0 + (uint32_t)(warp * G::NST * G::STAGE);

    for (int64_t x = x0; x < x1;) {
        // ---- the segment: sequence, row block, head, and its tiles in this CTA
        int s = 0;
        {
            int hi = p.n_seq;
            while (hi - s > 1) {
                const int mid = (s + hi) >> 1;
                if ((int64_t)s_pref[mid] * units <= x) s = mid;
                else hi = mid;
            }
        }
        AttnSeq sq;
        sq.set(attn_len(p, s), p);
        const int64_t seq0 = (int64_t)s_pref[s] * units;
        const int unit = (int)((x - seq0) / sq.n_tiles);
        const int rb = unit / p.n_kv, h = unit % p.n_kv;
        const int64_t seg0 = seq0 + (int64_t)unit * sq.n_tiles, seg1 = seg0 + sq.n_tiles;
        const int t0 = (int)(x - seg0), t1 = (int)(min(seg1, x1) - seg0);
        const int row0 = rb * rows_cta;
        const int n_steps = (t1 - t0 + NW - 1) / NW;
        const int32_t *tab = p.table + (int64_t)s * p.table_stride;
        x += t1 - t0;

        // ---- the ring: page entries one step ahead of the copies
        int pg_next = -1, slot_next = 0;
        auto fetch_page = [&](int step) {
            const int tile = t0 + step * NW + warp;
            pg_next = -1;
            if (step < n_steps && tile < t1 && lane < ATT_TILE) {
                const int j = sq.slot0(tile) + lane;
                slot_next = j;
                if (sq.seen(j)) {
                    const int pi = p.page_shift >= 0 ? j >> p.page_shift : j / p.page_size;
                    pg_next = __ldg(tab + pi);
                    if (pg_next < 0 || pg_next >= p.n_pages) {
                        atomicOr(p.err, 8 /* QMV_DEVERR_PAGE_ID */);
                        pg_next = -1;
                    }
                }
            }
        };
        auto issue = [&](int step) {
            const int tile = t0 + step * NW + warp;
            if (step < n_steps && tile < t1) {
                const int st = step % G::NST;
                const uint32_t dst = my_ring + (uint32_t)(st * G::STAGE);
                const int o = p.page_shift >= 0 ? slot_next & (p.page_size - 1) : slot_next % p.page_size;
                const long long e = pg_next < 0 ? -1
                                                : pg_next * p.page_stride + h * p.head_stride + o * p.slot_stride;
                const uint32_t mask = __ballot_sync(0xFFFFFFFFu, pg_next >= 0);
                if (lane == 0) s_mask[warp][st] = mask;
                constexpr int LPR = G::NCHUNK < 32 ? G::NCHUNK : 32;      // lanes of a row
                constexpr int RPI = 32 / LPR;                             // rows of a pass
                const int ch = lane % LPR;
#pragma unroll
                for (int r0 = 0; r0 < ATT_TILE; r0 += RPI) {
                    const int r = r0 + lane / LPR;
                    const long long er = __shfl_sync(0xFFFFFFFFu, e, r);
                    const uint32_t n = er >= 0 ? 16u : 0u;
                    const int64_t at = er >= 0 ? er * G::EB + ch * 16 : 0;
                    if (ch < nchunk) {
                        cp_async16(dst + G::at(r, ch), p.k + at, n);
                        cp_async16(dst + G::KV_BYTES + G::at(r, ch), p.v + at, n);
                    }
                }
                if (TYPE == KV_Q8_0) {
                    constexpr int WPR = DP / 64;                          // 4-byte words of a slot's scales
                    const int nw = p.dim / 64;
#pragma unroll
                    for (int i0 = 0; i0 < ATT_TILE * WPR; i0 += 32) {
                        const int r = (i0 + lane) / WPR, w = (i0 + lane) % WPR;
                        const long long er = __shfl_sync(0xFFFFFFFFu, e, r & 15);
                        const uint32_t n = er >= 0 ? 4u : 0u;
                        const int64_t at = er >= 0 ? er / 16 + w * 4 : 0;
                        if (r < ATT_TILE && w < nw) {
                            cp_async4(dst + 2 * G::KV_BYTES + r * G::SC_PITCH + w * 4, p.ks + at, n);
                            cp_async4(dst + 2 * G::KV_BYTES + G::SC_BYTES + r * G::SC_PITCH + w * 4, p.vs + at, n);
                        }
                    }
                }
            }
            cp_commit();
        };
        fetch_page(0);
#pragma unroll
        for (int i = 0; i < G::NST - 1; ++i) {
            issue(i);
            fetch_page(i + 1);
        }

        // ---- q as operand fragments: thread (g, c4) holds its row's values at
        // columns 2 c4, 2 c4 + 1 and + 8 of every 16 (Q8_0: 4 c4 .. 4 c4 + 3, the
        // order in which its k bytes come)
        uint32_t aq[G::QREG ? DP / 16 : 1][G::QS_WORDS];
        const int row = row0 + mi * 8 + g;
        const bool row_ok = row < p.rows;
        const int tok = row_ok ? row / p.group : 0;
        const int at = sq.first + tok;                                    // the query's slot
        float sfac = p.scale_log2;
        {
            const float *qr = p.q + (int64_t)(s * p.n_tok + tok) * p.q_stride + (int64_t)(h * p.group + (row_ok ? row % p.group : 0)) * p.dim;
            auto load4 = [&](int ks, float (&f)[4]) {
                const int d0 = ks * 16 + (TYPE == KV_Q8_0 ? 4 * c4 : 2 * c4), d1 = TYPE == KV_Q8_0 ? d0 + 2 : d0 + 8;
                const bool ok = row_ok && ks * 16 < p.dim;
                const float2 a = ok ? __ldg(reinterpret_cast<const float2 *>(qr + d0)) : make_float2(0.f, 0.f);
                const float2 b = ok ? __ldg(reinterpret_cast<const float2 *>(qr + d1)) : make_float2(0.f, 0.f);
                f[0] = a.x; f[1] = a.y; f[2] = b.x; f[3] = b.y;
            };
            float qmul = 1.f;
            if (TYPE != KV_BF16) {
                float mx = 0.f;
#pragma unroll
                for (int ks = 0; ks < DP / 16; ++ks) {
                    float f[4];
                    load4(ks, f);
                    mx = fmaxf(mx, fmaxf(fmaxf(fabsf(f[0]), fabsf(f[1])), fmaxf(fabsf(f[2]), fabsf(f[3]))));
                }
                mx = fmaxf(mx, __shfl_xor_sync(0xFFFFFFFFu, mx, 1));
                mx = fmaxf(mx, __shfl_xor_sync(0xFFFFFFFFu, mx, 2));
                const int ex = (int)(__float_as_uint(mx) >> 23) - 127;
                const int sh = mx > 0.f ? min(100, 12 - ex) : 0;
                qmul = __uint_as_float((uint32_t)(127 + sh) << 23);
                sfac *= __uint_as_float((uint32_t)(127 - sh) << 23);
            }
            uint32_t *qs = reinterpret_cast<uint32_t *>(smem + G::RING) + (size_t)mi * (DP / 16) * 32 * G::QS_WORDS;
            if (!G::QREG) __syncthreads();                                // the last segment's reads of it are done
#pragma unroll
            for (int ks = 0; ks < DP / 16; ++ks) {
                float f[4];
                load4(ks, f);
                uint32_t w[G::QS_WORDS];
                if constexpr (TYPE == KV_BF16) {
                    split_bf16(f[0], f[1], w[0], w[1], w[4]);
                    split_bf16(f[2], f[3], w[2], w[3], w[5]);
                } else {
                    split_f16(f[0] * qmul, f[1] * qmul, w[0], w[1]);
                    split_f16(f[2] * qmul, f[3] * qmul, w[2], w[3]);
                }
                if (G::QREG) {
#pragma unroll
                    for (int i = 0; i < G::QS_WORDS; ++i) aq[G::QREG ? ks : 0][i] = w[i];
                } else if (kg == 0) {
#pragma unroll
                    for (int i = 0; i < G::QS_WORDS; ++i) qs[(ks * G::QS_WORDS + i) * 32 + lane] = w[i];
                }
            }
            if (!G::QREG) __syncthreads();
        }
        auto q_frag = [&](int ks, uint32_t (&w)[G::QS_WORDS]) {
            if (G::QREG) {
#pragma unroll
                for (int i = 0; i < G::QS_WORDS; ++i) w[i] = aq[G::QREG ? ks : 0][i];
            } else {
                const uint32_t a = ring0 + G::RING + (uint32_t)((mi * (DP / 16) + ks) * G::QS_WORDS * 32 + lane) * 4u;
#pragma unroll
                for (int i = 0; i < G::QS_WORDS; ++i) w[i] = lds_u32(a + (uint32_t)i * 128u);
            }
        };

        float m = -INFINITY, l = 0.f;
        float o[DP / 8][4];
#pragma unroll
        for (int i = 0; i < DP / 8; ++i) o[i][0] = o[i][1] = o[i][2] = o[i][3] = 0.f;
        float *raw = p.score ? p.raw + ((int64_t)(s * p.n_kv + h) * p.rows + row) * p.raw_stride : nullptr;

        for (int step = 0; step < n_steps; ++step) {
            cp_wait<G::NST - 2>();
            if (mt == 1) __syncwarp();
            else named_bar_sync(1 + kg, 32 * mt);
            issue(step + G::NST - 1);
            fetch_page(step + G::NST);
            const int st = step % G::NST;
            for (int mm = 0; mm < mt; ++mm) {
                const int w = kg * mt + mm, tile = t0 + step * NW + w;
                if (tile >= t1) break;
                const uint32_t buf = ring0 + (uint32_t)((w * G::NST + st) * G::STAGE);
                const int j0 = sq.slot0(tile);
                const uint32_t use = s_mask[w][st];
                // -- scores of 16 slots: this thread's are slots 2 c4, 2 c4 + 1 and + 8
                float sc[2][4] = {};
                const uint32_t kaddr_r = (uint32_t)((lane >> 4) * 8 + (lane & 7)), kaddr_c = (uint32_t)((lane >> 3) & 1);
                if constexpr (TYPE == KV_Q8_0) {
#pragma unroll
                    for (int b = 0; b < DP / 32; ++b) {
                        uint32_t r[4];
                        ldsm4(r, buf + G::at(kaddr_r, 2 * b + kaddr_c));
                        float a[2][4] = {};
#pragma unroll
                        for (int k2 = 0; k2 < 2; ++k2) {
                            uint32_t q[G::QS_WORDS];
                            q_frag(2 * b + k2, q);
#pragma unroll
                            for (int nt = 0; nt < 2; ++nt) {
                                uint32_t b0, b1;
                                i8_to_f16(r[2 * nt + k2], b0, b1);
                                mma_f16(a[nt], q[0], q[1], q[2], q[3], b0, b1);
                            }
                        }
#pragma unroll
                        for (int nt = 0; nt < 2; ++nt)
#pragma unroll
                            for (int i = 0; i < 2; ++i) {
                                const float d = half_bits_to_float(lds_u16(buf + 2 * G::KV_BYTES + (uint32_t)((nt * 8 + 2 * c4 + i) * G::SC_PITCH + 2 * b)));
                                sc[nt][i] = fmaf(d, a[nt][i] + a[nt][i + 2], sc[nt][i]);
                            }
                    }
                } else {
#pragma unroll
                    for (int ks = 0; ks < DP / 16; ++ks) {
                        uint32_t r[4], q[G::QS_WORDS];
                        ldsm4(r, buf + G::at(kaddr_r, 2 * ks + kaddr_c));
                        q_frag(ks, q);
#pragma unroll
                        for (int nt = 0; nt < 2; ++nt) {
                            if constexpr (TYPE == KV_F16) {
                                mma_f16(sc[nt], q[0], q[1], q[2], q[3], r[2 * nt], r[2 * nt + 1]);
                            } else {
                                mma_bf16(sc[nt], q[0], q[1], q[2], q[3], r[2 * nt], r[2 * nt + 1]);
                                mma_bf16(sc[nt], q[4], 0u, q[5], 0u, r[2 * nt], r[2 * nt + 1]);
                            }
                        }
                    }
                }
                float sv[4];
                bool vis[4];
#pragma unroll
                for (int i = 0; i < 4; ++i) {
                    const int jj = (i >> 1) * 8 + 2 * c4 + (i & 1);
                    const float t = TYPE == KV_Q8_0 ? sc[i >> 1][i & 1] : sc[i >> 1][i & 1] + sc[i >> 1][(i & 1) + 2];
                    vis[i] = row_ok && ((use >> jj) & 1u) && attn_sees(p, at, j0 + jj);
                    sv[i] = vis[i] ? t * sfac : -INFINITY;
                }
                if (raw && row_ok) {
                    *reinterpret_cast<float2 *>(raw + j0 + 2 * c4) = make_float2(sv[0], sv[1]);
                    *reinterpret_cast<float2 *>(raw + j0 + 8 + 2 * c4) = make_float2(sv[2], sv[3]);
                }
                // -- the running maximum and sum
                float mx = fmaxf(fmaxf(sv[0], sv[1]), fmaxf(sv[2], sv[3]));
                mx = fmaxf(mx, __shfl_xor_sync(0xFFFFFFFFu, mx, 1));
                mx = fmaxf(mx, __shfl_xor_sync(0xFFFFFFFFu, mx, 2));
                const float mn = fmaxf(m, mx);
                if (__any_sync(0xFFFFFFFFu, mn > m)) {
                    const float f = m == mn ? 1.f : exp2f(m - mn);        // m = -inf: 0
                    l *= f;
#pragma unroll
                    for (int i = 0; i < DP / 8; ++i) {
                        o[i][0] *= f; o[i][1] *= f; o[i][2] *= f; o[i][3] *= f;
                    }
                    m = mn;
                }
                // f16 parts: weights times 2^15, so that their low parts stay normal
                const float mref = (m == -INFINITY ? 0.f : m) - p.l_shift;
                float pr[4];
#pragma unroll
                for (int i = 0; i < 4; ++i) {
                    pr[i] = exp2f(sv[i] - mref);
                    l += pr[i];
                }
                // -- output += weights x values
                const uint32_t va = buf + G::KV_BYTES;
                const uint32_t vaddr_r = (uint32_t)(((lane >> 3) & 1) * 8 + (lane & 7)), vaddr_c = (uint32_t)(lane >> 4);
                if constexpr (TYPE == KV_Q8_0) {
#pragma unroll
                    for (int b = 0; b < DP / 32; ++b) {
                        uint32_t r[4], a[6];
                        ldsm4t(r, va + G::at(vaddr_r, 2 * b + vaddr_c));
                        float pd[4];
#pragma unroll
                        for (int i = 0; i < 4; ++i) {
                            const int jj = (i >> 1) * 8 + 2 * c4 + (i & 1);
                            const float d = half_bits_to_float(lds_u16(buf + 2 * G::KV_BYTES + G::SC_BYTES + (uint32_t)(jj * G::SC_PITCH + 2 * b)));
                            pd[i] = vis[i] ? pr[i] * d : 0.f;
                        }
                        split_bf16(pd[0], pd[1], a[0], a[1], a[4]);
                        split_bf16(pd[2], pd[3], a[2], a[3], a[5]);
#pragma unroll
                        for (int k2 = 0; k2 < 2; ++k2) {
                            uint32_t e0, e1, d0, d1;                       // even and odd columns of 16
                            i8_to_bf16(r[2 * k2], e0, d0);
                            i8_to_bf16(r[2 * k2 + 1], e1, d1);
                            mma_bf16(o[4 * b + 2 * k2], a[0], a[1], a[2], a[3], e0, e1);
                            mma_bf16(o[4 * b + 2 * k2], a[4], 0u, a[5], 0u, e0, e1);
                            mma_bf16(o[4 * b + 2 * k2 + 1], a[0], a[1], a[2], a[3], d0, d1);
                            mma_bf16(o[4 * b + 2 * k2 + 1], a[4], 0u, a[5], 0u, d0, d1);
                        }
                    }
                } else {
                    uint32_t a[6];
                    if constexpr (TYPE == KV_F16) {
                        split_f16(pr[0], pr[1], a[0], a[1]);
                        split_f16(pr[2], pr[3], a[2], a[3]);
                    } else {
                        split_bf16(pr[0], pr[1], a[0], a[1], a[4]);
                        split_bf16(pr[2], pr[3], a[2], a[3], a[5]);
                    }
                    auto pv = [&](float (&acc)[4], uint32_t b0, uint32_t b1) {
                        if constexpr (TYPE == KV_F16) {
                            mma_f16(acc, a[0], a[1], a[2], a[3], b0, b1);
                        } else {
                            mma_bf16(acc, a[0], a[1], a[2], a[3], b0, b1);
                            mma_bf16(acc, a[4], 0u, a[5], 0u, b0, b1);
                        }
                    };
                    const bool mixed = p.n_tok > 1 && tile >= sq.sink_tiles &&
                                       (j0 + ATT_TILE - 1 > sq.first || (p.window > 0 && j0 <= sq.len - 1 - p.window));
                    if (!mixed) {
#pragma unroll
                        for (int i = 0; i < DP / 16; ++i) {
                            uint32_t r[4];
                            ldsm4t(r, va + G::at(vaddr_r, 2 * i + vaddr_c));
                            pv(o[2 * i], r[0], r[1]);
                            pv(o[2 * i + 1], r[2], r[3]);
                        }
                    } else {
                        // token by token, the values it does not see as zeros
                        const int tk0 = (row0 + mi * 8) / p.group, tk1 = min(row0 + mi * 8 + 7, p.rows - 1) / p.group;
                        for (int tk = tk0; tk <= tk1; ++tk) {
                            uint32_t z[2];
#pragma unroll
                            for (int i = 0; i < 2; ++i) {
                                const int j = j0 + 8 * i + 2 * c4;
                                z[i] = (attn_sees(p, sq.first + tk, j) ? 0xFFFFu : 0u) | (attn_sees(p, sq.first + tk, j + 1) ? 0xFFFF0000u : 0u);
                            }
#pragma unroll
                            for (int i = 0; i < DP / 16; ++i) {
                                uint32_t r[4];
                                ldsm4t(r, va + G::at(vaddr_r, 2 * i + vaddr_c));
#pragma unroll
                                for (int n2 = 0; n2 < 2; ++n2) {
                                    float acc[4] = {};
                                    pv(acc, r[2 * n2] & z[0], r[2 * n2 + 1] & z[1]);
                                    if (tk == tok) {
#pragma unroll
                                        for (int e = 0; e < 4; ++e) o[2 * i + n2][e] += acc[e];
                                    }
                                }
                            }
                        }
                    }
                }
            }
        }
        cp_wait<0>();
        l += __shfl_xor_sync(0xFFFFFFFFu, l, 1);
        l += __shfl_xor_sync(0xFFFFFFFFu, l, 2);
        if (c4 == 0) {
            s_m[warp][g] = m;
            s_l[warp][g] = l;
        }
        __syncthreads();                                                  // the ring is free

        // ---- join the key groups' parts (in the ring)
        float *so = reinterpret_cast<float *>(smem);
        {
            float mr = -INFINITY;
            for (int w = mi; w < NW / mt * mt; w += mt) mr = fmaxf(mr, s_m[w][g]);
            const float f = m == mr ? 1.f : exp2f(m - mr);
            float *ow = so + (size_t)(warp * 8 + g) * G::OPITCH;
#pragma unroll
            for (int i = 0; i < DP / 16; ++i) {
                const float v0 = (o[2 * i][0] + o[2 * i][2]) * f, v1 = (o[2 * i][1] + o[2 * i][3]) * f;
                const float u0 = (o[2 * i + 1][0] + o[2 * i + 1][2]) * f, u1 = (o[2 * i + 1][1] + o[2 * i + 1][3]) * f;
                if (TYPE == KV_Q8_0) {
                    *reinterpret_cast<float4 *>(ow + 16 * i + 4 * c4) = make_float4(v0, u0, v1, u1);
                } else {
                    *reinterpret_cast<float2 *>(ow + 16 * i + 2 * c4) = make_float2(v0, v1);
                    *reinterpret_cast<float2 *>(ow + 16 * i + 8 + 2 * c4) = make_float2(u0, u1);
                }
            }
            if (kg == 0 && c4 == 0) {
                float lr = 0.f;
                for (int w = mi; w < NW; w += mt) lr += s_m[w][g] == mr ? s_l[w][g] : s_l[w][g] * exp2f(s_m[w][g] - mr);
                s_mr[mi * 8 + g] = mr;
                s_lr[mi * 8 + g] = lr;
            }
        }
        __syncthreads();
        const int nrow = min(rows_cta, p.rows - row0);
        auto put = [&](int r, int d, float v) {
            const int rr = row0 + r, t = rr / p.group, hq = rr % p.group;
            p.out[(int64_t)(s * p.n_tok + t) * p.out_stride + (int64_t)(h * p.group + hq) * p.dim + d] = v;
        };
        auto put_stats = [&](int r, float mr, float lr) {
            if (p.score) {
                float *q = p.stats + 2 * ((int64_t)(s * p.n_kv + h) * p.rows + row0 + r);
                q[0] = mr;
                q[1] = lr;
            }
        };
        const bool whole = seg0 >= x0 && seg1 <= x1;
        const int slot = 2 * blockIdx.x + (seg0 >= x0 ? 1 : 0);
        for (int i = tid; i < nrow * p.dim; i += NT) {
            const int r = i / p.dim, d = i % p.dim;
            float v = 0.f;
            for (int k2 = 0; k2 < NW / mt; ++k2) v += so[(size_t)((k2 * mt + (r >> 3)) * 8 + (r & 7)) * G::OPITCH + d];
            if (whole) put(r, d, s_lr[r] != 0.f ? v / s_lr[r] : 0.f);
            else p.part_o[((int64_t)slot * rows_cta + r) * p.dim + d] = v;
        }
        if (tid < nrow) {
            if (whole) {
                put_stats(tid, s_mr[tid], s_lr[tid]);
            } else {
                float *q = p.part_ml + 2 * ((int64_t)slot * rows_cta + tid);
                q[0] = s_mr[tid];
                q[1] = s_lr[tid];
            }
        }
        if (!whole) {
            // ---- the last CTA of the segment joins its parts, in CTA order
            const int cta0 = (int)(seg0 / share), cta1 = (int)((seg1 - 1) / share), n = cta1 - cta0 + 1;
            __threadfence();
            __syncthreads();
            if (tid == 0) {
                const unsigned done = atomicAdd(p.counters + cta0, 1u);
                s_last = done == (unsigned)(n - 1);
                if (s_last) p.counters[cta0] = 0u;
            }
            __syncthreads();
            if (s_last) {
                __threadfence();
                auto slot_of = [&](int i) { return 2 * (cta0 + i) + (i == 0 ? 1 : 0); };
                float *fac = reinterpret_cast<float *>(smem);             // [n][nrow]
                for (int r = warp; r < nrow; r += NW) {
                    float mr = -INFINITY, lr = 0.f;
                    for (int i = lane; i < n; i += 32) mr = fmaxf(mr, __ldcg(p.part_ml + 2 * ((int64_t)slot_of(i) * rows_cta + r)));
                    for (int off = 16; off; off >>= 1) mr = fmaxf(mr, __shfl_xor_sync(0xFFFFFFFFu, mr, off));
                    for (int i = lane; i < n; i += 32) {
                        const float *q = p.part_ml + 2 * ((int64_t)slot_of(i) * rows_cta + r);
                        const float mc = __ldcg(q), f = mc == mr ? 1.f : exp2f(mc - mr);
                        fac[i * nrow + r] = f;
                        lr += f * __ldcg(q + 1);
                    }
                    for (int off = 16; off; off >>= 1) lr += __shfl_xor_sync(0xFFFFFFFFu, lr, off);
                    if (lane == 0) {
                        s_lr[r] = lr;
                        put_stats(r, mr, lr);
                    }
                }
                __syncthreads();
                for (int i = tid; i < nrow * p.dim; i += NT) {
                    const int r = i / p.dim, d = i % p.dim;
                    float v = 0.f;
                    for (int c = 0; c < n; ++c) v += fac[c * nrow + r] * __ldcg(p.part_o + ((int64_t)slot_of(c) * rows_cta + r) * p.dim + d);
                    put(r, d, s_lr[r] != 0.f ? v / s_lr[r] : 0.f);
                }
            }
        }
        __syncthreads();                                                  // the ring is refilled next
        if (p.dim < DP && x < x1) {                                       // and its unused columns were written over
            for (int i = tid; i < G::RING / 16; i += NT) reinterpret_cast<uint4 *>(smem)[i] = make_uint4(0, 0, 0, 0);
            __syncthreads();
        }
    }
}

// score[s][h][j] (+)= sum over the rows of 2^(s_j - m) / l, from the raw scores
// and the joined (m, l) that attn_decode_kernel left in the workspace.  One
// thread per slot, rows in order.
constexpr int ATT_SCORE_THREADS = 256;

static __global__ void __launch_bounds__(ATT_SCORE_THREADS) attn_score_kernel(const __grid_constant__ AttnParams p)
{
    const int s = blockIdx.z, h = blockIdx.y;
    AttnSeq sq;
    sq.set(attn_len(p, s), p);
    for (int64_t j64 = (int64_t)blockIdx.x * ATT_SCORE_THREADS + threadIdx.x; j64 < sq.len; j64 += (int64_t)gridDim.x * ATT_SCORE_THREADS) {
        const int j = (int)j64;
        if (!sq.seen(j)) continue;
        const int64_t sh = (int64_t)s * p.n_kv + h;
        const float *raw = p.raw + sh * p.rows * p.raw_stride + j;
        const float *st = p.stats + 2 * sh * p.rows;
        float v = 0.f;
        for (int r = 0; r < p.rows; ++r) {
            const float m = __ldg(st + 2 * r), l = __ldg(st + 2 * r + 1);
            if (l != 0.f) v += exp2f(__ldcg(raw + r * p.raw_stride) - m + p.l_shift) / l;
        }
        float *o = p.score + sh * p.score_stride + j;
        *o = j >= sq.first ? v : *o + v;
    }
}

// One launch of the instance that holds p.dim.
template <int TYPE>
static cudaError_t launch_attn(const AttnParams &p, int grid, cudaStream_t st)
{
    static SmemCfg configured[3];
    if (p.dim <= 64) return launch_with(attn_decode_kernel<TYPE, 64>, configured[0], p, dim3((unsigned)grid), AttnGeom<TYPE, 64>::SMEM, st, false, false, AttnGeom<TYPE, 64>::THREADS);
    if (p.dim <= 128) return launch_with(attn_decode_kernel<TYPE, 128>, configured[1], p, dim3((unsigned)grid), AttnGeom<TYPE, 128>::SMEM, st, false, false, AttnGeom<TYPE, 128>::THREADS);
    return launch_with(attn_decode_kernel<TYPE, 256>, configured[2], p, dim3((unsigned)grid), AttnGeom<TYPE, 256>::SMEM, st, false, false, AttnGeom<TYPE, 256>::THREADS);
}

}  // namespace qmv
