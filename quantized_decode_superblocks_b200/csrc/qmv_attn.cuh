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
// Work split.  The cache is cut into tiles of 16 or 32 slots of one kv head; one
// per warp of a CTA is a step.  The steps of all sequences, heads and row blocks
// are numbered through, and CTA c takes the c-th equal range of them, so that
// ragged batches and single long sequences load every SM alike; the lengths are
// only known on the device, so every CTA finds its own range from a prefix sum
// over them.  A (sequence, row block, head) that lies in several ranges leaves
// its parts in the workspace, and the last of its CTAs to arrive (a counter) joins
// them in CTA order.  Two or three CTAs share an SM where shared memory allows, so
// that one streams while another starts or joins a segment.
//
// In a CTA, each of 4 (6) warps streams every 4th (6th) tile through a ring of
// its own (cp.async, NST stages) and multiplies on the tensor cores (m16n8k16, f32
// accumulation) with the cache as the A operand:
//   S^T[16 slots][8 rows] = K q^T,   O^T[16 dims][8 rows] += V^T P^T,
// so a fragment of K or V is loaded (and, for Q8_0, unpacked) once for all rows
// of the CTA, and 8 rows fill the instruction.  The weights turn from the first
// product's C layout to the second's B layout by movmatrix.  f32 operands are
// split into parts that the tensor core multiplies exactly:
//   f16 cache:   q * 2^e (per row, so that the largest value is below 2^13) as two
//                f16 parts, 22 bits; 2^9 * p as one and 2^11 times what it leaves
//                as another, in two products: 22 bits of weights down to 2^-22 of
//                the largest (with a second part without a factor 12 bits are left there,
//                alike for alike weights, so that a long tail's errors add up);
//   bf16 cache:  q and p as three bf16 parts, 24 bits;
//   Q8_0 cache:  q as for f16 (int8 is exact in it), and p * scale as two f16
//                parts times a power of two of its own for every row, tile and
//                block of 32 dims, since scales may lie 2^40 apart.  (As three bf16
//                parts without a factor, which int8 is exact in too: one token for
//                16 sequences, 128 wide, 98 us instead of 84, 64 wide 56 instead of 50.)
// Tensor cores cut off the bits that an accumulation shifts out, so a long chain of
// them drifts: each tile's product starts from zero and is added to the
// running output by rounded f32 adds.
//
// The running maximum m is a reference: it only moves when a score passes it by
// more than a slack, so most tiles need no reduction across lanes.
//
// Slots that no query of the call sees are not loaded (their shared memory is
// zeroed by the copy).  A slot that only some of several queries see has weight 0
// for the others; 0 * NaN is NaN, so in tiles with such slots NaN and infinities
// among the values (Q8_0: the scales) are made finite first.
//
// Measured (32 query / 8 kv heads): f16, 64 wide, one token over 131071 slots
// 46.5 us, 5.8 TB/s; bf16, 128 wide, 32 ragged sequences up to 16384 slots 181 us,
// 6.5 TB/s, both bound by DRAM; Q8_0, 128 wide, 8 tokens over 4096 slots of 4 sequences
// 38 us, bound by dependent chains of instructions on under two warps a scheduler
// (0.41 issued a cycle); one token over 1000 slots 5.6 us, bound by the memory
// round trips that wait on each other.
#pragma once

#include <type_traits>

#include <cuda_bf16.h>

#include "qmv_device.cuh"
#include "qmv_launch.cuh"

namespace qmv {

enum { KV_F16 = 0, KV_BF16 = 1, KV_Q8_0 = 2 };

// Warps of a CTA; 6 where a stage is 16 KB and one CTA fills the SM.
__host__ __device__ constexpr int attn_warps(int type, int dp) { return dp > 128 && type != 2 ? 6 : 4; }
constexpr int ATT_MIN_NW = 4;
// Slots of a tile: 32 where its keys and values are short, so that a warp's work
// around a tile is spread over more of them.  Against 16 (32 query / 8 kv heads):
// f16, 64 wide, one token over 131071 slots 47.9 -> 46.4 us; Q8_0, 128 wide, for
// sequences of 3000 to 16000 slots, one token of 16 98 -> 84 us, four tokens of 8
// (two CTAs of two stages instead of three of three) 83 -> 70 us.
__host__ __device__ constexpr int attn_tile(int type, int dp) { return dp <= 64 || (type == 2 && dp <= 128) ? 32 : 16; }
constexpr int ATT_MIN_TILE = 16, ATT_MAX_TILE = 32;
// log2 of how far a weight may pass 1, and of the factors of an f16 cache's
// weights and of what their first part leaves of them (half a step at most):
// either stays below 2^15, and half a step of the second part's subnormals is
// 2^-45 of the reference.  Other caches' weights keep f32's range.
__host__ __device__ constexpr float attn_slack(int type) { return type == 0 ? 6.f : 12.f; }
constexpr float ATT_F16_SHIFT = 9.f;
constexpr float ATT_F16_LEFT = 2048.f;

// 8-row blocks that one CTA takes: up to 2.  (With 4, whose outputs and operands
// leave no registers to overlap anything, 32 rows over 4096 slots of 4 sequences
// take 48 us instead of 36 us in bf16 and 48 us instead of 38 us in Q8_0, 128 wide.)
__host__ __device__ constexpr int attn_mb(int rows) { return rows <= 8 ? 1 : 2; }
constexpr int ATT_MAX_SEQ = 1024;
constexpr int ATT_MAX_CTAS = 480;            // bound for the workspace's parts

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
    int32_t mb, n_rb;                                    // 8-row blocks of a CTA, row blocks of a head
    int32_t window, n_sink;
    float inv_group;                                     // 1 / group: row / group of up to 1024 rows by a product
    float scale_log2, l_shift;                           // l counts 2^l_shift times the weights
    unsigned *counters;                                  // [ATT_MAX_CTAS], zero between calls
    float *part_ml, *part_o;                             // [2 * CTAs][8 mb][2], [..][dim]
    float *raw, *stats;                                  // for `score`: scores s [..][slot][row]; (m - l_shift, 1 / l or 0) of every row
    int64_t raw_stride;                                  // slots
    int32_t raw_rows;                                    // rows, made even
    int *err;
};

// Which slots of a sequence the call's queries see, as tiles.
struct AttnSeq {
    int len, first;        // length; slot of the first query (may be negative)
    int lo, sinks;         // slots >= lo, and slots < sinks, are seen by some query
    int sink_tiles, base;  // tiles 0 .. sink_tiles - 1 start at slot 0, the others at slot base
    int n_tiles, n_steps;  // at least 1, so that every row gets written

    template <int TILE, int NW>
    __device__ __forceinline__ void set(int n, const AttnParams &p)
    {
        len = n;
        first = n - p.n_tok;
        lo = sinks = sink_tiles = base = 0;
        if (p.window > 0) {
            lo = max(0, max(first, 0) - p.window + 1);
            sinks = min(p.n_sink, lo);
            sink_tiles = (sinks + TILE - 1) / TILE;
            base = lo / TILE * TILE;
            if (sinks > 0 && sink_tiles * TILE >= base) sink_tiles = base = 0;   // the parts meet
        }
        n_tiles = max(1, sink_tiles + (len - base + TILE - 1) / TILE);
        n_steps = (n_tiles + NW - 1) / NW;
    }
    template <int TILE>
    __device__ __forceinline__ int slot0(int tile) const
    {
        return tile < sink_tiles ? tile * TILE : base + (tile - sink_tiles) * TILE;
    }
    __device__ __forceinline__ bool seen(int j) const { return j < len && (j >= lo || j < sinks); }
    // Slots j0 .. j0 + TILE - 1 are seen by every query (of several).
    template <int TILE>
    __device__ __forceinline__ bool by_all(int j0, const AttnParams &p) const
    {
        return j0 + TILE - 1 <= first && (p.window == 0 || j0 > len - 1 - p.window || j0 + TILE <= p.n_sink);
    }
};

__device__ __forceinline__ int attn_len(const AttnParams &p, int s)
{
    const int n = __ldg(p.kv_len + s);
    return min(max(n, 0), p.max_len);
}

// a / b where the quotient is below 2^20: the product with the reciprocal is off by at most one.
__device__ __forceinline__ int div_small(int a, int b)
{
    int q = (int)(__fdividef((float)a, (float)b));
    const int left = a - q * b;
    q += left < 0 ? -1 : left >= b ? 1 : 0;
    return q;
}
// row / group: (row + 1/2) / group is at least 1 / 2048 from a whole number, the product's error below 2^-13
__device__ __forceinline__ int attn_token(const AttnParams &p, int row) { return (int)(((float)row + 0.5f) * p.inv_group); }

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

// c = a b, without an addend.
template <bool BF16>
__device__ __forceinline__ void mma_16_0(float (&c)[4], const uint32_t (&a)[4], uint32_t b0, uint32_t b1)
{
    if constexpr (BF16)
        asm volatile("mma.sync.aligned.m16n8k16.row.col.f32.bf16.bf16.f32 {%0, %1, %2, %3}, {%4, %5, %6, %7}, {%8, %9}, {%10, %10, %10, %10};"
                     : "=f"(c[0]), "=f"(c[1]), "=f"(c[2]), "=f"(c[3])
                     : "r"(a[0]), "r"(a[1]), "r"(a[2]), "r"(a[3]), "r"(b0), "r"(b1), "f"(0.f));
    else
        asm volatile("mma.sync.aligned.m16n8k16.row.col.f32.f16.f16.f32 {%0, %1, %2, %3}, {%4, %5, %6, %7}, {%8, %9}, {%10, %10, %10, %10};"
                     : "=f"(c[0]), "=f"(c[1]), "=f"(c[2]), "=f"(c[3])
                     : "r"(a[0]), "r"(a[1]), "r"(a[2]), "r"(a[3]), "r"(b0), "r"(b1), "f"(0.f));
}
template <bool BF16>
__device__ __forceinline__ void mma_16(float (&c)[4], const uint32_t (&a)[4], uint32_t b0, uint32_t b1)
{
    if constexpr (BF16) mma_bf16(c, a[0], a[1], a[2], a[3], b0, b1);
    else mma_f16(c, a[0], a[1], a[2], a[3], b0, b1);
}
// Adds 1 and returns the old value; what this CTA wrote before (and a barrier
// ordered before this thread) is seen by who reads the sum, and the other way round.
__device__ __forceinline__ unsigned atomic_inc_acq_rel(unsigned *p)
{
    unsigned old;
    asm volatile("atom.add.acq_rel.gpu.global.u32 %0, [%1], 1;" : "=r"(old) : "l"(p) : "memory");
    return old;
}
// An 8x8 matrix of 16-bit values, two of a row per lane, transposed.
__device__ __forceinline__ uint32_t movm_t(uint32_t x)
{
    uint32_t y;
    asm volatile("movmatrix.sync.aligned.m8n8.trans.b16 %0, %1;" : "=r"(y) : "r"(x));
    return y;
}
__device__ __forceinline__ float ex2(float x)
{
    float y;
    asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
    return y;
}

// (x, y) as two f16 parts (the second times LEFT) / three bf16 parts, packed pairwise.
template <int LEFT = 1>
__device__ __forceinline__ void split_f16(float x, float y, uint32_t &hi, uint32_t &lo)
{
    const __half2 h = __floats2half2_rn(x, y);
    const float2 f = __half22float2(h);
    const __half2 l = __floats2half2_rn((x - f.x) * LEFT, (y - f.y) * LEFT);
    hi = *reinterpret_cast<const uint32_t *>(&h);
    lo = *reinterpret_cast<const uint32_t *>(&l);
}
// Each part is the leading 8 bits of what is left (cut off, not rounded: the
// rest of 24 bits always fits the next two).
__device__ __forceinline__ void split_bf16(float x, float y, uint32_t &hi, uint32_t &mid, uint32_t &lo)
{
    const uint32_t ux = __float_as_uint(x), uy = __float_as_uint(y);
    hi = __byte_perm(ux, uy, 0x7632);
    const float rx = x - __uint_as_float(ux & 0xFFFF0000u), ry = y - __uint_as_float(uy & 0xFFFF0000u);
    const uint32_t vx = __float_as_uint(rx), vy = __float_as_uint(ry);
    mid = __byte_perm(vx, vy, 0x7632);
    lo = __byte_perm(__float_as_uint(rx - __uint_as_float(vx & 0xFFFF0000u)), __float_as_uint(ry - __uint_as_float(vy & 0xFFFF0000u)), 0x7632);
}
// A pair of 16-bit values brought within the type's finite range; NaN becomes its
// lowest value (minimum and maximum return the operand that is a number).
template <int TYPE>
__device__ __forceinline__ uint32_t finite_pair(uint32_t x)
{
    if constexpr (TYPE == KV_F16) {
        const __half2 top = __half2half2(__ushort_as_half(0x7BFF)), y = __hmin2(__hmax2(*reinterpret_cast<const __half2 *>(&x), __hneg2(top)), top);
        return *reinterpret_cast<const uint32_t *>(&y);
    } else {
        const __nv_bfloat162 top = __bfloat162bfloat162(__ushort_as_bfloat16(0x7F7F)), y = __hmin2(__hmax2(*reinterpret_cast<const __nv_bfloat162 *>(&x), __hneg2(top)), top);
        return *reinterpret_cast<const uint32_t *>(&y);
    }
}
// (a, b) += (x, y), += (x, y) * f, += (x f, y g), *= (x, y): one instruction each.
__device__ __forceinline__ void add2(float &a, float &b, float x, float y)
{
    asm("{\n\t.reg .b64 u, v;\n\tmov.b64 u, {%0, %1};\n\tmov.b64 v, {%2, %3};\n\tadd.rn.f32x2 u, u, v;\n\tmov.b64 {%0, %1}, u;\n\t}"
        : "+f"(a), "+f"(b) : "f"(x), "f"(y));
}
__device__ __forceinline__ void fma2(float &a, float &b, float x, float y, float f)
{
    asm("{\n\t.reg .b64 u, v, w;\n\tmov.b64 u, {%0, %1};\n\tmov.b64 v, {%2, %3};\n\tmov.b64 w, {%4, %4};\n\tfma.rn.f32x2 u, v, w, u;\n\tmov.b64 {%0, %1}, u;\n\t}"
        : "+f"(a), "+f"(b) : "f"(x), "f"(y), "f"(f));
}
__device__ __forceinline__ void fma22(float &a, float &b, float x, float y, float f, float g)
{
    asm("{\n\t.reg .b64 u, v, w;\n\tmov.b64 u, {%0, %1};\n\tmov.b64 v, {%2, %3};\n\tmov.b64 w, {%4, %5};\n\tfma.rn.f32x2 u, v, w, u;\n\tmov.b64 {%0, %1}, u;\n\t}"
        : "+f"(a), "+f"(b) : "f"(x), "f"(y), "f"(f), "f"(g));
}
__device__ __forceinline__ void mul2(float &a, float &b, float x, float y)
{
    asm("{\n\t.reg .b64 u, v;\n\tmov.b64 u, {%0, %1};\n\tmov.b64 v, {%2, %3};\n\tmul.rn.f32x2 u, u, v;\n\tmov.b64 {%0, %1}, u;\n\t}"
        : "+f"(a), "+f"(b) : "f"(x), "f"(y));
}

// Four int8 of a word as two pairs of exact f16 (bytes 0 and 1, 2 and 3 or as
// the selectors say): the byte, its sign bit flipped, under the exponent of
// 1024 is 1024 + 128 + value.
template <int S0 = 0x4140, int S1 = 0x4342>
__device__ __forceinline__ void i8_to_f16(uint32_t w, uint32_t &p0, uint32_t &p1)
{
    w ^= 0x80808080u;
    const __half2 off = __halves2half2(__ushort_as_half(0x6480), __ushort_as_half(0x6480));   // 1152
    uint32_t a = __byte_perm(w, 0x64646464u, S0), b = __byte_perm(w, 0x64646464u, S1);
    const __half2 x = __hsub2(*reinterpret_cast<__half2 *>(&a), off), y = __hsub2(*reinterpret_cast<__half2 *>(&b), off);
    p0 = *reinterpret_cast<const uint32_t *>(&x);
    p1 = *reinterpret_cast<const uint32_t *>(&y);
}

// Shared-memory geometry of one instance: MB 8-row blocks of a DP-wide head.
template <int TYPE, int DP, int MB>
struct AttnGeom {
    static constexpr int TILE = attn_tile(TYPE, DP), SUB = TILE / 16;     // slots of a tile, and products of 16
    static constexpr uint32_t ALL = 0xFFFFFFFFu >> (32 - TILE);
    static constexpr int EB = TYPE == KV_Q8_0 ? 1 : 2;           // bytes of a value
    static constexpr int PITCH = DP * EB;                        // bytes of a slot's k (or v)
    static constexpr int NCHUNK = PITCH / 16;
    static constexpr int KV_BYTES = TILE * PITCH;            // a tile's k (or v)
    static constexpr int SC_PITCH = DP / 32 * 2;                 // a slot's scales
    static constexpr int SC_BYTES = TYPE == KV_Q8_0 ? TILE * SC_PITCH : 0;
    static constexpr int STAGE = 2 * (KV_BYTES + SC_BYTES);      // one warp's stage: k | v | k scales | v scales
    static constexpr int ROWS = 8 * MB;
    static constexpr int NW = attn_warps(TYPE, DP), THREADS = NW * 32;
    // Stages and CTAs a SM: three CTAs with up to 70 KB of shared memory for narrow
    // heads and one row block of Q8_0, else two with up to 110 KB, one where a stage
    // is 16 KB.  Three against two (32 query / 8 kv heads): f16, 64 wide, one token
    // over 131071 slots 47.5 -> 46.4 us, 8 tokens over 4096 slots of 4 sequences 20.2
    // -> 19.2 us; Q8_0, 128 wide, one token for 16 sequences 84 us either way.  bf16,
    // 64 wide, 16 rows have two, the 8 tokens 23.9 us (22.4 us with three); 16 rows
    // of Q8_0 or of 128 wide heads do not fit three times.
    static constexpr bool THREE = (DP <= 64 && (MB == 1 || DP <= 32 || TYPE == KV_F16)) || (TYPE == KV_Q8_0 && DP == 128 && MB == 1);
    static constexpr int NST = DP > 128 ? 2 : THREE ? (STAGE >= 8 * 1024 ? 2 : 4) : STAGE > 8 * 1024 ? 2 : STAGE == 8 * 1024 ? 3 : 5;
    static constexpr int RING = NW * NST * STAGE;
    static constexpr int NPQ = TYPE == KV_BF16 ? 3 : 2;          // parts of q
    static constexpr int NPP = TYPE == KV_BF16 ? 3 : 2;          // parts of the weights
    static constexpr bool QREG = MB == 1 && DP <= 128;           // q's operand fragments in registers
    static constexpr int QW = 2 * NPQ;                           // words of q per lane and 16 columns
    static constexpr int Q_BYTES = QREG ? 0 : MB * (DP / 16) * 32 * QW * 4;
    static constexpr int OPITCH = DP + 4;                        // floats: a store's rows in different banks
    static_assert(NW * ROWS * OPITCH * 4 <= RING, "the warps' outputs are joined in the ring");
    static constexpr int SMEM = RING + Q_BYTES;
    static constexpr int CTAS = THREE ? 3 : SMEM <= 110 * 1024 ? 2 : 1;           // on a SM
    static_assert(!THREE || SMEM <= 70 * 1024, "three CTAs' shared memory");
    static_assert(SMEM <= 222 * 1024, "one CTA's shared memory");
    // 16-byte chunk c of slot r, so that 8 slots' chunks fall in different banks
    static __device__ __forceinline__ int mix(int r) { return NCHUNK >= 8 ? (r & 7) : ((r >> 1) & 3); }
    static __device__ __forceinline__ uint32_t at(int r, int c) { return (uint32_t)(r * PITCH + ((c ^ mix(r)) << 4)); }
};

template <int TYPE, int DP, int MB>
__global__ void __launch_bounds__(AttnGeom<TYPE, DP, MB>::THREADS, AttnGeom<TYPE, DP, MB>::CTAS) attn_decode_kernel(const __grid_constant__ AttnParams p)
{
    using G = AttnGeom<TYPE, DP, MB>;
    constexpr int NW = G::NW, NT = G::THREADS, NPQ = G::NPQ, NPP = G::NPP, QW = G::QW, TILE = G::TILE, SUB = G::SUB;
    constexpr bool PBF = TYPE == KV_BF16;                        // type of the second product's parts
    extern __shared__ __align__(128) uint8_t smem[];
    __shared__ int s_pref[ATT_MAX_SEQ + 1];                      // steps of one head before each sequence
    __shared__ int4 s_warp[NW];
    __shared__ float s_m[NW][G::ROWS], s_l[NW][G::ROWS];
    __shared__ float s_lr[G::ROWS], s_sf[G::ROWS];
    __shared__ int s_at[G::ROWS];                                // the slot of each row's query, -1 for rows past the end
    __shared__ uint32_t s_mask[NW][G::NST];                      // per warp and stage: slots to use
    __shared__ int s_last;
    const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
    const int g = lane >> 2, c4 = lane & 3;
    const uint32_t ring0 = smem_addr(smem);
    const int units = p.n_rb * p.n_kv;
    if (p.score) asm volatile("griddepcontrol.launch_dependents;" ::: "memory");          // attn_score_kernel, which waits for this one's end

    // ---- where this CTA's steps lie.  Every CTA gets `share` steps; where a little
    // more than the equal share lets each CTA stay within one segment (sequence, row
    // block, head), segments are padded to whole shares: a CTA then neither drains
    // its ring nor joins twice.
    auto steps_of = [&](int s) {
        AttnSeq q;
        q.set<TILE, NW>(attn_len(p, s), p);
        return q.n_steps;
    };
    auto prefix = [&](auto &&length) {                                    // s_pref[s] = sum of the lengths before sequence s
        int run = 0;
        for (int s0 = 0; s0 < p.n_seq; s0 += NT) {
            const int s = s0 + tid, n = s < p.n_seq ? length(s) : 0;
            int x = n;
            for (int o = 1; o < 32; o <<= 1) {
                const int y = __shfl_up_sync(0xFFFFFFFFu, x, o);
                if (lane >= o) x += y;
            }
            if (lane == 31) s_warp[warp].x = x;
            __syncthreads();
            int before = run, upto = run;
            for (int w = 0; w < NW; ++w) {
                if (w < warp) before += s_warp[w].x;
                upto += s_warp[w].x;
            }
            if (s < p.n_seq) s_pref[s] = before + x - n;
            run = upto;
            if (s0 + NT < p.n_seq) __syncthreads();
        }
        if (tid == 0) s_pref[p.n_seq] = run;
        __syncthreads();
        return (unsigned)run * (unsigned)units;                           // below 2^31
    };
    unsigned total;
    int share;
    bool padded = false;
    auto choose = [&](int4 n) {                                           // n: CTAs at shares of share .. share + 3
        const int most = (int)gridDim.x, more = n.x * units <= most ? 0 : n.y * units <= most ? 1 : n.z * units <= most ? 2 : n.w * units <= most ? 3 : 4;
        padded = more < 4 && more <= share / 8 + 1;
        if (padded) share += more;
    };
    auto ctas_of = [&](int n) {
        const int k = n - 1;
        return n == 0 ? make_int4(0, 0, 0, 0) : make_int4(div_small(k, share) + 1, div_small(k, share + 1) + 1, div_small(k, share + 2) + 1, div_small(k, share + 3) + 1);
    };
    auto reduce = [&](int4 n) {
        return make_int4(__reduce_add_sync(0xFFFFFFFFu, n.x), __reduce_add_sync(0xFFFFFFFFu, n.y), __reduce_add_sync(0xFFFFFFFFu, n.z), __reduce_add_sync(0xFFFFFFFFu, n.w));
    };
    auto length_of = [&](int n) { return padded ? div_small(n + share - 1, share) * share : n; };
    const bool few = p.n_seq <= 32;                                       // sequences: one a lane, every warp by itself
    int my_len = 0, my_length = 0, my_pref = 0;
    if (few) {
        const int raw = lane < p.n_seq ? __ldg(p.kv_len + lane) : 0;
        if ((raw < 0 || raw > p.max_len) && blockIdx.x == 0) atomicOr(p.err, 16 /* QMV_DEVERR_SEQ_LEN */);
        my_len = min(max(raw, 0), p.max_len);
        AttnSeq q;
        q.set<TILE, NW>(my_len, p);
        const int n = lane < p.n_seq ? q.n_steps : 0;
        total = (unsigned)__reduce_add_sync(0xFFFFFFFFu, n) * (unsigned)units;
        share = total <= gridDim.x ? 1 : (int)((total + gridDim.x - 1) / gridDim.x);
        if (share > 1 && p.n_seq * units <= (int)gridDim.x) choose(reduce(ctas_of(n)));
        my_length = length_of(n);
        int x = my_length;
        for (int o = 1; o < p.n_seq; o <<= 1) {
            const int y = __shfl_up_sync(0xFFFFFFFFu, x, o);
            if (lane >= o) x += y;
        }
        my_pref = x - my_length;
        total = (unsigned)__shfl_sync(0xFFFFFFFFu, x, p.n_seq - 1) * (unsigned)units;
    } else {
        total = prefix([&](int s) {
            const int raw = __ldg(p.kv_len + s);
            if ((raw < 0 || raw > p.max_len) && blockIdx.x == 0) atomicOr(p.err, 16 /* QMV_DEVERR_SEQ_LEN */);
            return steps_of(s);
        });
        share = total <= gridDim.x ? 1 : (int)((total + gridDim.x - 1) / gridDim.x);
        if (share > 1 && p.n_seq * units <= (int)gridDim.x) {
            int4 n = make_int4(0, 0, 0, 0);
            for (int s = tid; s < p.n_seq; s += NT) {
                const int4 c = ctas_of(steps_of(s));
                n = make_int4(n.x + c.x, n.y + c.y, n.z + c.z, n.w + c.w);
            }
            n = reduce(n);
            if (lane == 0) s_warp[warp] = n;
            __syncthreads();
            n = make_int4(0, 0, 0, 0);
#pragma unroll
            for (int w = 0; w < NW; ++w) n = make_int4(n.x + s_warp[w].x, n.y + s_warp[w].y, n.z + s_warp[w].z, n.w + s_warp[w].w);
            __syncthreads();
            choose(n);
        }
        if (padded) total = prefix([&](int s) { return length_of(steps_of(s)); });
    }
    const int x0 = (int)min(total, (unsigned)share * blockIdx.x), x1 = (int)min(total, (unsigned)x0 + share);

    const int nchunk = p.dim * G::EB / 16;
    const uint32_t my_ring = ring0 + (uint32_t)(warp * G::NST * G::STAGE);
    const bool one_page = p.page_size % 16 == 0;                 // 16 slots never leave their page
    constexpr int LPR = G::NCHUNK < 32 ? G::NCHUNK : 32, RPI = 32 / LPR;         // copies: lanes of a slot, slots of a pass
    const int ch = lane % LPR;
    const uint32_t lane_bytes = ch < nchunk ? 16u : 0u;          // chunks behind the head are zeroed by the copy
    const int64_t lane_at = (lane / LPR) * p.slot_stride * G::EB + min(ch, nchunk - 1) * 16, pass_step = RPI * p.slot_stride * G::EB;
    const uint32_t k_row = ((lane >> 3) & 1) * 8 + (lane & 7), k_chunk = lane >> 4;       // ldmatrix addresses: K
    const uint32_t v_row = TYPE == KV_Q8_0 ? k_row : (lane >> 4) * 8 + (lane & 7);        // and V
    const uint32_t v_chunk = TYPE == KV_Q8_0 ? k_chunk : (lane >> 3) & 1;

    for (int x = x0; x < x1;) {
        // ---- the segment: sequence, row block, head, and its steps in this CTA
        int s = 0, len, length, seq0;
        if (few) {
            s = __popc(__ballot_sync(0xFFFFFFFFu, lane < p.n_seq && my_pref * units <= x)) - 1;
            len = __shfl_sync(0xFFFFFFFFu, my_len, s);
            length = __shfl_sync(0xFFFFFFFFu, my_length, s);
            seq0 = __shfl_sync(0xFFFFFFFFu, my_pref, s) * units;
        } else {
            int hi = p.n_seq;
            while (hi - s > 1) {
                const int mid = (s + hi) >> 1;
                if (s_pref[mid] * units <= x) s = mid;
                else hi = mid;
            }
            len = attn_len(p, s);
            length = length_of(steps_of(s));
            seq0 = s_pref[s] * units;
        }
        AttnSeq sq;
        sq.set<TILE, NW>(len, p);
        const int unit = div_small(x - seq0, length);
        const int h = p.n_rb == 1 ? unit : div_small(unit, p.n_rb), rb = unit - h * p.n_rb;        // a head's row blocks follow each other: the cache is in L2
        const int seg0 = seq0 + unit * length, seg1 = seg0 + length;
        const int row0 = rb * G::ROWS;
        const int tile0 = (x - seg0) * NW + warp;                         // this warp's first tile
        const int k0 = x - seg0, k1 = min(min(seg1, x1) - seg0, sq.n_steps);          // steps of the segment
        const int n_steps = max(0, min(k1, (sq.n_tiles - warp + NW - 1) / NW) - k0);      // this warp has a tile in
        const int32_t *tab = p.table + (int64_t)s * p.table_stride;
        x = min(seg1, x1);

        // ---- the warp's q rows (all warps' are the same 8, or those of block `warp`)
        // before the copies, behind which their loads would wait
        constexpr bool Q_EARLY = DP <= 128;
        const int q_nb = G::QREG ? 0 : warp;
        float qraw[Q_EARLY ? DP / 16 : 1][4];
        auto q_row = [&](int row) {
            const int tok = row < p.rows ? attn_token(p, row) : 0;
            return p.q + (int64_t)(s * p.n_tok + tok) * p.q_stride + (int64_t)(h * p.group + (row < p.rows ? row - tok * p.group : 0)) * p.dim;
        };
        auto q_load4 = [&](const float *x, bool row_ok, int ks, float (&f)[4]) {
            const int d0 = ks * 16 + (TYPE == KV_Q8_0 ? 4 * c4 : 2 * c4), d1 = TYPE == KV_Q8_0 ? d0 + 2 : d0 + 8;
            const bool ok = row_ok && ks * 16 < p.dim;
            const float2 a = ok ? __ldg(reinterpret_cast<const float2 *>(x + d0)) : make_float2(0.f, 0.f);
            const float2 b = ok ? __ldg(reinterpret_cast<const float2 *>(x + d1)) : make_float2(0.f, 0.f);
            f[0] = a.x; f[1] = a.y; f[2] = b.x; f[3] = b.y;
        };
        if constexpr (Q_EARLY) {
            const int row = row0 + q_nb * 8 + g;
            const bool ok = q_nb < MB && row < p.rows;
            const float *x = q_row(ok ? row : 0);
#pragma unroll
            for (int ks = 0; ks < DP / 16; ++ks) q_load4(x, ok, ks, qraw[ks]);
        }

        // ---- the ring: page entries one step ahead of the copies
        auto fetch_page = [&](int step) {
            int pg = -1;
            if (step < n_steps) {
                const int j = sq.slot0<TILE>(tile0 + step * NW) + (one_page ? lane & (TILE - 16) : lane & (TILE - 1));
                if (one_page ? j < sq.len : sq.seen(j)) {
                    pg = __ldg(tab + (p.page_shift >= 0 ? j >> p.page_shift : j / p.page_size));
                }
            }
            return pg;
        };
        auto issue = [&](int step, int st, int pg) {
            if (step < n_steps) {
                const uint32_t dst = my_ring + (uint32_t)(st * G::STAGE);
                const int j0 = sq.slot0<TILE>(tile0 + step * NW), j = j0 + (one_page ? lane & (TILE - 16) : lane & (TILE - 1));
                const int o = p.page_shift >= 0 ? j & (p.page_size - 1) : j % p.page_size;
                const long long e = pg * p.page_stride + h * p.head_stride + o * p.slot_stride;
                const bool bad = pg < 0 || pg >= p.n_pages, want = lane < TILE && sq.seen(j0 + lane);
                const uint32_t use = __ballot_sync(0xFFFFFFFFu, want && !bad);
                if (want && bad) atomicOr(p.err, 8 /* QMV_DEVERR_PAGE_ID */);
                if (lane == 0) s_mask[warp][st] = use;
                // rows' addresses: from the first of their 16 where those lie in one page, else from the lane of the row
                static_assert(RPI <= 16, "a pass's rows lie in one group of 16");
                const uint32_t to = dst + (uint32_t)(lane / LPR * G::PITCH);
                if (one_page && use == G::ALL) {
#pragma unroll
                    for (int u = 0; u < SUB; ++u) {
                        const int64_t at = (SUB == 1 ? e : __shfl_sync(0xFFFFFFFFu, e, 16 * u)) * G::EB + lane_at;
                        const uint8_t *k = p.k + at, *v = p.v + at;
#pragma unroll
                        for (int i = 0; i < 16 / RPI; ++i) {
                            const uint32_t x = to + (uint32_t)((16 * u + i * RPI) * G::PITCH) + ((uint32_t)(ch ^ G::mix(i * RPI + lane / LPR)) << 4);
                            cp_async16(x, k, lane_bytes);
                            cp_async16(x + G::KV_BYTES, v, lane_bytes);
                            k += pass_step;
                            v += pass_step;
                        }
                    }
                } else {
                    int64_t e16[SUB];
#pragma unroll
                    for (int u = 0; u < SUB; ++u) e16[u] = SUB == 1 ? e : __shfl_sync(0xFFFFFFFFu, e, 16 * u);
#pragma unroll
                    for (int i = 0; i < TILE / RPI; ++i) {
                        const int r = i * RPI + lane / LPR;
                        const bool ok = ((use >> r) & 1u) && ch < nchunk;
                        int64_t at = (e16[i * RPI / 16] + (r & 15) * p.slot_stride) * G::EB + ch * 16;
                        if (!one_page) at = __shfl_sync(0xFFFFFFFFu, e, r) * G::EB + ch * 16;
                        if (!ok) at = 0;
                        cp_async16(dst + G::at(r, ch), p.k + at, ok ? 16u : 0u);
                        cp_async16(dst + G::KV_BYTES + G::at(r, ch), p.v + at, ok ? 16u : 0u);
                    }
                }
                if constexpr (TYPE == KV_Q8_0) {
                    constexpr int WPR = DP / 64;                          // 4-byte words of a slot's scales
                    const int nw = p.dim / 64;
#pragma unroll
                    for (int i0 = 0; i0 < TILE * WPR; i0 += 32) {
                        const int r = (i0 + lane) / WPR, w = (i0 + lane) % WPR;
                        const long long from = __shfl_sync(0xFFFFFFFFu, e, one_page ? r & (TILE - 16) : r & (TILE - 1));
                        const bool ok = r < TILE && ((use >> r) & 1u) && w < nw;
                        const int64_t at = ok ? (one_page ? from + (r & 15) * p.slot_stride : from) / 16 + w * 4 : 0;
                        if (r < TILE) {
                            cp_async4(dst + 2 * G::KV_BYTES + r * G::SC_PITCH + w * 4, p.ks + at, ok ? 4u : 0u);
                            cp_async4(dst + 2 * G::KV_BYTES + G::SC_BYTES + r * G::SC_PITCH + w * 4, p.vs + at, ok ? 4u : 0u);
                        }
                    }
                }
            }
            cp_commit();
        };
        int pg_next;
        {
            int pg[G::NST];
#pragma unroll
            for (int i = 0; i < G::NST; ++i) pg[i] = fetch_page(i);
#pragma unroll
            for (int i = 0; i < G::NST - 1; ++i) issue(i, i, pg[i]);
            pg_next = pg[G::NST - 1];
        }

        // ---- q as B fragments: lane (g, c4) holds row g's values at columns
        // 2 c4, 2 c4 + 1 and + 8 of every 16 (Q8_0: 4 c4 .. 4 c4 + 3, the order in
        // which its k bytes come).  In registers for 8 narrow rows, else in shared memory.
        uint32_t qr[G::QREG ? DP / 16 : 1][QW];
        const uint32_t qs0 = ring0 + G::RING;
        auto q_block = [&](int nb, auto &&put) {                          // returns the row's factor of the scores
            const int row = row0 + nb * 8 + g;
            const float *x = q_row(row);
            auto load4 = [&](int ks, float (&f)[4]) {
                if constexpr (Q_EARLY) {
                    f[0] = qraw[ks][0]; f[1] = qraw[ks][1]; f[2] = qraw[ks][2]; f[3] = qraw[ks][3];
                } else {
                    q_load4(x, row < p.rows, ks, f);
                }
            };
            float qmul = 1.f, sf = p.scale_log2;
            if constexpr (TYPE != KV_BF16) {
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
                sf *= __uint_as_float((uint32_t)(127 - sh) << 23);
            }
#pragma unroll
            for (int ks = 0; ks < DP / 16; ++ks) {
                float f[4];
                load4(ks, f);
                uint32_t w[QW];
                if constexpr (TYPE == KV_BF16) {
                    split_bf16(f[0], f[1], w[0], w[2], w[4]);
                    split_bf16(f[2], f[3], w[1], w[3], w[5]);
                } else {
                    split_f16(f[0] * qmul, f[1] * qmul, w[0], w[2]);
                    split_f16(f[2] * qmul, f[3] * qmul, w[1], w[3]);
                }
                put(ks, w);
            }
            return sf;
        };
        for (int r = tid; r < G::ROWS; r += NT) s_at[r] = row0 + r < p.rows ? sq.first + attn_token(p, row0 + r) : -1;
        float sf[MB][2];                                                  // of rows 2 c4, 2 c4 + 1 of every block
        if constexpr (G::QREG) {
            const float f = q_block(0, [&](int ks, const uint32_t (&w)[QW]) {
#pragma unroll
                for (int i = 0; i < QW; ++i) qr[ks][i] = w[i];
            });
            sf[0][0] = __shfl_sync(0xFFFFFFFFu, f, 8 * c4);
            sf[0][1] = __shfl_sync(0xFFFFFFFFu, f, 8 * c4 + 4);
            __syncthreads();
        } else {
            for (int nb = warp; nb < MB; nb += NW) {
                const float f = q_block(nb, [&](int ks, const uint32_t (&w)[QW]) {
                    const uint32_t a = qs0 + (uint32_t)((nb * (DP / 16) + ks) * 32 * QW * 4);
                    sts_v4(a + lane * 16, make_uint4(w[0], w[1], w[2], w[3]));
                    if constexpr (QW == 6) sts_v2(a + 512 + lane * 8, make_uint2(w[4], w[5]));
                });
                if (c4 == 0) s_sf[nb * 8 + g] = f;
            }
            __syncthreads();
#pragma unroll
            for (int nb = 0; nb < MB; ++nb) {
                sf[nb][0] = s_sf[nb * 8 + 2 * c4];
                sf[nb][1] = s_sf[nb * 8 + 2 * c4 + 1];
            }
        }
        auto q_frag = [&](int nb, int ks, uint32_t (&w)[QW]) {
            if constexpr (G::QREG) {
#pragma unroll
                for (int i = 0; i < QW; ++i) w[i] = qr[ks][i];
            } else {
                const uint32_t a = qs0 + (uint32_t)((nb * (DP / 16) + ks) * 32 * QW * 4);
                const uint4 u = lds_v4(a + lane * 16);
                w[0] = u.x; w[1] = u.y; w[2] = u.z; w[3] = u.w;
                if constexpr (QW == 6) {
                    const uint2 v = lds_v2(a + 512 + lane * 8);
                    w[4] = v.x; w[5] = v.y;
                }
            }
        };

        float m[MB][2], l[MB][2], acc[MB][DP / 16][4];
#pragma unroll
        for (int nb = 0; nb < MB; ++nb) {
            m[nb][0] = m[nb][1] = -INFINITY;
            l[nb][0] = l[nb][1] = 0.f;
#pragma unroll
            for (int i = 0; i < DP / 16; ++i) acc[nb][i][0] = acc[nb][i][1] = acc[nb][i][2] = acc[nb][i][3] = 0.f;
        }

        int st = 0;
        for (int step = 0; step < n_steps; ++step) {
            cp_wait<G::NST - 2>();
            __syncwarp();
            issue(step + G::NST - 1, st == 0 ? G::NST - 1 : st - 1, pg_next);
            pg_next = fetch_page(step + G::NST);
            const int j0 = sq.slot0<TILE>(tile0 + step * NW);
            const uint32_t buf = my_ring + (uint32_t)(st * G::STAGE), use = s_mask[warp][st];
            if (++st == G::NST) st = 0;
            // -- scores: this lane's are slots g (values 0, 1) and g + 8 (2, 3), rows 2 c4 and 2 c4 + 1 of every block
            float sc[MB][SUB][4];
            if constexpr (TYPE == KV_Q8_0) {
#pragma unroll
                for (int nb = 0; nb < MB; ++nb)
#pragma unroll
                    for (int u = 0; u < SUB; ++u) sc[nb][u][0] = sc[nb][u][1] = sc[nb][u][2] = sc[nb][u][3] = 0.f;
#pragma unroll
                for (int b = 0; b < DP / 32; ++b)
#pragma unroll
                    for (int u = 0; u < SUB; ++u) {
                        uint32_t r[4], a[2][4];
                        ldsm4(r, buf + G::at(16 * u + k_row, 2 * b + k_chunk));
#pragma unroll
                        for (int k2 = 0; k2 < 2; ++k2) {
                            i8_to_f16(r[2 * k2], a[k2][0], a[k2][2]);
                            i8_to_f16(r[2 * k2 + 1], a[k2][1], a[k2][3]);
                        }
                        const uint32_t sa = buf + 2 * G::KV_BYTES + 2 * b + (16 * u + g) * G::SC_PITCH;
                        const float d0 = half_bits_to_float(lds_u16(sa)), d1 = half_bits_to_float(lds_u16(sa + 8 * G::SC_PITCH));
#pragma unroll
                        for (int nb = 0; nb < MB; ++nb) {
                            float hi[4], lo[4];
                            uint32_t q[QW];
                            q_frag(nb, 2 * b, q);
                            mma_16_0<false>(hi, a[0], q[0], q[1]);
                            mma_16_0<false>(lo, a[0], q[2], q[3]);
                            q_frag(nb, 2 * b + 1, q);
                            mma_16<false>(hi, a[1], q[0], q[1]);
                            mma_16<false>(lo, a[1], q[2], q[3]);
                            add2(hi[0], hi[1], lo[0], lo[1]);
                            add2(hi[2], hi[3], lo[2], lo[3]);
                            fma2(sc[nb][u][0], sc[nb][u][1], hi[0], hi[1], d0);
                            fma2(sc[nb][u][2], sc[nb][u][3], hi[2], hi[3], d1);
                        }
                    }
            } else {
                constexpr int PAR = MB * SUB == 1 ? 2 : 1;                // chains per part: their sums wait on the one before
                float a[MB][SUB][NPQ][PAR][4];
#pragma unroll
                for (int ks = 0; ks < DP / 16; ++ks) {
                    uint32_t r[SUB][4];
#pragma unroll
                    for (int u = 0; u < SUB; ++u) ldsm4(r[u], buf + G::at(16 * u + k_row, 2 * ks + k_chunk));
#pragma unroll
                    for (int nb = 0; nb < MB; ++nb) {
                        uint32_t q[QW];
                        q_frag(nb, ks, q);
#pragma unroll
                        for (int i = 0; i < NPQ; ++i)
#pragma unroll
                            for (int u = 0; u < SUB; ++u) {
                                if (ks < PAR) mma_16_0<TYPE == KV_BF16>(a[nb][u][i][ks % PAR], r[u], q[2 * i], q[2 * i + 1]);
                                else mma_16<TYPE == KV_BF16>(a[nb][u][i][ks % PAR], r[u], q[2 * i], q[2 * i + 1]);
                            }
                    }
                }
#pragma unroll
                for (int nb = 0; nb < MB; ++nb)
#pragma unroll
                    for (int u = 0; u < SUB; ++u)
#pragma unroll
                        for (int e = 0; e < 4; ++e) {
                            float t = 0.f;
#pragma unroll
                            for (int i = NPQ - 1; i >= 0; --i) t += PAR == 2 ? a[nb][u][i][0][e] + a[nb][u][i][PAR - 1][e] : a[nb][u][i][0][e];
                            sc[nb][u][e] = t;
                        }
            }
#pragma unroll
            for (int nb = 0; nb < MB; ++nb)
#pragma unroll
                for (int u = 0; u < SUB; ++u)
#pragma unroll
                    for (int e = 0; e < 4; ++e) sc[nb][u][e] *= sf[nb][e & 1];
            const bool mixed = p.n_tok > 1 && (use != G::ALL || !sq.by_all<TILE>(j0, p));
            if (mixed) {
#pragma unroll
                for (int nb = 0; nb < MB; ++nb)
#pragma unroll
                    for (int u = 0; u < SUB; ++u)
#pragma unroll
                        for (int e = 0; e < 4; ++e) {
                            const int jj = 16 * u + g + (e >> 1) * 8;
                            if (!((use >> jj) & 1u) || !attn_sees(p, s_at[nb * 8 + 2 * c4 + (e & 1)], j0 + jj)) sc[nb][u][e] = -INFINITY;
                        }
            } else if (use != G::ALL) {                                   // one query: what it sees was loaded
#pragma unroll
                for (int u = 0; u < SUB; ++u) {
                    const bool u0 = (use >> (16 * u + g)) & 1u, u1 = (use >> (16 * u + g + 8)) & 1u;
#pragma unroll
                    for (int nb = 0; nb < MB; ++nb) {
                        if (!u0) sc[nb][u][0] = sc[nb][u][1] = -INFINITY;
                        if (!u1) sc[nb][u][2] = sc[nb][u][3] = -INFINITY;
                    }
                }
            }
            if (p.score) {
                float *raw = p.raw + ((int64_t)(s * p.n_kv + h) * p.raw_stride + j0 + g) * p.raw_rows + row0 + 2 * c4;
#pragma unroll
                for (int nb = 0; nb < MB; ++nb)
                    if (row0 + nb * 8 + 2 * c4 < p.raw_rows) {
#pragma unroll
                        for (int u = 0; u < SUB; ++u) {
                            *reinterpret_cast<float2 *>(raw + nb * 8 + 16 * u * (int64_t)p.raw_rows) = make_float2(sc[nb][u][0], sc[nb][u][1]);
                            *reinterpret_cast<float2 *>(raw + nb * 8 + (16 * u + 8) * (int64_t)p.raw_rows) = make_float2(sc[nb][u][2], sc[nb][u][3]);
                        }
                    }
            }
            // -- the running maximum: moved only when a score is well above it
            float mx[MB][2];
            bool up = false;
#pragma unroll
            for (int nb = 0; nb < MB; ++nb)
#pragma unroll
                for (int e = 0; e < 2; ++e) {
                    mx[nb][e] = fmaxf(sc[nb][0][e], sc[nb][0][e + 2]);
#pragma unroll
                    for (int u = 1; u < SUB; ++u) mx[nb][e] = fmaxf(mx[nb][e], fmaxf(sc[nb][u][e], sc[nb][u][e + 2]));
                    up |= mx[nb][e] > m[nb][e] + attn_slack(TYPE);
                }
            if (__any_sync(0xFFFFFFFFu, up)) {
#pragma unroll
                for (int nb = 0; nb < MB; ++nb) {
                    float f[2];
#pragma unroll
                    for (int e = 0; e < 2; ++e) {
                        float top = mx[nb][e];
                        top = fmaxf(top, __shfl_xor_sync(0xFFFFFFFFu, top, 4));
                        top = fmaxf(top, __shfl_xor_sync(0xFFFFFFFFu, top, 8));
                        top = fmaxf(top, __shfl_xor_sync(0xFFFFFFFFu, top, 16));
                        const float mn = fmaxf(m[nb][e], top);
                        f[e] = m[nb][e] == mn ? 1.f : ex2(m[nb][e] - mn);         // m = -inf: 0
                        m[nb][e] = mn;
                        l[nb][e] *= f[e];
                    }
#pragma unroll
                    for (int i = 0; i < DP / 16; ++i) {
                        mul2(acc[nb][i][0], acc[nb][i][1], f[0], f[1]);
                        mul2(acc[nb][i][2], acc[nb][i][3], f[0], f[1]);
                    }
                }
            }
            // -- the weights
#pragma unroll
            for (int nb = 0; nb < MB; ++nb)
#pragma unroll
                for (int e = 0; e < 2; ++e) {
                    const float mref = (m[nb][e] == -INFINITY ? 0.f : m[nb][e]) - p.l_shift;
#pragma unroll
                    for (int u = 0; u < SUB; ++u) {
                        sc[nb][u][e] = ex2(sc[nb][u][e] - mref);
                        sc[nb][u][e + 2] = ex2(sc[nb][u][e + 2] - mref);
                        l[nb][e] += sc[nb][u][e] + sc[nb][u][e + 2];
                    }
                }
            // -- output += values x weights
            const uint32_t va = buf + G::KV_BYTES;
            if constexpr (TYPE == KV_Q8_0) {
                // weights transposed to lane (row g, slots 2 c4, 2 c4 + 1 and + 8) as halves of 16 bits, then scaled per block of 32
                float pw[MB][SUB][4];
#pragma unroll
                for (int nb = 0; nb < MB; ++nb)
#pragma unroll
                    for (int u = 0; u < SUB; ++u)
#pragma unroll
                        for (int i = 0; i < 2; ++i) {
                            const uint32_t u0 = __float_as_uint(sc[nb][u][2 * i]), u1 = __float_as_uint(sc[nb][u][2 * i + 1]);
                            const uint32_t hi = movm_t(__byte_perm(u0, u1, 0x7632)), lo = movm_t(__byte_perm(u0, u1, 0x5410));
                            pw[nb][u][2 * i] = __uint_as_float(__byte_perm(lo, hi, 0x5410));
                            pw[nb][u][2 * i + 1] = __uint_as_float(__byte_perm(lo, hi, 0x7632));
                        }
#pragma unroll
                for (int b = 0; b < DP / 32; ++b) {
                    const uint32_t sa = buf + 2 * G::KV_BYTES + G::SC_BYTES + 2 * b;
                    float d[SUB][4];
#pragma unroll
                    for (int u = 0; u < SUB; ++u)
#pragma unroll
                        for (int i = 0; i < 4; ++i) {
                            d[u][i] = half_bits_to_float(lds_u16(sa + (16 * u + 2 * c4 + (i & 1) + (i >> 1) * 8) * G::SC_PITCH));
                            // NaN or infinity of a slot that a row may not see: its weight is 0
                            if (mixed && !(fabsf(d[u][i]) < INFINITY)) d[u][i] = 0.f;
                        }
                    uint32_t a[SUB][2][4];
#pragma unroll
                    for (int u = 0; u < SUB; ++u) {
                        uint32_t r[4];
                        ldsm4t(r, va + G::at(16 * u + v_row, 2 * b + v_chunk));
#pragma unroll
                        for (int k2 = 0; k2 < 2; ++k2) {                  // rows g and g + 8: dims 2 g and 2 g + 1 of 16
                            i8_to_f16<0x4240, 0x4341>(r[2 * k2], a[u][k2][0], a[u][k2][1]);
                            i8_to_f16<0x4240, 0x4341>(r[2 * k2 + 1], a[u][k2][2], a[u][k2][3]);
                        }
                    }
#pragma unroll
                    for (int nb = 0; nb < MB; ++nb) {
                        uint32_t pb[SUB][2][2];
                        float pd[SUB][4], top = 0.f;
#pragma unroll
                        for (int u = 0; u < SUB; ++u) {
#pragma unroll
                            for (int i = 0; i < 4; ++i) pd[u][i] = pw[nb][u][i];
                            mul2(pd[u][0], pd[u][1], d[u][0], d[u][1]);
                            mul2(pd[u][2], pd[u][3], d[u][2], d[u][3]);
#pragma unroll
                            for (int i = 0; i < 4; ++i) top = fmaxf(top, fabsf(pd[u][i]));
                        }
                        // the row's products times the power of two that brings the largest below 2^15: what the parts
                        // leave of the others is at most 2^-39 of it, whatever the scales of slots without weight are
                        top = fmaxf(top, __shfl_xor_sync(0xFFFFFFFFu, top, 1));
                        top = fmaxf(top, __shfl_xor_sync(0xFFFFFFFFu, top, 2));
                        const uint32_t ex = max(__float_as_uint(top) & 0x7F800000u, 15u << 23);
                        const float down = __uint_as_float((268u << 23) - ex), own = __uint_as_float(ex - (14u << 23));
                        const float back0 = __shfl_sync(0xFFFFFFFFu, own, 8 * c4), back1 = __shfl_sync(0xFFFFFFFFu, own, 8 * c4 + 4);
#pragma unroll
                        for (int u = 0; u < SUB; ++u) {
                            mul2(pd[u][0], pd[u][1], down, down);
                            mul2(pd[u][2], pd[u][3], down, down);
                            split_f16(pd[u][0], pd[u][1], pb[u][0][0], pb[u][1][0]);
                            split_f16(pd[u][2], pd[u][3], pb[u][0][1], pb[u][1][1]);
                        }
#pragma unroll
                        for (int k2 = 0; k2 < 2; ++k2) {
                            float t[4];
                            mma_16_0<false>(t, a[0][k2], pb[0][1][0], pb[0][1][1]);
#pragma unroll
                            for (int u = 1; u < SUB; ++u) mma_16<false>(t, a[u][k2], pb[u][1][0], pb[u][1][1]);
#pragma unroll
                            for (int u = 0; u < SUB; ++u) mma_16<false>(t, a[u][k2], pb[u][0][0], pb[u][0][1]);
                            fma22(acc[nb][2 * b + k2][0], acc[nb][2 * b + k2][1], t[0], t[1], back0, back1);
                            fma22(acc[nb][2 * b + k2][2], acc[nb][2 * b + k2][3], t[2], t[3], back0, back1);
                        }
                    }
                }
            } else {
                uint32_t pb[MB][SUB][NPP][2];
#pragma unroll
                for (int nb = 0; nb < MB; ++nb)
#pragma unroll
                    for (int u = 0; u < SUB; ++u)
#pragma unroll
                        for (int i = 0; i < 2; ++i) {
                            uint32_t w[3];
                            if constexpr (TYPE == KV_F16) split_f16<(int)ATT_F16_LEFT>(sc[nb][u][2 * i], sc[nb][u][2 * i + 1], w[0], w[1]);
                            else split_bf16(sc[nb][u][2 * i], sc[nb][u][2 * i + 1], w[0], w[1], w[2]);
#pragma unroll
                            for (int k = 0; k < NPP; ++k) pb[nb][u][k][i] = movm_t(w[k]);
                        }
                auto chain = [&](float (&t)[4], const uint32_t (&r)[SUB][4], int nb, int k0, int k1) {     // parts k0 down to k1
                    mma_16_0<PBF>(t, r[0], pb[nb][0][k0][0], pb[nb][0][k0][1]);
#pragma unroll
                    for (int k = k0; k >= k1; --k)
#pragma unroll
                        for (int u = 0; u < SUB; ++u)
                            if (k < k0 || u > 0) mma_16<PBF>(t, r[u], pb[nb][u][k][0], pb[nb][u][k][1]);
                };
                auto product = [&](float (&t)[4], const uint32_t (&r)[SUB][4], int nb) {
                    if constexpr (TYPE == KV_F16) {
                        float left[4];
                        chain(left, r, nb, 1, 1);
                        chain(t, r, nb, 0, 0);
                        fma2(t[0], t[1], left[0], left[1], 1.f / ATT_F16_LEFT);
                        fma2(t[2], t[3], left[2], left[3], 1.f / ATT_F16_LEFT);
                    } else {
                        chain(t, r, nb, NPP - 1, 0);
                    }
                };
                auto values = [&](auto &&each) {
#pragma unroll
                    for (int i = 0; i < DP / 16; ++i) {
                        uint32_t r[SUB][4];
#pragma unroll
                        for (int u = 0; u < SUB; ++u) {
                            ldsm4t(r[u], va + G::at(16 * u + v_row, 2 * i + v_chunk));
#pragma unroll
                            for (int k = 0; k < 4; ++k) each(r[u][k]);
                        }
#pragma unroll
                        for (int nb = 0; nb < MB; ++nb) {
                            float t[4];
                            product(t, r, nb);
                            add2(acc[nb][i][0], acc[nb][i][1], t[0], t[1]);
                            add2(acc[nb][i][2], acc[nb][i][3], t[2], t[3]);
                        }
                    }
                };
                if (mixed) values([](uint32_t &x) { x = finite_pair<TYPE>(x); });
                else values([](uint32_t &) {});
            }
        }
        cp_wait<0>();
#pragma unroll
        for (int nb = 0; nb < MB; ++nb)
#pragma unroll
            for (int e = 0; e < 2; ++e) {
                float t = l[nb][e];
                t += __shfl_xor_sync(0xFFFFFFFFu, t, 4);
                t += __shfl_xor_sync(0xFFFFFFFFu, t, 8);
                t += __shfl_xor_sync(0xFFFFFFFFu, t, 16);
                if (g == 0) {
                    s_m[warp][nb * 8 + 2 * c4 + e] = m[nb][e];
                    s_l[warp][nb * 8 + 2 * c4 + e] = t;
                }
            }
        __syncthreads();                                                  // the ring is free

        // ---- join the warps' parts (in the ring); one without a tile has m = -inf, l = 0, o = 0
        float *so = reinterpret_cast<float *>(smem);
#pragma unroll
        for (int nb = 0; nb < MB; ++nb)
#pragma unroll
            for (int e = 0; e < 2; ++e) {
                const int r = nb * 8 + 2 * c4 + e;
                float mr = s_m[0][r];
#pragma unroll
                for (int w = 1; w < NW; ++w) mr = fmaxf(mr, s_m[w][r]);
                const float f = m[nb][e] == mr ? 1.f : ex2(m[nb][e] - mr);
                float *ow = so + (size_t)(warp * G::ROWS + r) * G::OPITCH;
#pragma unroll
                for (int i = 0; i < DP / 16; ++i) {
                    const float v0 = acc[nb][i][e] * f, v1 = acc[nb][i][e + 2] * f;
                    if constexpr (TYPE == KV_Q8_0) {
                        *reinterpret_cast<float2 *>(ow + 16 * i + 2 * g) = make_float2(v0, v1);
                    } else {
                        ow[16 * i + g] = v0;
                        ow[16 * i + 8 + g] = v1;
                    }
                }
            }
        const int nrow = min(G::ROWS, p.rows - row0);
        auto out_row = [&](int r) {
            const int t = s_at[r] - sq.first;
            return p.out + (int64_t)(s * p.n_tok + t) * p.out_stride + (int64_t)(h * p.group + row0 + r - t * p.group) * p.dim;
        };
        auto put_stats = [&](int r, float mr, float lr) {
            if (p.score) *reinterpret_cast<float2 *>(p.stats + 2 * ((int64_t)(s * p.n_kv + h) * p.raw_rows + row0 + r)) = make_float2(mr - p.l_shift, lr != 0.f ? __fdiv_rn(1.f, lr) : 0.f);
        };
        const bool whole = seg0 >= x0 && seg1 <= x1;
        const int slot = 2 * blockIdx.x + (seg0 >= x0 ? 1 : 0);
        if (tid < nrow) {
            float mr = s_m[0][tid], lr = 0.f;
#pragma unroll
            for (int w = 1; w < NW; ++w) mr = fmaxf(mr, s_m[w][tid]);
#pragma unroll
            for (int w = 0; w < NW; ++w) lr += s_m[w][tid] == mr ? s_l[w][tid] : s_l[w][tid] * ex2(s_m[w][tid] - mr);
            s_lr[tid] = lr;
            if (whole) put_stats(tid, mr, lr);
            else __stcg(reinterpret_cast<float2 *>(p.part_ml) + (int64_t)slot * G::ROWS + tid, make_float2(mr, lr));
        }
        __syncthreads();
        constexpr int D4 = DP / 4;                                        // a thread takes 4 dims of a row
        auto put = [&](int r, int d, float4 v, float lr) {
            float *o = out_row(r) + 4 * d;
            const float f = lr != 0.f ? __frcp_rn(lr) : 0.f;
            o[0] = v.x * f;
            o[1] = v.y * f;
            o[2] = v.z * f;
            o[3] = v.w * f;
        };
        for (int i = tid; i < nrow * D4; i += NT) {
            const int r = i / D4, d = i % D4;
            if (4 * d >= p.dim) continue;
            float4 v = make_float4(0.f, 0.f, 0.f, 0.f);
#pragma unroll
            for (int w = 0; w < NW; ++w) {
                const float4 u = *reinterpret_cast<const float4 *>(so + (size_t)(w * G::ROWS + r) * G::OPITCH + 4 * d);
                v.x += u.x; v.y += u.y; v.z += u.z; v.w += u.w;
            }
            if (whole) put(r, d, v, s_lr[r]);
            else __stcg(reinterpret_cast<float4 *>(p.part_o + ((int64_t)slot * G::ROWS + r) * p.dim) + d, v);
        }
        if (!whole) {
            // ---- the last CTA of the segment joins its parts, in CTA order
            const int cta0 = div_small(seg0, share), cta1 = div_small(seg1 - 1, share), n = cta1 - cta0 + 1;
            __syncthreads();
            if (tid == 0) s_last = atomic_inc_acq_rel(p.counters + cta0) == (unsigned)(n - 1);
            __syncthreads();
            if (s_last) {
                if (tid == 0) p.counters[cta0] = 0u;
                // part c: the second of CTA cta0's two slots for c = 0, else the first of CTA cta0 + c's
                const int64_t po_step = (int64_t)G::ROWS * p.dim;
                auto join = [&](auto in_flight, int r, int d, int c_first, int c_step, float4 &v, float &mr, float &lr) {
                    constexpr int CH = decltype(in_flight)::value;        // parts in flight
                    const float2 *ml = reinterpret_cast<const float2 *>(p.part_ml) + (int64_t)2 * cta0 * G::ROWS + r;
                    const float *po = p.part_o + ((int64_t)2 * cta0 * G::ROWS + r) * p.dim + 4 * d;
                    v = make_float4(0.f, 0.f, 0.f, 0.f);
                    mr = -INFINITY;
                    lr = 0.f;
                    for (int c0 = c_first; c0 < n; c0 += CH * c_step) {
                        float2 q[CH];
                        float4 u[CH];
#pragma unroll
                        for (int k = 0; k < CH; ++k) {
                            const int c = c0 + k * c_step, sl = c == 0 ? 1 : 2 * c;
                            q[k] = make_float2(-INFINITY, 0.f);
                            u[k] = make_float4(0.f, 0.f, 0.f, 0.f);
                            if (c < n) {
                                q[k] = __ldcg(ml + sl * G::ROWS);
                                u[k] = __ldcg(reinterpret_cast<const float4 *>(po + sl * po_step));
                            }
                        }
                        float mn = mr;
#pragma unroll
                        for (int k = 0; k < CH; ++k) mn = fmaxf(mn, q[k].x);
                        const float f0 = mr == mn ? 1.f : ex2(mr - mn);
                        v.x *= f0; v.y *= f0; v.z *= f0; v.w *= f0;
                        lr *= f0;
                        mr = mn;
#pragma unroll
                        for (int k = 0; k < CH; ++k) {
                            const float f = q[k].x == mn ? 1.f : ex2(q[k].x - mn);
                            lr += f * q[k].y;
                            v.x += f * u[k].x; v.y += f * u[k].y; v.z += f * u[k].z; v.w += f * u[k].w;
                        }
                    }
                };
                float4 v;
                float mr, lr;
                if (nrow * D4 <= NT / 2 && n > 16) {                      // many parts of few rows: two threads take every other one
                    float4 *sv = reinterpret_cast<float4 *>(smem);
                    float2 *sm = reinterpret_cast<float2 *>(smem + NT / 2 * sizeof(float4));
                    const int half = tid / (NT / 2), i = tid % (NT / 2), r = i / D4, d = i % D4;
                    const bool in = i < nrow * D4 && 4 * d < p.dim;
                    if (in) {
                        join(std::integral_constant<int, 16>(), r, d, half, 2, v, mr, lr);
                        if (half) {
                            sv[i] = v;
                            sm[i] = make_float2(mr, lr);
                        }
                    }
                    __syncthreads();
                    if (in && !half) {
                        const float4 w = sv[i];
                        const float2 q = sm[i];
                        const float mn = fmaxf(mr, q.x), f = mr == mn ? 1.f : ex2(mr - mn), g2 = q.x == mn ? 1.f : ex2(q.x - mn);
                        lr = f * lr + g2 * q.y;
                        put(r, d, make_float4(f * v.x + g2 * w.x, f * v.y + g2 * w.y, f * v.z + g2 * w.z, f * v.w + g2 * w.w), lr);
                        if (d == 0) put_stats(r, mn, lr);
                    }
                } else {
                    for (int i = tid; i < nrow * D4; i += NT) {
                        const int r = i / D4, d = i % D4;
                        if (4 * d >= p.dim) continue;
                        if (n <= 8) join(std::integral_constant<int, 8>(), r, d, 0, 1, v, mr, lr);
                        else join(std::integral_constant<int, 16>(), r, d, 0, 1, v, mr, lr);
                        put(r, d, v, lr);
                        if (d == 0) put_stats(r, mr, lr);
                    }
                }
            }
        }
        __syncthreads();                                                  // the ring is refilled next
    }
}

// score[s][h][j] (+)= sum over the rows of 2^(s_j - m) / l, from the raw scores
// and the joined (m, l) that attn_decode_kernel left in the workspace.  Two
// slots a thread, rows in order.  It starts while that kernel ends, and what does
// not come from it is read before the wait.  Plain loads: a slot's rows lie in few
// lines, which the row by row reads find in L1.
constexpr int ATT_SCORE_THREADS = 256, ATT_SCORE_SLOTS = 2 * ATT_SCORE_THREADS;

static __global__ void __launch_bounds__(ATT_SCORE_THREADS) attn_score_kernel(const __grid_constant__ AttnParams p)
{
    const int s = blockIdx.z, h = blockIdx.y;
    AttnSeq sq;
    sq.set<ATT_MIN_TILE, ATT_MIN_NW>(attn_len(p, s), p);
    const int64_t sh = (int64_t)s * p.n_kv + h;
    const float4 *st = reinterpret_cast<const float4 *>(p.stats + 2 * sh * p.raw_rows);      // of two rows
    bool waited = false;
    for (int64_t base = (int64_t)blockIdx.x * ATT_SCORE_SLOTS; base < sq.len; base += (int64_t)gridDim.x * ATT_SCORE_SLOTS) {
        int j[2];
        bool in[2];
        float v[2], given[2] = {0.f, 0.f};
#pragma unroll
        for (int k = 0; k < 2; ++k) {
            j[k] = (int)min(base + k * ATT_SCORE_THREADS + threadIdx.x, (int64_t)sq.len);
            in[k] = sq.seen(j[k]);
            v[k] = in[k] && j[k] < sq.first ? p.score[sh * p.score_stride + j[k]] : 0.f;
        }
        if (!waited) asm volatile("griddepcontrol.wait;" ::: "memory");   // attn_decode_kernel is done
        waited = true;
#pragma unroll 4
        for (int r = 0; r < p.rows; r += 2) {
            const float4 w = st[r / 2];
#pragma unroll
            for (int k = 0; k < 2; ++k) {
                const float2 u = in[k] ? *reinterpret_cast<const float2 *>(p.raw + (sh * p.raw_stride + j[k]) * p.raw_rows + r) : make_float2(0.f, 0.f);
                given[k] += w.y != 0.f ? ex2(u.x - w.x) * w.y : 0.f;
                if (r + 1 < p.rows) given[k] += w.w != 0.f ? ex2(u.y - w.z) * w.w : 0.f;
            }
        }
#pragma unroll
        for (int k = 0; k < 2; ++k)
            if (in[k]) p.score[sh * p.score_stride + j[k]] = v[k] + given[k];
    }
    if (!waited) asm volatile("griddepcontrol.wait;" ::: "memory");
}

// One launch of the instance that holds p.dim and p.mb, on as many CTAs as run at
// once and have a step by the longest lengths.
template <int TYPE, int DP, int MB>
static cudaError_t launch_attn_mb(const AttnParams &p, int sms, int64_t steps, cudaStream_t st)
{
    using G = AttnGeom<TYPE, DP, MB>;
    static SmemCfg configured;
    const int most = sms * G::CTAS < ATT_MAX_CTAS ? sms * G::CTAS : ATT_MAX_CTAS;
    return launch_with(attn_decode_kernel<TYPE, DP, MB>, configured, p, dim3((unsigned)(steps < most ? steps : most)), G::SMEM, st, false, false, G::THREADS);
}

template <int TYPE>
static cudaError_t launch_attn(const AttnParams &p, int sms, int64_t steps, cudaStream_t st)
{
    if constexpr (TYPE != KV_Q8_0)
        if (p.dim <= 32) return p.mb == 1 ? launch_attn_mb<TYPE, 32, 1>(p, sms, steps, st) : launch_attn_mb<TYPE, 32, 2>(p, sms, steps, st);
    if (p.dim <= 64) return p.mb == 1 ? launch_attn_mb<TYPE, 64, 1>(p, sms, steps, st) : launch_attn_mb<TYPE, 64, 2>(p, sms, steps, st);
    if (p.dim <= 128) return p.mb == 1 ? launch_attn_mb<TYPE, 128, 1>(p, sms, steps, st) : launch_attn_mb<TYPE, 128, 2>(p, sms, steps, st);
    return p.mb == 1 ? launch_attn_mb<TYPE, 256, 1>(p, sms, steps, st) : launch_attn_mb<TYPE, 256, 2>(p, sms, steps, st);
}

}  // namespace qmv
