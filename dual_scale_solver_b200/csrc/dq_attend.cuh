// dq_attend.cuh — attention of few query rows over the 4-bit cache.
//
//   out = softmax(scale q . k_hat) v_hat,  k_hat = c_k s_k,  v_hat = c_v s_v
//
// For single tokens (and drafts of a few) the work is the streaming of codes:
// each code byte is used for at most 8 query rows.  Tensor-core products
// keep the arithmetic per code low enough to stay near the memory's pace:
//
//  S^T = K Q^T   A = 16 tokens x 16 channels of codes as fp16 (exact), B = 8
//                query rows as fp16, scaled by a power of two per row (exact
//                but for elements 2^-38 below the row's largest); float32
//                accumulation per group of G channels, then one multiply-add
//                with the group's scale.
//  O^T = V^T P^T A = 16 channels x 16 tokens of codes as fp16, B = the
//                probabilities times the tokens' group scales, fp16 both and
//                their product.  With 2^E the largest value scale of a tile,
//                scales enter as s 2^(6 - E) (below 2^7), probabilities as p
//                2^(E + 7 .. 9) against a running maximum that holds E, so
//                the products stay below 2^16 - 2^8 and what lies 2^-28 below
//                the largest is lost; roundings 2^-12 each, below the output
//                type's 2^-9.
//
// A query row is one (token, head of the group) pair, so the g heads of a
// group share every code.  The probabilities pass from the layout of the
// first product's result to the second's operand with movmatrix.
//
// Work: (sequence, cache head, tile of 8 rows) segments of 256-token units
// (whole ones in batches of short sequences), numbered through the batch; CTA i of n
// takes units [U i / n, U (i+1) / n) (found by a scan over the sequences'
// lengths on the device, so lengths may differ freely and the call needs no
// host copy of them).  A segment that one CTA covers is written at once; the
// pieces of one that is cut go to the workspace, at most two per CTA, and a
// second kernel joins them in order.
// A warp takes 32 tokens at a time through its own cp.async ring.
//
// Measured (64 query over 8 cache heads, D = 128): 16 sequences of 32768,
// MXFP4, 103 us, 4.1 TB/s; 32 of 8192 (32 query heads), INT4 G 64, 55 us, 3.4
// TB/s.  No unit is full: issue 65% of the slots (16 warps a SM of 128
// registers each, 511 warp instructions per 32 positions), the pipe of
// conversions 57%, products 24%; the products alone would take 60 us of the
// first, the codes 65 at the memory's rate.  A call of one token over 511
// positions (3 heads of 64) takes 6.3 us, the latency of two steps.
#pragma once

#include <cuda_runtime.h>

#include "dq_kv.cuh"

namespace dq {

constexpr int kAttWarps = 8;
constexpr int kAttThreads = 32 * kAttWarps;
constexpr int kAttTile = 32;                       // tokens per warp step
constexpr int kAttUnit = kAttTile * kAttWarps;     // tokens per step of a CTA, and per unit of work
// But where every sequence has few steps, segments are whole: up to
// kAttWhole steps, or half of that where there are not enough segments to give
// every second SM one.  A step takes 1 to 1.5 us, writing and joining pieces 2 to
// 3.  One token each, 8 heads of 128, us, cut against whole: 1 sequence of 500
// positions 8.5, 7.0, of 1000 8.8, 9.8; 4 of 1000 8.9, 12.0; 16 of 1000 14.8, 13.5;
// 32 17.1, 13.9; 128 47.4, 45.6; 16 of 1500 14.6, 14.8; 48 26.3, 32.5.
constexpr int kAttWhole = 4;
__host__ __device__ inline int att_whole(int64_t segments) {
    return (segments >= 74 ? kAttWhole : kAttWhole / 2) * kAttUnit;
}
constexpr int kAttCtas = 2 * 148;

// Sequences of up to 32 query rows (new tokens x heads of a group) are this
// file's, longer ones the tcgen05 kernel's, which takes 256 rows at a time.
// 8 sequences of 8 cache heads, D = 128: 32 rows each over 4001 positions 31
// us (MXFP4) and 35 (NVFP4) here against 40 there, over 16000 87 and 101
// against 91 and 97; 16 rows 22 to 69 us against 39 to 96.
constexpr int kAttFew = 32;
enum { ATT_FEW = 1, ATT_MANY = 2 };

// The kernels of a call; which of two takes a sequence is decided on the
// device, where its length is known.  Calls of a token per sequence in the mean
// (or fewer) are single tokens: the other kernel's launch is saved.  A long
// sequence among empty ones is then taken in tiles of 8 rows.  us, 32 query
// heads over 8 of 128, MXFP4, this kernel alone against both: 32 single tokens
// over 200 positions 7.9, 9.3; 128 over 2000 80.4, 82.3; 50 over 2000 with a
// prompt of 200 tokens and 205 empty sequences 67.0, 65.4 (the prompt over 4000:
// 142, 134); with a prompt of 1000 over 4000 and 1049 empty ones 533, 151.
inline int attend_kernels(int64_t tokens, int32_t q_heads, int32_t heads, int32_t seqs) {
    const int64_t group = q_heads / heads;
    if (tokens * group <= kAttFew) return ATT_FEW;
    if (seqs == 1 || group > kAttFew) return ATT_MANY;
    return tokens <= seqs ? ATT_FEW : ATT_FEW | ATT_MANY;
}

// What CTA i leaves for the joining kernel: the segment that starts (and
// does not end) in its share.
struct AttMeta {
    int last;               // the last share with a piece of the segment
    int rows;               // of the segment; 0: nothing to join
    int row0;               // its first row in the sequence
    int head;
    int token0;             // the sequence's first token row
};

struct AttArgs {
    const uint16_t *q;
    int64_t q_token, q_head;
    uint16_t *out;
    int64_t out_token, out_head;
    int64_t tokens;
    int group;              // query heads per cache head
    int few;                // sequences of up to so many rows are dq_attend.cuh's
    float scale_log2;       // scale * log2(e)
    uint32_t k16;           // 16
    int causal;
    dq_kv_cache cache;
    dq_kv_batch batch;
    float *part;            // [2 n][rows][D]
    float2 *part_ml;        // [2 n][rows]  (running maximum, sum)
    AttMeta *meta;          // [n]
    unsigned int *status;
};

struct AttSpan {            // a sequence's segments and units
    int qt;                 // row tiles
    int kvt;                // units per segment
    long long units;
};

template <int ROWS>
__device__ __forceinline__ AttSpan att_span(const AttArgs &A, const KvSeq &s, int unit) {
    AttSpan a;
    const long long rows = (long long)s.n * A.group;
    a.qt = rows > A.few ? 0 : (int)((rows + ROWS - 1) / ROWS);
    a.kvt = max(1, (s.len + unit - 1) / unit);
    a.units = (long long)a.qt * A.cache.heads * a.kvt;
    return a;
}

// ---- small wrappers
__device__ __forceinline__ uint32_t att_smem(const void *p) {
    return (uint32_t)__cvta_generic_to_shared(p);
}
__device__ __forceinline__ void cp16(uint32_t dst, const void *src, bool ok) {
    asm volatile("cp.async.cg.shared.global [%0], [%1], 16, %2;"
                 :: "r"(dst), "l"(src), "r"(ok ? 16 : 0) : "memory");
}
__device__ __forceinline__ void cp_commit() { asm volatile("cp.async.commit_group;" ::: "memory"); }
template <int N>
__device__ __forceinline__ void cp_wait() { asm volatile("cp.async.wait_group %0;" :: "n"(N) : "memory"); }

template <bool TRANS>
__device__ __forceinline__ void ldsm4(uint32_t (&w)[4], uint32_t addr) {
    if constexpr (TRANS)
        asm volatile("ldmatrix.sync.aligned.m8n8.x4.trans.shared.b16 {%0, %1, %2, %3}, [%4];"
                     : "=r"(w[0]), "=r"(w[1]), "=r"(w[2]), "=r"(w[3]) : "r"(addr) : "memory");
    else
        asm volatile("ldmatrix.sync.aligned.m8n8.x4.shared.b16 {%0, %1, %2, %3}, [%4];"
                     : "=r"(w[0]), "=r"(w[1]), "=r"(w[2]), "=r"(w[3]) : "r"(addr) : "memory");
}
__device__ __forceinline__ void mma_f16(float (&d)[4], uint32_t a0, uint32_t a1, uint32_t a2, uint32_t a3,
                                        uint32_t b0, uint32_t b1) {
    asm("mma.sync.aligned.m16n8k16.row.col.f32.f16.f16.f32 {%0, %1, %2, %3}, {%4, %5, %6, %7}, "
        "{%8, %9}, {%0, %1, %2, %3};"
        : "+f"(d[0]), "+f"(d[1]), "+f"(d[2]), "+f"(d[3])
        : "r"(a0), "r"(a1), "r"(a2), "r"(a3), "r"(b0), "r"(b1));
}
__device__ __forceinline__ uint32_t movm(uint32_t x) {
    uint32_t r;
    asm("movmatrix.sync.aligned.m8n8.trans.b16 %0, %1;" : "=r"(r) : "r"(x));
    return r;
}
__device__ __forceinline__ uint32_t f16x2_rn(float lo, float hi) {
    uint32_t r;
    asm("cvt.rn.f16x2.f32 %0, %1, %2;" : "=r"(r) : "f"(hi), "f"(lo));
    return r;
}
__device__ __forceinline__ float ex2(float x) {
    float r;
    asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(r) : "f"(x));
    return r;
}
__device__ __forceinline__ uint32_t prmt(uint32_t a, uint32_t b, uint32_t sel) {
    uint32_t r;
    asm("prmt.b32 %0, %1, %2, %3;" : "=r"(r) : "r"(a), "r"(b), "r"(sel));
    return r;
}
__device__ __forceinline__ uint32_t mul_lo(uint32_t a, uint32_t b) {
    uint32_t r;
    asm("mul.lo.u32 %0, %1, %2;" : "=r"(r) : "r"(a), "r"(b));
    return r;
}
// (x & m) | (y & ~m)
__device__ __forceinline__ uint32_t bit_select(uint32_t x, uint32_t y, uint32_t m) {
    uint32_t r;
    asm("lop3.b32 %0, %1, %2, %3, 0xE4;" : "=r"(r) : "r"(x), "r"(y), "r"(m));
    return r;
}
__device__ __forceinline__ uint32_t hfma2(uint32_t a, uint32_t b, uint32_t c) {
    uint32_t r;
    asm("fma.rn.f16x2 %0, %1, %2, %3;" : "=r"(r) : "r"(a), "r"(b), "r"(c));
    return r;
}
__device__ __forceinline__ uint32_t hmul2(uint32_t a, uint32_t b) {
    uint32_t r;
    asm("mul.rn.f16x2 %0, %1, %2;" : "=r"(r) : "r"(a), "r"(b));
    return r;
}
__device__ __forceinline__ uint32_t hsub2(uint32_t a, uint32_t b) {
    uint32_t r;
    asm("sub.rn.f16x2 %0, %1, %2;" : "=r"(r) : "r"(a), "r"(b));
    return r;
}

// (x & m) ^ v
__device__ __forceinline__ uint32_t and_xor(uint32_t x, uint32_t m, uint32_t v) {
    uint32_t r;
    asm("lop3.b32 %0, %1, %2, %3, 0x6A;" : "=r"(r) : "r"(x), "r"(m), "r"(v));
    return r;
}
// Eight INT4 codes of a word: out[i] holds nibbles i (low) and i + 4 (high)
// as fp16.  With u = c + 8, 0x6400 | u is 1024 + u; for the nibbles in bits 4
// to 7 it is 1024 + 16 u, brought down by a multiply-add; all exact.
__device__ __forceinline__ void int4_halves(uint32_t w, uint32_t (&out)[4]) {
    const uint32_t w8 = w >> 8;
    out[0] = hsub2(and_xor(w, 0x000F000Fu, 0x64086408u), 0x64086408u);
    out[1] = hfma2(and_xor(w, 0x00F000F0u, 0x64806480u), 0x2C002C00u, 0xD480D480u);   // / 16, - 72
    out[2] = hsub2(and_xor(w8, 0x000F000Fu, 0x64086408u), 0x64086408u);
    out[3] = hfma2(and_xor(w8, 0x00F000F0u, 0x64806480u), 0x2C002C00u, 0xD480D480u);
}
// Eight E2M1 codes of a word by bytes: out[i] holds nibbles 2i (low) and 2i + 1.
__device__ __forceinline__ void e2m1_bytes(uint32_t w, uint32_t (&out)[4]) {
    asm("{ .reg .b8 p, q, r, s; mov.b32 {p, q, r, s}, %4;\n\t"
        "cvt.rn.f16x2.e2m1x2 %0, p; cvt.rn.f16x2.e2m1x2 %1, q;\n\t"
        "cvt.rn.f16x2.e2m1x2 %2, r; cvt.rn.f16x2.e2m1x2 %3, s; }"
        : "=r"(out[0]), "=r"(out[1]), "=r"(out[2]), "=r"(out[3]) : "r"(w));
}
// Two halves of 4 nibbles each (a token each): out[i] holds nibble i of the
// low half and nibble i of the high half.
// (k16: 16, a value the compiler does not know)
template <int CODES>
__device__ __forceinline__ void nibble_pairs(uint32_t x, uint32_t (&out)[4], uint32_t k16) {
    if constexpr (CODES == CODES_INT4) {
        int4_halves(x, out);
    } else {
        // bytes 2 and 3 of e: nibbles 0, 2; of o: nibbles 1, 3 (the second
        // token's in the upper half).  The shifts go to the left and are
        // multiplications: the kernel is bound by the pipe of logic, shifts
        // and conversions, not by that of the multipliers.
        const uint32_t e = bit_select(mul_lo(x, k16), mul_lo(x, k16 * 4096u), 0xF0F0F0F0u);
        const uint32_t o = bit_select(x, mul_lo(x, k16 * 256u), 0xF0F0F0F0u);
        asm("{ .reg .b8 p, q, r, s, t; mov.b32 {t, t, p, q}, %4; mov.b32 {t, t, r, s}, %5;\n\t"
            "cvt.rn.f16x2.e2m1x2 %0, p; cvt.rn.f16x2.e2m1x2 %2, q;\n\t"
            "cvt.rn.f16x2.e2m1x2 %1, r; cvt.rn.f16x2.e2m1x2 %3, s; }"
            : "=r"(out[0]), "=r"(out[1]), "=r"(out[2]), "=r"(out[3]) : "r"(e), "r"(o));
    }
}

// Two tokens' words of 8 codes, channels 8 c .. of a block of 32, where the
// lanes of a quad (c = 0..3) hold the first group of 16 in its lower half and
// the second in its upper: lanes c and c + 2 exchange halves, so that each
// holds 4 channels of both groups, at 8 c (upper lanes: 8 c - 12) and 8 c + 16
// (8 c + 4).  The halves of the word become the first and the last two results
// of the conversion: the two groups.
template <int CODES>
__device__ __forceinline__ void k_order(uint32_t &a, uint32_t &b, bool upper) {
    const uint32_t give = prmt(a, b, upper ? 0x5410u : 0x7632u);
    const uint32_t got = __shfl_xor_sync(0xffffffffu, give, 2);
    if constexpr (CODES == CODES_INT4) {            // (nibbles i and i + 4 go together)
        a = prmt(a, got, upper ? 0x3524u : 0x5140u);
        b = prmt(b, got, upper ? 0x3726u : 0x7160u);
    } else {
        a = prmt(a, got, upper ? 0x3254u : 0x5410u);
        b = prmt(b, got, upper ? 0x3276u : 0x7610u);
    }
}

// A token's group scales in shared memory: SB bytes as words.
template <int SB>
struct ScaleWords {
    static constexpr int N = SB < 4 ? 1 : SB / 4;
    uint32_t w[N];
    __device__ __forceinline__ void load(const uint8_t *p) {
        if constexpr (SB == 1) w[0] = *p;
        else if constexpr (SB == 2) w[0] = *reinterpret_cast<const uint16_t *>(p);
        else if constexpr (SB == 4) w[0] = *reinterpret_cast<const uint32_t *>(p);
        else if constexpr (SB == 8) {
            const uint2 v = *reinterpret_cast<const uint2 *>(p);
            w[0] = v.x, w[1] = v.y;
        } else {
            const uint4 v = *reinterpret_cast<const uint4 *>(p);
            w[0] = v.x, w[1] = v.y, w[2] = v.z, w[3] = v.w;
        }
    }
    // Scale of group g (a constant after unrolling).
    template <int GS>
    __device__ __forceinline__ float get(int g) const {
        if constexpr (GS == SC_BF16) {
            const uint32_t v = w[g / 2];
            return __uint_as_float((g & 1) ? (v & 0xFFFF0000u) : (v << 16));
        } else if constexpr (GS == SC_E8M0) {
            const uint32_t v = w[g / 4];
            const int b = g % 4;
            return __uint_as_float((b == 3 ? v >> 1 : v << (23 - 8 * b)) & 0x7F800000u);
        } else {
            const uint16_t v = (uint16_t)((g & 2) ? (w[g / 4] >> 16) : w[g / 4]);
            uint32_t h2;
            asm("cvt.rn.f16x2.e4m3x2 %0, %1;" : "=r"(h2) : "h"(v));
            float f;
            if (g & 1) asm("{ .reg .f16 l, h; mov.b32 {l, h}, %1; cvt.f32.f16 %0, h; }" : "=f"(f) : "r"(h2));
            else asm("{ .reg .f16 l, h; mov.b32 {l, h}, %1; cvt.f32.f16 %0, l; }" : "=f"(f) : "r"(h2));
            return f;
        }
    }
    // floor(log2) of the largest scale (E4M3: at least its normal range's);
    // -200 if all are zero.
    template <int GS>
    __device__ __forceinline__ int top() const {
        uint32_t m = w[0];
        if constexpr (GS == SC_BF16) {
#pragma unroll
            for (int i = 1; i < N; ++i) m = __vmaxu2(m, w[i]);
            const uint32_t v = max(m & 0x7FFFu, (m >> 16) & 0x7FFFu);
            return v == 0 ? -200 : (int)(v >> 7) - 127;
        } else {
#pragma unroll
            for (int i = 1; i < N; ++i) m = __vmaxu4(m, w[i]);
            m = __vmaxu4(m, m >> 16);
            const uint32_t v = max(m & 0xFFu, (m >> 8) & 0xFFu);
            if constexpr (GS == SC_E8M0) return v == 0 ? -200 : (int)v - 127;
            else return v == 0 ? -200 : max((int)((v & 0x7Fu) >> 3), 1) - 7;
        }
    }
};

template <int CODES, int GS, int G, int D>
struct AttShape {
    static constexpr int ROWS = 8;
    static constexpr int NG = D / G;
    static constexpr int SB = NG * (GS == SC_BF16 ? 2 : 1);      // scale bytes of a token
    static constexpr int CB = kAttTile * D / 2;                  // code bytes of a warp tile
    static constexpr int TB = kAttTile * SB;                     // scale bytes of a warp tile
    static constexpr int STAGE = 2 * CB + 2 * TB;
    // a warp tile's scales by group and token: values' as fp16, keys' as float32
    static constexpr int VS_BYTES = NG * kAttTile * 6;
    static constexpr int RING_MAX = (112 * 1024 / kAttWarps - VS_BYTES - 64) / STAGE;
    static constexpr int RING = RING_MAX > 5 ? 5 : RING_MAX;
    static constexpr int RING_BYTES = kAttWarps * RING * STAGE;
    static constexpr int OST = D + 4;                            // row stride of the joining buffer
    static constexpr int JOIN_BYTES = kAttWarps * ROWS * OST * 4;
    static constexpr int BODY = RING_BYTES > JOIN_BYTES ? RING_BYTES : JOIN_BYTES;
    static constexpr int BYTES = BODY + kAttWarps * (ROWS * 8 + VS_BYTES);
    static_assert(RING >= 2, "ring");
};

// Byte offset of 16-byte chunk `ch` of token row `t` in a code tile: rows of
// D / 2 bytes, chunks exchanged so that the 8 rows of an 8x8 matrix load fall
// on different banks.
template <int D>
__device__ __forceinline__ uint32_t code_off(int t, int ch) {
    if constexpr (D == 128) return (uint32_t)(t * 64 + ((ch ^ ((t >> 1) & 3)) << 4));
    else return (uint32_t)(t * 32 + ((ch ^ ((t >> 2) & 1)) << 4));
}

template <int CODES, int GS, int G, int D>
__global__ void __launch_bounds__(kAttThreads, 2)
attend_split_kernel(const AttArgs A) {
    using Sh = AttShape<CODES, GS, G, D>;
    using Sw = ScaleWords<Sh::SB>;
    constexpr int ROWS = Sh::ROWS, RING = Sh::RING, NJ = D / 32;
    grid_dependency_begin();
    extern __shared__ __align__(128) uint8_t att_smem_raw[];
    float *const join = reinterpret_cast<float *>(att_smem_raw);
    float2 *const join_ml = reinterpret_cast<float2 *>(att_smem_raw + Sh::BODY);
    __shared__ long long s_scan[kAttWarps + 1];
    __shared__ long long s_first;
    __shared__ int s_seq;
    const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
    const int r = lane >> 2, c = lane & 3;
    const bool upper = c >= 2;
    const int me = blockIdx.x;
    const int heads = A.cache.heads, seqs = A.batch.seqs;

    // ---- this CTA's share: units [u0, u1) of the batch
    const int most = att_whole((int64_t)seqs * heads);
    bool longer = false;
    for (int b = tid; b < seqs; b += kAttThreads) {
        const KvSeq s = kv_seq(A.batch, A.cache.page_size, A.tokens, b);
        if (!s.ok && me == 0) atomicOr(A.status, STATUS_INDEX);
        longer |= s.len > most;
    }
    const int unit = __syncthreads_or(longer) ? kAttUnit : most;
    long long mine = 0, total = 0;
    for (int b = tid; b < seqs; b += kAttThreads) {
        const KvSeq s = kv_seq(A.batch, A.cache.page_size, A.tokens, b);
        mine = att_span<ROWS>(A, s, unit).units;
        total += mine;
    }
    const auto block_scan = [&](long long v, long long &all) {     // inclusive
#pragma unroll
        for (int o = 1; o < 32; o <<= 1) {
            const long long y = __shfl_up_sync(0xffffffffu, v, o);
            if (lane >= o) v += y;
        }
        __syncthreads();
        if (lane == 31) s_scan[warp] = v;
        __syncthreads();
        long long before = 0;
        all = 0;
#pragma unroll
        for (int w = 0; w < kAttWarps; ++w) {
            if (w < warp) before += s_scan[w];
            all += s_scan[w];
        }
        return v + before;
    };
    long long units, incl = block_scan(total, units);
    if (tid == 0) A.meta[me] = AttMeta{};
    const int n = (int)min((long long)gridDim.x, units);       // shares, none of them empty
    if (me >= n) return;
    const long long u0 = units * me / n, u1 = units * (me + 1) / n;
    if (seqs <= kAttThreads) {
        if (tid < seqs && incl - mine <= u0 && u0 < incl) {
            s_seq = tid;
            s_first = incl - mine;
        }
    } else {
        long long base = 0;
        for (int b0 = 0; b0 < seqs; b0 += kAttThreads) {
            const int b = b0 + tid;
            long long v = 0, all;
            if (b < seqs) v = att_span<ROWS>(A, kv_seq(A.batch, A.cache.page_size, A.tokens, b), unit).units;
            const long long in = base + block_scan(v, all);
            if (v > 0 && in - v <= u0 && u0 < in) {
                s_seq = b;
                s_first = in - v;
            }
            base += all;
            if (base > u0) break;
        }
    }
    __syncthreads();
    int seq = s_seq;
    long long first = s_first;

    uint8_t *const ring = att_smem_raw + warp * RING * Sh::STAGE;
    uint16_t *const vs16 = reinterpret_cast<uint16_t *>(att_smem_raw + Sh::BODY + kAttWarps * ROWS * 8) +
                           warp * (Sh::VS_BYTES / 2);
    float *const ks32 = reinterpret_cast<float *>(vs16 + Sh::NG * kAttTile);
    const uint32_t ring_s = att_smem(ring);
    // byte of this lane's row in a matrix load: token (lane & 7) + 8 of matrix 1, 3; chunk + 1 of 2, 3
    const int lm_t = (lane & 7) + ((lane >> 3) & 1) * 8, lm_c = lane >> 4;

    for (long long u = u0; u < u1;) {
        const KvSeq s = kv_seq(A.batch, A.cache.page_size, A.tokens, seq);
        const AttSpan sp = att_span<ROWS>(A, s, unit);
        if (u >= first + sp.units) {
            first += sp.units;
            ++seq;
            continue;
        }
        const long long local = u - first;
        const int seg = (int)(local / sp.kvt);
        const int t0 = (int)(local - (long long)seg * sp.kvt);
        const int t1 = (int)min((long long)sp.kvt, t0 + (u1 - u));
        const int head = seg / sp.qt, row0 = (seg - head * sp.qt) * ROWS;
        const int nrows = s.n * A.group;                       // of the sequence
        const int rows = min(ROWS, nrows - row0);              // of this tile
        // positions below limit(row) are seen by the row
        const auto limit = [&](int row) {
            return A.causal ? min(max(s.len - s.n + row / A.group + 1, 0), s.len) : s.len;
        };
        const int lim_min = limit(row0), lim_max = limit(row0 + rows - 1);
        const int lo = t0 * unit, hi = min(t1 * unit, lim_max);

        // ---- tokens, 32 at a time; the first loads go out before anything else
        const int base0 = lo + kAttTile * warp;
        const int nt = hi > base0 ? (hi - base0 + kAttUnit - 1) / kAttUnit : 0;
        // a tile is two runs of 16 tokens, each inside a page; lane 0 (16) and
        // its neighbours follow the first (second): its page and slot, tile by tile
        const int ps = A.cache.page_size, hop_pages = kAttUnit / ps, hop_slots = kAttUnit - hop_pages * ps;
        const int32_t *const table = A.batch.block_table + seq * A.batch.table_stride;
        int at_pos = base0 + (lane & 16), at_page = at_pos / ps, at_slot = at_pos - at_page * ps;
        // row in the cache of this lane's run of the next tile, or -1
        const auto next_row = [&]() -> int64_t {
            int64_t row = -1;
            if (at_pos < hi) {
                const int page = __ldg(table + at_page);
                if (page >= 0 && (int64_t)page < A.cache.pages) row = ((int64_t)page * heads + head) * ps + at_slot;
                else atomicOr(A.status, STATUS_INDEX);
            }
            at_pos += kAttUnit;
            at_page += hop_pages;
            at_slot += hop_slots;
            if (at_slot >= ps) at_slot -= ps, ++at_page;
            return row;
        };
        const auto issue = [&](int i, int64_t row) {
            if (i < nt) {
                const uint32_t st = ring_s + (i % RING) * Sh::STAGE;
                const int64_t row_a = __shfl_sync(0xffffffffu, row, 0), row_b = __shfl_sync(0xffffffffu, row, 16);
                // codes: 16 bytes per lane and step, in the order of the rows
                constexpr int CPR = D / 32;                     // 16-byte chunks per code row
                const uint32_t dst = st + code_off<D>(lane / CPR, lane % CPR);
                const bool ok_a = row_a >= 0, ok_b = row_b >= 0;
                const int64_t off_a = (ok_a ? row_a * (D / 2) : 0) + lane * 16;
                const int64_t off_b = (ok_b ? row_b * (D / 2) : 0) + lane * 16;
                const uint8_t *const ka = A.cache.k_codes + off_a, *const kb = A.cache.k_codes + off_b;
                const uint8_t *const va = A.cache.v_codes + off_a, *const vb = A.cache.v_codes + off_b;
#pragma unroll
                for (int k = 0; k < CPR / 2; ++k) {             // (nothing is read where !ok)
                    cp16(dst + k * 512, ka + k * 512, ok_a);
                    cp16(dst + (k + CPR / 2) * 512, kb + k * 512, ok_b);
                    cp16(dst + k * 512 + Sh::CB, va + k * 512, ok_a);
                    cp16(dst + (k + CPR / 2) * 512 + Sh::CB, vb + k * 512, ok_b);
                }
                // scales: SB chunks of 16 bytes per run, keys then values
#pragma unroll
                for (int k = 0; k < (4 * Sh::SB + 31) / 32; ++k) {
                    const int x = k * 32 + lane;
                    if (4 * Sh::SB % 32 == 0 || x < 4 * Sh::SB) {
                        const int64_t row = (x / Sh::SB) % 2 ? row_b : row_a;
                        cp16(st + 2 * Sh::CB + x * 16,
                             reinterpret_cast<const uint8_t *>(x < 2 * Sh::SB ? A.cache.k_scales : A.cache.v_scales) +
                                 (row < 0 ? 0 : row * Sh::SB + (x % Sh::SB) * 16),
                             row >= 0);
                    }
                }
            }
            cp_commit();
        };
        // (every load that depends on nothing else first)
        uint4 raw[NJ];
        const int row = row0 + r, tok = row / A.group;
        const uint16_t *p = A.q + (s.s0 + tok) * A.q_token +
                            (int64_t)(head * A.group + row - tok * A.group) * A.q_head;
#pragma unroll
        for (int j = 0; j < NJ; ++j) {
            raw[j] = make_uint4(0, 0, 0, 0);
            if (r >= rows) continue;
            if constexpr (G == 16) {                            // 4 channels of each group (k_order)
                const uint2 a = __ldg(reinterpret_cast<const uint2 *>(p + 32 * j + (upper ? 8 * c - 12 : 8 * c)));
                const uint2 b = __ldg(reinterpret_cast<const uint2 *>(p + 32 * j + (upper ? 8 * c + 4 : 8 * c + 16)));
                raw[j] = make_uint4(a.x, a.y, b.x, b.y);
            } else {
                raw[j] = __ldg(reinterpret_cast<const uint4 *>(p + 32 * j + 8 * c));
            }
        }
        int64_t first_rows[RING];
#pragma unroll
        for (int i = 0; i < RING; ++i) first_rows[i] = next_row();
        int64_t row_next = first_rows[RING - 1];
#pragma unroll
        for (int i = 0; i < RING - 1; ++i) issue(i, first_rows[i]);

        // ---- the query rows: B operands, and the factor that takes a
        // product of scaled operands to log2 units
        uint32_t qf[NJ][4];
        float fac[2];
        int lim[2];
        uint32_t top = 0;
#pragma unroll
        for (int j = 0; j < NJ; ++j) {
            const uint32_t v[4] = {raw[j].x, raw[j].y, raw[j].z, raw[j].w};
#pragma unroll
            for (int k = 0; k < 4; ++k) top = __vmaxu2(top, v[k] & 0x7FFF7FFFu);
        }
        top = max(top & 0xFFFFu, top >> 16);
        top = max(top, __shfl_xor_sync(0xffffffffu, top, 1));
        top = max(top, __shfl_xor_sync(0xffffffffu, top, 2));
        const int e = max((int)(top >> 7) - 127, -100);     // of the row's largest element
        const float up = pow2f(13 - e);
#pragma unroll
        for (int j = 0; j < NJ; ++j) {
            const uint32_t v[4] = {raw[j].x, raw[j].y, raw[j].z, raw[j].w};
            float x[8];
#pragma unroll
            for (int k = 0; k < 4; ++k) {
                x[2 * k] = __uint_as_float(v[k] << 16) * up;
                x[2 * k + 1] = __uint_as_float(v[k] & 0xFFFF0000u) * up;
            }
            if constexpr (CODES == CODES_INT4) {
#pragma unroll
                for (int k = 0; k < 4; ++k) {
                    if constexpr (G == 16) qf[j][k] = f16x2_rn(x[k + (k & 2)], x[k + (k & 2) + 2]);
                    else qf[j][k] = f16x2_rn(x[k], x[k + 4]);
                }
            } else {
#pragma unroll
                for (int k = 0; k < 4; ++k) qf[j][k] = f16x2_rn(x[2 * k], x[2 * k + 1]);
            }
        }
        // (above zero, so that a masked -inf stays -inf; a finite score times the
        // smallest float32 is below 5e-7)
        const float f = fmaxf(A.scale_log2 * pow2f(e - 13), __uint_as_float(1));
        fac[0] = __shfl_sync(0xffffffffu, f, 8 * c);         // row 2c of the tile
        fac[1] = __shfl_sync(0xffffffffu, f, 8 * c + 4);     // row 2c + 1
#pragma unroll
        for (int h = 0; h < 2; ++h) lim[h] = limit(min(row0 + 2 * c + h, row0 + rows - 1));

        float o[NJ][2][4];
        float m[2], l[2];
#pragma unroll
        for (int j = 0; j < NJ; ++j)
#pragma unroll
            for (int k = 0; k < 8; ++k) o[j][k >> 2][k & 3] = 0.0f;
        m[0] = m[1] = -INFINITY;
        l[0] = l[1] = 0.0f;
        for (int it = 0; it < nt; ++it) {
            {
                const int64_t row = row_next;
                row_next = next_row();
                issue(it + RING - 1, row);
            }
            cp_wait<RING - 1>();
            __syncwarp();
            uint8_t *const st = ring + (it % RING) * Sh::STAGE;
            const uint32_t st_s = ring_s + (it % RING) * Sh::STAGE;
            uint8_t *const ks = st + 2 * Sh::CB, *const vs = ks + Sh::TB;
            const int base = base0 + it * kAttUnit;
            // scales, token by token: keys' as float32, values' as fp16
            // relative to the largest; values' of tokens that no row sees are
            // zero
            int ev;                                             // its exponent
            {
                Sw v;
                v.load(vs + lane * Sh::SB);
                if (base + lane >= hi) {
#pragma unroll
                    for (int i = 0; i < Sw::N; ++i) v.w[i] = 0;
                }
                ev = max(__reduce_max_sync(0xffffffffu, v.template top<GS>()), -90);
                const float down = pow2f(6 - ev);
#pragma unroll
                for (int g = 0; g < Sh::NG; ++g) {
                    const uint32_t h = f16x2_rn(v.template get<GS>(g) * down, 0.0f);
                    vs16[g * kAttTile + lane] = (uint16_t)h;
                }
                Sw k;
                k.load(ks + lane * Sh::SB);
#pragma unroll
                for (int g = 0; g < Sh::NG; ++g) ks32[g * kAttTile + lane] = k.template get<GS>(g);
                __syncwarp();
            }
            // ---- scores
            float sc[2][4];
#pragma unroll
            for (int mb = 0; mb < 2; ++mb) {
                const float *const sk = ks32 + mb * 16 + r;
#pragma unroll
                for (int k = 0; k < 4; ++k) sc[mb][k] = 0.0f;
#pragma unroll
                for (int j = 0; j < NJ; j += 2) {
                    uint32_t w[4];
                    ldsm4<false>(w, st_s + code_off<D>(mb * 16 + lm_t, j + lm_c));
                    float acc[4];
#pragma unroll
                    for (int jj = 0; jj < 2; ++jj) {
                        uint32_t x[4], y[4];
                        if constexpr (G == 16) k_order<CODES>(w[2 * jj], w[2 * jj + 1], upper);
                        if constexpr (CODES == CODES_INT4) {
                            int4_halves(w[2 * jj], x);
                            int4_halves(w[2 * jj + 1], y);
                        } else {
                            e2m1_bytes(w[2 * jj], x);
                            e2m1_bytes(w[2 * jj + 1], y);
                        }
                        const uint32_t(&q)[4] = qf[j + jj];
                        if constexpr (G == 16) {
#pragma unroll
                            for (int half = 0; half < 2; ++half) {
                                const int g = 2 * (j + jj) + half;
                                float d[4] = {0.0f, 0.0f, 0.0f, 0.0f};
                                mma_f16(d, x[2 * half], y[2 * half], x[2 * half + 1], y[2 * half + 1], q[2 * half],
                                        q[2 * half + 1]);
                                const float s0 = sk[g * kAttTile], s8 = sk[g * kAttTile + 8];
                                sc[mb][0] = fmaf(d[0], s0, sc[mb][0]);
                                sc[mb][1] = fmaf(d[1], s0, sc[mb][1]);
                                sc[mb][2] = fmaf(d[2], s8, sc[mb][2]);
                                sc[mb][3] = fmaf(d[3], s8, sc[mb][3]);
                            }
                        } else {
                            if (G == 32 || jj == 0) {
#pragma unroll
                                for (int k = 0; k < 4; ++k) acc[k] = 0.0f;
                            }
                            mma_f16(acc, x[0], y[0], x[1], y[1], q[0], q[1]);
                            mma_f16(acc, x[2], y[2], x[3], y[3], q[2], q[3]);
                            if (G == 32 || jj == 1) {
                                const int g = (j + jj) * 32 / G;
                                const float s0 = sk[g * kAttTile], s8 = sk[g * kAttTile + 8];
                                sc[mb][0] = fmaf(acc[0], s0, sc[mb][0]);
                                sc[mb][1] = fmaf(acc[1], s0, sc[mb][1]);
                                sc[mb][2] = fmaf(acc[2], s8, sc[mb][2]);
                                sc[mb][3] = fmaf(acc[3], s8, sc[mb][3]);
                            }
                        }
                    }
                }
            }
            // ---- softmax: the running maximum carries the exponent of the
            // tiles' value scales, p 2^E is what the products take.  It is
            // raised, to the largest score + exponent - 7, only where that is
            // more than 2 above it: p stays at most 2^9
            const bool cut = base + kAttTile > lim_min;
            float top[2];
            bool raise = false;
#pragma unroll
            for (int h = 0; h < 2; ++h) {
                float t = -INFINITY;
#pragma unroll
                for (int mb = 0; mb < 2; ++mb)
#pragma unroll
                    for (int k = 0; k < 2; ++k) {
                        float &x = sc[mb][2 * k + h];
                        if (cut && base + mb * 16 + 8 * k + r >= lim[h]) x = -INFINITY;
                        t = max_nan(t, x);
                    }
                top[h] = fmaf(t, fac[h], (float)(ev - 7));
                raise |= top[h] > m[h] + 2.0f;
            }
            if (__any_sync(0xffffffffu, raise)) {
                float alpha[2];
#pragma unroll
                for (int h = 0; h < 2; ++h) {
                    float t = top[h];
                    t = max_nan(t, __shfl_xor_sync(0xffffffffu, t, 4));
                    t = max_nan(t, __shfl_xor_sync(0xffffffffu, t, 8));
                    t = max_nan(t, __shfl_xor_sync(0xffffffffu, t, 16));
                    const float now = t > m[h] + 2.0f ? t : m[h];
                    alpha[h] = now == m[h] ? 1.0f : ex2(m[h] - now);
                    m[h] = now;
                    l[h] *= alpha[h];
                }
#pragma unroll
                for (int j = 0; j < NJ; ++j)
#pragma unroll
                    for (int k = 0; k < 8; ++k) o[j][k >> 2][k & 3] *= alpha[k & 1];
            }
            uint32_t pt[2][2];                              // transposed: tokens 2c, 2c + 1 (+ 8) of row r
            float sum[2] = {0.0f, 0.0f}, off[2];
#pragma unroll
            for (int h = 0; h < 2; ++h) off[h] = (float)ev - (m[h] == -INFINITY ? 0.0f : m[h]);
#pragma unroll
            for (int mb = 0; mb < 2; ++mb) {
                float p[4];
#pragma unroll
                for (int k = 0; k < 4; ++k) {
                    p[k] = ex2(fmaf(sc[mb][k], fac[k & 1], off[k & 1]));
                    sum[k & 1] += p[k];
                }
                pt[mb][0] = movm(f16x2_rn(p[0], p[1]));
                pt[mb][1] = movm(f16x2_rn(p[2], p[3]));
            }
            const float up = pow2f(6 - ev);                 // (as the scales)
            l[0] = fmaf(sum[0], up, l[0]);
            l[1] = fmaf(sum[1], up, l[1]);
            // ---- values
#pragma unroll
            for (int mb = 0; mb < 2; ++mb) {
                uint32_t p0, p1, p2, p3;        // B operands of the group(s) at hand
                const auto probs = [&](int g, uint32_t &b0, uint32_t &b1) {
                    const uint32_t *const s2 = reinterpret_cast<const uint32_t *>(vs16 + g * kAttTile + mb * 16);
                    const uint32_t s0 = s2[c], s8 = s2[c + 4];
                    b0 = hmul2(pt[mb][0], s0);
                    b1 = hmul2(pt[mb][1], s8);
                };
#pragma unroll
                for (int j = 0; j < NJ; j += 2) {
                    uint32_t w[4];
                    ldsm4<true>(w, st_s + Sh::CB + code_off<D>(mb * 16 + lm_t, j + lm_c));
#pragma unroll
                    for (int jj = 0; jj < 2; ++jj) {
                        uint32_t wa = w[2 * jj], wb = w[2 * jj + 1];
                        if constexpr (G == 16) {
                            // a lane of the lower four rows holds nibbles of the first
                            // group, one of the upper four of the second; half of them
                            // change places, so that nibbles 0, 1 are the first group's
                            // and 2, 3 the second's in every lane
                            const bool up = (r & 4) != 0;
                            const uint32_t give = prmt(wa, wb, up ? 0x6420u : 0x7531u);
                            const uint32_t got = __shfl_xor_sync(0xffffffffu, give, 16);
                            wa = prmt(wa, got, up ? 0x3514u : 0x5240u);
                            wb = prmt(wb, got, up ? 0x3716u : 0x7260u);
                            probs(2 * (j + jj), p0, p1);
                            probs(2 * (j + jj) + 1, p2, p3);
                        } else if (G == 32 || jj == 0) {
                            probs((j + jj) * 32 / G, p0, p1);
                        }
                        uint32_t x[4], y[4];
                        nibble_pairs<CODES>(wa, x, A.k16);
                        nibble_pairs<CODES>(wb, y, A.k16);
                        mma_f16(o[j + jj][0], x[0], x[1], y[0], y[1], p0, p1);
                        if constexpr (G == 16)
                            mma_f16(o[j + jj][1], x[2], x[3], y[2], y[3], p2, p3);
                        else
                            mma_f16(o[j + jj][1], x[2], x[3], y[2], y[3], p0, p1);
                    }
                }
            }
            __syncwarp();
        }
        cp_wait<0>();
        __syncthreads();                                        // the ring becomes the joining buffer

        // ---- join the warps
#pragma unroll
        for (int h = 0; h < 2; ++h) {
            float t = l[h];
            t += __shfl_xor_sync(0xffffffffu, t, 4);
            t += __shfl_xor_sync(0xffffffffu, t, 8);
            t += __shfl_xor_sync(0xffffffffu, t, 16);
            const int row = 2 * c + h;
            if (r == 0) join_ml[warp * ROWS + row] = make_float2(m[h], t);
            float *const dst = join + (warp * ROWS + row) * Sh::OST;
#pragma unroll
            for (int j = 0; j < NJ; ++j) {
                if constexpr (G == 16) {
#pragma unroll
                    for (int blk = 0; blk < 2; ++blk)
                        *reinterpret_cast<float2 *>(dst + 32 * j + 16 * blk + 4 * (r & 3) + 2 * (r >> 2)) =
                            make_float2(o[j][blk][h], o[j][blk][2 + h]);
                } else {
                    *reinterpret_cast<float4 *>(dst + 32 * j + 4 * r) =
                        make_float4(o[j][0][h], o[j][0][2 + h], o[j][1][h], o[j][1][2 + h]);
                }
            }
        }
        __syncthreads();
        const bool whole = t0 == 0 && t1 == sp.kvt;
        const int slot = 2 * me + (t0 == 0 ? 1 : 0);
        for (int x = tid; x < rows * (D / 4); x += kAttThreads) {
            const int row = x / (D / 4), d = 4 * (x % (D / 4));
            float mx = -INFINITY;
#pragma unroll
            for (int w = 0; w < kAttWarps; ++w) mx = max_nan(mx, join_ml[w * ROWS + row].x);
            const float base = mx == -INFINITY ? 0.0f : mx;
            float4 acc = make_float4(0.0f, 0.0f, 0.0f, 0.0f);
            float sum = 0.0f;
#pragma unroll
            for (int w = 0; w < kAttWarps; ++w) {
                const float2 ml = join_ml[w * ROWS + row];
                const float f = ex2(ml.x - base);
                const float4 v = *reinterpret_cast<const float4 *>(join + (w * ROWS + row) * Sh::OST + d);
                sum = fmaf(ml.y, f, sum);
                acc.x = fmaf(v.x, f, acc.x);
                acc.y = fmaf(v.y, f, acc.y);
                acc.z = fmaf(v.z, f, acc.z);
                acc.w = fmaf(v.w, f, acc.w);
            }
            if (whole) {
                const float inv = sum == 0.0f ? 0.0f : 1.0f / sum;
                const int rr = row0 + row, tok = rr / A.group;
                uint2 v;
                asm("cvt.rn.bf16x2.f32 %0, %1, %2;" : "=r"(v.x) : "f"(acc.y * inv), "f"(acc.x * inv));
                asm("cvt.rn.bf16x2.f32 %0, %1, %2;" : "=r"(v.y) : "f"(acc.w * inv), "f"(acc.z * inv));
                *reinterpret_cast<uint2 *>(A.out + (s.s0 + tok) * A.out_token +
                                           (int64_t)(head * A.group + rr - tok * A.group) * A.out_head + d) = v;
            } else {
                *reinterpret_cast<float4 *>(A.part + ((int64_t)slot * ROWS + row) * D + d) = acc;
                if (d == 0) A.part_ml[slot * ROWS + row] = make_float2(mx, sum);
            }
        }
        if (!whole && t0 == 0 && tid == 0) {
            const long long end = first + (long long)(seg + 1) * sp.kvt;    // (its last unit, plus 1)
            AttMeta mt;
            mt.last = (int)min((long long)n - 1, (end * n - 1) / units);
            mt.rows = rows;
            mt.row0 = row0;
            mt.head = head;
            mt.token0 = s.s0;
            A.meta[me] = mt;
        }
        __syncthreads();
        u += t1 - t0;
    }
}

// Joins the pieces of the segments that were cut: CTA (i, row) takes the one
// that starts in share i.  Four warps take every fourth piece each; their
// sums are added in a fixed order.
template <int D>
__global__ void __launch_bounds__(128)
attend_join_kernel(const AttArgs A) {
    grid_dependency_begin();
    constexpr int ROWS = 8;
    __shared__ float4 s_acc[4][D / 4];
    __shared__ float s_sum[4];
    const AttMeta mt = A.meta[blockIdx.x];
    const int row = blockIdx.y, warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    if (row >= mt.rows) return;
    // shares i, i + 1, ..., last hold pieces
    const int i0 = blockIdx.x, last = mt.last;
    const auto piece = [&](int i) { return 2 * i + (i == i0 ? 1 : 0); };     // its slot
    float mx = -INFINITY;
    for (int i = i0 + lane; i <= last; i += 32)
        mx = max_nan(mx, A.part_ml[piece(i) * ROWS + row].x);
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) mx = max_nan(mx, __shfl_xor_sync(0xffffffffu, mx, o));
    const float base = mx == -INFINITY ? 0.0f : mx;
    float4 acc = make_float4(0.0f, 0.0f, 0.0f, 0.0f);
    float sum = 0.0f;
#pragma unroll 4
    for (int i = i0 + warp; i <= last; i += 4) {
        const int k = piece(i);
        const float2 ml = A.part_ml[k * ROWS + row];
        const float f = ex2(ml.x - base);
        sum = fmaf(ml.y, f, sum);
        if (4 * lane < D) {
            const float4 v = *reinterpret_cast<const float4 *>(A.part + ((int64_t)k * ROWS + row) * D + 4 * lane);
            acc.x = fmaf(v.x, f, acc.x);
            acc.y = fmaf(v.y, f, acc.y);
            acc.z = fmaf(v.z, f, acc.z);
            acc.w = fmaf(v.w, f, acc.w);
        }
    }
    if (4 * lane < D) s_acc[warp][lane] = acc;
    if (lane == 0) s_sum[warp] = sum;
    __syncthreads();
    if (warp != 0 || 4 * lane >= D) return;
#pragma unroll
    for (int w = 1; w < 4; ++w) {
        const float4 v = s_acc[w][lane];
        acc.x += v.x;
        acc.y += v.y;
        acc.z += v.z;
        acc.w += v.w;
        sum += s_sum[w];
    }
    const float inv = sum == 0.0f ? 0.0f : 1.0f / sum;
    const int rr = mt.row0 + row, tok = rr / A.group;
    uint2 v;
    asm("cvt.rn.bf16x2.f32 %0, %1, %2;" : "=r"(v.x) : "f"(acc.y * inv), "f"(acc.x * inv));
    asm("cvt.rn.bf16x2.f32 %0, %1, %2;" : "=r"(v.y) : "f"(acc.w * inv), "f"(acc.z * inv));
    *reinterpret_cast<uint2 *>(A.out + (mt.token0 + tok) * A.out_token +
                               (int64_t)(mt.head * A.group + rr - tok * A.group) * A.out_head + 4 * lane) = v;
}

// ---- launch

inline AttArgs att_args(const AttendLaunch &L, int slots, int rows, int few) {
    AttArgs A;
    A.q = static_cast<const uint16_t *>(L.q);
    A.q_token = L.q_token;
    A.q_head = L.q_head;
    A.out = static_cast<uint16_t *>(L.out);
    A.out_token = L.out_token;
    A.out_head = L.out_head;
    A.tokens = L.tokens;
    A.group = L.q_heads / L.cache.heads;
    A.scale_log2 = L.scale * 1.44269504088896341f;
    A.few = few;
    A.causal = L.causal;
    A.k16 = 16;
    A.cache = L.cache;
    A.batch = L.batch;
    uint8_t *w = static_cast<uint8_t *>(L.workspace);
    A.part = reinterpret_cast<float *>(w);
    w += (size_t)slots * rows * L.cache.head_dim * sizeof(float);
    A.part_ml = reinterpret_cast<float2 *>(w);
    w += (size_t)slots * rows * sizeof(float2);
    A.meta = reinterpret_cast<AttMeta *>(w);
    A.status = L.status;
    return A;
}

template <int CODES, int GS, int G, int D>
cudaError_t launch_attend_split(AttendLaunch &L, int few) {
    using Sh = AttShape<CODES, GS, G, D>;
    const AttArgs A = att_args(L, 2 * kAttCtas, Sh::ROWS, few);
    const auto kern = attend_split_kernel<CODES, GS, G, D>;
    static std::atomic<bool> done[64];
    cudaError_t e = smem_opt_in(kern, Sh::BYTES, done);
    if (e != cudaSuccess) return e;
    e = launch_k(kern, dim3(kAttCtas), dim3(kAttThreads), Sh::BYTES, L.stream, A);
    if (e != cudaSuccess) return e;
    L.launches += 1;
    // (nothing is cut where no sequence can be longer)
    if ((int64_t)L.batch.max_pages * L.cache.page_size <= att_whole((int64_t)L.batch.seqs * L.cache.heads))
        return cudaSuccess;
    L.launches += 1;
    return launch_k(attend_join_kernel<D>, dim3(kAttCtas, Sh::ROWS), dim3(128), 0, L.stream, A);
}

}  // namespace dq
