// dq_kv_cache.cu — writing new keys and values into the paged 4-bit cache and
// reading them back.
//
// Both move a token's row of one head (head_dim channels) at a time: a lane
// takes 8 channels (16 bytes of bf16, 4 bytes of codes), so a row is 8 or 16
// lanes and a group of G channels G / 8 of them; the quantizer is the one of
// the activation mode (Quant::run with b = 1), so the cache holds exactly
// what dq_quantize writes.  A warp looks its token's sequence up once (32
// starts at a time) and then walks the heads of keys and values.
//
// Moves 2 bytes per channel in (or out) and half a byte of codes.  16
// sequences of 2048 new tokens, 8 heads of 128, MXFP4: append 40 us, read 38
// (3.7 TB/s): both are bound by instructions (issue 66% in the read), the
// append by the quantizer's (NVFP4, whose scales are divided by, 95 us).
#include <cuda_runtime.h>

#include "dq_kv.cuh"

namespace dq {

namespace {

struct KvCopyArgs {
    uint16_t *k, *v;
    int64_t k_token, k_head, v_token, v_head;
    int64_t tokens;
    dq_kv_cache cache;
    dq_kv_batch batch;
    int splits;              // warps that share a token's rows
    unsigned int *status;
};

// Sequence and position of token row t; false if it has none in the cache.
__device__ __forceinline__ bool place_of(const KvCopyArgs &A, int64_t t, int &seq, int &pos) {
    seq = kv_find(A.batch, t);
    if (seq >= A.batch.seqs) return false;             // behind the last sequence
    bool bad = seq < 0;
    if (!bad) {
        const KvSeq s = kv_seq(A.batch, A.cache.page_size, A.tokens, seq);
        pos = s.len - s.n + (int)(t - s.s0);
        bad = !s.ok || t >= (int64_t)s.s0 + s.n || pos < 0;
    }
    if (bad && (threadIdx.x & 31) == 0) atomicOr(A.status, STATUS_INDEX);
    return !bad;
}

template <int CODES, int GS, int G, int D, bool READ>
__global__ void __launch_bounds__(256)
kv_copy_kernel(const KvCopyArgs A) {
    grid_dependency_begin();
    constexpr int LPR = D / 8;                          // lanes per row
    constexpr int RPW = 32 / LPR;                       // rows per warp step
    const int lane = threadIdx.x & 31;
    const int64_t nwarps = ((int64_t)gridDim.x * blockDim.x) >> 5;
    const int64_t units = A.tokens * A.splits;
    for (int64_t u = ((int64_t)blockIdx.x * blockDim.x + threadIdx.x) >> 5; u < units; u += nwarps) {
        const int64_t t = u / A.splits;
        const int part = (int)(u - t * A.splits);
        int seq, pos;
        if (!place_of(A, t, seq, pos)) continue;
        const int64_t row0 = kv_row(A.cache, A.batch, seq, pos, 0);
        if (row0 < 0) {
            if (lane == 0) atomicOr(A.status, STATUS_INDEX);
            if (!READ) continue;
        }
        const int rows = 2 * A.cache.heads;             // keys, then values
        // UN steps at a time, their loads first: a warp's rows are few, and
        // one load after the other would leave the memory idle (at the size
        // above: one step 52 us, two 40, four 41 to 44, eight 49)
        constexpr int UN = 2;
        const int hop = A.splits * RPW;
        for (int r0 = part * RPW; r0 < rows; r0 += UN * hop) {
            uint16_t *x[UN];
            uint8_t *codes[UN];
            void *scales[UN];
            int64_t gi[UN];
            bool ok[UN];
            uint4 in[UN];
            float sc[UN];
            const int c = lane % LPR;
#pragma unroll
            for (int i = 0; i < UN; ++i) {
                const int r = r0 + i * hop + lane / LPR;
                ok[i] = r < rows;
                const bool val = r >= A.cache.heads;
                const int head = ok[i] ? (val ? r - A.cache.heads : r) : 0;
                x[i] = (val ? A.v + t * A.v_token + head * A.v_head : A.k + t * A.k_token + head * A.k_head) + 8 * c;
                const int64_t row = row0 + (int64_t)head * A.cache.page_size;
                codes[i] = (val ? A.cache.v_codes : A.cache.k_codes) + row * (D / 2) + 4 * c;
                scales[i] = val ? A.cache.v_scales : A.cache.k_scales;
                gi[i] = row * (D / G) + c / (G / 8);
                in[i] = make_uint4(0, 0, 0, 0);
                sc[i] = 0.0f;
                if constexpr (READ) {
                    if (ok[i] && row0 >= 0) {
                        in[i].x = *reinterpret_cast<const uint32_t *>(codes[i]);
                        sc[i] = scale_value<GS>(scales[i], gi[i]);
                    }
                } else {
                    if (ok[i]) in[i] = __ldg(reinterpret_cast<const uint4 *>(x[i]));
                }
            }
#pragma unroll
            for (int i = 0; i < UN; ++i) {
                if (r0 + i * hop >= rows) break;        // (the whole warp)
                if constexpr (READ) {
                    uint32_t p[4];
#pragma unroll
                    for (int k = 0; k < 4; ++k) {
                        const uint32_t b = (in[i].x >> (8 * k)) & 0xFFu;
                        const float2 v = CODES == CODES_INT4
                                             ? make_float2((float)((int)((b & 15u) ^ 8u) - 8),
                                                           (float)((int)((b >> 4) ^ 8u) - 8))
                                             : e2m1x2_to_f32(b);
                        asm("cvt.rn.bf16x2.f32 %0, %1, %2;" : "=r"(p[k]) : "f"(v.y * sc[i]), "f"(v.x * sc[i]));
                    }
                    if (ok[i]) *reinterpret_cast<uint4 *>(x[i]) = make_uint4(p[0], p[1], p[2], p[3]);
                } else {
                    Chunk<Bf16Tag> ch;
                    ch.raw = in[i];
                    f2 z[4], code[4];
                    ch.unpack2(z);
                    float s, s_eff;
                    uint32_t cw[2], mbits;
                    bool nonzero;
                    Quant<CODES, GS, SC_BF16, true, 4, G / 8>::template run<true>(
                        z, z, 1.0f, 1.0f, z, 1.0f, 1.0f, A.status, code, s, s_eff, cw, nonzero, mbits);
                    if (!ok[i]) continue;
                    *reinterpret_cast<uint32_t *>(codes[i]) = cw[0];
                    if (c % (G / 8) == 0) {
                        if constexpr (GS == SC_BF16)
                            reinterpret_cast<uint16_t *>(scales[i])[gi[i]] = (uint16_t)(__float_as_uint(s) >> 16);
                        else if constexpr (GS == SC_E8M0)
                            reinterpret_cast<uint8_t *>(scales[i])[gi[i]] = (uint8_t)(__float_as_uint(s) >> 23);
                        else
                            reinterpret_cast<uint8_t *>(scales[i])[gi[i]] = (uint8_t)e4m3_bits(s);
                    }
                }
            }
        }
    }
}

template <int CODES, int GS, bool READ>
cudaError_t launch_fmt(const KvCopyLaunch &L) {
    KvCopyArgs A;
    A.k = static_cast<uint16_t *>(const_cast<void *>(L.k));
    A.v = static_cast<uint16_t *>(const_cast<void *>(L.v));
    A.k_token = L.k_token;
    A.k_head = L.k_head;
    A.v_token = L.v_token;
    A.v_head = L.v_head;
    A.tokens = L.tokens;
    A.cache = L.cache;
    A.batch = L.batch;
    A.status = L.status;
    // A token's rows are shared by as many warps as it takes to give every SM
    // 16 of them; a warp per token where there are more (fewer lookups).
    const int steps = (2 * L.cache.heads * (L.cache.head_dim / 8) + 31) / 32;
    int splits = 1;
    while (splits < steps && L.tokens * splits < 148 * 16) splits *= 2;
    A.splits = splits;
    const int64_t blocks = (L.tokens * splits + 7) / 8;
    const dim3 grid((unsigned)blocks), block(256);
#define DQ_KV(GG, DD)                                                                           \
    if (L.group == GG && L.cache.head_dim == DD)                                                \
        return launch_k(kv_copy_kernel<CODES, GS, GG, DD, READ>, grid, block, 0, L.stream, A);
    DQ_KV(16, 64) DQ_KV(32, 64) DQ_KV(64, 64) DQ_KV(16, 128) DQ_KV(32, 128) DQ_KV(64, 128)
#undef DQ_KV
    return cudaErrorInvalidValue;
}

template <bool READ>
cudaError_t launch_copy(const KvCopyLaunch &L) {
    if (L.gscale == DQ_SCALE_BF16) return launch_fmt<CODES_INT4, SC_BF16, READ>(L);
    if (L.gscale == DQ_SCALE_E4M3) return launch_fmt<CODES_E2M1, SC_E4M3, READ>(L);
    if (L.codes == DQ_CODES_INT4) return launch_fmt<CODES_INT4, SC_E8M0, READ>(L);
    return launch_fmt<CODES_E2M1, SC_E8M0, READ>(L);
}

}  // namespace

cudaError_t launch_kv_append(const KvCopyLaunch &L) { return launch_copy<false>(L); }
cudaError_t launch_kv_read(const KvCopyLaunch &L) { return launch_copy<true>(L); }

}  // namespace dq
