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
// sequences of up to 2048 new tokens (28,300 in all), 8 heads of 128: append in MXFP4 35 us (4.2 TB/s; issue 64%, ALU 59%), MXINT4 38, INT4 with
// BF16 scales 59, NVFP4 90; read 31 (4.8 TB/s).  The last two settle values that
// lie next to a border in branches that were made for float32 products, where
// they are rare.  bf16 values have so few bits that they tie: on random normal
// rows 1.2% of the elements and 6.4% of the groups' scales in NVFP4, so that 96%
// and 65% of the warps' steps take the branches; in INT4 0.24%, 41% of the steps.
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
        // a head's key and value row together: their places differ by the
        // arrays' addresses only, and both loads are under way at once
        const int c = lane % LPR, heads = A.cache.heads, hop = A.splits * RPW;
        const int h0 = part * RPW;                      // (the warp's first head; a lane's is up to RPW - 1 more)
        const int64_t row = row0 + (int64_t)(h0 + lane / LPR) * A.cache.page_size;
        int64_t co = row * (D / 2) + 4 * c, so = row * (D / G) + c / (G / 8);
        const int64_t co_hop = (int64_t)hop * A.cache.page_size * (D / 2);
        const int64_t so_hop = (int64_t)hop * A.cache.page_size * (D / G);
        uint16_t *x[2] = {A.k + t * A.k_token + (h0 + lane / LPR) * A.k_head + 8 * c,
                          A.v + t * A.v_token + (h0 + lane / LPR) * A.v_head + 8 * c};
        const int64_t x_hop[2] = {hop * A.k_head, hop * A.v_head};
        uint8_t *const codes[2] = {A.cache.k_codes, A.cache.v_codes};
        void *const scales[2] = {A.cache.k_scales, A.cache.v_scales};
        for (int h = h0; h < heads; h += hop, co += co_hop, so += so_hop, x[0] += x_hop[0], x[1] += x_hop[1]) {
            const bool ok = h + lane / LPR < heads;
            uint4 in[2];
            float sc[2];
#pragma unroll
            for (int i = 0; i < 2; ++i) {
                in[i] = make_uint4(0, 0, 0, 0);
                sc[i] = 0.0f;
                if constexpr (READ) {
                    if (ok && row0 >= 0) {
                        in[i].x = *reinterpret_cast<const uint32_t *>(codes[i] + co);
                        sc[i] = scale_value<GS>(scales[i], so);
                    }
                } else {
                    if (ok) in[i] = __ldg(reinterpret_cast<const uint4 *>(x[i]));
                }
            }
#pragma unroll
            for (int i = 0; i < 2; ++i) {
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
                    if (ok) *reinterpret_cast<uint4 *>(x[i]) = make_uint4(p[0], p[1], p[2], p[3]);
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
                    if (!ok) continue;
                    *reinterpret_cast<uint32_t *>(codes[i] + co) = cw[0];
                    if (c % (G / 8) == 0) {
                        if constexpr (GS == SC_BF16)
                            static_cast<uint16_t *>(scales[i])[so] = (uint16_t)(__float_as_uint(s) >> 16);
                        else if constexpr (GS == SC_E8M0)
                            static_cast<uint8_t *>(scales[i])[so] = (uint8_t)(__float_as_uint(s) >> 23);
                        else
                            static_cast<uint8_t *>(scales[i])[so] = (uint8_t)e4m3_bits(s);
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
    const int steps = (L.cache.heads * (L.cache.head_dim / 8) + 31) / 32;
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
