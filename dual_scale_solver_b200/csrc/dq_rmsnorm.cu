// dq_rmsnorm.cu — residual addition, root-mean-square norm and activation
// quantization in one pass over a token's row:
//
//   h = x + r,  r' = bf16(h),  y = h / sqrt(mean h^2 + eps) * w * b,  Q(y)
//
// The step in front of every quantized linear.  It is bound by memory: a row
// is read once (x and r, 4 bytes per element), held in registers as float32
// while its sum of squares is reduced over the CTA, and leaves as r' (2
// bytes) and codes (1 byte or less) with their scales.  A CTA takes one row;
// a thread holds C chunks of 8 consecutive elements (16-byte loads), so a
// group of G elements spans G / 8 neighbouring lanes and its maximum is a
// shuffle butterfly, as in the activation mode of the tile kernel, whose
// quantizer (Quant::run) makes the decisions.  The sum of squares is added
// per thread in element order (at most 32 of them in float32), then over lanes
// and (in 64 bits) warps in a fixed order.
// 32768 rows of 8192 with a residual, MXFP8 E5M2: 350 us, 5.4 TB/s, 82% of a
// copy's rate (347 with the last sums and the root in float32).  Of these 268
// million codes 62 to 124 are not those of the exact y (six inputs, 81 in the
// mean; with elementary float32 operations 70 to 117, 93 in the mean).  Forming
// a y next to a border again in 64 bits left 1 to 16 of them, at 394 us.
#include <cuda_runtime.h>

#include <type_traits>

#include "dq_launch.h"
#include "dq_serving.h"

namespace dq {

namespace {

constexpr int kNormMaxThreads = 1024;

struct NormArgs {
    const uint16_t *x, *res;
    int64_t x_stride, res_stride;
    const void *weight;
    int weight_f32;
    const float *b;
    float eps;
    double per_k;            // 1 / K
    int64_t tokens;
    int K;
    uint16_t *res_out;
    int64_t res_out_stride;
    uint8_t *codes;
    void *scales;
    unsigned int *status;
};

__device__ __forceinline__ void unpack8(const uint4 &v, f2 (&w)[4]) {
    const uint32_t u[4] = {v.x, v.y, v.z, v.w};
#pragma unroll
    for (int k = 0; k < 4; ++k)
        w[k] = make_float2(__uint_as_float(u[k] << 16), __uint_as_float(u[k] & 0xFFFF0000u));
}

__device__ __forceinline__ uint32_t bf16x2_rn(float lo, float hi) {
    uint32_t r;
    asm("cvt.rn.bf16x2.f32 %0, %1, %2;" : "=r"(r) : "f"(hi), "f"(lo));
    return r;
}

// h = x + r of one chunk
__device__ __forceinline__ void load_h(const NormArgs &A, int64_t row, int c, f2 (&h)[4]) {
    // (plain loads, not the read-only path: residual_out may be either buffer)
    unpack8(*reinterpret_cast<const uint4 *>(A.x + row * A.x_stride + 8 * (int64_t)c), h);
    if (A.res) {
        f2 r[4];
        unpack8(*reinterpret_cast<const uint4 *>(A.res + row * A.res_stride + 8 * (int64_t)c), r);
#pragma unroll
        for (int k = 0; k < 4; ++k) h[k] = __fadd2_rn(h[k], r[k]);
    }
}

// One chunk's y, its quantization and the stores.
template <int CODES, int GS, int G>
__device__ __forceinline__ void finish_chunk(const NormArgs &A, int64_t row, int c, bool ok, float inv,
                                             const f2 (&h)[4]) {
    constexpr int LPG = G / 8;
    constexpr int BITS = CodeTraits<CODES>::kBits;
    f2 y[4];
#pragma unroll
    for (int k = 0; k < 4; ++k) y[k] = make_float2(0.0f, 0.0f);
    if (ok) {
        f2 w[4];
        if (A.weight_f32) {
            const float4 *p = reinterpret_cast<const float4 *>(A.weight) + 2 * (int64_t)c;
            const float4 p0 = __ldg(p), p1 = __ldg(p + 1);
            w[0] = make_float2(p0.x, p0.y);
            w[1] = make_float2(p0.z, p0.w);
            w[2] = make_float2(p1.x, p1.y);
            w[3] = make_float2(p1.z, p1.w);
        } else {
            unpack8(__ldg(reinterpret_cast<const uint4 *>(A.weight) + c), w);
        }
#pragma unroll
        for (int k = 0; k < 4; ++k) y[k] = mul2(mul2(h[k], bcast(inv)), w[k]);
        if (A.b) {
            const float4 *p = reinterpret_cast<const float4 *>(A.b) + 2 * (int64_t)c;
            const float4 p0 = __ldg(p), p1 = __ldg(p + 1);
            y[0] = mul2(y[0], make_float2(p0.x, p0.y));
            y[1] = mul2(y[1], make_float2(p0.z, p0.w));
            y[2] = mul2(y[2], make_float2(p1.x, p1.y));
            y[3] = mul2(y[3], make_float2(p1.z, p1.w));
        }
        if (A.res_out) {
            uint4 o;
            o.x = bf16x2_rn(h[0].x, h[0].y);
            o.y = bf16x2_rn(h[1].x, h[1].y);
            o.z = bf16x2_rn(h[2].x, h[2].y);
            o.w = bf16x2_rn(h[3].x, h[3].y);
            *reinterpret_cast<uint4 *>(A.res_out + row * A.res_out_stride + 8 * (int64_t)c) = o;
        }
    }
    // every lane of the warp takes part (group shuffles)
    f2 code[4];
    float s, s_eff;
    uint32_t cw[2], mbits;
    bool nonzero;
    Quant<CODES, GS, SC_BF16, true, 4, LPG>::template run<true>(y, y, 1.0f, 1.0f, y, 1.0f, 1.0f,
                                                                A.status, code, s, s_eff, cw,
                                                                nonzero, mbits);
    if (!ok) return;
    uint8_t *cp = A.codes + row * ((int64_t)A.K * BITS / 8) + (int64_t)c * BITS;
    if constexpr (BITS == 4) {
        *reinterpret_cast<uint32_t *>(cp) = cw[0];
    } else if constexpr (BITS == 8) {
        *reinterpret_cast<uint2 *>(cp) = make_uint2(cw[0], cw[1]);
    } else {
        uint16_t *p = reinterpret_cast<uint16_t *>(cp);
        p[0] = (uint16_t)cw[0];
        p[1] = (uint16_t)(cw[0] >> 16);
        p[2] = (uint16_t)cw[1];
    }
    if (c % LPG == 0) {
        const int64_t gi = row * (A.K / G) + c / LPG;
        const uint32_t sb = __float_as_uint(s);
        if constexpr (GS == SC_BF16)
            reinterpret_cast<uint16_t *>(A.scales)[gi] = (uint16_t)(sb >> 16);
        else if constexpr (GS == SC_E8M0)
            reinterpret_cast<uint8_t *>(A.scales)[gi] = (uint8_t)(sb >> 23);
        else
            reinterpret_cast<uint8_t *>(A.scales)[gi] = (uint8_t)e4m3_bits(s);
    }
}

// Sum over the CTA in a fixed order (lanes by butterfly, then warps); every
// thread gets it.  The warps' sums are added in 64 bits: the last few
// additions hold most of the sum's rounding.  T: the type of the threads' sums.
template <typename T>
__device__ __forceinline__ double block_sum(T v, T *part) {
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) v += __shfl_xor_sync(0xffffffffu, v, o);
    const int nw = blockDim.x >> 5;
    if (nw == 1) return v;
    if ((threadIdx.x & 31) == 0) part[threadIdx.x >> 5] = v;
    __syncthreads();
    double d = (int)(threadIdx.x & 31) < nw ? part[threadIdx.x & 31] : T(0);
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) d += __shfl_xor_sync(0xffffffffu, d, o);
    return d;
}

// 1 / sqrt(v) to little more than half a step: a float32 estimate and one
// Newton step whose residual is formed in 64 bits.
__device__ __forceinline__ float rsqrt_near(double v) {
    const float r = 1.0f / sqrtf((float)v);
    const double d = fma(v * (double)r, (double)r, -1.0);
    return fmaf(-0.5f * r, (float)d, r);
}

// C > 0: a row is at most C * blockDim.x chunks, held in registers.
// C == 0: any K; the row is read a second time for the quantization (from L2).
// A thread then has K / 1024 squares, up to 2^18: its sum is taken to 64 bits
// after each chunk, since 2^14 equal squares already lose 6e-5 in float32.
template <int CODES, int GS, int G, int C>
__global__ void __launch_bounds__(kNormMaxThreads)
rmsnorm_quant_kernel(const NormArgs A) {
    grid_dependency_begin();
    using Sum = typename std::conditional<(C > 0), float, double>::type;
    __shared__ Sum part[32];
    const int nch = A.K / 8;
    const int64_t row = blockIdx.x;
    constexpr int CH = C > 0 ? C : 1;
    f2 h[CH][4];
    Sum ss = 0;
    const int loops = C > 0 ? C : (nch + (int)blockDim.x - 1) / (int)blockDim.x;
#pragma unroll
    for (int i = 0; i < loops; ++i) {
        const int c = (int)threadIdx.x + i * (int)blockDim.x;
        f2(&hh)[4] = h[C > 0 ? i : 0];
#pragma unroll
        for (int k = 0; k < 4; ++k) hh[k] = make_float2(0.0f, 0.0f);
        if (c < nch) load_h(A, row, c, hh);
        if constexpr (C == 0) {
            float chunk = 0.0f;
#pragma unroll
            for (int k = 0; k < 4; ++k) chunk = fmaf(hh[k].y, hh[k].y, fmaf(hh[k].x, hh[k].x, chunk));
            ss += chunk;
        }
    }
    if constexpr (C > 0) {
#pragma unroll
        for (int i = 0; i < C; ++i)
#pragma unroll
            for (int k = 0; k < 4; ++k) ss = fmaf(h[i][k].y, h[i][k].y, fmaf(h[i][k].x, h[i][k].x, ss));
    }
    const double sum = block_sum(ss, part);
    if (threadIdx.x == 0 && !(sum <= 3.4028234663852886e38))
        atomicOr(A.status, STATUS_NONFINITE);
    const float inv = rsqrt_near(fma(sum, A.per_k, (double)A.eps));
#pragma unroll
    for (int i = 0; i < loops; ++i) {
        const int c = (int)threadIdx.x + i * (int)blockDim.x;
        f2(&hh)[4] = h[C > 0 ? i : 0];
        if constexpr (C == 0) {
            if (c < nch) load_h(A, row, c, hh);
        }
        finish_chunk<CODES, GS, G>(A, row, c, c < nch, inv, hh);
    }
}

template <int CODES, int GS, int G, int C>
cudaError_t launch_c(const NormLaunch &L, const NormArgs &A, int threads) {
    return launch_k(rmsnorm_quant_kernel<CODES, GS, G, C>, dim3((unsigned)L.tokens), dim3(threads), 0,
                    L.stream, A);
}

template <int CODES, int GS, int G>
cudaError_t launch_g(const NormLaunch &L) {
    NormArgs A;
    A.x = static_cast<const uint16_t *>(L.x);
    A.res = static_cast<const uint16_t *>(L.residual);
    A.x_stride = L.x_stride;
    A.res_stride = L.res_stride;
    A.weight = L.weight;
    A.weight_f32 = L.weight_f32;
    A.b = L.b;
    A.eps = L.eps;
    A.tokens = L.tokens;
    A.K = (int)L.K;
    A.per_k = 1.0 / (double)L.K;
    A.res_out = static_cast<uint16_t *>(L.residual_out);
    A.res_out_stride = L.res_out_stride;
    A.codes = L.out_codes;
    A.scales = L.out_scales;
    A.status = L.status;
    const int64_t nch = L.K / 8;
    const auto round32 = [](int64_t n) { return (int)((n + 31) / 32 * 32); };
    if (nch > 4 * kNormMaxThreads) return launch_c<CODES, GS, G, 0>(L, A, kNormMaxThreads);
    // 8 elements a thread while rows are few or short (a row's latency counts),
    // 32 where many wide rows come one after the other on an SM (more loads in
    // flight, fewer reductions).  MXFP8, us, 8 against 32: 61 x 8192 2.8, 4.0;
    // 592 x 4096 3.8, 4.5; 1184 x 4096 6.6, 5.9; 592 x 8192 6.9, 6.0; 8192 x
    // 2048 25.2, 26.0; 8192 x 1024 11.7, 13.2; 8192 x 8192 112, 94; 32768 x 8192
    // 429, 347 (16 elements: 409, 64: 501).  MXFP4 with b: 592 x 4096 4.6, 4.7;
    // 592 x 8192 9.9, 8.2; 2048 x 4096 17.2, 16.4; 8192 x 2048 26.9, 27.5; 32768 x
    // 8192 435, 351.  NVFP4 with b: 592 x 4096 6.0, 5.6; 2048 x 4096 24.2, 18.5;
    // 8192 x 1024 18.7, 17.8; 8192 x 2048 35.8, 30.5 (the one that the rule costs
    // most); 32768 x 8192 762, 391.
    if (nch > kNormMaxThreads || (L.K >= 4096 && L.tokens * L.K > (1 << 22)))
        return launch_c<CODES, GS, G, 4>(L, A, round32((nch + 3) / 4));
    return launch_c<CODES, GS, G, 1>(L, A, round32(nch));
}

template <int CODES, int GS>
cudaError_t launch_fmt(const NormLaunch &L) {
    switch (L.group) {
        case 16: return launch_g<CODES, GS, 16>(L);
        case 32: return launch_g<CODES, GS, 32>(L);
        case 64: return launch_g<CODES, GS, 64>(L);
    }
    return cudaErrorInvalidValue;
}

}  // namespace

cudaError_t launch_rmsnorm_quant(const NormLaunch &L) {
    if (L.gscale == DQ_SCALE_BF16) return launch_fmt<CODES_INT4, SC_BF16>(L);
    if (L.gscale == DQ_SCALE_E4M3) return launch_fmt<CODES_E2M1, SC_E4M3>(L);
    switch (L.codes) {
        case DQ_CODES_INT4: return launch_fmt<CODES_INT4, SC_E8M0>(L);
        case DQ_CODES_E2M1: return launch_fmt<CODES_E2M1, SC_E8M0>(L);
        case DQ_CODES_INT8: return launch_fmt<CODES_INT8, SC_E8M0>(L);
        case DQ_CODES_E4M3: return launch_fmt<CODES_E4M3, SC_E8M0>(L);
        case DQ_CODES_E5M2: return launch_fmt<CODES_E5M2, SC_E8M0>(L);
        case DQ_CODES_E2M3: return launch_fmt<CODES_E2M3, SC_E8M0>(L);
        case DQ_CODES_E3M2: return launch_fmt<CODES_E3M2, SC_E8M0>(L);
    }
    return cudaErrorInvalidValue;
}

}  // namespace dq
