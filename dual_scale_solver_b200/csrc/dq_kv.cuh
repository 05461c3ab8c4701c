// dq_kv.cuh — device side shared by the 4-bit cache's kernels: the batch's
// sequences, the places of their tokens, group scales.
#pragma once

#include "dq_launch.h"
#include "dq_serving.h"

namespace dq {

// One sequence of a batch, checked: new tokens [s0, s0 + n), `len` positions
// in all.  ok is false (and n = 0) for a sequence whose starts or length are
// out of range.
struct KvSeq {
    int s0, n, len;
    bool ok;
};

__device__ __forceinline__ KvSeq kv_seq(const dq_kv_batch &b, int page_size, int64_t tokens, int i) {
    KvSeq s;
    const int a = __ldg(b.starts + i), e = __ldg(b.starts + i + 1);
    s.s0 = a;
    s.n = e - a;
    s.len = __ldg(b.kv_lens + i);
    s.ok = a >= 0 && e >= a && (int64_t)e <= tokens && s.len >= 0 &&
           (int64_t)s.len <= (int64_t)b.max_pages * page_size;
    if (!s.ok) s.n = 0, s.len = 0;
    return s;
}

// Row of the cache (in units of one token's codes or scales of one head) of
// position `pos`, or -1 if its page is out of range.
__device__ __forceinline__ int64_t kv_row(const dq_kv_cache &c, const dq_kv_batch &b, int seq,
                                          int pos, int head) {
    const int pi = pos / c.page_size;
    const int page = __ldg(b.block_table + seq * b.table_stride + pi);
    if (page < 0 || (int64_t)page >= c.pages) return -1;
    return ((int64_t)page * c.heads + head) * c.page_size + (pos - pi * c.page_size);
}

// Sequence that holds token row t (the warp looks 32 starts at a time): the
// last i in [0, seqs] with starts[i] <= t, which is seqs for the rows behind
// the last sequence.  -1 if t lies before the first one.  All lanes call it
// with the same t.
__device__ __forceinline__ int kv_find(const dq_kv_batch &b, int64_t t) {
    int lo = 0, n = b.seqs + 1;                        // the answer is below lo + n
    const int lane = threadIdx.x & 31;
    while (true) {
        const int step = (n + 31) >> 5;
        const int i = lo + lane * step;
        const bool le = lane * step < n && (int64_t)__ldg(b.starts + i) <= t;
        const int k = __popc(__ballot_sync(0xffffffffu, le));
        if (k == 0) return lo - 1;
        const int next = lo + (k - 1) * step;
        if (step == 1) return next;
        n = min(step, lo + n - next);
        lo = next;
    }
}

template <int GS>
__device__ __forceinline__ float scale_value(const void *scales, int64_t i) {
    if constexpr (GS == SC_BF16) {
        return __uint_as_float((uint32_t)reinterpret_cast<const uint16_t *>(scales)[i] << 16);
    } else if constexpr (GS == SC_E8M0) {
        return __uint_as_float((uint32_t)reinterpret_cast<const uint8_t *>(scales)[i] << 23);
    } else {
        const uint16_t u = reinterpret_cast<const uint8_t *>(scales)[i];
        uint32_t h2;
        asm("cvt.rn.f16x2.e4m3x2 %0, %1;" : "=r"(h2) : "h"(u));
        float f;
        asm("{ .reg .f16 l, h; mov.b32 {l, h}, %1; cvt.f32.f16 %0, l; }" : "=f"(f) : "r"(h2));
        return f;
    }
}

}  // namespace dq
