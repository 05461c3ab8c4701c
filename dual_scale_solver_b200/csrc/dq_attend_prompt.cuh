// dq_attend_prompt.cuh — attention of many query rows over the 4-bit cache on
// the tcgen05 tensor cores.
//
// A CTA takes 256 query rows (two tiles of 128; a row is one token and one
// head of the group, so a group's heads share every code) of one sequence
// and cache head, and walks the positions in tiles of 128:
//
//   S = Q K^T    tcgen05.mma, 128 x 128 x D, both operands fp16 in shared
//                memory, float32 in TMEM
//   P = 2^(S f - m)  by the rows' threads (TMEM -> registers -> TMEM, fp16)
//   O += P V     tcgen05.mma, 128 x D x 128, P from TMEM, V fp16 in shared
//                memory, float32 in TMEM
//
// and the two row tiles take turns, so that one tile's softmax runs while the
// tensor core works for the other.  The products are bound by the tensor
// core (4 D flops per pair of row and position, 4096 multiply-adds per clock
// and SM), closely followed by the exponentials (16 per clock and SM).
//
// Codes become fp16 exactly: a code times its group scale has at most 11
// significant bits, and the scales of a warp's 32 tokens are taken relative
// to 2^E, E the exponent of the largest of them (what lies 2^-24 or further
// below is lost to fp16's smallest step).  E of the keys is part of the
// factor that takes scores to log2 units; E of the values is part of the
// exponent that P is formed with, and of the running maximum, so that P stays
// at most 2^15.  The maximum is raised only when it has to grow by more than
// 2^8 (O is then rescaled in TMEM); P is rounded to fp16 (2^-12 at most), its
// sum is float32.
//
//   warps 0-3, 4-7   softmax of row tile 0, 1: a thread per row; they also
//                    bring in the row of Q and write the row of the output
//   warps 8-11       codes -> fp16 tiles: a thread per token, 64 bytes of
//                    codes in registers while the previous tile is expanded
//   warps 12, 13     issue the MMAs of row tile 0, 1
// Every wait is bounded (dq_tc.cuh).
//
// Scores are taken in steps of 64 positions, two steps' columns in turn, so
// that the products of one step run during the softmax of the next (one step
// of 128: 1.13 against 1.07 ms).  Measured (64 query over 8 cache heads, D =
// 128, MXFP4): 2 sequences of 1000 new tokens over 16384 positions 952 us, 1.04
// PFLOP/s; 2048 new tokens alone (32 query heads, MXFP4) 55 us, 0.62 PFLOP/s.
// Scores 64 columns wide run at two thirds of the tensor core's rate, so the
// products fill 55% of its time; exponentials fill 44% of theirs.  More warps
// (eight that expand codes, or two softmax teams) were slower, 1.2 ms: the
// registers a thread keeps fall below 96.  At 128 each instantiation spills 5 to 9
// of them (20 to 36 bytes).
#pragma once

#include "dq_attend.cuh"
#include "dq_tc.cuh"

namespace dq {

constexpr int kPromptRows = 256;                 // query rows of a CTA
constexpr int kPromptTile = 128;                 // positions of a tile of keys or values
constexpr int kPromptStep = 64;                  // positions of a step of the softmax
constexpr int kPromptThreads = 448;
constexpr int kPromptCtas = 148;
constexpr int kPromptPlan = 64;                  // sequences, and
constexpr int kPromptRounds = 8;                 // rounds of the grid, that cutting is planned for
constexpr int kPromptItem = 2;                   // position tiles that an item costs beside its own
constexpr int kPromptJoin = 6;                   // position tiles that cutting items costs a CTA
constexpr int kPromptK0 = 12;                    // fp16 code x scale: at most 7 * 2^13

// Byte of 16-byte chunk c (8 elements) of a row in a tile of 128 rows.
__device__ __forceinline__ uint32_t prompt_off(int row, int c) {
    return (uint32_t)((c >> 3) * (128 * 128) + row * 128 + (((c & 7) ^ (row & 7)) << 4));
}

// A piece of work: 256 query rows of a sequence and cache head over the
// position tiles [t0, t1) of the `steps` that the rows see.
struct PromptItem {
    KvSeq s;
    int seq, head, row0;
    int rows[2], nt[2];                          // valid rows and steps of 64 positions of each row tile
    int steps, t0, t1;
};

// A warp's way through the CTA's pieces.  Either whole items: a sequence's row
// tiles from the last (longest, when causal) to the first, all heads of each;
// rounds of the grid run forwards and backwards in turn, so that long and
// short ones pair up.  Or (left >= 0) an equal share of all position tiles in
// that order (and of kPromptItem more behind each item's, for its beginning
// and end), its first and last item cut where need be.
struct PromptWalk {
    int seq, round, tile, head, t;
    long long first, left;
    PromptItem it;
    // The next piece, for the whole warp whose walk this is (in shared memory,
    // worked out by one lane: registers are short elsewhere).
    __device__ __forceinline__ bool next(const AttArgs &A, bool report) {
        __syncwarp();
        skip(A, report);
        if ((threadIdx.x & 31) == 0) step(A);
        __syncwarp();
        // a share may begin behind an item's last tile
        if (it.seq >= 0 && it.t0 == it.t1 && it.steps > 0) {
            skip(A, report);
            if ((threadIdx.x & 31) == 0) step(A);
            __syncwarp();
        }
        return it.seq >= 0;
    }
    // row tile pairs of a sequence (none of one that the other kernel takes)
    __device__ __forceinline__ static int tiles(const AttArgs &A, const KvSeq &s) {
        const long long rows = (long long)s.n * A.group;
        return rows <= A.few ? 0 : (int)((rows + kPromptRows - 1) / kPromptRows);
    }
    // The place of the next whole item.
    __device__ __forceinline__ long long index() const {
        const long long n = gridDim.x;
        return round * n + ((round & 1) ? n - 1 - blockIdx.x : blockIdx.x);
    }
    // Passes over the sequences that have no part in the next piece, 32 at a
    // time (the whole warp).
    __device__ __forceinline__ void skip(const AttArgs &A, bool report) {
        const int lane = threadIdx.x & 31, seqs = A.batch.seqs;
        const bool cut = left >= 0, stay = cut && tile >= 0;
        const long long idx = index();
        int at = seq;
        long long before = first;
        __syncwarp();
        while (!stay && at < seqs) {
            long long cnt = 0;
            if (at + lane < seqs) {
                const KvSeq s = kv_seq(A.batch, A.cache.page_size, A.tokens, at + lane);
                if (!s.ok && report) atomicOr(A.status, STATUS_INDEX);
                cnt = (long long)tiles(A, s) * A.cache.heads;
            }
            long long incl = cnt;
#pragma unroll
            for (int o = 1; o < 32; o <<= 1) {
                const long long y = __shfl_up_sync(0xffffffffu, incl, o);
                if (lane >= o) incl += y;
            }
            const uint32_t hit = __ballot_sync(0xffffffffu, cut ? cnt > 0 : idx < before + incl);
            const int k = hit ? __ffs(hit) - 1 : 31;
            before += __shfl_sync(0xffffffffu, hit ? incl - cnt : incl, k);
            at += hit ? k : 32;
            if (hit) break;
        }
        if (lane == 0) seq = at, first = before;
    }
    // position tiles that row tile pair `tile` sees
    __device__ __forceinline__ static int span(const AttArgs &A, const KvSeq &s, int tile) {
        const int last = (int)min((long long)(tile + 1) * kPromptRows, (long long)s.n * A.group) - 1;
        return (limit(A, s, last) + kPromptTile - 1) / kPromptTile;
    }
    __device__ __forceinline__ void fill(const AttArgs &A, const KvSeq &s, int tl, int hd) {
        const int all = s.n * A.group;
        it.s = s;
        it.seq = seq;
        it.head = hd;
        it.row0 = tl * kPromptRows;
        it.steps = 0;
        for (int i = 0; i < 2; ++i) {
            const int r0 = it.row0 + 128 * i;
            it.rows[i] = min(max(all - r0, 0), 128);
            it.nt[i] = it.rows[i] == 0 ? 0 : (limit(A, s, r0 + it.rows[i] - 1) + kPromptStep - 1) / kPromptStep;
            it.steps = max(it.steps, (it.nt[i] + 1) / 2);
        }
        it.t0 = 0;
        it.t1 = it.steps;
    }
    __device__ __forceinline__ void step(const AttArgs &A) {
        const long long local = index() - first;
        ++round;
        it.seq = -1;
        if (seq >= A.batch.seqs || left == 0) return;
        const KvSeq s = kv_seq(A.batch, A.cache.page_size, A.tokens, seq);
        if (left < 0) {
            const int up = (int)(local / A.cache.heads);
            fill(A, s, tiles(A, s) - 1 - up, (int)(local - (long long)up * A.cache.heads));
            return;
        }
        if (tile < 0) tile = tiles(A, s) - 1;              // a new sequence
        fill(A, s, tile, head);
        const int len = max(it.steps, 1) + kPromptItem, take = (int)min(left, (long long)len - t);
        it.t0 = min(t, it.steps);
        it.t1 = min(t + take, it.steps);
        left -= take;
        t += take;
        if (t >= len) {
            t = 0;
            if (++head == A.cache.heads) {
                head = 0;
                if (--tile < 0) ++seq;
            }
        }
    }
    // positions below it are seen by the row
    __device__ __forceinline__ static int limit(const AttArgs &A, const KvSeq &s, int row) {
        return A.causal ? min(max(s.len - s.n + row / A.group + 1, 0), s.len) : s.len;
    }
};

template <int D>
struct __align__(1024) PromptSmem {
    uint8_t q[2][128 * D * 2];
    uint8_t k[2][128 * D * 2];
    uint8_t v[2][128 * D * 2];
    uint64_t q_full[2];                                      // by row tile
    uint64_t s_full[2][2], p_full[2][2], o_full[2][2];       // by row tile and half of its score columns
    uint64_t k_full[2], k_empty[2], v_full[2], v_empty[2];   // by stage
    uint64_t drained[2];
    // of a position tile (mod 8) and 32 of its tokens: 2^(E - k0) of the
    // keys, E and 2^-E of the values
    float kf[8][4], ve[8][4], vi[8][4];
    PromptWalk walk[14];                         // of each warp
    unsigned long long plan_units, plan_items, plan_most;
    long long plan[kPromptPlan];                 // position tiles of each sequence
    uint32_t tmem;
    int abort;
};

// One token's codes of one head (passing L1 by), and its scales (zeros for
// row < 0).
__device__ __forceinline__ uint4 prompt_load(const uint4 *p) {
    uint4 v;
    asm volatile("ld.global.nc.L1::no_allocate.v4.u32 {%0, %1, %2, %3}, [%4];"
                 : "=r"(v.x), "=r"(v.y), "=r"(v.z), "=r"(v.w) : "l"(p));
    return v;
}
template <int D>
__device__ __forceinline__ void prompt_codes(uint4 (&c)[D / 32], const uint8_t *codes, int64_t row) {
    const uint4 *p = reinterpret_cast<const uint4 *>(codes + row * (D / 2));
#pragma unroll
    for (int i = 0; i < D / 32; ++i) c[i] = row >= 0 ? prompt_load(p + i) : make_uint4(0, 0, 0, 0);
}
template <int SB>
__device__ __forceinline__ void prompt_scales(ScaleWords<SB> &s, const void *scales, int64_t row) {
    if (row >= 0) {
        s.load(static_cast<const uint8_t *>(scales) + row * SB);
    } else {
#pragma unroll
        for (int i = 0; i < ScaleWords<SB>::N; ++i) s.w[i] = 0;
    }
}

// Expands a token's row into a tile, with scales relative to 2^e; the order of
// the 8 elements of a chunk is the one the code conversion gives
// (prompt_order).
template <int CODES, int GS, int G, int D, int SB>
__device__ __forceinline__ void prompt_expand(const uint4 (&c)[D / 32], const ScaleWords<SB> &sw, int e,
                                              uint8_t *tile, int row) {
    const float down = pow2f(kPromptK0 - e);
    uint32_t s2[D / G];
#pragma unroll
    for (int g = 0; g < D / G; ++g) {
        const float s = sw.template get<GS>(g) * down;
        s2[g] = f16x2_rn(s, s);
    }
#pragma unroll
    for (int i = 0; i < D / 32; ++i) {
        const uint32_t w[4] = {c[i].x, c[i].y, c[i].z, c[i].w};
#pragma unroll
        for (int k = 0; k < 4; ++k) {
            uint32_t h[4];
            if constexpr (CODES == CODES_INT4) int4_halves(w[k], h);
            else e2m1_bytes(w[k], h);
            const uint32_t f = s2[(32 * i + 8 * k) / G];
            *reinterpret_cast<uint4 *>(tile + prompt_off(row, 4 * i + k)) =
                make_uint4(hmul2(h[0], f), hmul2(h[1], f), hmul2(h[2], f), hmul2(h[3], f));
        }
    }
}

// Channel (0..7 of a chunk) at place p of a chunk in the tiles.
template <int CODES>
__host__ __device__ constexpr int prompt_order(int p) {
    return CODES == CODES_INT4 ? (p & 1) * 4 + (p >> 1) : p;
}

// Whether this call's items are cut into equal shares, and where this CTA's
// share begins.  In tiles, whole items take what the CTA with the most of them
// has; shares the mean and kPromptJoin for writing and joining the pieces (256
// rows of float32 each).  MXFP4, 32 query over 8 heads of 128, us, whole
// against cut: 512 new tokens over 8192 148, 89; 128 over 2048 47, 31; 4 x 512
// over 4096 150, 137; 2 x 1000 over 16384 (64 query heads) 1071, 952; 300 over
// 20000 (8 query heads) 342, 67; 1000 over 1000 (9 over 3 heads of 64) 23.5,
// 21.6; 16 x 100 over 3000 82, 89; 4096 over 4096 165, and 403 before an item's
// beginning and end counted.
template <class Smem>
__device__ __forceinline__ void prompt_plan(const AttArgs &A, Smem &sm, int warp, int lane) {
    const int seqs = A.batch.seqs, heads = A.cache.heads, n = gridDim.x;
    const auto length = [&](const KvSeq &s, int tile) { return max(1, PromptWalk::span(A, s, tile)) + kPromptItem; };
    __syncthreads();                             // (the sums are zero)
    for (int b = warp; b < seqs; b += kPromptThreads / 32) {
        const KvSeq s = kv_seq(A.batch, A.cache.page_size, A.tokens, b);
        if (!s.ok && blockIdx.x == 0 && lane == 0) atomicOr(A.status, STATUS_INDEX);
        const int tiles = PromptWalk::tiles(A, s);
        long long sum = 0;
        for (int i = lane; i < tiles; i += 32) sum += length(s, i);
#pragma unroll
        for (int o = 16; o > 0; o >>= 1) sum += __shfl_xor_sync(0xffffffffu, sum, o);
        if (lane == 0) {
            sm.plan[b] = sum * heads;
            atomicAdd(&sm.plan_units, (unsigned long long)(sum * heads));
            atomicAdd(&sm.plan_items, (unsigned long long)tiles * heads);
        }
    }
    __syncthreads();
    const long long units = sm.plan_units, items = sm.plan_items;
    if (items == 0 || items > (long long)kPromptRounds * n) return;
    for (int i = threadIdx.x; i < n; i += kPromptThreads) {
        // the whole items of CTA i (as PromptWalk::index)
        long long load = 0, first = 0;
        int b = 0;
        KvSeq s = kv_seq(A.batch, A.cache.page_size, A.tokens, b);
        for (int r = 0; (long long)r * n < items; ++r) {
            const long long idx = (long long)r * n + ((r & 1) ? n - 1 - i : i);
            if (idx >= items) break;
            while (idx >= first + (long long)PromptWalk::tiles(A, s) * heads) {
                first += (long long)PromptWalk::tiles(A, s) * heads;
                s = kv_seq(A.batch, A.cache.page_size, A.tokens, ++b);
            }
            load += length(s, PromptWalk::tiles(A, s) - 1 - (int)((idx - first) / heads));
        }
        atomicMax(&sm.plan_most, (unsigned long long)load);
    }
    __syncthreads();
    if ((long long)sm.plan_most * n <= units + (long long)kPromptJoin * n) return;
    // the place of unit u0, by one thread of each warp for its own walk
    const int shares = (int)min((long long)n, units);          // (none of them empty)
    const long long u0 = units * blockIdx.x / shares, u1 = units * (blockIdx.x + 1) / shares;
    if (lane == 0) {
        PromptWalk &w = sm.walk[warp];
        w.left = (int)blockIdx.x < shares ? u1 - u0 : 0;
        long long at = u0;
        int b = 0;
        while (b < seqs && at >= sm.plan[b]) at -= sm.plan[b++];       // (b = seqs behind the last share)
        w.seq = b;
        if (b < seqs && w.left > 0) {
            const KvSeq s = kv_seq(A.batch, A.cache.page_size, A.tokens, b);
            int tile = PromptWalk::tiles(A, s) - 1;
            long long len = length(s, tile);
            while (at >= len * heads) {
                at -= len * heads;
                --tile;
                len = length(s, tile);
            }
            w.tile = tile;
            w.head = (int)(at / len);
            w.t = (int)(at - w.head * len);
        }
    }
}

template <int CODES, int GS, int G, int D>
__global__ void __launch_bounds__(kPromptThreads, 1)
attend_prompt_kernel(const AttArgs A, int split) {
    using Smem = PromptSmem<D>;
    constexpr int SB = D / G * (GS == SC_BF16 ? 2 : 1);
    grid_dependency_begin();
    extern __shared__ uint8_t prompt_smem_raw[];
    Smem &sm = *reinterpret_cast<Smem *>(
        (reinterpret_cast<uintptr_t>(prompt_smem_raw) + 1023) & ~uintptr_t(1023));
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    volatile int *abort = &sm.abort;
    if (threadIdx.x == 0) A.meta[blockIdx.x] = AttMeta{};
    if (A.few) {
        // nothing to do where every sequence has few rows
        bool any = false;
        for (int b = threadIdx.x; b < A.batch.seqs; b += kPromptThreads)
            any |= PromptWalk::tiles(A, kv_seq(A.batch, A.cache.page_size, A.tokens, b)) > 0;
        if (!__syncthreads_or(any)) return;
    }
    if (threadIdx.x == 0) {
        for (int i = 0; i < 2; ++i) {
            tc::bar_init(&sm.q_full[i], 128);
            for (int b = 0; b < 2; ++b) {
                tc::bar_init(&sm.s_full[i][b], 1);
                tc::bar_init(&sm.p_full[i][b], 128);
                tc::bar_init(&sm.o_full[i][b], 1);
            }
            tc::bar_init(&sm.drained[i], 1);
            tc::bar_init(&sm.k_full[i], 4);
            tc::bar_init(&sm.k_empty[i], 2);
            tc::bar_init(&sm.v_full[i], 4);
            tc::bar_init(&sm.v_empty[i], 2);
        }
        sm.abort = 0;
        asm volatile("fence.mbarrier_init.release.cluster;" ::: "memory");
    }
    if (lane == 0) {
        PromptWalk &w = sm.walk[warp];
        w.seq = w.round = w.head = w.t = 0;
        w.tile = -1;
        w.first = 0;
        w.left = -1;
    }
    if (threadIdx.x == 0) {
        sm.plan_units = sm.plan_items = sm.plan_most = 0;
    }
    const PromptItem &it = sm.walk[warp].it;
    if (warp == 12) tc::tmem_alloc<512>(&sm.tmem);
    tc::fence_before();
    __syncthreads();
    tc::fence_after();
    const uint32_t tmem = sm.tmem;
    if (split) prompt_plan(A, sm, warp, lane);
    // TMEM columns: S (and P over it) of row tile 0, of row tile 1, O of both

    if (warp < 8) {
        // ---------------- softmax: thread = row ----------------
        const int t = warp >> 2;
        const int row_in = (warp & 3) * 32 + lane;
        const uint32_t lanes = (uint32_t)((warp & 3) * 32) << 16;
        const uint32_t s_addr = tmem + 128 * t + lanes, o_addr = tmem + 256 + D * t + lanes;
        int done = 0;                               // position tiles of this CTA so far (all items)
        int mine = 0;                               // steps of this row tile so far
        bool live = true;
        // the product of the step before this one is in O (of the two steps'
        // barriers in turn: the one before that is, since its scores' columns
        // have been used again)
        const auto summed = [&]() {
            return tc::bar_wait(&sm.o_full[t][(mine - 1) & 1], ((mine - 1) >> 1) & 1, abort, A.status);
        };
        while (live && sm.walk[warp].next(A, false)) {
            const int row = it.row0 + 128 * t + row_in;
            // steps of this piece (none where the row tile sees less than its start)
            const int nt = max(min(it.nt[t], 2 * it.t1) - 2 * it.t0, 0);
            const bool valid = row_in < it.rows[t];
            const int tok = row / A.group;
            const int64_t qrow = it.s.s0 + tok, qhead = (int64_t)it.head * A.group + row - tok * A.group;
            float m = -INFINITY, l = 0.0f;
            if (nt > 0) {
                // this row of Q, as fp16 scaled so that its largest element is in [2^13, 2^14)
                uint32_t top = 0;
                const uint4 *src = reinterpret_cast<const uint4 *>(A.q + qrow * A.q_token + qhead * A.q_head);
                uint4 raw[D / 8];                               // (in the registers that scores take later)
#pragma unroll
                for (int i = 0; i < D / 8; ++i) raw[i] = valid ? __ldg(src + i) : make_uint4(0, 0, 0, 0);
#pragma unroll
                for (int i = 0; i < D / 8; ++i) {
                    const uint4 v = raw[i];
                    top = __vmaxu2(__vmaxu2(top, v.x & 0x7FFF7FFFu), __vmaxu2(v.y & 0x7FFF7FFFu, __vmaxu2(v.z & 0x7FFF7FFFu, v.w & 0x7FFF7FFFu)));
                }
                const int e = max((int)(max(top & 0xFFFFu, top >> 16) >> 7) - 127, -100);
                const float up = pow2f(13 - e);
#pragma unroll
                for (int i = 0; i < D / 8; ++i) {
                    const uint4 v = raw[i];
                    const uint32_t w[4] = {v.x, v.y, v.z, v.w};
                    float x[8];
#pragma unroll
                    for (int k = 0; k < 4; ++k) {
                        x[2 * k] = __uint_as_float(w[k] << 16) * up;
                        x[2 * k + 1] = __uint_as_float(w[k] & 0xFFFF0000u) * up;
                    }
                    uint32_t h[4];
#pragma unroll
                    for (int k = 0; k < 4; ++k)
                        h[k] = f16x2_rn(x[prompt_order<CODES>(2 * k)], x[prompt_order<CODES>(2 * k + 1)]);
                    *reinterpret_cast<uint4 *>(sm.q[t] + prompt_off(row_in, i)) = make_uint4(h[0], h[1], h[2], h[3]);
                }
                const float fac = A.scale_log2 * pow2f(e - 13);
                tc::fence_async();
                tc::bar_arrive(&sm.q_full[t]);
                int seen = valid ? PromptWalk::limit(A, it.s, row) - it.t0 * kPromptTile : 0x7fffffff;   // columns below it count

                for (int j = 0; j < nt; ++j, seen -= kPromptStep) {
                    const int half = mine & 1;                          // of the score columns, in turn
                    const uint32_t cols = s_addr + 64 * half;
                    bool ok = tc::bar_wait(&sm.s_full[t][half], (mine >> 1) & 1, abort, A.status);
                    if (!__all_sync(0xffffffffu, ok)) { live = false; break; }
                    if ((warp & 3) * 32 >= it.rows[t]) {                // no row of this warp's: P may be anything
                        tc::bar_arrive(&sm.p_full[t][half]);
                        ++mine;
                        continue;
                    }
                    tc::fence_after();
                    uint32_t x[2][32];
#pragma unroll
                    for (int c = 0; c < 2; ++c) tc::tmem_load(cols + 32 * c, x[c]);
                    const int slot = (done + (j >> 1)) & 7, quarter = 2 * (j & 1);
                    float f[2], ev[2];
#pragma unroll
                    for (int c = 0; c < 2; ++c) {
                        // (above zero, so that a masked -inf stays -inf; scores here are
                        // below 2^37)
                        f[c] = fmaxf(fac * sm.kf[slot][quarter + c], 1e-37f);
                        ev[c] = sm.ve[slot][quarter + c];
                    }
#pragma unroll
                    for (int c = 0; c < 2; ++c) tc::tmem_load_wait(x[c]);
                    if (seen < 64) {
#pragma unroll
                        for (int c = 0; c < 2; ++c)
#pragma unroll
                            for (int i = 0; i < 32; ++i)
                                if (32 * c + i >= seen) x[c][i] = 0xFF800000u;
                    }
                    // row maximum, each 32 positions with their factor and exponent
                    float want = -INFINITY;
#pragma unroll
                    for (int c = 0; c < 2; ++c) {
                        float a = -INFINITY, b = -INFINITY;
#pragma unroll
                        for (int i = 0; i < 32; i += 4) {
                            a = max3_nan(a, __uint_as_float(x[c][i]), __uint_as_float(x[c][i + 1]));
                            b = max3_nan(b, __uint_as_float(x[c][i + 2]), __uint_as_float(x[c][i + 3]));
                        }
                        want = max_nan(want, fmaf(max_nan(a, b), f[c], ev[c]));
                    }
                    // P is at most 2^7 when the maximum is new, 2^15 before it is raised
                    want -= 7.0f;
                    if (__any_sync(0xffffffffu, want > m + 8.0f)) {
                        const float now = want > m + 8.0f ? want : m;
                        const float alpha = now == m ? 1.0f : ex2(m - now);
                        m = now;
                        l *= alpha;
                        if (j > 0) {
                            ok = summed();
                            if (!__all_sync(0xffffffffu, ok)) { live = false; break; }
                            tc::fence_after();
#pragma unroll 1
                            for (int c = 0; c < D / 8; ++c) {
                                uint32_t o[8];
                                tc::tmem_load8(o_addr + 8 * c, o);
#pragma unroll
                                for (int i = 0; i < 8; ++i) o[i] = __float_as_uint(__uint_as_float(o[i]) * alpha);
                                tc::tmem_store8(o_addr + 8 * c, o);
                            }
                        }
                    }
                    const float mu = m == -INFINITY ? 0.0f : m;
#pragma unroll
                    for (int c = 0; c < 2; ++c) {
                        const float off = ev[c] - mu;
                        float sum0 = 0.0f, sum1 = 0.0f;
#pragma unroll
                        for (int g = 0; g < 2; ++g) {
                            uint32_t p[8];                              // over columns already read
#pragma unroll
                            for (int i = 0; i < 8; ++i) {
                                const float p0 = ex2(fmaf(__uint_as_float(x[c][16 * g + 2 * i]), f[c], off));
                                const float p1 = ex2(fmaf(__uint_as_float(x[c][16 * g + 2 * i + 1]), f[c], off));
                                sum0 += p0;
                                sum1 += p1;
                                p[i] = f16x2_rn(p0, p1);
                            }
                            tc::tmem_store8(cols + 16 * c + 8 * g, p);
                        }
                        l = fmaf(sum0 + sum1, sm.vi[slot][quarter + c], l);
                    }
                    tc::tmem_store_wait();
                    tc::fence_before();
                    tc::bar_arrive(&sm.p_full[t][half]);
                    ++mine;
                }
                if (!live) break;
                const bool ok = summed();
                if (!__all_sync(0xffffffffu, ok)) break;
                tc::fence_after();
            }
            done += it.t1 - it.t0;
            // ---- the row of the output
            const bool whole = it.t0 == 0 && it.t1 == it.steps;
            if (!whole) {
                // a piece: the unnormalized row, its maximum and sum, for the
                // join; columns of 4 channels by rows, so that a warp's stores
                // are contiguous
                const int slot = 2 * (int)blockIdx.x + (it.t0 == 0 ? 1 : 0), prow = 128 * t + row_in;
                float4 *const dst = reinterpret_cast<float4 *>(A.part) + (int64_t)slot * (D / 4) * kPromptRows + prow;
                if ((warp & 3) * 32 < it.rows[t]) {
#pragma unroll 1
                    for (int b = 0; b < D / 32; ++b) {
                        uint32_t o[32];
                        tc::tmem_load(o_addr + 32 * b, o);      // (anything where nt is 0)
                        tc::tmem_load_wait(o);
#pragma unroll
                        for (int c = 0; c < 4; ++c) {
                            float y[8];
#pragma unroll
                            for (int k = 0; k < 8; ++k)
                                y[prompt_order<CODES>(k)] =
                                    nt > 0 ? __uint_as_float(o[8 * c + k]) * pow2f(-kPromptK0) : 0.0f;
                            dst[(8 * b + 2 * c) * kPromptRows] = make_float4(y[0], y[1], y[2], y[3]);
                            dst[(8 * b + 2 * c + 1) * kPromptRows] = make_float4(y[4], y[5], y[6], y[7]);
                        }
                    }
                    A.part_ml[slot * kPromptRows + prow] = make_float2(m, l);
                }
                if (threadIdx.x == 0 && it.t0 == 0) {
                    // the last share with a piece of this item: the one of its last tile
                    const long long units = sm.plan_units, n = min((long long)gridDim.x, units);
                    const long long end = units * (blockIdx.x + 1) / n - it.t1 + it.steps;
                    AttMeta mt;
                    mt.last = (int)min(n - 1, (end * n - 1) / units);
                    mt.rows = it.rows[0] + it.rows[1];
                    mt.row0 = it.row0;
                    mt.head = it.head;
                    mt.token0 = it.s.s0;
                    A.meta[blockIdx.x] = mt;
                }
                tc::fence_before();
            } else if (it.rows[t] > 0) {
                const float inv = l == 0.0f ? 0.0f : pow2f(-kPromptK0) / l;      // (l is NaN where Q is)
                uint16_t *const dst = A.out + qrow * A.out_token + qhead * A.out_head;
#pragma unroll 1
                for (int b = 0; b < D / 32; ++b) {
                    uint32_t o[32];
                    tc::tmem_load(o_addr + 32 * b, o);          // (anything where nt is 0)
                    tc::tmem_load_wait(o);
#pragma unroll
                    for (int c = 0; c < 4; ++c) {
                        float y[8];
#pragma unroll
                        for (int k = 0; k < 8; ++k)
                            y[prompt_order<CODES>(k)] = inv == 0.0f ? 0.0f : __uint_as_float(o[8 * c + k]) * inv;
                        uint32_t h[4];
#pragma unroll
                        for (int k = 0; k < 4; ++k)
                            asm("cvt.rn.bf16x2.f32 %0, %1, %2;" : "=r"(h[k]) : "f"(y[2 * k + 1]), "f"(y[2 * k]));
                        if (valid) *reinterpret_cast<uint4 *>(dst + 32 * b + 8 * c) = make_uint4(h[0], h[1], h[2], h[3]);
                    }
                }
                tc::fence_before();                 // (these reads before the next item's products)
            }
        }
    } else if (warp < 12) {
        // ---------------- codes -> fp16 tiles: thread = token ----------------
        const int w = warp - 8, row = w * 32 + lane;
        int done = 0;
        bool live = true;
        while (live && sm.walk[warp].next(A, blockIdx.x == 0 && w == 0)) {
            if (it.t1 == it.t0) continue;
            const int last = it.row0 + it.rows[0] + it.rows[1] - 1;
            const int hi = PromptWalk::limit(A, it.s, last);
            const auto place = [&](int j) -> int64_t {
                const int pos = j * kPromptTile + row;
                if (pos >= hi) return -1;
                const int64_t r = kv_row(A.cache, A.batch, it.seq, pos, it.head);
                if (r < 0) atomicOr(A.status, STATUS_INDEX);
                return r;
            };
            // loads run ahead: a tile's rows are looked up two tiles before
            // it is expanded, its scales and key codes loaded one before
            int64_t at = place(it.t0), at_next = place(it.t0 + 1);
            uint4 kc[D / 32], vc[D / 32];
            ScaleWords<SB> ks, vs, vs_next;
            prompt_codes<D>(kc, A.cache.k_codes, at);
            prompt_scales(ks, A.cache.k_scales, at);
            prompt_scales(vs, A.cache.v_scales, at);
            const int t0 = it.t0, tiles = it.t1 - t0;
            for (int j = 0; j < tiles; ++j) {
                const int n = done + j, st = n & 1, ph = ((n >> 1) & 1) ^ 1;
                prompt_codes<D>(vc, A.cache.v_codes, at);
                // the exponents of both go with the keys: the softmax that
                // needs them may run before the values are expanded
                const int ek = max(__reduce_max_sync(0xffffffffu, ks.template top<GS>()), -90);
                const int ev = max(__reduce_max_sync(0xffffffffu, vs.template top<GS>()), -90);
                bool ok = n < 2 || tc::bar_wait(&sm.k_empty[st], ph, abort, A.status);
                if (!__all_sync(0xffffffffu, ok)) { live = false; break; }
                prompt_expand<CODES, GS, G, D, SB>(kc, ks, ek, sm.k[st], row);
                if (lane == 0) {
                    sm.kf[n & 7][w] = pow2f(ek - kPromptK0);
                    sm.ve[n & 7][w] = (float)ev;
                    sm.vi[n & 7][w] = pow2f(-ev);
                }
                tc::fence_async();
                __syncwarp();
                if (lane == 0) tc::bar_arrive(&sm.k_full[st]);
                at = at_next;
                prompt_codes<D>(kc, A.cache.k_codes, at);
                prompt_scales(ks, A.cache.k_scales, at);
                prompt_scales(vs_next, A.cache.v_scales, at);
                at_next = place(t0 + j + 2);
                ok = n < 2 || tc::bar_wait(&sm.v_empty[st], ph, abort, A.status);
                if (!__all_sync(0xffffffffu, ok)) { live = false; break; }
                prompt_expand<CODES, GS, G, D, SB>(vc, vs, ev, sm.v[st], row);
                tc::fence_async();
                __syncwarp();
                if (lane == 0) tc::bar_arrive(&sm.v_full[st]);
                vs = vs_next;
            }
            done += tiles;
        }
    } else {
        // ---------------- MMA issue ----------------
        constexpr uint32_t id_s = tc::idesc_f16(128, 64, false), id_o = tc::idesc_f16(128, D, true);
        const int t = warp - 12;
        int done = 0, mine = 0;                      // position tiles of the CTA, steps of this row tile so far
        uint32_t q_phase = 0;
        bool live = true;
        const auto wait = [&](uint64_t *bar, int phase) {
            live = live && __all_sync(0xffffffffu, tc::bar_wait(bar, phase & 1, abort, A.status));
        };
        constexpr uint32_t kStage = 128 * D * 2 / 16;                // one tile, in descriptor units
        const uint64_t q_desc = tc::desc_k_major(tc::smem_addr(sm.q[t])), k_desc = tc::desc_k_major(tc::smem_addr(sm.k[0]));
        const uint64_t v_desc = tc::desc_n_major(tc::smem_addr(sm.v[0]), 16384);
        const uint32_t s_col = tmem + 128 * t, o_col = tmem + 256 + D * t;
        while (live && sm.walk[warp].next(A, false)) {
            const int steps = it.t1 - it.t0, nt = max(min(it.nt[t], 2 * it.t1) - 2 * it.t0, 0);
            // S = Q K^T of step i (64 positions) into its half of the columns
            const auto scores = [&](int i) {
                const int n = done + (i >> 1);
                if (!(i & 1)) wait(&sm.k_full[n & 1], n >> 1);
                if (live && tc::elect()) {
                    uint64_t a = q_desc, b = k_desc + (n & 1) * kStage + (i & 1) * 512;
                    const uint32_t d = s_col + 64 * ((mine + i) & 1);
#pragma unroll 1
                    for (int h = 0; h < D / 64; ++h, a += 1024, b += 1024) {
#pragma unroll
                        for (int kk = 0; kk < 4; ++kk) tc::mma_ss(d, a + 2 * kk, b + 2 * kk, id_s, h + kk != 0);
                    }
                    tc::commit(&sm.s_full[t][(mine + i) & 1]);
                    if ((i & 1) || i + 1 == nt) tc::commit(&sm.k_empty[n & 1]);
                }
                __syncwarp();
            };
            if (nt > 0) {
                wait(&sm.q_full[t], q_phase);
                q_phase ^= 1;
                tc::fence_after();
                scores(0);
                if (nt > 1) scores(1);
            }
            for (int i = 0; i < nt && live; ++i) {
                // O += P V of step i, then the scores two steps ahead, over P
                const int n = done + (i >> 1), half = (mine + i) & 1;
                if (!(i & 1)) wait(&sm.v_full[n & 1], n >> 1);
                wait(&sm.p_full[t][half], (mine + i) >> 1);
                tc::fence_after();
                if (live && tc::elect()) {
                    const uint64_t b = v_desc + (n & 1) * kStage + (i & 1) * 512;
#pragma unroll
                    for (int kk = 0; kk < 4; ++kk)
                        tc::mma_ts(o_col, s_col + 64 * half + 8 * kk, b + 128 * kk, id_o, i > 0 || kk > 0);
                    tc::commit(&sm.o_full[t][half]);
                    if ((i & 1) || i + 1 == nt) tc::commit(&sm.v_empty[n & 1]);
                }
                __syncwarp();
                if (live && i + 2 < nt) scores(i + 2);
            }
            // tiles that only the other row tile needs
            for (int j = (nt + 1) / 2; j < steps && live; ++j) {
                const int n = done + j;
                wait(&sm.k_full[n & 1], n >> 1);
                if (live && lane == 0) tc::bar_arrive(&sm.k_empty[n & 1]);
                wait(&sm.v_full[n & 1], n >> 1);
                if (live && lane == 0) tc::bar_arrive(&sm.v_empty[n & 1]);
            }
            mine += nt;
            done += steps;
        }
        // after an abort, products may still be running on this CTA's memory
        if (tc::elect()) tc::commit(&sm.drained[t]);
        __syncwarp();
        const uint64_t t0 = tc::now_ns();
        while (!tc::bar_test(tc::smem_addr(&sm.drained[t]), 0) && tc::now_ns() - t0 <= tc::kWaitLimitNs) {
        }
        __syncwarp();
    }
    tc::fence_before();
    __syncthreads();
    if (warp == 12) {
        tc::fence_after();
        tc::tmem_free<512>(tmem);
    }
}

// Joins the pieces of the items that were cut: CTA (i, g) takes rows 32 g ..
// of the one that starts in share i; lane = row, a warp takes a quarter of the
// channels.
template <int D>
__global__ void __launch_bounds__(128)
attend_prompt_join_kernel(const AttArgs A) {
    grid_dependency_begin();
    constexpr int COLS = D / 16;                 // of 4 channels, per warp
    const AttMeta mt = A.meta[blockIdx.x];
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31, row = 32 * blockIdx.y + lane;
    if ((int)(32 * blockIdx.y) >= mt.rows) return;
    const bool valid = row < mt.rows;
    const int i0 = blockIdx.x, last = mt.last;
    const auto piece = [&](int i) { return 2 * i + (i == i0 ? 1 : 0); };     // its slot
    float mx = -INFINITY;
    for (int i = i0; i <= last; ++i) {
        if (valid) mx = max_nan(mx, A.part_ml[piece(i) * kPromptRows + row].x);
    }
    const float base = mx == -INFINITY ? 0.0f : mx;
    float4 acc[COLS];
#pragma unroll
    for (int c = 0; c < COLS; ++c) acc[c] = make_float4(0.0f, 0.0f, 0.0f, 0.0f);
    float sum = 0.0f;
    for (int i = i0; i <= last; ++i) {
        if (!valid) continue;
        const int k = piece(i);
        const float2 ml = A.part_ml[k * kPromptRows + row];
        const float f = ex2(ml.x - base);
        sum = fmaf(ml.y, f, sum);
        const float4 *const src = reinterpret_cast<const float4 *>(A.part) +
                                  ((int64_t)k * (D / 4) + warp * COLS) * kPromptRows + row;
#pragma unroll
        for (int c = 0; c < COLS; ++c) {
            const float4 v = src[c * kPromptRows];
            acc[c].x = fmaf(v.x, f, acc[c].x);
            acc[c].y = fmaf(v.y, f, acc[c].y);
            acc[c].z = fmaf(v.z, f, acc[c].z);
            acc[c].w = fmaf(v.w, f, acc[c].w);
        }
    }
    if (!valid) return;
    const float inv = sum == 0.0f ? 0.0f : 1.0f / sum;
    const int rr = mt.row0 + row, tok = rr / A.group;
    uint16_t *const dst = A.out + (mt.token0 + tok) * A.out_token +
                          (int64_t)(mt.head * A.group + rr - tok * A.group) * A.out_head + warp * (D / 4);
#pragma unroll
    for (int c = 0; c < COLS; c += 2) {
        uint32_t h[4];
        asm("cvt.rn.bf16x2.f32 %0, %1, %2;" : "=r"(h[0]) : "f"(acc[c].y * inv), "f"(acc[c].x * inv));
        asm("cvt.rn.bf16x2.f32 %0, %1, %2;" : "=r"(h[1]) : "f"(acc[c].w * inv), "f"(acc[c].z * inv));
        asm("cvt.rn.bf16x2.f32 %0, %1, %2;" : "=r"(h[2]) : "f"(acc[c + 1].y * inv), "f"(acc[c + 1].x * inv));
        asm("cvt.rn.bf16x2.f32 %0, %1, %2;" : "=r"(h[3]) : "f"(acc[c + 1].w * inv), "f"(acc[c + 1].z * inv));
        *reinterpret_cast<uint4 *>(dst + 4 * c) = make_uint4(h[0], h[1], h[2], h[3]);
    }
}

template <int CODES, int GS, int G, int D>
cudaError_t launch_attend_prompt(AttendLaunch &L, int few) {
    const AttArgs A = att_args(L, 2 * kPromptCtas, kPromptRows, few);
    const auto kern = attend_prompt_kernel<CODES, GS, G, D>;
    constexpr size_t bytes = sizeof(PromptSmem<D>) + 1024;
    static_assert(bytes <= 232448, "shared memory of the prompt kernel");
    static std::atomic<bool> done[64];
    cudaError_t e = smem_opt_in(kern, bytes, done);
    if (e != cudaSuccess) return e;
    // Whether items may be cut at all, by what the host knows (the kernel
    // decides): at least lo items of at most `longest` tiles, so whole items
    // lose at most (n - 1) / lo of the time (exactly known for one sequence).
    // Where lo is 0 (32 rows a sequence in the mean, or fewer) there may be no
    // item at all: batches of drafts, which are not to pay the joining kernel's
    // launch, and mixed ones are then whole, as all batches of more than
    // kPromptPlan sequences are.  us, whole against cut, 32 query heads over 8
    // of 128: 8 x 5 of 4001 NVFP4 31.0, 33.5; MXFP4: 30 single tokens with a piece
    // of 40, all over 500 positions, 30.4, 36.1, all over 2000, 76, 65; 50 over 2000
    // with 200 over 4000 130, 94; 60 over 2000 with 300 over 20000 410, 187.
    const int64_t n = kPromptCtas, heads = L.cache.heads, seqs = L.batch.seqs, rows = L.tokens * A.group;
    const int64_t lo = std::max<int64_t>((rows - few * seqs + kPromptRows - 1) / kPromptRows, 0) * heads;
    const int64_t hi = ((rows + kPromptRows - 1) / kPromptRows + seqs - 1) * heads;
    const int64_t longest = ((int64_t)L.batch.max_pages * L.cache.page_size + kPromptTile - 1) / kPromptTile;
    const double loss = lo == 0 ? 0.0 : seqs == 1 ? (double)((lo + n - 1) / n * n) / lo - 1.0 : (double)(n - 1) / lo;
    const int split = seqs <= kPromptPlan && longest > 1 && lo <= kPromptRounds * n && loss > (double)kPromptJoin * n / (hi * longest);
    L.launches += split ? 2 : 1;
    e = launch_k(kern, dim3((unsigned)(split ? n : std::min(hi, n))), dim3(kPromptThreads), bytes, L.stream, A, split);
    if (e != cudaSuccess || !split) return e;
    return launch_k(attend_prompt_join_kernel<D>, dim3((unsigned)n, kPromptRows / 32), dim3(128), 0, L.stream, A);
}

template <int CODES, int GS, int G, int D>
cudaError_t launch_attend_d(AttendLaunch &L) {
    const int by = attend_kernels(L.tokens, L.q_heads, L.cache.heads, L.batch.seqs);
    cudaError_t e = cudaSuccess;
    if (by & ATT_MANY) e = launch_attend_prompt<CODES, GS, G, D>(L, by & ATT_FEW ? kAttFew : 0);
    if (e != cudaSuccess || !(by & ATT_FEW)) return e;
    return launch_attend_split<CODES, GS, G, D>(L, by & ATT_MANY ? kAttFew : INT32_MAX);
}

template <int CODES, int GS>
cudaError_t launch_attend_fmt(AttendLaunch &L) {
#define DQ_ATT(GG, DD) \
    if (L.group == GG && L.cache.head_dim == DD) return launch_attend_d<CODES, GS, GG, DD>(L);
    DQ_ATT(16, 64) DQ_ATT(32, 64) DQ_ATT(64, 64) DQ_ATT(16, 128) DQ_ATT(32, 128) DQ_ATT(64, 128)
#undef DQ_ATT
    return cudaErrorInvalidValue;
}

}  // namespace dq
