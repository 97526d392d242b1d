// Attention over a paged cache for few rows per KV head (bf16): decoding and short verifications.
//
// With up to 32 rows per KV head the work is reading K and V once: 2 d bf16 values per key against 4 d M flops, 16 to 32
// flops a byte, far below what the tensor cores could do with it.  So the kernel is built around the loads:
//   last warp    producer: every tile of 64 or 128 keys, K and V, comes by TMA from its pages into a ring of stages
//   4 MT warps   a group of four per 16 rows, each warp with 16 or 32 keys of each tile: S = Q K^T (m16n8k16, Q in
//                registers), the running maximum and sum of the softmax, O += P V -- no warp waits for another while keys go
//                by; a group's four partial results are joined through shared memory where a piece ends.
// Up to 16 rows: two CTAs per SM, so that one loads while the other joins, stores or begins a piece.  Up to 32: one CTA with
// twice the stages (four warps with 32 rows each, two CTAs, spilled: 123 us for five tokens of 16 sequences).
//
// The pool is one tensor map (column, KV head, token of the page, page); a box holds min(page_size, 32) tokens, so that a
// tile is 2 to 8 boxes per 64 columns, issued by as many lanes.  Boxes without a visible key, or of a page that the pool
// does not have, are not loaded: their keys are left out by the warps that own them.
//
// Measured, 32 query and 8 KV heads of 128 values, whole calls with their merge (in brackets this kernel alone, caches cold): one
// token of one sequence of 131072 in 87 us, 6.2 TB/s (85); of 64 sequences of 17 to 32768 in 155 us, 6.5 TB/s (157); five
// tokens of 16 sequences in 84 us, 5.8 TB/s (80, 6.1 TB/s).
#include <cmath>

#include <cuda_bf16.h>

#include "paged.cuh"
#include "ptx.cuh"

namespace usp {

namespace {

constexpr int kGroup = 4;  // warps that share 16 rows
// Keys of a box at most.  Smaller boxes read less beyond a sequence's ends (200 sequences of about 750 own keys behind a prefix:
// 128 us against 133 with boxes of 64), but boxes of 16 keep the producer too busy where one CTA has the SM (107 us against 91
// for five tokens of 16 sequences).
constexpr int kBox = 32;
constexpr float kLn2 = 0.6931471805599453f;
constexpr float kRescale = 8.0f;  // log2 units: O is rescaled only when the maximum grows by more than 2^8

template <int D, int MT>
struct Cfg {
    static constexpr UnitShape kUnit = mma_unit(D, MT);
    static constexpr int M = kUnit.rows;
    // Steps of 16 keys of a warp per tile.  Two hide each other's latency and share the maximum's exchange, where the ring
    // allows for larger tiles: five tokens of 16 sequences 84.0 us against 88.0, one of 64 sequences with heads of 64 values 85.7
    // against 100.  (16 rows of 128 values would have stages of 64 KB, one and a half per CTA.)
    static constexpr int KS = mma_steps(D, MT);
    static constexpr int kKeyTile = kUnit.keys;
    static_assert(M == 16 * MT && kKeyTile == 16 * KS * kGroup, "the unit's shape");
    // Places that a piece's beginning and end (rows of Q, the join, the stores) count, in tiles.  It takes about 3 us, a tile of
    // 64 keys 1.5 us at the memory's rate where two CTAs share the SM.  With two steps: 88.4, 84.5, 84.0, 83.8, 84.3 us for
    // five tokens of 16 sequences at 1 to 5, and 37.8 at 2, 38.0 at 3, 39.6 at 4 for those of 64 short ones.
    static constexpr int kPieceCost = kUnit.piece;
    static constexpr int kConsumers = kGroup * MT;
    static constexpr int kThreads = 32 * (kConsumers + 1);
    static constexpr int kCtasPerSm = kUnit.ctas_per_sm;
    static constexpr int kChunks = D / 64;                                    // 64-column boxes per row
    static constexpr int kTileBytes = kKeyTile * D * 2;                       // K or V of a tile
    static constexpr int kStages = D == 64 ? 3 * MT : 3;                      // 192 KB in flight per SM
    static constexpr int kJoinStride = D + 8;                                 // float32 per row: rows in different banks
    static constexpr int kJoinBytes = 16 * kJoinStride * 4;                   // per group
    static constexpr int kOffJoin = kStages * 2 * kTileBytes;
    static constexpr int kOffStat = kOffJoin + MT * kJoinBytes;               // per group m, sum, sum of rounded: 3 x [4][16]
    static constexpr int kOffBar = kOffStat + MT * 3 * kGroup * 16 * 4;
    static constexpr int kSmem = kOffBar + 2 * (kStages + kSegs) * 8 + 1024;
};

__device__ __forceinline__ void ldsm4(uint32_t addr, uint32_t (&r)[4]) {
    asm volatile("ldmatrix.sync.aligned.m8n8.x4.shared.b16 {%0,%1,%2,%3}, [%4];"
                 : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3]) : "r"(addr) : "memory");
}
__device__ __forceinline__ void ldsm4t(uint32_t addr, uint32_t (&r)[4]) {
    asm volatile("ldmatrix.sync.aligned.m8n8.x4.trans.shared.b16 {%0,%1,%2,%3}, [%4];"
                 : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3]) : "r"(addr) : "memory");
}
__device__ __forceinline__ void mma16816(float (&c)[4], const uint32_t (&a)[4], uint32_t b0, uint32_t b1) {
    asm volatile("mma.sync.aligned.m16n8k16.row.col.f32.bf16.bf16.f32 {%0,%1,%2,%3}, {%4,%5,%6,%7}, {%8,%9}, {%0,%1,%2,%3};"
                 : "+f"(c[0]), "+f"(c[1]), "+f"(c[2]), "+f"(c[3])
                 : "r"(a[0]), "r"(a[1]), "r"(a[2]), "r"(a[3]), "r"(b0), "r"(b1));
}
// Barrier of a group's warps, and the same with whether all of them say yes.
__device__ __forceinline__ void bar_group(int group) {
    asm volatile("bar.sync %0, %1;" ::"r"(group + 1), "n"(32 * kGroup) : "memory");
}
__device__ __forceinline__ bool bar_group_all(int group, bool yes) {
    uint32_t all;
    asm volatile("{\n\t.reg .pred p, q;\n\tsetp.ne.u32 p, %1, 0;\n\tbar.red.and.pred q, %2, %3, p;\n\tselp.u32 %0, 1, 0, q;\n\t}"
                 : "=r"(all) : "r"((uint32_t)yes), "r"(group + 1), "n"(32 * kGroup) : "memory");
    return all != 0;
}

template <int D, int MT, bool PREFIX>
__global__ void __launch_bounds__(Cfg<D, MT>::kThreads, Cfg<D, MT>::kCtasPerSm)
    paged_mma_kernel(const __grid_constant__ CUtensorMap tm_k, const __grid_constant__ CUtensorMap tm_v,
                     const PagedArgs a) {
    using C = Cfg<D, MT>;
    constexpr int M = C::M, kThreads = C::kThreads, kConsumers = C::kConsumers, kKeyTile = C::kKeyTile, KS = C::KS;
    extern __shared__ uint8_t smem_raw[];
    uint8_t* smem = reinterpret_cast<uint8_t*>((reinterpret_cast<uintptr_t>(smem_raw) + 1023) & ~uintptr_t(1023));
    const uint32_t sbase = smem_u32(smem);
    __shared__ Share share;
    __shared__ int abort_flag;
    __shared__ uint32_t s_boxes[C::kStages];  // boxes of the stage that were loaded
    __shared__ Seg s_seg[kSegs];
    const uint32_t full0 = sbase + C::kOffBar, empty0 = full0 + 8 * C::kStages;
    const uint32_t seg_full0 = empty0 + 8 * C::kStages, seg_empty0 = seg_full0 + 8 * kSegs;
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31, cta = blockIdx.x;
    begin_kernel(PREFIX);
    Seg pre{};
    if constexpr (PREFIX) pre = prefix_piece<M, kKeyTile>(a, cta);
    if (threadIdx.x == 32 * kConsumers) {
        tma_prefetch_desc(&tm_k);
        tma_prefetch_desc(&tm_v);
    }
    if (threadIdx.x == 0) {
        abort_flag = 0;
        for (int s = 0; s < C::kStages; ++s) {
            mbar_init(full0 + 8 * s, 1);
            mbar_init(empty0 + 8 * s, kConsumers);
        }
        for (int s = 0; s < kSegs; ++s) {
            mbar_init(seg_full0 + 8 * s, 1);
            mbar_init(seg_empty0 + 8 * s, kConsumers);
        }
        fence_mbar_init();
    }
    if constexpr (PREFIX) {
        __syncthreads();
    } else {
        // (holds the barrier that publishes the set-up, too)
        find_share<M, kKeyTile, C::kPieceCost, kThreads>(a, cta, a.ctas, &share);
        finish_empty_rows<__nv_bfloat16, M, kKeyTile, kThreads>(a, cta, a.ctas);
        __syncthreads();
    }
    volatile int* abort_p = &abort_flag;

    if (warp == kConsumers) {
        // ---------------------------------------------------------------- producer
        const int psize = 1 << a.page_log2, box = min(psize, kBox), nb = kKeyTile / box;
        const int my_box = lane % nb, my_chunk = lane / nb % C::kChunks, my_kv = lane / nb / C::kChunks;
        int it = 0, n_seg = 0;
        bool ok = true;
        auto publish = [&](const Seg& g) {
            if (PREFIX) return;
            const int i = n_seg % kSegs;
            if (n_seg >= kSegs)
                ok = __all_sync(~0u, mbar_wait(seg_empty0 + 8 * i, (n_seg / kSegs - 1) & 1, abort_p, 24, a.status));
            if (ok && lane == 0) {
                s_seg[i] = g;
                mbar_arrive(seg_full0 + 8 * i);
            }
            ++n_seg;
            __syncwarp();
        };
        auto piece = [&](const Seg& g) {
            publish(g);
            const int first = PREFIX ? 0 : a.key_begin, end = seg_key_end<PREFIX>(a, g);
            auto page_of = [&](int tile) {  // of this lane's box, -1: not loaded
                const int j = tile * kKeyTile + my_box * box;
                return my_kv < 2 && j < end && j + box > first ? seg_page<PREFIX>(a, g, j >> a.page_log2) : -1;
            };
            int page = page_of(g.tile0);
            for (int x = 0; ok && x < g.n_tiles; ++x, ++it) {
                const int next = x + 1 < g.n_tiles ? page_of(g.tile0 + x + 1) : -1;  // on its way during the wait
                const int st = it % C::kStages;
                if (it >= C::kStages &&
                    !__all_sync(~0u, mbar_wait(empty0 + 8 * st, (it / C::kStages - 1) & 1, abort_p, 21, a.status))) {
                    ok = false;
                    break;
                }
                const uint32_t live = __ballot_sync(~0u, page >= 0);
                if (lane == 0) {
                    s_boxes[st] = live;
                    mbar_arrive_expect_tx(full0 + 8 * st, __popc(live) * box * 128);
                }
                __syncwarp();
                if (page >= 0) {
                    const int j = (g.tile0 + x) * kKeyTile + my_box * box;
                    tma_load_4d(sbase + (st * 2 + my_kv) * C::kTileBytes + my_chunk * (kKeyTile * 128) +
                                    my_box * box * 128,
                                my_kv ? &tm_v : &tm_k, my_chunk * 64, g.h, j & (psize - 1), page, full0 + 8 * st);
                }
                page = next;
            }
            return ok;
        };
        Seg g = pre;
        if constexpr (PREFIX) {
            piece(g);
        } else {
            OwnWalk<M, kKeyTile, C::kPieceCost> walk(a, share);
            while (walk.next(g) && piece(g)) {}
        }
        g.n_tiles = 0;
        if (ok) publish(g);
        if (lane == 0) drain_ring(full0, C::kStages, it, 22, a.status);  // every load has landed before the CTA exits
    } else {
        // ---------------------------------------------------------------- consumers
        const int group = warp / kGroup, kw = warp % kGroup;  // rows 16 * group .., keys 16 KS * kw .. of each tile
        const int r0 = lane >> 2, c0 = (lane & 3) * 2;        // this lane's first row and column of a fragment
        const int box_log2 = min(a.page_log2, 5);  // of kBox
        float* s_m = reinterpret_cast<float*>(smem + C::kOffStat) + group * 3 * kGroup * 16;
        float* s_l = s_m + kGroup * 16;
        float* s_lr = s_l + kGroup * 16;
        float* s_join = reinterpret_cast<float*>(smem + C::kOffJoin + group * C::kJoinBytes);
        // ldmatrix rows of this lane: K (key, 16-byte column) and V transposed
        const int k_key = kw * 16 * KS + ((lane >> 4) << 3) + (lane & 7), k_c = (lane >> 3) & 1;
        const int v_key = kw * 16 * KS + (((lane >> 3) & 1) << 3) + (lane & 7), v_c = lane >> 4;
        int it = 0;
        bool ok = true;
        for (int n_seg = 0; !PREFIX || n_seg == 0; ++n_seg) {
            const int si = n_seg % kSegs;
            ok = PREFIX || ok && mbar_wait(seg_full0 + 8 * si, (n_seg / kSegs) & 1, abort_p, 25, a.status);
            // (one answer for the group's warps, which meet at barriers below; a wait that gives up within a piece lets its
            // warp run on to the next one without waiting)
            if (!PREFIX && !bar_group_all(group, ok)) break;
            const Seg& g = PREFIX ? pre : s_seg[si];
            if (g.n_tiles == 0) break;
            const int first = PREFIX ? 0 : a.key_begin, end = seg_key_end<PREFIX>(a, g);
            const int tile0 = g.tile0, n_tiles = g.n_tiles;
            const bool rows_here = MT == 1 || group * 16 < g.n_rows;
            // ---- rows: Q, limits
            uint32_t q[D / 16][4];
            int lim[2];
#pragma unroll
            for (int hh = 0; hh < 2; ++hh) {
                const int r = group * 16 + hh * 8 + r0;
                const bool live = r < g.n_rows;
                const int R = g.row0 + (live ? r : 0), i = R / a.g;
                const uint32_t* src = reinterpret_cast<const uint32_t*>(
                    static_cast<const __nv_bfloat16*>(a.q) +
                    ((int64_t)(g.t0 + i) * a.Hq + g.h * a.g + (R - i * a.g)) * D + c0);
#pragma unroll
                for (int kk = 0; kk < D / 16; ++kk) {
                    q[kk][hh] = live ? *(src + kk * 8) : 0u;
                    q[kk][hh + 2] = live ? *(src + kk * 8 + 4) : 0u;
                }
                lim[hh] = live ? row_limit<PREFIX>(a, g, r) : INT_MAX;
            }
            const int lim_min = __reduce_min_sync(~0u, min(lim[0], lim[1]));
            float o[D / 8][4], m[2] = {-INFINITY, -INFINITY}, l[2] = {0.f, 0.f}, lr[2] = {0.f, 0.f};
#pragma unroll
            for (int n = 0; n < D / 8; ++n)
#pragma unroll
                for (int e = 0; e < 4; ++e) o[n][e] = 0.f;
            // ---- keys
            for (int x = 0; x < n_tiles; ++x, ++it) {
                const int st = it % C::kStages;
                ok = ok && mbar_wait(full0 + 8 * st, (it / C::kStages) & 1, abort_p, 23, a.status);
                ok = __all_sync(~0u, ok);
                const int key0 = (tile0 + x) * kKeyTile + kw * 16 * KS;  // this warp's keys key0 .. key0 + 16 KS - 1
                uint32_t live = 0;  // steps whose box was loaded
                if (ok && rows_here && key0 < end && key0 + 16 * KS > first) {
                    const uint32_t boxes = s_boxes[st];
#pragma unroll
                    for (int u = 0; u < KS; ++u) live |= (boxes >> ((kw * KS + u) * 16 >> box_log2) & 1u) << u;
                }
                if (live) {
                    const uint32_t kb = sbase + st * 2 * C::kTileBytes, vb = kb + C::kTileBytes;
                    float s[2 * KS][4];
#pragma unroll
                    for (int n = 0; n < 2 * KS; ++n)
#pragma unroll
                        for (int e = 0; e < 4; ++e) s[n][e] = 0.f;
#pragma unroll
                    for (int kk = 0; kk < D / 16; ++kk)
#pragma unroll
                        for (int u = 0; u < KS; ++u) {
                            uint32_t b[4];
                            ldsm4(kb + (kk / 4) * (kKeyTile * 128) + (k_key + u * 16) * 128 +
                                      ((((kk & 3) * 2 + k_c) ^ (k_key & 7)) << 4), b);
                            mma16816(s[2 * u], q[kk], b[0], b[1]);
                            mma16816(s[2 * u + 1], q[kk], b[2], b[3]);
                        }
                    // ---- masks: only where one of these keys is hidden from some row
                    uint32_t vm[KS][2];
#pragma unroll
                    for (int u = 0; u < KS; ++u) vm[u][0] = vm[u][1] = ~0u;
                    if (key0 + 16 * KS > lim_min || key0 + 16 * KS > end || key0 < first || live != (1u << KS) - 1u) {
#pragma unroll
                        for (int n = 0; n < 2 * KS; ++n) {
                            const bool there = live >> (n / 2) & 1u;
                            const int key = key0 + n * 8 + c0;
#pragma unroll
                            for (int e = 0; e < 4; ++e)
                                if (!there || key + (e & 1) >= lim[e >> 1] || key + (e & 1) < first) s[n][e] = -INFINITY;
                            // what lies beyond the sequence in its last page may be NaN: 0 * NaN must not reach O
                            if (!there || key >= end || key < first) vm[n / 2][n & 1] &= 0xffff0000u;
                            if (!there || key + 1 >= end || key + 1 < first) vm[n / 2][n & 1] &= 0x0000ffffu;
                        }
                    }
                    // ---- softmax
                    uint32_t p[KS][4];
                    bool grew = false;
                    float al[2];
#pragma unroll
                    for (int hh = 0; hh < 2; ++hh) {
                        float mx = fmaxf(s[0][2 * hh], s[0][2 * hh + 1]);
#pragma unroll
                        for (int n = 1; n < 2 * KS; ++n) mx = fmaxf(mx, fmaxf(s[n][2 * hh], s[n][2 * hh + 1]));
                        mx = fmaxf(mx, __shfl_xor_sync(~0u, mx, 1));
                        mx = fmaxf(mx, __shfl_xor_sync(~0u, mx, 2));
                        mx *= a.scale_log2;
                        const bool up = mx > m[hh] + kRescale;
                        al[hh] = up ? ex2_approx(m[hh] - mx) : 1.f;
                        if (up) m[hh] = mx;
                        grew |= up;
                        const float ms = m[hh] == -INFINITY ? 0.f : m[hh];
                        float sum = 0.f, sum_r = 0.f;
#pragma unroll
                        for (int u = 0; u < KS; ++u) {
                            const float e0 = ex2_approx(fmaf(s[2 * u][2 * hh], a.scale_log2, -ms));
                            const float e1 = ex2_approx(fmaf(s[2 * u][2 * hh + 1], a.scale_log2, -ms));
                            const float e2 = ex2_approx(fmaf(s[2 * u + 1][2 * hh], a.scale_log2, -ms));
                            const float e3 = ex2_approx(fmaf(s[2 * u + 1][2 * hh + 1], a.scale_log2, -ms));
                            p[u][hh] = pack_bf16(e0, e1);
                            p[u][hh + 2] = pack_bf16(e2, e3);
                            sum += (e0 + e1) + (e2 + e3);
                            // P is rounded to bf16, V's type: each p is off by up to 2^-8 of itself.  O is divided by the sum of
                            // what the product uses, the rounded p, so that o is off by up to 2^-8 sum p|v - o| / sum p (measured
                            // 2.0e-3 to 2.3e-3 of the output, with the output's own rounding, 1.7e-3 by itself)
                            const float f0 = __uint_as_float(p[u][hh] << 16), f1 = __uint_as_float(p[u][hh] & 0xffff0000u),
                                        f2 = __uint_as_float(p[u][hh + 2] << 16),
                                        f3 = __uint_as_float(p[u][hh + 2] & 0xffff0000u);
                            sum_r += (f0 + f1) + (f2 + f3);
                        }
                        l[hh] = l[hh] * al[hh] + sum;
                        lr[hh] = lr[hh] * al[hh] + sum_r;
                    }
                    if (__any_sync(~0u, grew)) {
#pragma unroll
                        for (int n = 0; n < D / 8; ++n) {
                            o[n][0] *= al[0];
                            o[n][1] *= al[0];
                            o[n][2] *= al[1];
                            o[n][3] *= al[1];
                        }
                    }
                    // ---- O += P V
#pragma unroll
                    for (int nn = 0; nn < D / 16; ++nn)
#pragma unroll
                        for (int u = 0; u < KS; ++u) {
                            uint32_t b[4];
                            ldsm4t(vb + (nn / 4) * (kKeyTile * 128) + (v_key + u * 16) * 128 +
                                       ((((nn & 3) * 2 + v_c) ^ (v_key & 7)) << 4), b);
                            mma16816(o[2 * nn], p[u], b[0] & vm[u][0], b[1] & vm[u][1]);
                            mma16816(o[2 * nn + 1], p[u], b[2] & vm[u][0], b[3] & vm[u][1]);
                        }
                }
                __syncwarp();
                if (lane == 0) mbar_arrive(empty0 + 8 * st);
            }
            // ---- join the group's four warps (in an order fixed per column quarter), normalise, store
#pragma unroll
            for (int hh = 0; hh < 2; ++hh) {
                float s1 = l[hh], s2 = lr[hh];
                s1 += __shfl_xor_sync(~0u, s1, 1);
                s2 += __shfl_xor_sync(~0u, s2, 1);
                s1 += __shfl_xor_sync(~0u, s1, 2);
                s2 += __shfl_xor_sync(~0u, s2, 2);
                if ((lane & 3) == 0) {
                    const int r = kw * 16 + hh * 8 + r0;
                    s_m[r] = m[hh];
                    s_l[r] = s1;
                    s_lr[r] = s2;
                }
            }
            bar_group(group);
            float f[2];
#pragma unroll
            for (int hh = 0; hh < 2; ++hh) {
                float mx = -INFINITY;
#pragma unroll
                for (int w = 0; w < kGroup; ++w) mx = fmaxf(mx, s_m[w * 16 + hh * 8 + r0]);
                f[hh] = mx == -INFINITY ? 0.f : ex2_approx(m[hh] - mx);
            }
#pragma unroll
            for (int round = 0; round < kGroup; ++round) {
                const int part = (kw + round) % kGroup;
#pragma unroll
                for (int n = 0; n < D / 8; ++n)
                    if (n / (D / 32) == part) {
#pragma unroll
                        for (int hh = 0; hh < 2; ++hh) {
                            float2* dst = reinterpret_cast<float2*>(s_join + (hh * 8 + r0) * C::kJoinStride + n * 8 + c0);
                            float2 w = round ? *dst : make_float2(0.f, 0.f);
                            w.x += o[n][2 * hh] * f[hh];
                            w.y += o[n][2 * hh + 1] * f[hh];
                            *dst = w;
                        }
                    }
                bar_group(group);
            }
            // eight threads per row, D/8 columns each
            const int rr = (threadIdx.x % (32 * kGroup)) >> 3, cc = (threadIdx.x & 7) * (D / 8), r = group * 16 + rr;
            if (r < g.n_rows) {
                float mx = -INFINITY;
#pragma unroll
                for (int w = 0; w < kGroup; ++w) mx = fmaxf(mx, s_m[w * 16 + rr]);
                float sum = 0.f, sum_r = 0.f;
#pragma unroll
                for (int w = 0; w < kGroup; ++w) {
                    const float e = mx == -INFINITY ? 0.f : ex2_approx(s_m[w * 16 + rr] - mx);
                    sum += e * s_l[w * 16 + rr];
                    sum_r += e * s_lr[w * 16 + rr];
                }
                const bool has = sum_r != 0.f;  // (NaN, too, which has to show)
                const float inv = has ? 1.f / sum_r : 0.f;
                const float lse2 = has ? mx + log2f(sum) : -INFINITY;
                const float* src = s_join + rr * C::kJoinStride + cc;
                const RowDst dst = row_dst<M, PREFIX>(a, g, r, cta);
                if (dst.out) {
                    uint4* w = reinterpret_cast<uint4*>(static_cast<__nv_bfloat16*>(dst.out) + cc);
#pragma unroll
                    for (int e = 0; e < D / 64; ++e) {
                        const float* y = src + e * 8;
                        w[e] = has ? make_uint4(pack_bf16(y[0] * inv, y[1] * inv), pack_bf16(y[2] * inv, y[3] * inv),
                                                pack_bf16(y[4] * inv, y[5] * inv), pack_bf16(y[6] * inv, y[7] * inv))
                                   : make_uint4(0, 0, 0, 0);
                    }
                    if ((threadIdx.x & 7) == 0) *dst.lse = lse2 * kLn2;
                } else {
                    float4* w = reinterpret_cast<float4*>(dst.part + cc);
#pragma unroll
                    for (int e = 0; e < D / 32; ++e) {
                        const float* y = src + e * 4;
                        w[e] = has ? make_float4(y[0] * inv, y[1] * inv, y[2] * inv, y[3] * inv)
                                   : make_float4(0.f, 0.f, 0.f, 0.f);
                    }
                    if ((threadIdx.x & 7) == 0) *dst.lse = lse2;
                }
                if (!PREFIX && g.ends && (threadIdx.x & 7) == 0) note_row<M>(a, g, r, cta);
            }
            // (the next piece's first barrier comes before anyone writes the join buffer or the statistics again)
            __syncwarp();
            if (!PREFIX && lane == 0) mbar_arrive(seg_empty0 + 8 * si);
        }
    }
    if constexpr (PREFIX) grid_dependency_wait();  // end after the own kernel
}

template <int D, int MT, bool PREFIX>
cudaError_t launch_t(const PagedArgs& a, cudaStream_t s) {
    using C = Cfg<D, MT>;
    const int psize = 1 << a.page_log2, box = psize < kBox ? psize : kBox;
    const int64_t page = (int64_t)psize * D;
    CUtensorMap tk, tv;
    const Tensor4 k{const_cast<void*>(a.k_pages), page, D, page * a.Hkv, a.Hkv, psize, a.n_pages};
    Tensor4 v = k;
    v.ptr = const_cast<void*>(a.v_pages);
    if (!make_tmap_bf16(&tk, k, D, box) || !make_tmap_bf16(&tv, v, D, box)) return cudaErrorInvalidValue;
    auto kern = paged_mma_kernel<D, MT, PREFIX>;
    const cudaError_t e = allow_smem<paged_mma_kernel<D, MT, PREFIX>>(C::kSmem);
    if (e != cudaSuccess) return e;
    return launch_dependent(kern, dim3(PREFIX ? a.p_ctas : a.ctas), C::kThreads, C::kSmem, s, tk, tv, a);
}

template <int D, bool PREFIX>
cudaError_t launch_d(const PagedArgs& a, cudaStream_t s) {
    return (PREFIX ? a.p_rows : a.rows) == 16 ? launch_t<D, 1, PREFIX>(a, s) : launch_t<D, 2, PREFIX>(a, s);
}

}  // namespace

cudaError_t launch_paged_mma(const PagedArgs& a, bool prefix, cudaStream_t s) {
    if (a.d == 64) return prefix ? launch_d<64, true>(a, s) : launch_d<64, false>(a, s);
    return prefix ? launch_d<128, true>(a, s) : launch_d<128, false>(a, s);
}

}  // namespace usp
