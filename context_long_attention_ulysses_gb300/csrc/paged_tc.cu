// Attention over a paged cache for many rows per KV head (bf16): chunks of prompts, and the prefix that a batch shares.
//
// 33 rows per KV head and more are a matrix product: with M rows a key costs 4 d M flops per 4 d bytes, and from about 260
// rows on the tensor cores bound it (1735 TFLOP/s against 6.7 TB/s).  One CTA per SM owns a unit of 128 rows (one stream) or
// 256 (two streams A and B that share every K/V tile); rows are (token, query head of the group) pairs, of one sequence or,
// over a prefix, of the whole batch:
//   warp 4 NS      TMA producer: K and V of each tile of 128 keys, page by page, into two rings
//   warps 4 NS + 1 (and + 2)  one thread each issues tcgen05.mma (the first of these warps owns the TMEM)
//   warps 0-3 (A), 4-7 (B)  Q rows into shared memory, softmax (thread = row = TMEM lane; log2 domain, O rescaled only when
//                  the maximum grows by more than 2^8), normalisation, stores
// With two streams the tensor core runs one stream's products while the other's softmax works.  Each stream has an issuer of
// its own, and they take turns, QK(0) and then [PV(j), QK(j+1)] being a turn: while one's products run, the other does its
// waits and the commits of its last turn.  (One issuer for both streams spent 1470 of the 3517 clocks of a tile in those,
// with nothing queued; two issuers without turns mix the streams' products, both softmaxes then work at the same time and
// the tensor core waits for both: 1991 us against 1570 for 2048 tokens at 64K.)  Where TMEM has room for one more
// buffer of scores (one stream, or d = 64), a turn is PV(n), QK(n + NS + 1) over n = NS j + stream: a softmax finds its next
// scores made, and is no longer a chain with the products (2048 tokens over 67584 keys, d = 64: 1305 -> 1130 us; 64 and 96
// rows of 16 sequences of 1000 to 20000 tokens 97 -> 93 and 101 -> 97).  A CTA walks its share piece by piece (paged.cuh); the rings run on
// across pieces, so the next piece's keys arrive during the epilogue.
// Measured, 32 query and 8 KV heads of 128 values: 2048 tokens over 67584 keys in 1.42 ms, 1570 TFLOP/s (1.51 ms when run on
// end, under the power cap), the tensor pipe active 67 % of the time: a stream's own chain, S to P (1360 clocks) and two
// products, is what a tile takes.  With heads of 64 values 1.12 ms, the tensor pipe active 42 %, issue slots 51 %: the two
// softmax warps per scheduler wait for their own instructions.  A prefix of 32768 under 64 tokens (256 rows per KV head):
// 35 us for 134 MB, of which 6 pass before the first scores.
// TMEM columns: S_A [0,128), S_B [128,256), O_A [256,256+D), O_B [384,384+D); with three S O_A [384,448), O_B [448,512);
// P (bf16) lies over its own S.
#include <cmath>

#include <cuda_bf16.h>

#include "paged.cuh"
#include "ptx.cuh"

namespace usp {

namespace {

constexpr int kKeyTile = 128;
// A piece's beginning and end (Q, the first products, the stores) against a tile's 1.5 to 2 us.
constexpr int kPieceCost = tc_unit(1).piece;
static_assert(tc_unit(1).keys == kKeyTile && tc_unit(2).keys == kKeyTile && tc_unit(2).piece == kPieceCost, "the unit's shape");
constexpr float kLn2 = 0.6931471805599453f;
constexpr float kRescale = 8.0f;  // log2 units
constexpr int kSoftmaxRegs = 208, kOtherRegs = 88;  // of 168 at launch (NS = 2): 2 * 208 + 88 <= 3 * 168
static_assert(2 * kSoftmaxRegs + kOtherRegs <= 3 * 168, "register split exceeds the launch allocation");
constexpr int kFlags = 8;  // ring of loaded-box masks; longer than the K ring by what the softmax may lag behind

template <int D, int NS>
struct Cfg {
    static constexpr int M = tc_unit(NS).rows;
    static_assert(M == 128 * NS && tc_unit(NS).ctas_per_sm == 1, "the unit's shape");
    static constexpr int kThreads = (4 * NS + 4) * 32;
    static constexpr int kChunks = D / 64;
    static constexpr int kTileBytes = kChunks * 128 * 128;  // 128 rows of bf16
    static constexpr int kKStages = D == 64 ? 4 : 3;
    static constexpr int kVStages = D == 64 ? 4 : (NS == 2 ? 2 : 3);
    // One buffer of scores more than streams where O leaves the columns for it: a stream's next scores are made while it works
    // on these.
    static constexpr bool kAhead = NS == 1 || D == 64;
    static constexpr int kBufs = kAhead ? NS + 1 : NS;
    static constexpr int kDbl = kAhead ? 2 : 1;  // barriers of a stream's scores, of its P and of its O, used in turn
    static constexpr int kOffQ = 0;
    static constexpr int kOffK = NS * kTileBytes;
    static constexpr int kOffV = kOffK + kKStages * kTileBytes;
    static constexpr int kOffBar = kOffV + kVStages * kTileBytes;
    static constexpr int kBars = 2 * kKStages + 2 * kVStages + (2 + 3 * kDbl) * NS + 1 + 2 * kSegs;
    static constexpr int kSmem = kOffBar + kBars * 8 + 16 + 1024;
};

// Bits lo .. hi-1 of word w (32 bits each) of a mask.
__device__ __forceinline__ uint32_t range_bits(int lo, int hi, int w) {
    lo = min(max(lo - 32 * w, 0), 32);
    hi = min(max(hi - 32 * w, 0), 32);
    if (lo >= hi) return 0u;
    return (0xffffffffu >> (32 - (hi - lo))) << lo;
}

// Row r of a piece's queries, zero beyond its last row.
template <int N>
__device__ __forceinline__ void load_q_row(const PagedArgs& a, const Seg& g, int r, uint4 (&w)[N]) {
    const bool live = r < g.n_rows;
    const int R = g.row0 + r, i = R / a.g;
    const uint4* src = reinterpret_cast<const uint4*>(static_cast<const __nv_bfloat16*>(a.q) +
                                                      ((int64_t)(g.t0 + i) * a.Hq + g.h * a.g + (R - i * a.g)) * (N * 8));
#pragma unroll
    for (int c = 0; c < N; ++c) w[c] = live ? *(src + c) : make_uint4(0, 0, 0, 0);
}

template <int D, int NS, bool PREFIX>
__global__ void __launch_bounds__(Cfg<D, NS>::kThreads, 1)
    paged_tc_kernel(const __grid_constant__ CUtensorMap tm_k, const __grid_constant__ CUtensorMap tm_v,
                    const PagedArgs a) {
    using C = Cfg<D, NS>;
    constexpr int M = C::M, KS = C::kKStages, VS = C::kVStages;
    extern __shared__ uint8_t smem_raw[];
    uint8_t* smem = reinterpret_cast<uint8_t*>((reinterpret_cast<uintptr_t>(smem_raw) + 1023) & ~uintptr_t(1023));
    const uint32_t sbase = smem_u32(smem);
    uint32_t* tmem_slot = reinterpret_cast<uint32_t*>(smem + C::kOffBar + C::kBars * 8);
    __shared__ Share share;
    __shared__ int abort_flag;
    __shared__ uint32_t s_boxes[kFlags];  // boxes of a tile that were loaded
    __shared__ Seg s_seg[kSegs], s_tail;
    auto BAR = [&](int i) { return sbase + C::kOffBar + 8u * (uint32_t)i; };
    const int kKFull = 0, kKEmpty = KS, kVFull = 2 * KS, kVEmpty = kVFull + VS;
    constexpr int DB = C::kDbl;
    const int kQFull = kVEmpty + VS, kSFull = kQFull + NS, kPReady = kSFull + NS * DB, kOReady = kPReady + NS * DB;  // per stream
    const int kTurn = kOReady + NS * DB;  // per stream: its issuer may issue
    const int kDrain = kTurn + NS, kSegFull = kDrain + 1, kSegEmpty = kSegFull + kSegs;
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31, cta = blockIdx.x;
    constexpr int kProducer = 4 * NS, kIssuer = 4 * NS + 1;

    begin_kernel(PREFIX);
    Seg pre{};
    uint4 first_q[PREFIX ? D / 8 : 1];  // prefix: a softmax thread's row of Q
    if constexpr (PREFIX) {
        pre = prefix_piece<M, kKeyTile>(a, cta);
        if (warp < 4 * NS) load_q_row(a, pre, threadIdx.x, first_q);
    }
    if (threadIdx.x == 32 * kProducer) {
        tma_prefetch_desc(&tm_k);
        tma_prefetch_desc(&tm_v);
    }
    if (threadIdx.x == 0) {
        abort_flag = 0;
        for (int s = 0; s < KS; ++s) { mbar_init(BAR(kKFull + s), 1); mbar_init(BAR(kKEmpty + s), NS); }
        for (int s = 0; s < VS; ++s) { mbar_init(BAR(kVFull + s), 1); mbar_init(BAR(kVEmpty + s), NS); }
        for (int st = 0; st < NS; ++st) {
            mbar_init(BAR(kQFull + st), 128);
            for (int b = 0; b < DB; ++b) {
                mbar_init(BAR(kSFull + st * DB + b), 1);
                mbar_init(BAR(kPReady + st * DB + b), 128);
                mbar_init(BAR(kOReady + st * DB + b), 1);
            }
            mbar_init(BAR(kTurn + st), 1);
        }
        mbar_init(BAR(kDrain), NS);
        for (int s = 0; s < kSegs; ++s) { mbar_init(BAR(kSegFull + s), 1); mbar_init(BAR(kSegEmpty + s), 5 * NS); }
        fence_mbar_init();
    }
    if (warp == kIssuer) {
        tmem_alloc(smem_u32(tmem_slot), 512);
        tmem_relinquish();
    }
    if constexpr (!PREFIX) {
        find_share<M, kKeyTile, kPieceCost, C::kThreads>(a, cta, a.ctas, &share);
        finish_empty_rows<__nv_bfloat16, M, kKeyTile, C::kThreads>(a, cta, a.ctas);
    }
    tc_fence_before();
    __syncthreads();
    tc_fence_after();
    const uint32_t tmem = *tmem_slot;
    volatile int* abort_p = &abort_flag;

    // the barrier of a stream's n-th scores (or P, or product with V), and its phase
    auto DBAR = [&](int first, int st, uint32_t n) { return BAR(first + st * DB + (int)(n % DB)); };
    auto phase = [](uint32_t n) { return (n / DB) & 1u; };

    // tiles of a piece that hold a key which some row of stream st sees
    auto stream_tiles = [&](const Seg& g, int st) {
        if (st * 128 >= g.n_rows) return 0;
        if (PREFIX) return g.n_tiles;
        const int last = min(g.n_rows, st * 128 + 128) - 1;
        const int end = visible(a, SeqRows{g.t0, g.n, g.len}, (g.row0 + last) / a.g);
        return min(max((end + kKeyTile - 1) / kKeyTile - g.tile0, 0), g.n_tiles);
    };

    if (warp >= 4 * NS) {
        if constexpr (NS == 2) setmaxnreg_dec<kOtherRegs>();
        if (warp == kProducer) {
            // ---------------------------------------------------------------- TMA producer
            const int psize = 1 << a.page_log2, box = min(psize, kKeyTile), nb = kKeyTile / box;
            const int my_box = lane % nb, my_chunk = lane / nb;
            int it = 0, nv = 0, n_seg = 0;
            auto publish = [&](const Seg& g) {
                if (PREFIX) return true;
                const int i = n_seg % kSegs;
                if (n_seg >= kSegs &&
                    !__all_sync(~0u, mbar_wait(BAR(kSegEmpty + i), (n_seg / kSegs - 1) & 1, abort_p, 43, a.status)))
                    return false;
                if (lane == 0) {
                    s_seg[i] = g;
                    mbar_arrive(BAR(kSegFull + i));
                }
                ++n_seg;
                __syncwarp();
                return true;
            };
            auto piece = [&](const Seg& g) {  // false: a wait gave up
                if (!publish(g)) return false;
                const int first = PREFIX ? 0 : a.key_begin, end = seg_key_end<PREFIX>(a, g);
                auto page_of = [&](int tile) {  // of this lane's box, -1: not loaded
                    const int j = tile * kKeyTile + my_box * box;
                    return my_chunk < C::kChunks && j < end && j + box > first
                               ? seg_page<PREFIX>(a, g, j >> a.page_log2) : -1;
                };
                int page = page_of(g.tile0);
                for (int x = 0; x < g.n_tiles; ++x, ++it) {
                    const int next = x + 1 < g.n_tiles ? page_of(g.tile0 + x + 1) : -1;  // on its way during the waits
                    const uint32_t live = __ballot_sync(~0u, page >= 0);
                    const uint32_t bytes = __popc(live) * box * 128;
                    const int j = (g.tile0 + x) * kKeyTile + my_box * box;
                    const uint32_t off = my_chunk * 16384 + my_box * box * 128;
                    const int ks = it % KS, vs = it % VS;
                    if (it >= KS &&
                        !__all_sync(~0u, mbar_wait(BAR(kKEmpty + ks), (it / KS - 1) & 1, abort_p, 31, a.status)))
                        return false;
                    if (lane == 0) {
                        s_boxes[it % kFlags] = live;
                        mbar_arrive_expect_tx(BAR(kKFull + ks), bytes);
                    }
                    __syncwarp();
                    if (page >= 0)
                        tma_load_4d(sbase + C::kOffK + ks * C::kTileBytes + off, &tm_k, my_chunk * 64, g.h,
                                    j & (psize - 1), page, BAR(kKFull + ks));
                    if (it >= VS &&
                        !__all_sync(~0u, mbar_wait(BAR(kVEmpty + vs), (it / VS - 1) & 1, abort_p, 32, a.status))) {
                        ++it;  // this K tile was issued, its V tile was not
                        return false;
                    }
                    if (lane == 0) mbar_arrive_expect_tx(BAR(kVFull + vs), bytes);
                    __syncwarp();
                    if (page >= 0)
                        tma_load_4d(sbase + C::kOffV + vs * C::kTileBytes + off, &tm_v, my_chunk * 64, g.h,
                                    j & (psize - 1), page, BAR(kVFull + vs));
                    nv = it + 1;
                    page = next;
                }
                return true;
            };
            Seg g = pre;
            bool ok = true;
            if constexpr (PREFIX) {
                ok = piece(g);
            } else {
                OwnWalk<M, kKeyTile, kPieceCost> walk(a, share);
                // The end of a unit that an earlier CTA began comes last.  All shares being equally long, the CTAs of a
                // head are then at the same key tile, or at one of two, at any time, and read it from L2 together.
                bool has_tail = false;
                while (ok && walk.next(g)) {
                    if (g.ordinal == 0 && !g.begins) {
                        if (lane == 0) s_tail = g;
                        has_tail = true;
                    } else {
                        ok = piece(g);
                    }
                }
                __syncwarp();
                if (ok && has_tail) ok = piece(s_tail);
            }
            g.n_tiles = 0;
            if (ok) publish(g);
            __syncwarp();
            if (lane == 0) {  // every issued load lands before the CTA can exit
                drain_ring(BAR(kKFull), KS, it, 33, a.status);
                drain_ring(BAR(kVFull), VS, nv, 34, a.status);
            }
        } else if (warp < kIssuer + NS && lane == 0) {
            // ---------------------------------------------------------------- MMA issuer
            constexpr uint32_t kIdS = idesc_bf16(128, kKeyTile, 0, 0);  // S = Q K^T, both K-major
            constexpr uint32_t kIdO = idesc_bf16(128, D, 0, 1);         // O += P V, V MN-major
            const int st = warp - kIssuer;
            const uint64_t dq0 = sdesc_sw128(sbase + C::kOffQ, 16, 1024), dk0 = sdesc_sw128(sbase + C::kOffK, 16, 1024),
                           dv0 = sdesc_sw128(sbase + C::kOffV, 16384, 1024);
            int base = 0;                           // tiles so far
            uint32_t cnt = 0, turn = 0;             // tiles of this stream, and turns waited for, so far
            auto products_pv = [&](uint32_t o_col, uint32_t p_col, int vs, bool first) {
                const uint64_t dv = dv0 + (uint32_t)(vs * C::kTileBytes >> 4);
#pragma unroll
                for (int kk = 0; kk < kKeyTile / 16; ++kk)
                    mma_ts(o_col, p_col + kk * 8, dv + (kk * 2048 >> 4), kIdO, (!first || kk > 0) ? 1u : 0u);
            };
            auto products_qk = [&](uint32_t s_col, int stream, int ks) {
                const uint64_t dq = dq0 + (uint32_t)(stream * C::kTileBytes >> 4), dk = dk0 + (uint32_t)(ks * C::kTileBytes >> 4);
#pragma unroll
                for (int kk = 0; kk < D / 16; ++kk) {
                    const uint32_t off = ((kk / 4) * 16384 + (kk % 4) * 32) >> 4;
                    mma_ss(s_col, dq + off, dk + off, kIdS, kk > 0);
                }
            };
            // (a tile that a stream does not see is released, once it is there, without a product)
            auto release = [&](uint32_t bar, bool used) { if (used) mma_commit(bar); else mbar_arrive(bar); };
            uint32_t q_pieces = 0;                  // pieces with Q of the stream whose scores this issuer makes
            uint32_t cnt_q = 0;                     // and their tiles
            const int sq = C::kAhead ? NS - 1 - st : st;
            // Turn j of stream st: PV(j), QK(j + 1), for a piece of n_tiles tiles of which the stream sees the first nt
            // (j = -1: the first QK only); false: a wait gave up.
            auto turn_in_chain = [&](int j, int n_tiles, int nt) {
                const bool has_v = j >= 0, has_k = j + 1 < n_tiles, pv = has_v && j < nt, qk = has_k && j + 1 < nt;
                const int iv = base + j, ik = iv + 1, vs = iv % VS, ks = ik % KS;
                if (has_v && !mbar_wait(BAR(kVFull + vs), (iv / VS) & 1, abort_p, 37, a.status)) return false;
                if (has_k && !mbar_wait(BAR(kKFull + ks), (ik / KS) & 1, abort_p, 36, a.status)) return false;
                if (pv && !mbar_wait(DBAR(kPReady, st, cnt + j), phase(cnt + j), abort_p, 38, a.status)) return false;
                if (NS == 2 && (st == 1 || turn > 0) &&
                    !mbar_wait(BAR(kTurn + st), (turn - 1 + st) & 1, abort_p, 46, a.status))
                    return false;
                ++turn;
                tc_fence_after();
                const uint32_t s_col = tmem + st * 128;
                if (pv) products_pv(tmem + 256 + st * 128, s_col, vs, j == 0);
                if (qk) products_qk(s_col, st, ks);  // in issue order after the product that read P from the columns of S
                if (NS == 2) mbar_arrive(BAR(kTurn + 1 - st));
                if (qk) mma_commit(DBAR(kSFull, st, cnt + j + 1));
                if (pv && j == nt - 1) mma_commit(BAR(kOReady + st));
                if (has_v) release(BAR(kVEmpty + vs), pv);
                if (has_k) release(BAR(kKEmpty + ks), qk);
                return true;
            };
            // Turn n = NS j + st with a buffer more than streams: PV(n), and into the columns that it leaves QK(n + NS + 1), with
            // two streams the other's.  From n = -NS - 1 on, the turns of a piece end with the last stream, as they began with two,
            // and buffers rotate on across pieces, so that a buffer is always refilled by the thread that issued the product
            // before.
            auto turn_ahead = [&](int n, int n_tiles, int nt, int nt_q) {
                constexpr int NB = C::kBufs;
                const int j = NS == 2 ? n >> 1 : n, jk = NS == 2 ? (n + NB) >> 1 : n + NB;
                const bool has_v = n >= 0, has_k = jk < n_tiles, pv = has_v && j < nt, qk = has_k && jk < nt_q;
                const int iv = base + j, ik = base + jk, vs = iv % VS, ks = ik % KS;
                if (has_v && !mbar_wait(BAR(kVFull + vs), (iv / VS) & 1, abort_p, 37, a.status)) return false;
                if (has_k && !mbar_wait(BAR(kKFull + ks), (ik / KS) & 1, abort_p, 36, a.status)) return false;
                if (pv && !mbar_wait(DBAR(kPReady, st, cnt + j), phase(cnt + j), abort_p, 38, a.status)) return false;
                if (NS == 2 && n != -NB && !mbar_wait(BAR(kTurn + st), turn++ & 1, abort_p, 46, a.status)) return false;
                // (where this stream sees no tile the columns are those of the other's product three tiles before, and another
                // thread's: it has to be complete.  In a piece's first turns that follows from Q being there.)
                if (NS == 2 && qk && !pv && jk >= 3 &&
                    !mbar_wait(DBAR(kOReady, sq, cnt_q + jk - 3), phase(cnt_q + jk - 3), abort_p, 47, a.status))
                    return false;
                tc_fence_after();
                const uint32_t col = tmem + (uint32_t)((NS * base + n + NB) % NB) * 128;
                if (pv) products_pv(tmem + NB * 128 + st * 64, col, vs, j == 0);
                if (qk) products_qk(col, sq, ks);
                if (NS == 2 && n != 2 * n_tiles - 1) mbar_arrive(BAR(kTurn + 1 - st));
                if (qk) mma_commit(DBAR(kSFull, sq, cnt_q + jk));
                if (pv) mma_commit(DBAR(kOReady, st, cnt + j));
                if (has_v) release(BAR(kVEmpty + vs), pv);
                if (has_k) release(BAR(kKEmpty + ks), qk);
                return true;
            };
            for (int n_seg = 0; !PREFIX || n_seg == 0; ++n_seg) {
                const int si = n_seg % kSegs;
                if (!PREFIX && !mbar_wait(BAR(kSegFull + si), (n_seg / kSegs) & 1, abort_p, 44, a.status)) break;
                const int n_tiles = PREFIX ? pre.n_tiles : s_seg[si].n_tiles;
                if (n_tiles == 0) break;
                const int nt = PREFIX ? stream_tiles(pre, st) : stream_tiles(s_seg[si], st);
                const int nt_q = !C::kAhead ? nt : PREFIX ? stream_tiles(pre, sq) : stream_tiles(s_seg[si], sq);
                if (!PREFIX) mbar_arrive(BAR(kSegEmpty + si));
                if (nt_q > 0 && !mbar_wait(BAR(kQFull + sq), q_pieces++ & 1, abort_p, 35, a.status)) break;
                bool ok = true;
                if constexpr (C::kAhead) {
                    for (int n = -2 - st; ok && n < NS * n_tiles; n += NS) ok = turn_ahead(n, n_tiles, nt, nt_q);
                } else {
                    for (int j = -1; ok && j < n_tiles; ++j) ok = turn_in_chain(j, n_tiles, nt);
                }
                if (!ok) break;
                base += n_tiles;
                cnt += nt;
                cnt_q += nt_q;
            }
            // every issued MMA completes before TMEM is freed (after an abort, too)
            mma_commit(BAR(kDrain));
            mbar_drain(BAR(kDrain), 0, 39, a.status);
        }
    } else {
        if constexpr (NS == 2) setmaxnreg_inc<kSoftmaxRegs>();
        // ---------------------------------------------------------------- softmax warps
        const int st = warp >> 2;                    // stream
        const int row = (warp & 3) * 32 + lane;      // row of the stream = TMEM lane
        const uint32_t lane_base = tmem + ((uint32_t)((warp & 3) * 32) << 16);
        const uint32_t ocol = lane_base + (C::kAhead ? C::kBufs * 128 + st * 64 : 256 + st * 128);
        const int box_log2 = min(a.page_log2, 7);
        const uint32_t all_boxes = (1u << (kKeyTile >> box_log2)) - 1u;
        auto warp_wait = [&](uint32_t bar, uint32_t parity, int site) {  // one answer for the warp: TMEM access is collective
            return __all_sync(~0u, mbar_wait(bar, parity, abort_p, site, a.status)) != 0;
        };
        auto o_wait = [&](uint32_t n) {  // ahead: for the stream's n-th product with V; in a chain: for its n-th piece
            if (!warp_wait(DBAR(kOReady, st, n), phase(n), 42)) return false;
            tc_fence_after();
            return true;
        };
        uint32_t base = 0, cnt = 0, pieces = 0;
        auto piece = [&](const Seg& g) {  // false: a wait gave up
            const int r = st * 128 + row;
            const bool valid = r < g.n_rows;
            const int n_tiles = stream_tiles(g, st), tile0 = g.tile0;
            if (n_tiles > 0) {  // this row of Q, swizzled as a TMA load would place it; rows beyond the unit are zero
                uint8_t* dst = smem + C::kOffQ + st * C::kTileBytes + row * 128;
                uint4 w[D / 8];
                if constexpr (!PREFIX) load_q_row(a, g, r, w);
#pragma unroll
                for (int c = 0; c < D / 8; ++c)
                    *reinterpret_cast<uint4*>(dst + (c / 8) * 16384 + (((c & 7) ^ (row & 7)) << 4)) =
                        PREFIX ? first_q[PREFIX ? c : 0] : w[c];
                fence_proxy_async_smem();
                mbar_arrive(BAR(kQFull + st));
            }
            const int lim = valid ? row_limit<PREFIX>(a, g, r) : INT_MAX;
            // (a warp without a valid row has its rows of V to clear, too)
            const int lim_min = min(__reduce_min_sync(~0u, lim), seg_key_end<PREFIX>(a, g));
            float m_run = -INFINITY, l_run = 0.f;
            uint32_t buf = C::kAhead ? (NS * base + st) % C::kBufs : st;  // of the scores
            for (int j = 0; j < n_tiles; ++j) {
                if (!warp_wait(DBAR(kSFull, st, cnt + j), phase(cnt + j), 40)) return false;
                tc_fence_after();
                const uint32_t scol = lane_base + buf * 128;
                uint32_t r0r[32], r1r[32], r2r[32], r3r[32];
                tmem_ld32(scol, r0r);
                tmem_ld32(scol + 32, r1r);
                tmem_ld32(scol + 64, r2r);
                tmem_ld32(scol + 96, r3r);
                const int key0 = (tile0 + j) * kKeyTile;
                const uint32_t live = s_boxes[(base + j) % kFlags] & all_boxes;
                tmem_wait_ld();
                float s[kKeyTile];
#pragma unroll
                for (int c = 0; c < 32; ++c) {
                    s[c] = __uint_as_float(r0r[c]);
                    s[32 + c] = __uint_as_float(r1r[c]);
                    s[64 + c] = __uint_as_float(r2r[c]);
                    s[96 + c] = __uint_as_float(r3r[c]);
                }
                if (key0 + kKeyTile > lim_min || (!PREFIX && key0 < a.key_begin) || live != all_boxes) {
                    const int first = PREFIX ? 0 : a.key_begin, end = seg_key_end<PREFIX>(a, g);
                    // (own keys: the limit again, as the registers are short in the loop)
                    const int mine = PREFIX ? lim : st * 128 + row < g.n_rows ? row_limit<PREFIX>(a, g, st * 128 + row) : INT_MAX;
                    const int lo = first - key0, hi = min(mine, end) - key0;
#pragma unroll
                    for (int w = 0; w < 4; ++w) {
                        uint32_t see = 0u;
                        for (int b = 0; b < kKeyTile >> box_log2; ++b)
                            if (live >> b & 1u) see |= range_bits(b << box_log2, (b + 1) << box_log2, w);
                        see &= range_bits(lo, hi, w);
#pragma unroll
                        for (int c = 0; c < 32; ++c)
                            if (!(see >> c & 1u)) s[32 * w + c] = -INFINITY;
                    }
                    // V rows that are no key of this piece may hold anything, NaN too, and 0 * NaN must not reach O:
                    // thread = row of the V tile (both streams write the same zeros)
                    const uint32_t vs = (base + j) % VS;
                    if (!warp_wait(BAR(kVFull + vs), ((base + j) / VS) & 1, 41)) return false;
                    const bool real = key0 + row >= first && key0 + row < end && (live >> (row >> box_log2) & 1u);
                    if (!real) {
                        uint8_t* v = smem + C::kOffV + vs * C::kTileBytes + row * 128;
#pragma unroll
                        for (int c = 0; c < D / 8; ++c)
                            *reinterpret_cast<uint4*>(v + (c / 8) * 16384 + (c & 7) * 16) = make_uint4(0, 0, 0, 0);
                    }
                    fence_proxy_async_smem();
                }
                // row max as eight independent chains of three-input maxima
                float m8[8];
#pragma unroll
                for (int c = 0; c < 8; ++c) m8[c] = s[c];
#pragma unroll
                for (int c = 8; c < kKeyTile; c += 2) m8[(c / 2) & 7] = max3f(m8[(c / 2) & 7], s[c], s[c + 1]);
                float mx = max3f(max3f(m8[0], m8[1], m8[2]), max3f(m8[3], m8[4], m8[5]), fmaxf(m8[6], m8[7]));
                mx *= a.scale_log2;
                const bool up = mx > m_run + kRescale;
                const float alpha = up ? ex2_approx(m_run - mx) : 1.f;
                if (up) m_run = mx;
                const float msub = m_run == -INFINITY ? 0.f : m_run;
                const float2 c2 = make_float2(a.scale_log2, a.scale_log2), nm2 = make_float2(-msub, -msub);
                float2 sum2[2] = {make_float2(0.f, 0.f), make_float2(0.f, 0.f)};
#pragma unroll
                for (int h = 0; h < 4; ++h) {
                    uint32_t pk[16];
#pragma unroll
                    for (int c = 0; c < 16; ++c) {
                        const float2 x = fma2(make_float2(s[h * 32 + 2 * c], s[h * 32 + 2 * c + 1]), c2, nm2);
                        const float2 pv = make_float2(ex2_approx(x.x), ex2_approx(x.y));
                        sum2[c & 1] = add2(sum2[c & 1], pv);
                        pk[c] = pack_bf16(pv.x, pv.y);
                    }
                    tmem_st16(scol + h * 16, pk);  // P over S: this row's S is in registers
                }
                // P is rounded to bf16: both operands of the product have V's type.  Each p is off by up to 2^-8 of itself, o by up to
                // 2^-8 sum p|v| / sum p (measured 2.3e-3 of the output, with the output's own rounding, 1.7e-3 by itself; a second
                // product with what the rounding leaves would be half as much tensor work again).  O is divided by the sum of
                // the unrounded p: the sum of the rounded ones, as in paged_mma.cu, is two more operations per pair in the warps
                // that this kernel waits for.
                l_run = l_run * alpha + ((sum2[0].x + sum2[0].y) + (sum2[1].x + sum2[1].y));
                // Made ahead, S_j was signalled before the product of tile j - 1, even j - 2, had to be complete.  Each is
                // waited for, in order (a phase that is skipped could be taken for the one after next), the last but one always.
                if (C::kAhead && j > 1 && !o_wait(cnt + j - 2)) return false;
                if (j > 0 && __any_sync(~0u, up)) {
                    // (in a chain the products of earlier tiles completed before S_j was signalled) scale O in place
                    if (C::kAhead && !o_wait(cnt + j - 1)) return false;
#pragma unroll
                    for (int c = 0; c < D / 32; ++c) {
                        uint32_t o[32];
                        tmem_ld32(ocol + c * 32, o);
                        tmem_wait_ld();
#pragma unroll
                        for (int e = 0; e < 32; ++e) o[e] = __float_as_uint(__uint_as_float(o[e]) * alpha);
                        tmem_st32(ocol + c * 32, o);
                    }
                }
                tmem_wait_st();
                tc_fence_before();
                mbar_arrive(DBAR(kPReady, st, cnt + j));
                if constexpr (C::kAhead) buf = buf == 0 ? C::kBufs - 1 : buf - 1;  // NS buffers on
            }
            // ---------------------------------------------------------------- the piece's result
            if (n_tiles > 0) {
                if (C::kAhead && n_tiles > 1 && !o_wait(cnt + n_tiles - 2)) return false;
                if (!o_wait(C::kAhead ? cnt + n_tiles - 1 : pieces)) return false;
                ++pieces;
            }
            const bool has = n_tiles > 0 && l_run != 0.f;  // (NaN, too, which has to show)
            const float inv = has ? 1.f / l_run : 0.f;
            const float lse2 = has ? m_run + log2f(l_run) : -INFINITY;
            const RowDst dst = row_dst<M, PREFIX, true>(a, g, valid ? r : 0, cta);
#pragma unroll
            for (int c = 0; c < D / 32; ++c) {
                uint32_t o[32];
                if (n_tiles > 0) {
                    tmem_ld32(ocol + c * 32, o);
                    tmem_wait_ld();
                }
                if (!has) {
#pragma unroll
                    for (int e = 0; e < 32; ++e) o[e] = 0u;
                }
                if (valid && dst.out) {
                    uint4* y = reinterpret_cast<uint4*>(static_cast<__nv_bfloat16*>(dst.out) + c * 32);
#pragma unroll
                    for (int e = 0; e < 4; ++e) {
                        uint4 v;
                        v.x = pack_bf16(__uint_as_float(o[8 * e + 0]) * inv, __uint_as_float(o[8 * e + 1]) * inv);
                        v.y = pack_bf16(__uint_as_float(o[8 * e + 2]) * inv, __uint_as_float(o[8 * e + 3]) * inv);
                        v.z = pack_bf16(__uint_as_float(o[8 * e + 4]) * inv, __uint_as_float(o[8 * e + 5]) * inv);
                        v.w = pack_bf16(__uint_as_float(o[8 * e + 6]) * inv, __uint_as_float(o[8 * e + 7]) * inv);
                        y[e] = v;
                    }
                } else if (valid) {
                    float* y = dst.part + c * 32 * dst.step;
#pragma unroll
                    for (int e = 0; e < 8; ++e)
                        *reinterpret_cast<float4*>(y + 4 * e * dst.step) =
                            make_float4(__uint_as_float(o[4 * e]) * inv, __uint_as_float(o[4 * e + 1]) * inv,
                                           __uint_as_float(o[4 * e + 2]) * inv, __uint_as_float(o[4 * e + 3]) * inv);
                }
            }
            tc_fence_before();  // O is read: the next piece's first product may overwrite it once P is ready
            if (valid) {
                *dst.lse = dst.out ? lse2 * kLn2 : lse2;
                if (!PREFIX && g.ends) note_row<M>(a, g, r, cta);
            }
            base += g.n_tiles;
            cnt += n_tiles;
            return true;
        };
        if constexpr (PREFIX) {
            piece(pre);
        } else {
            for (int n_seg = 0;; ++n_seg) {
                const int si = n_seg % kSegs;
                if (!warp_wait(BAR(kSegFull + si), (n_seg / kSegs) & 1, 45)) break;
                if (s_seg[si].n_tiles == 0 || !piece(s_seg[si])) break;
                __syncwarp();
                if (lane == 0) mbar_arrive(BAR(kSegEmpty + si));
            }
        }
    }
    // ---------------------------------------------------------------- teardown
    tc_fence_before();
    __syncthreads();
    if (warp == kIssuer) {
        __syncwarp();
        tc_fence_after();
        tmem_dealloc(tmem, 512);
    }
    if constexpr (PREFIX) grid_dependency_wait();  // end after the own kernel
}

template <int D, int NS, bool PREFIX>
cudaError_t launch_t(const PagedArgs& a, cudaStream_t s) {
    using C = Cfg<D, NS>;
    const int psize = 1 << a.page_log2, box = psize < kKeyTile ? psize : kKeyTile;
    const int64_t page = (int64_t)psize * D;
    CUtensorMap tk, tv;
    const Tensor4 k{const_cast<void*>(a.k_pages), page, D, page * a.Hkv, a.Hkv, psize, a.n_pages};
    Tensor4 v = k;
    v.ptr = const_cast<void*>(a.v_pages);
    if (!make_tmap_bf16(&tk, k, D, box) || !make_tmap_bf16(&tv, v, D, box)) return cudaErrorInvalidValue;
    auto kern = paged_tc_kernel<D, NS, PREFIX>;
    const cudaError_t e = allow_smem<paged_tc_kernel<D, NS, PREFIX>>(C::kSmem);
    if (e != cudaSuccess) return e;
    return launch_dependent(kern, dim3(PREFIX ? a.p_ctas : a.ctas), C::kThreads, C::kSmem, s, tk, tv, a);
}

template <int D, bool PREFIX>
cudaError_t launch_d(const PagedArgs& a, cudaStream_t s) {
    return (PREFIX ? a.p_rows : a.rows) == 128 ? launch_t<D, 1, PREFIX>(a, s) : launch_t<D, 2, PREFIX>(a, s);
}

}  // namespace

cudaError_t launch_paged_tc(const PagedArgs& a, bool prefix, cudaStream_t s) {
    if (a.d == 64) return prefix ? launch_d<64, true>(a, s) : launch_d<64, false>(a, s);
    return prefix ? launch_d<128, true>(a, s) : launch_d<128, false>(a, s);
}

}  // namespace usp
