// Attention over a paged cache: what its kernels share -- how the work is cut
// into equal shares, and where a row's result goes.
//
// A unit is (sequence, KV head, tile of M consecutive rows), a row being one
// (token, query head of the group): K and V of the head are read once for all
// M rows.  A unit's keys are cut into tiles of KT.  All tiles of all
// units, in the order sequence, head, row tile, key tile, form one line, in
// which a unit takes PC places before its first tile: beginning and ending a
// unit costs about as much as that many tiles (without them, 16 sequences of
// one tile each fell to one CTA and decided the time of the whole launch).  Of
// the W places CTA c of G takes [c*W/G, (c+1)*W/G).  So every CTA has the same
// work whatever the lengths are, one sequence of 128K tokens spreads over all
// SMs, and the lengths are read on the device (a captured graph replays with
// new ones).  A unit that lies in one share is finished by its CTA; the
// rows of a unit cut by a border leave partial results (normalised output and
// log-sum-exp) in the workspace, which paged_merge_kernel joins in the order
// of the keys.  A share holds at most two cut units: its first (slot 0, begun
// by an earlier CTA) and its last (slot 1).
#pragma once

#include <atomic>
#include <cmath>
#include <cstdint>

#include <cuda_bf16.h>
#include <cuda_runtime.h>

#include "kernels.h"

namespace usp {

// The kernels follow each other by programmatic dependent launch: a kernel lets its successor's CTAs start as soon as its own
// have all begun, so that the successor's set-up overlaps with it, and every kernel waits for its predecessor's end, and
// everything it wrote, before it reads or overwrites any of that.  The prefix kernel, which comes second, needs nothing of the
// own kernel: it waits at its end only, so that the merge after it sees what both wrote (and the own kernel lets it start only
// after its own wait, so that it has what came before the call).  What a predecessor may have written is read by plain loads, not
// through the read-only path, which holds what it likes from before the wait.
__device__ __forceinline__ void let_dependents_start() { asm volatile("griddepcontrol.launch_dependents;" ::: "memory"); }
__device__ __forceinline__ void grid_dependency_wait() { asm volatile("griddepcontrol.wait;" ::: "memory"); }

template <typename... P, typename... A>
cudaError_t launch_dependent(void (*kernel)(P...), dim3 grid, unsigned threads, size_t smem, cudaStream_t stream,
                             const A&... args) {
    cudaLaunchAttribute attr{};
    attr.id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attr.val.programmaticStreamSerializationAllowed = 1;
    cudaLaunchConfig_t cfg{};
    cfg.gridDim = grid;
    cfg.blockDim = dim3(threads);
    cfg.dynamicSmemBytes = smem;
    cfg.stream = stream;
    cfg.attrs = &attr;
    cfg.numAttrs = 1;
    return cudaLaunchKernelEx(&cfg, kernel, args...);
}

// To be called by all threads, before anything is read; the prefix kernel waits at its end instead.
__device__ __forceinline__ void begin_kernel(bool prefix) {
    if (!prefix) grid_dependency_wait();
    let_dependents_start();
}

// Allows a kernel its dynamic shared memory, once per device (asked for on every call it shows in the smallest ones).
template <auto Kernel>
cudaError_t allow_smem(int bytes) {
    static std::atomic<uint64_t> done{0};
    int dev = 0;
    cudaError_t e = cudaGetDevice(&dev);
    if (e != cudaSuccess) return e;
    const uint64_t bit = dev < 64 ? (uint64_t)1 << dev : 0;
    if (done.load(std::memory_order_relaxed) & bit) return cudaSuccess;
    e = cudaFuncSetAttribute(Kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, bytes);
    if (e == cudaSuccess) done.fetch_or(bit, std::memory_order_relaxed);
    return e;
}

// A kernel's unit: rows, keys of a tile, CTAs that an SM holds, and the places on the line that its beginning and end count
// (below).  The kernels are built with these, and paged_plan cuts the prefix and lays out the workspace by them.
struct UnitShape {
    int rows, keys, ctas_per_sm, piece;
};
constexpr int mma_steps(int d, int mt) { return d == 64 ? 2 : mt; }  // steps of 16 keys of a warp per tile
constexpr UnitShape mma_unit(int d, int mt) {                        // paged_mma.cu, 16 mt rows
    return {16 * mt, 64 * mma_steps(d, mt), mt == 1 ? 2 : 1, mma_steps(d, mt) == 1 ? 2 : 3};
}
constexpr UnitShape tc_unit(int ns) { return {128 * ns, 128, 1, 3}; }        // paged_tc.cu, ns streams
constexpr UnitShape f32_unit(int d) { return {8, 8 * (1024 / d), 1, 2}; }    // paged_f32.cu

// What paged_merge_kernel does with a row: word x = kind | row in the tile << 2, y = first CTA | last CTA << 16.
enum RowKind : uint32_t {
    kRowDone = 0,   // nothing (finished, or a row of no sequence)
    kRowNone = 1,   // no own keys (prefix only)
    kRowWhole = 2,  // own part in own_o, own_lse (prefix only)
    kRowSplit = 3   // own part in the slots of the CTAs named in y
};

// Rows of one sequence in this call.
struct SeqRows {
    int t0, n, len;  // first token (row of q), tokens, cached tokens
};

__device__ __forceinline__ SeqRows seq_rows(const PagedArgs& a, int b) {
    SeqRows s;
    if (a.q_start) {
        s.t0 = min(max(*(a.q_start + b), 0), a.n_tokens);
        s.n = min(max(*(a.q_start + b + 1), s.t0), a.n_tokens) - s.t0;
    } else {
        s.t0 = b;
        s.n = 1;
    }
    s.len = min(max(*(a.seq_lens + b), 0), a.max_pages << a.page_log2);
    return s;
}

// Keys [0, vis) are seen by token i of the sequence.
__device__ __forceinline__ int visible(const PagedArgs& a, const SeqRows& s, int i) {
    return a.causal ? max(s.len - s.n + i + 1, 0) : s.len;
}

// Key tiles of row tile rt of a sequence: those that hold a key in [key_begin, vis of the tile's last row).
template <int M, int KT>
__device__ __forceinline__ int unit_tiles(const PagedArgs& a, const SeqRows& s, int rt) {
    const int last = min(((rt + 1) * M - 1) / a.g, s.n - 1);
    const int end = visible(a, s, last);
    return end > a.key_begin ? (end + KT - 1) / KT - a.key_begin / KT : 0;
}

template <int M>
__device__ __forceinline__ int row_tiles(const PagedArgs& a, const SeqRows& s) {
    return (s.n * a.g + M - 1) / M;
}

// The first row tile with a key, row_tiles if none has one (limits grow with the row, so all from it on have keys): that of the
// first token that sees a key from key_begin on.
template <int M>
__device__ __forceinline__ int first_row_tile(const PagedArgs& a, const SeqRows& s) {
    const int keys = s.len - a.key_begin;
    if (keys <= 0 || s.n == 0) return row_tiles<M>(a, s);
    return a.causal ? max(s.n - keys, 0) * a.g / M : 0;
}

// Places of a unit of ut tiles on the line.
template <int PC>
__device__ __forceinline__ int unit_places(int ut) {
    return ut > 0 ? ut + PC : 0;
}

// Places of all row tiles of one head of a sequence.
template <int M, int KT, int PC>
__device__ __forceinline__ int64_t head_places(const PagedArgs& a, int b) {
    const SeqRows s = seq_rows(a, b);
    const int nrt = row_tiles<M>(a, s);
    if (nrt == 0) return 0;
    if (!a.causal || s.n == 1) return (int64_t)nrt * unit_places<PC>(unit_tiles<M, KT>(a, s, 0));
    int64_t sum = 0;
    for (int rt = first_row_tile<M>(a, s); rt < nrt; ++rt) sum += unit_places<PC>(unit_tiles<M, KT>(a, s, rt));
    return sum;
}

// A CTA's share of the line: [pos, end), beginning `off` places into sequence b, whose heads take per_head places each.
// Of W (total) places over n CTAs the first W % n CTAs take one more than the others; no share is empty (so that every CTA
// between those of a unit's first and last tile holds a part of it).
struct Cut {
    int64_t each;  // places of a share, rounded down
    int more;      // CTAs that take one more
};
struct Share {
    int64_t pos, end, off, per_head;
    Cut cut;
    int b;
};

__device__ __forceinline__ int64_t share_begin(const Cut& c, int cta) { return c.each * cta + min(cta, c.more); }

// The CTA that owns place x.
__device__ __forceinline__ int share_owner(const Cut& c, int64_t x) {
    const int64_t big = (c.each + 1) * c.more;
    return x < big ? (int)(x / (c.each + 1)) : c.more + (int)((x - big) / c.each);
}

// Computed by all threads of the CTA (a scan over the sequences; NT threads), result in *out (shared memory).
template <int M, int KT, int PC, int NT>
__device__ void find_share(const PagedArgs& a, int cta, int n_cta, Share* out) {
    constexpr int kWarps = NT / 32;
    __shared__ int64_t part[kWarps];
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
    if (threadIdx.x == 0) *out = Share{0, 0, 0, 0, Cut{0, 0}, a.n_seqs};
    // sequence b0 + threadIdx.x: its places of a head, and the inclusive sum of all heads' places from b0 on
    int64_t per_head, inc, sum;
    auto scan = [&](int b0) {
        const int b = b0 + threadIdx.x;
        per_head = b < a.n_seqs ? head_places<M, KT, PC>(a, b) : 0;
        inc = per_head * a.Hkv;
        for (int o = 1; o < 32; o <<= 1) {
            const int64_t up = __shfl_up_sync(~0u, inc, o);
            if (lane >= o) inc += up;
        }
        __syncthreads();  // (the warp sums of the scan before are read)
        if (lane == 31) part[warp] = inc;
        __syncthreads();
        sum = 0;
        for (int w = 0; w < kWarps; ++w) {
            if (w < warp) inc += part[w];
            sum += part[w];
        }
    };
    int64_t total = 0;
    int b0 = 0;
    for (;; b0 += NT) {
        scan(b0);
        total += sum;
        if (b0 + NT >= a.n_seqs) break;
    }
    if (n_cta > total) n_cta = (int)total;
    if (cta >= n_cta) return;
    const Cut cut = total <= INT_MAX ? Cut{(int)total / n_cta, (int)total % n_cta}
                                     : Cut{total / n_cta, (int)(total % n_cta)};
    const int64_t pos = share_begin(cut, cta), end = share_begin(cut, cta + 1);
    int64_t before = 0;
    if (b0 > 0) {  // more than one chunk of sequences: find the one
        for (b0 = 0;; b0 += NT) {
            scan(b0);
            if (before + sum > pos || b0 + NT >= a.n_seqs) break;  // (the second only if the lengths changed meanwhile)
            before += sum;
        }
    }
    const int64_t lo = before + inc - per_head * a.Hkv;
    if (lo <= pos && pos < before + inc) *out = Share{pos, end, pos - lo, per_head, cut, b0 + (int)threadIdx.x};
    __syncthreads();
}

// A piece of one unit: the rows row0 .. row0 + n_rows of a sequence's n*g rows (prefix: of the batch's n_tokens*g
// rows) against key tiles tile0 .. tile0 + n_tiles.
struct Seg {
    int b, h, row0, n_rows;
    int t0, n, len;        // the sequence (prefix: the whole batch, t0 = 0)
    int tile0, n_tiles;    // tile numbers from key 0
    bool begins, ends;     // the piece holds the unit's first / last tile
    int ordinal;           // own keys: pieces of this CTA before it
    int first_cta;         // of a cut unit, known where it ends
};

// The first sequence from b on that has a row with a key, n_seqs if there is none.  Called by whole warps, which look at 32
// sequences at a time.  (One by one, and each of their eight heads, 0.18 us each: 60 us against 23 for eight sequences in 256
// slots, 770 against 92 in 4096; 1.4 million idle slots on end are the 2 s that the other warps wait for a piece.)
__device__ __forceinline__ int next_sequence(const PagedArgs& a, int b) {
    for (; b < a.n_seqs; b += 32) {
        const int mine = b + (int)(threadIdx.x & 31);
        bool has = false;
        if (mine < a.n_seqs) {
            const SeqRows s = seq_rows(a, mine);
            has = s.n > 0 && s.len > a.key_begin;
        }
        const uint32_t some = __ballot_sync(~0u, has);
        if (some) return b + __ffs(some) - 1;
    }
    return a.n_seqs;
}

// Walks a CTA's share piece by piece (own keys).  Uniform over the threads that call it, whole warps.
template <int M, int KT, int PC>
struct OwnWalk {
    const PagedArgs& a;
    int64_t pos, end, base;  // base: the place of the unit's first tile
    Cut cut;
    SeqRows s;
    int b, h, rt, nrt, ut, ordinal;

    __device__ OwnWalk(const PagedArgs& args, const Share& sh)
        : a(args), pos(sh.pos), end(sh.end), cut(sh.cut), b(sh.b), ordinal(0) {
        if (pos >= end) return;
        s = seq_rows(a, b);
        nrt = row_tiles<M>(a, s);
        h = (int)(sh.off / sh.per_head);
        int64_t off = sh.off - h * sh.per_head;
        rt = first_row_tile<M>(a, s);
        ut = unit_tiles<M, KT>(a, s, rt);
        while (off >= unit_places<PC>(ut) && rt + 1 < nrt) {
            off -= unit_places<PC>(ut);
            ++rt;
            ut = unit_tiles<M, KT>(a, s, rt);
        }
        base = pos - off + PC;
    }

    __device__ bool next(Seg& g) {
        for (;;) {
            pos = max(pos, base);  // past the unit's places without a tile
            if (pos >= end) return false;
            if (ut > 0 && pos < base + ut) break;
            base += ut;  // on to the next unit that has keys
            if (++rt >= nrt) {
                if (++h >= a.Hkv) {
                    h = 0;
                    b = next_sequence(a, b + 1);
                    if (b >= a.n_seqs) return false;
                    s = seq_rows(a, b);
                    nrt = row_tiles<M>(a, s);
                }
                rt = first_row_tile<M>(a, s);
            }
            ut = unit_tiles<M, KT>(a, s, rt);
            base += PC;
        }
        const int64_t to = min(end, base + ut);
        g.b = b;
        g.h = h;
        g.row0 = rt * M;
        g.n_rows = min(M, s.n * a.g - g.row0);
        g.t0 = s.t0;
        g.n = s.n;
        g.len = s.len;
        g.tile0 = a.key_begin / KT + (int)(pos - base);
        g.n_tiles = (int)(to - pos);
        g.begins = pos == base;
        g.ends = to == base + ut;
        g.ordinal = ordinal++;
        g.first_cta = g.begins || !g.ends ? -1 : share_owner(cut, base);  // noted where the unit ends
        pos = to;
        return true;
    }
};

// The keys of a shared prefix: units are (row tile of the whole batch, head), all alike, so the host cuts each into
// p_split parts (what it weighs is said in paged_plan), one per CTA: CTA (head * row tiles + row tile) * p_split + part.
template <int M, int KT>
__device__ __forceinline__ Seg prefix_piece(const PagedArgs& a, int cta) {
    const int tiles = (a.prefix_len + KT - 1) / KT, nrt = (a.n_tokens * a.g + M - 1) / M;
    const int unit = cta / a.p_split, part = cta - unit * a.p_split;
    const int each = tiles / a.p_split, more = tiles - each * a.p_split;  // the first `more` parts have one tile more
    Seg g;
    g.b = -1;
    g.h = unit / nrt;
    g.row0 = (unit - g.h * nrt) * M;
    g.n_rows = min(M, a.n_tokens * a.g - g.row0);
    g.t0 = 0;
    g.n = a.n_tokens;
    g.len = 0;
    g.tile0 = part * each + min(part, more);
    g.n_tiles = each + (part < more ? 1 : 0);
    g.begins = part == 0;
    g.ends = part == a.p_split - 1;
    g.ordinal = 0;
    g.first_cta = 0;
    return g;
}

// The producer warp walks the share and hands each piece to the other warps through a ring of kSegs entries, so that the
// walk's divisions and registers are paid once; a piece without tiles ends it.  (The one piece of a prefix CTA follows from
// its number: every warp finds it for itself, and Q and the first pages are on their way before anything else is set up.)
constexpr int kSegs = 4;

// Keys that row r of a piece sees: below this limit (0 for a row of no sequence).
template <bool PREFIX>
__device__ __forceinline__ int row_limit(const PagedArgs& a, const Seg& g, int r) {
    const int i = (g.row0 + r) / a.g;
    if constexpr (!PREFIX) {
        return visible(a, SeqRows{g.t0, g.n, g.len}, i);
    } else {
        int lo = i;  // the sequence of token i
        if (a.q_start) {
            int hi = a.n_seqs;
            lo = 0;
            while (lo < hi) {  // first b with q_start[b + 1] > i
                const int mid = (lo + hi) >> 1;
                if (*(a.q_start + mid + 1) > i) hi = mid; else lo = mid + 1;
            }
        }
        if (lo >= a.n_seqs) return 0;
        const SeqRows s = seq_rows(a, lo);
        if (i < s.t0 || i >= s.t0 + s.n) return 0;
        return min(visible(a, s, i - s.t0), a.prefix_len);
    }
}

// First and last key (exclusive) that some row of a piece may see.
template <bool PREFIX>
__device__ __forceinline__ int seg_key_end(const PagedArgs& a, const Seg& g) {
    if constexpr (PREFIX) return a.prefix_len;
    return visible(a, SeqRows{g.t0, g.n, g.len}, (g.row0 + g.n_rows - 1) / a.g);
}

// Pages of a piece's keys; an entry outside the pool reads as -1.
template <bool PREFIX>
__device__ __forceinline__ int seg_page(const PagedArgs& a, const Seg& g, int j) {
    const int id = *((PREFIX ? a.prefix_pages : a.page_table + (int64_t)g.b * a.max_pages) + j);
    return (unsigned)id < (unsigned)a.n_pages ? id : -1;
}

// Where the result of row r of a piece goes: `out` (final, dtype of q) or `part` (float32), and its log-sum-exp
// (natural log in lse, log2 units elsewhere).  The four values from column c (a multiple of 4) on lie at part + c * step: a
// row of d values has step 1; slots written with a thread per row (GROUPS) are [d/4][M][4], so that a warp's stores of one
// group of columns are 512 contiguous bytes, and have step M.
struct RowDst {
    void* out;
    float* part;
    float* lse;
    int step;
};

template <int M, bool PREFIX, bool GROUPS = false>
__device__ __forceinline__ RowDst row_dst(const PagedArgs& a, const Seg& g, int r, int cta) {
    if (!PREFIX && g.begins && g.ends) {
        const int R = g.row0 + r, i = R / a.g;
        const int64_t row = (int64_t)(g.t0 + i) * a.Hq + g.h * a.g + (R - i * a.g);
        if (a.prefix_len == 0)
            return {static_cast<char*>(a.o) + row * a.d * a.elem, nullptr, a.lse + row, 1};
        return {nullptr, a.own_o + row * a.d, a.own_lse + row, 1};
    }
    const int64_t slot = PREFIX ? (int64_t)cta : (int64_t)cta * 2 + (g.begins ? 1 : 0);
    float* o = (PREFIX ? a.pslot_o : a.slot_o) + slot * M * a.d;
    float* l = (PREFIX ? a.pslot_l : a.slot_l) + slot * M + r;
    return GROUPS ? RowDst{nullptr, o + r * 4, l, M} : RowDst{nullptr, o + (int64_t)r * a.d, l, 1};
}

// Tells paged_merge_kernel about row r of a piece; called by the CTA that holds the unit's last tile.
template <int M>
__device__ __forceinline__ void note_row(const PagedArgs& a, const Seg& g, int r, int cta) {
    const int R = g.row0 + r, i = R / a.g;
    const int64_t row = (int64_t)(g.t0 + i) * a.Hq + g.h * a.g + (R - i * a.g);
    uint2 w;
    if (g.begins) {
        w = make_uint2(a.prefix_len ? kRowWhole : kRowDone, 0);
    } else {
        w = make_uint2(kRowSplit | (uint32_t)r << 2, (uint32_t)g.first_cta | (uint32_t)cta << 16);
    }
    a.row_info[row] = w;
}

// Rows that no unit covers: those of sequences whose row tiles have no keys (o = 0, lse = -inf, or left to the prefix),
// and rows of no sequence (not touched).  Spread over the CTAs; all threads of the CTA (NT) call it.
template <typename T, int M, int KT, int NT>
__device__ void finish_empty_rows(const PagedArgs& a, int cta, int n_cta) {
    const int lo = a.q_start ? min(max(*a.q_start, 0), a.n_tokens) : 0;
    const int hi = a.q_start ? min(max(*(a.q_start + a.n_seqs), lo), a.n_tokens) : a.n_tokens;
    for (int64_t x = (int64_t)cta * NT + threadIdx.x; x < (int64_t)(a.n_tokens - (hi - lo)) * a.Hq;
         x += (int64_t)n_cta * NT) {
        const int64_t row = x < (int64_t)lo * a.Hq ? x : x + (int64_t)(hi - lo) * a.Hq;
        a.row_info[row] = make_uint2(kRowDone, 0);
    }
    // (as many CTAs per sequence as there are: three whose 290 tokens mostly see nothing: 51 us with one each, 27 so)
    const int per_seq = max(n_cta / a.n_seqs, 1), part = cta % per_seq;
    for (int b = cta / per_seq; b < a.n_seqs; b += n_cta / per_seq) {
        const SeqRows s = seq_rows(a, b);
        const int rt = first_row_tile<M>(a, s);
        const uint32_t rows = rt < row_tiles<M>(a, s) ? rt * M : s.n * a.g;
        for (uint32_t x = part * NT + threadIdx.x; x < rows * a.Hkv; x += per_seq * NT) {
            const int h = x / rows, R = x % rows, i = R / a.g;
            const int64_t row = (int64_t)(s.t0 + i) * a.Hq + h * a.g + (R - i * a.g);
            a.row_info[row] = make_uint2(a.prefix_len ? kRowNone : kRowDone, 0);
            if (a.prefix_len == 0) {
                a.lse[row] = -INFINITY;
                uint4* o = reinterpret_cast<uint4*>(static_cast<T*>(a.o) + row * a.d);
                for (int c = 0; c < a.d * (int)sizeof(T) / 16; ++c) o[c] = make_uint4(0, 0, 0, 0);
            }
        }
    }
}

}  // namespace usp
