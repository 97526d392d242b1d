// Pages of the paged cache: who holds them (forking, truncating, freeing, growing and compacting, on the device, so that lengths
// which only the device knows, accepted drafts say, need no wait of the host) and copies of them.
//
// The state is the page table, the lengths and a count per page of the table's entries that name it (and of the user's own holds);
// a page whose count is 0 is free.  There is no list of free pages: pages are handed out lowest first, found by going over
// the counts, so that the same state gives the same pages and a pool fills from its beginning.
//
// usp_pages_update is bound by latency (64 conversations in a pool of 4568 pages need 20 KB): one launch of one cluster, whose CTAs
// each take a share of the slots and of the pages, with a barrier of the cluster where all have to have counted:
//   1 the counts are copied to the workspace and what the slots do is worked out: what they hold is counted off, what they go
//     on with is counted on (what stays is left alone), rows that come from another slot are put aside, and a page that
//     ends inside and is about to be written counts its writers and remembers the first;
//   2 a writer that must not keep such a page takes a copy; new pages and copies are numbered slot by slot, free pages page by page;
//   3 if there are enough: rows, counts and lengths are written, and the list of copies.
#include <algorithm>

#include "cluster.cuh"
#include "paged.cuh"

namespace usp {

namespace {

constexpr int kThreads = 1024;
constexpr int kWarps = kThreads / 32;
constexpr int kCtas = 8;          // of a cluster

// Exclusive running sum over the CTA's threads, and the total to all.
__device__ __forceinline__ uint64_t block_scan(uint64_t x, uint64_t* total, uint64_t (&part)[kWarps]) {
    const int warp = threadIdx.x / 32, lane = threadIdx.x % 32;
    uint64_t to = x;
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
        const uint64_t y = __shfl_up_sync(~0u, to, o);
        if (lane >= o) to += y;
    }
    __syncthreads();  // (part may still be read from the last time)
    if (lane == 31) part[warp] = to;
    __syncthreads();
    uint64_t sum = part[lane], before = lane < warp ? sum : 0;
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) {
        sum += __shfl_xor_sync(~0u, sum, o);
        before += __shfl_xor_sync(~0u, before, o);
    }
    *total = sum;
    return before + to - x;
}

// Share `rank` of n things among kCtas, and of a CTA's share among its warps.
__device__ __forceinline__ int share(int n, int rank) { return (int)((int64_t)n * rank / kCtas); }
__device__ __forceinline__ int warp_share(int i0, int i1, int warp) { return i0 + (int)((int64_t)(i1 - i0) * warp / kWarps); }

// The places of [i0, i1) (a warp's) for which `is` holds, in order: f(place, number of those before it).  Returns how many.
template <typename Is, typename F>
__device__ __forceinline__ int each_of(int i0, int i1, Is&& is, F&& f) {
    const int lane = threadIdx.x % 32;
    int n = 0;
#pragma unroll 4
    for (int i = i0; i < i1; i += 32) {
        const bool x = i + lane < i1 && is(i + lane);
        const uint32_t m = __ballot_sync(~0u, x);
        if (x) f(i + lane, n + __popc(m & ((1u << lane) - 1)));
        n += __popc(m);
    }
    return n;
}

struct UpdateSpace {
    int32_t *count, *writers, *free_ids;  // [n_pages]
    uint32_t* first;                      // [n_pages]
    int4* slot;                                    // [n_seqs]: kept, new, pages held, place of what it needs
    int32_t* copy;                                 // [n_seqs]: its copy's place in the list, -1: none
    int32_t* stage;                                // [n_seqs][max_pages]: rows that come from another slot
};

__host__ __device__ inline size_t layout(int n_seqs, int max_pages, int n_pages, char* ws, UpdateSpace* u) {
    size_t at = 0;
    auto take = [&](size_t bytes) {
        char* p = ws + at;
        at += (bytes + 255) / 256 * 256;
        return p;
    };
    u->count = reinterpret_cast<int32_t*>(take(4 * (size_t)n_pages));
    u->writers = reinterpret_cast<int32_t*>(take(4 * (size_t)n_pages));
    u->first = reinterpret_cast<uint32_t*>(take(4 * (size_t)n_pages));
    u->free_ids = reinterpret_cast<int32_t*>(take(4 * (size_t)n_pages));
    u->slot = reinterpret_cast<int4*>(take(16 * (size_t)n_seqs));
    u->copy = reinterpret_cast<int32_t*>(take(4 * (size_t)n_seqs));
    u->stage = reinterpret_cast<int32_t*>(take(4 * (size_t)n_seqs * max_pages));
    return at;
}

__global__ void __launch_bounds__(kThreads) pages_update_kernel(const PagesUpdateParams p, const UpdateSpace u) {
    __shared__ uint64_t part[kWarps];
    __shared__ uint64_t said[3];  // to the cluster: what its slots need, their copies, its free pages | those before << 32
    const int rank = (int)cluster_rank(), warp = threadIdx.x / 32, lane = threadIdx.x % 32;
    const int page = 1 << p.page_log2, cap = p.max_pages << p.page_log2;
    const int p0 = share(p.n_pages, rank), p1 = share(p.n_pages, rank + 1);
    const int s0 = share(p.n_seqs, rank), s1 = share(p.n_seqs, rank + 1);
    auto pages = [&](int tokens) { return (tokens + page - 1) >> p.page_log2; };
    auto inside = [&](int id) { return id >= 0 && id < p.n_pages; };
    auto length = [&](int b) { return min(max(__ldcg(p.seq_lens + b), 0), cap); };
    auto parent = [&](int b) { return p.parent ? __ldcg(p.parent + b) : b; };
    // of the writers of a page the one that holds it already is the first, then the lowest slot
    auto order = [](int a, int b) { return a == b ? (uint32_t)b : (uint32_t)b | 0x80000000u; };
    begin_kernel(false);
    int held = 0;  // pages that are free before
    for (int i = p0 + threadIdx.x; i < p1; i += kThreads) {
        const int c = __ldcg(p.ref + i);
        u.count[i] = c;
        u.writers[i] = 0;
        u.first[i] = ~0u;
        held += c <= 0;
    }
    cluster_sync();

    // (warps of all CTAs in turn: rows are of any length)
    for (int64_t b0 = warp * kCtas + rank; b0 < p.n_seqs; b0 += kWarps * kCtas) {
        const int b = (int)b0, a = parent(b);
        const bool known = a >= 0 && a < p.n_seqs;
        const int old = length(b), most = known ? length(a) : 0;
        const int kept = p.keep ? min(max(__ldcg(p.keep + b), 0), most) : most;
        const int grow = p.grow ? max(__ldcg(p.grow + b), 0) : 0;
        const int now = kept + min(grow, cap - kept);
        const int kept_n = pages(kept);
        if (lane == 0) u.slot[b] = make_int4(kept, now, pages(old), 0);
        const int32_t* mine = p.page_table + (int64_t)b * p.max_pages;
        const int32_t* from = known ? p.page_table + (int64_t)a * p.max_pages : mine;
#pragma unroll 4
        for (int j = (a == b ? kept_n : 0) + lane; j < pages(old); j += 32) {
            const int id = __ldcg(mine + j);
            if (inside(id)) atomicAdd(u.count + id, -1);
        }
        if (a != b) {
            int32_t* stage = u.stage + (int64_t)b * p.max_pages;
#pragma unroll 4
            for (int j = lane; j < kept_n; j += 32) {
                const int id = __ldcg(from + j);
                stage[j] = id;
                if (inside(id)) atomicAdd(u.count + id, 1);
            }
        }
        if (lane == 0 && now > kept && (kept & (page - 1))) {
            const int id = __ldcg(from + kept_n - 1);
            if (inside(id)) {
                atomicAdd(u.writers + id, 1);
                atomicMin(u.first + id, order(a, b));
            }
        }
    }
    cluster_sync();

    uint64_t needs = 0, copying = 0;  // of this CTA's slots
    for (int64_t b0 = s0; b0 < s1; b0 += kThreads) {
        const int b = (int)b0 + threadIdx.x;
        const bool some = b0 + threadIdx.x < s1;
        uint64_t x = 0;  // pages that the slot needs (2^27 at most), and 2^40 if one of them is a copy
        bool copies = false;
        if (some) {
            const int4 s = __ldcg(u.slot + b);
            if (s.y > s.x && (s.x & (page - 1))) {
                const int a = parent(b);
                const int id = __ldcg(p.page_table + (int64_t)a * p.max_pages + (s.x >> p.page_log2));
                if (inside(id))
                    copies = __ldcg(u.count + id) != __ldcg(u.writers + id) || __ldcg(u.first + id) != order(a, b);
            }
            x = (uint64_t)(pages(s.y) - pages(s.x) + copies) | (uint64_t)copies << 40;
        }
        uint64_t sum;
        const uint64_t at = block_scan(x, &sum, part);
        if (some) {
            u.slot[b].w = (int)(needs + (at & ((1ull << 40) - 1)));
            u.copy[b] = copies ? (int)(copying + (at >> 40)) : -1;
        }
        needs += sum & ((1ull << 40) - 1);
        copying += sum >> 40;
    }
    const int w0 = warp_share(p0, p1, warp), w1 = warp_share(p0, p1, warp + 1);
    auto is_free = [&](int i) { return __ldcg(u.count + i) <= 0; };
    const int mine = each_of(w0, w1, is_free, [](int, int) {});
    uint64_t sum;
    const int before = (int)(block_scan((lane == 0 ? mine : 0) | (uint64_t)held << 32, &sum, part) & 0xffffffffu);
    const int at = p0 + __shfl_sync(~0u, before, 0);
    each_of(w0, w1, is_free, [&](int i, int k) { u.free_ids[at + k] = i; });
    if (threadIdx.x == 0) {
        said[0] = needs;
        said[1] = copying;
        said[2] = sum;
    }
    cluster_sync();

    uint64_t told[3];
#pragma unroll
    for (int k = 0; k < 3; ++k) told[k] = lane < kCtas ? cluster_read(&said[k], lane) : 0;
    cluster_arrive();  // (waited for at the end: others may still read what this CTA says)
    int64_t need = 0, copies = 0, free_n = 0, left = 0, need_before = 0, copies_before = 0, free_before[kCtas];
#pragma unroll
    for (int c = 0; c < kCtas; ++c) {
        const uint64_t x = __shfl_sync(~0u, told[0], c), y = __shfl_sync(~0u, told[1], c), z = __shfl_sync(~0u, told[2], c);
        if (c < rank) {
            need_before += x;
            copies_before += y;
        }
        free_before[c] = free_n;
        need += x;
        copies += y;
        free_n += (uint32_t)z;
        left += z >> 32;
    }
    const bool enough = need <= free_n;
    if (rank == 0 && threadIdx.x == 0)
        *reinterpret_cast<int4*>(p.copies) = enough ? make_int4((int)copies, 0, (int)(free_n - need), 0)
                                                    : make_int4(0, (int)min(need - free_n, (int64_t)INT32_MAX), (int)left, 0);
    if (enough) {
        auto free_page = [&](int64_t k) {  // the k-th free page
            int c = 0;
            int64_t first = 0;
#pragma unroll
            for (int i = 1; i < kCtas; ++i)
                if (free_before[i] <= k) {
                    c = i;
                    first = free_before[i];
                }
            return __ldcg(u.free_ids + share(p.n_pages, c) + (k - first));
        };
        for (int64_t b0 = s0 + warp; b0 < s1; b0 += kWarps) {
            const int b = (int)b0;
            const int4 s = __ldcg(u.slot + b);
            const int copy = __ldcg(u.copy + b), kept_n = pages(s.x), new_n = pages(s.y);
            const bool other = parent(b) != b;
            int32_t* row = p.page_table + (int64_t)b * p.max_pages;
            const int32_t* had = other ? u.stage + (int64_t)b * p.max_pages : row;
            int64_t k = need_before + s.w;
            if (copy >= 0) {
                const int from = __ldcg(had + kept_n - 1), to = free_page(k);
                __syncwarp();  // (the row's entry is read before it is written)
                if (lane == 0) {
                    row[kept_n - 1] = to;
                    *reinterpret_cast<int4*>(p.copies + 4 * (1 + copies_before + copy)) = make_int4(from, to, s.x & (page - 1), 0);
                }
                ++k;
            }
            if (other) {
#pragma unroll 4
                for (int j = lane; j < kept_n - (copy >= 0); j += 32) row[j] = __ldcg(had + j);
            }
            for (int j = kept_n + lane; j < new_n; j += 32) row[j] = free_page(k + (j - kept_n));
            for (int j = new_n + lane; j < s.z; j += 32) row[j] = -1;
            if (lane == 0) p.seq_lens[b] = s.y;
        }
        // the free pages up to `last` of this CTA's are taken
        int64_t taken = need, here = 0;
#pragma unroll
        for (int c = 0; c < kCtas; ++c)
            if (c == rank) {
                taken -= free_before[c];
                here = (c + 1 < kCtas ? free_before[c + 1 < kCtas ? c + 1 : c] : free_n) - free_before[c];
            }
        taken = min(taken, here);
        const int last = taken > 0 ? __ldcg(u.free_ids + p0 + (taken - 1)) : -1;
        for (int i = p0 + threadIdx.x; i < p1; i += kThreads) {
            const int c = __ldcg(u.count + i), w = __ldcg(u.writers + i);
            p.ref[i] = c <= 0 ? i <= last : c - w + (w > 0 && c == w);  // (where all write, one stays)
        }
    }
    cluster_wait();
}

// Live pages with ids from their number on go, lowest first, to the free ids below it, lowest first.
__global__ void __launch_bounds__(kThreads) pages_compact_kernel(const PagesCompactParams p) {
    __shared__ uint64_t part[kWarps];
    __shared__ uint64_t said[2];  // to the cluster: its live pages; those that move | free ids that are filled << 32
    const int rank = (int)cluster_rank(), warp = threadIdx.x / 32, lane = threadIdx.x % 32;
    const int p0 = share(p.n_pages, rank), p1 = share(p.n_pages, rank + 1);
    const int w0 = warp_share(p0, p1, warp), w1 = warp_share(p0, p1, warp + 1);
    begin_kernel(false);
    auto live = [&](int i) { return __ldcg(p.ref + i) > 0; };
    const int mine = each_of(w0, w1, live, [](int, int) {});
    uint64_t sum;
    block_scan(lane == 0 ? mine : 0, &sum, part);
    if (threadIdx.x == 0) said[0] = sum;
    cluster_sync();
    uint64_t x = lane < kCtas ? cluster_read(&said[0], lane) : 0;
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) x += __shfl_xor_sync(~0u, x, o);
    const int n_live = (int)x;
    auto moves = [&](int i) { return i >= n_live && live(i); };
    auto filled = [&](int i) { return i < n_live && !live(i); };
    const uint64_t movers = each_of(w0, w1, moves, [](int, int) {}), holes = each_of(w0, w1, filled, [](int, int) {});
    uint64_t before = block_scan(lane == 0 ? movers | holes << 32 : 0, &sum, part);
    before = __shfl_sync(~0u, before, 0);
    if (threadIdx.x == 0) said[1] = sum;
    cluster_sync();
    x = lane < kCtas ? cluster_read(&said[1], lane) : 0;
    uint64_t all = x, mine_at = lane < rank ? x : 0;
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) {
        all += __shfl_xor_sync(~0u, all, o);
        mine_at += __shfl_xor_sync(~0u, mine_at, o);
    }
    before += mine_at;
    const int at_moves = (int)(uint32_t)before, at_holes = (int)(before >> 32);
    int4* rows = reinterpret_cast<int4*>(p.copies) + 1;
    if (rank == 0 && threadIdx.x == 0) rows[-1] = make_int4((int)(uint32_t)all, 0, p.n_pages - n_live, 0);
    each_of(w0, w1, filled, [&](int i, int k) { rows[at_holes + k].y = i; });
    for (int i = w0 + lane; i < w1; i += 32) {
        const int c = __ldcg(p.ref + i);
        if (c <= 0) {
            p.new_id[i] = -1;
            if (i >= n_live) p.ref_out[i] = 0;
        } else if (i < n_live) {
            p.new_id[i] = i;
            p.ref_out[i] = c;
        }
    }
    cluster_sync();
    // (from here on counts of pages that move are read, each by the warp that writes them: ref_out may be ref)
    each_of(w0, w1, moves, [&](int i, int k) {
        const int to = __ldcg(&rows[at_moves + k].y);
        rows[at_moves + k].x = i;
        rows[at_moves + k].z = 1 << p.page_log2;
        rows[at_moves + k].w = 0;
        p.new_id[i] = to;
        p.ref_out[to] = __ldcg(p.ref + i);
        p.ref_out[i] = 0;
    });
}

// Entries of the page table by their pages' new ids (those that name no live page stay).
__global__ void __launch_bounds__(256) pages_rename_kernel(const PagesCompactParams p) {
    begin_kernel(false);
    const int64_t n = (int64_t)p.n_seqs * p.max_pages;
    for (int64_t i = blockIdx.x * 256ll + threadIdx.x; i < n; i += gridDim.x * 256ll) {
        const int id = __ldcg(p.page_table + i);
        const int to = id >= 0 && id < p.n_pages ? __ldcg(p.new_id + id) : -1;
        p.page_table_out[i] = to >= 0 ? to : id;
    }
}

// The pages' data.  A page of K, or of V, in pieces of kCopyThreads * kCopyAhead vectors of 16 bytes; those of tokens that the
// copy leaves out are passed over.  Bound by HBM.
constexpr int kCopyThreads = 256;
constexpr int kCopyAhead = 8;

__global__ void __launch_bounds__(kCopyThreads) pages_copy_kernel(const PagesCopyParams p, int head_log2, int pieces) {
    begin_kernel(false);
    const int n = min(max(__ldcg(p.copies), 0), p.max_copies);
    const int64_t items = (int64_t)n * p.n_layers * 2 * pieces;
    const int head = 1 << head_log2;                              // vectors of a page's head
    const int64_t page = (int64_t)p.Hkv << head_log2;
    const int row_log2 = head_log2 - p.page_log2;                 // vectors of a token
    for (int64_t item = blockIdx.x; item < items; item += gridDim.x) {
        const int piece = (int)(item % pieces);
        const int64_t rest = item / pieces;
        const int layer = (int)((rest >> 1) % p.n_layers);
        const int4 c = __ldcg(reinterpret_cast<const int4*>(p.copies) + 1 + (rest >> 1) / p.n_layers);
        if (c.x < 0 || c.x >= p.n_pages || c.y < 0 || c.y >= p.n_pages || c.x == c.y) continue;
        uint4* pool = reinterpret_cast<uint4*>(static_cast<char*>(rest & 1 ? p.v_pages : p.k_pages) + layer * p.layer_bytes);
        const uint4* from = pool + c.x * page;
        uint4* to = pool + c.y * page;
        const int64_t v0 = (int64_t)piece * (kCopyThreads * kCopyAhead) + threadIdx.x;
        auto wanted = [&](int64_t v) { return v < page && (int)(v & (head - 1)) >> row_log2 < c.z; };
        uint4 w[kCopyAhead];
#pragma unroll
        for (int e = 0; e < kCopyAhead; ++e)
            if (wanted(v0 + e * kCopyThreads)) w[e] = __ldcs(from + v0 + e * kCopyThreads);
#pragma unroll
        for (int e = 0; e < kCopyAhead; ++e)
            if (wanted(v0 + e * kCopyThreads)) __stcs(to + v0 + e * kCopyThreads, w[e]);
    }
}

}  // namespace

size_t pages_update_workspace(int n_seqs, int max_pages, int n_pages) {
    UpdateSpace u;
    return layout(n_seqs, max_pages, n_pages, nullptr, &u);
}

cudaError_t launch_pages_update(const PagesUpdateParams& p, cudaStream_t stream) {
    UpdateSpace u;
    layout(p.n_seqs, p.max_pages, p.n_pages, static_cast<char*>(p.ws), &u);
    return launch_clusters(pages_update_kernel, 1, kCtas, kThreads, 0, stream, p, u);
}

cudaError_t launch_pages_compact(const PagesCompactParams& p, cudaStream_t stream) {
    cudaError_t e = launch_clusters(pages_compact_kernel, 1, kCtas, kThreads, 0, stream, p);
    const int64_t n = (int64_t)p.n_seqs * p.max_pages;
    if (e != cudaSuccess || n == 0) return e;
    return launch_dependent(pages_rename_kernel, dim3((unsigned)std::min<int64_t>((n + 255) / 256, 8 * 152)), 256, 0, stream, p);
}

cudaError_t launch_pages_copy(const PagesCopyParams& p, cudaStream_t stream) {
    int row_log2 = 0;
    while (16 << row_log2 < p.row_bytes) ++row_log2;
    const int head_log2 = row_log2 + p.page_log2;
    const int64_t per = kCopyThreads * kCopyAhead, pieces = (((int64_t)p.Hkv << head_log2) + per - 1) / per;
    const int64_t items = (int64_t)p.max_copies * p.n_layers * 2 * pieces;
    return launch_dependent(pages_copy_kernel, dim3((unsigned)std::min<int64_t>(items, 6 * 152)), kCopyThreads, 0, stream, p,
                            head_log2, (int)pieces);
}

}  // namespace usp
