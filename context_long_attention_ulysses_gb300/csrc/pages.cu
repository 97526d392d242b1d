// Pages of the paged cache: who holds them (forking, truncating, freeing, growing and compacting, on the device, so that lengths
// which only the device knows, accepted drafts say, need no wait of the host) and copies of them.
//
// The state is the page table, the lengths and a count per page of the table's entries that name it (and of the user's own holds);
// a page whose count is 0 is free.  There is no list of free pages: pages are handed out lowest first, found by going over
// the counts, so that the same state gives the same pages and a pool fills from its beginning.
//
// usp_pages_update is bound by latency (64 conversations in a pool of 4568 pages need 20 KB), its steps are
//   init    the pages' counts;
//   enter, move   what the slots hold is counted off, what they go on with is counted on (what stays is left alone).  A page that
//           ends inside and is about to be written is not counted but remembers the first of its writers: if its count is 0
//           then, the writers alone hold it, and the first keeps it;
//   number  new pages and copies slot by slot, free pages page by page;
//   write   rows, lengths, the list of copies, counts, if there are pages enough.
// Small caches take one CTA with all counts in its shared memory (64 conversations 4.7 us in a captured graph; 11.4 as one cluster
// of eight CTAs with the counts in L2, where a step's few dependent accesses and a barrier cost 1 to 4 us), others a launch for each
// step, which follow each other by dependent launch.
#include <algorithm>

#include "cluster.cuh"
#include "paged.cuh"

namespace usp {

namespace {

constexpr int kThreads = 1024;
constexpr int kWarps = kThreads / 32;
constexpr int kCtas = 8;           // of a cluster

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

// Share `k` of `n` in [i0, i1).
__device__ __forceinline__ int share(int i0, int i1, int k, int n) { return i0 + (int)((int64_t)(i1 - i0) * k / n); }

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

constexpr uint32_t kNobody = ~0u;

// What the update's steps keep between them: in the shared memory of the one CTA, or in the workspace.
struct Books {
    int32_t* count;     // [n_pages]: holders, without those that are about to write the page
    uint32_t* first;    // [n_pages]: the first of those, kNobody
    int32_t* free_ids;  // [n_pages]: free pages, lowest first
    int4* slot;         // [n_seqs]: tokens kept, tokens afterwards, pages held before, the page that ends inside (-1: none)
    int4* place;        // [n_seqs]: where the pages it gets begin, its copy's place in the list (-1: none), kSlot flags, parent
    int32_t* stage;     // [n_seqs][max_pages]: rows of slots that change places (workspace in any case)
    int64_t* totals;    // pages needed, free pages (as many at least, or fewer)
};
enum : int { kSlotOther = 1, kSlotStaged = 2, kSlotWrites = 4 };

__host__ __device__ inline size_t books_bytes(int n_seqs, int n_pages) { return 12 * (size_t)n_pages + 32 * (size_t)n_seqs; }

// n_pages and n_seqs of the caches that one CTA takes and, where `parent` is given, the table's entries, which it may then have to
// copy.  In a captured graph, one CTA and the launches: eight samples of 360 entries in all 4.6 and 7.3 us, 64 of 16000 8.7 and
// 8.3, 120 of 61600 23.5 and 10.8, 256 of 131000 43 and 11.8; with a parent that is every slot itself 4.7 and 7.4, whatever the
// table.  (Entries that are dropped without `parent` play no part in the rule: a table of 131000 released at once takes the CTA 36 us,
// the launches would take 10.3; a step that drops little 4.8 and 7.2.)
constexpr int kOnePages = 16384, kOneSeqs = 1024;
constexpr int64_t kOneEntries = 1 << 16;
__host__ __device__ inline bool one_cta(const PagesUpdateParams& p) {
    return p.n_pages <= kOnePages && p.n_seqs <= kOneSeqs && (!p.parent || (int64_t)p.n_seqs * p.max_pages <= kOneEntries);
}

__host__ __device__ inline size_t layout(int n_seqs, int max_pages, int n_pages, char* ws, Books* u) {
    size_t at = 0;
    auto take = [&](size_t bytes) {
        char* p = ws + at;
        at += (bytes + 255) / 256 * 256;
        return p;
    };
    u->totals = reinterpret_cast<int64_t*>(take(2 * sizeof(int64_t)));
    u->count = reinterpret_cast<int32_t*>(take(4 * (size_t)n_pages));
    u->first = reinterpret_cast<uint32_t*>(take(4 * (size_t)n_pages));
    u->free_ids = reinterpret_cast<int32_t*>(take(4 * (size_t)n_pages));
    u->slot = reinterpret_cast<int4*>(take(16 * (size_t)n_seqs));
    u->place = reinterpret_cast<int4*>(take(16 * (size_t)n_seqs));
    u->stage = reinterpret_cast<int32_t*>(take(4 * (size_t)n_seqs * max_pages));
    return at;
}

// The steps, for PagesUpdateParams p and Books u that more than one CTA uses (ONE: one CTA, the books in its shared memory).
template <bool ONE>
struct Update {
    const PagesUpdateParams& p;
    const Books u;

    template <typename T>
    __device__ __forceinline__ static T get(const T* x) {
        if constexpr (ONE) return *x;
        return __ldcg(x);
    }
    __device__ __forceinline__ int pages(int tokens) const { return (tokens + (1 << p.page_log2) - 1) >> p.page_log2; }
    __device__ __forceinline__ bool inside(int id) const { return id >= 0 && id < p.n_pages; }
    __device__ __forceinline__ bool slot_exists(int b) const { return b >= 0 && b < p.n_seqs; }
    __device__ __forceinline__ int length(int b) const { return min(max(__ldcg(p.seq_lens + b), 0), p.max_pages << p.page_log2); }
    __device__ __forceinline__ int parent(int b) const { return p.parent ? __ldcg(p.parent + b) : b; }
    __device__ __forceinline__ int kept(int b, int most) const { return p.keep ? min(max(__ldcg(p.keep + b), 0), most) : most; }
    __device__ __forceinline__ int32_t* row(int b) const { return p.page_table + (int64_t)b * p.max_pages; }
    __device__ __forceinline__ int32_t* stage(int b) const { return u.stage + (int64_t)b * p.max_pages; }
    // of the writers of a page the one that holds it already is the first, then the lowest slot
    __device__ __forceinline__ static uint32_t order(int a, int b) { return a == b ? (uint32_t)b : (uint32_t)b | 0x80000000u; }
    __device__ __forceinline__ bool is_free(int i) const { return get(u.count + i) <= 0 && get(u.first + i) == kNobody; }

    // The pages' counts, every n-th from k on.
    __device__ __forceinline__ void init(int k, int n) const {
#pragma unroll 4
        for (int i = k; i < p.n_pages; i += n) {
            const int c = __ldcg(p.ref + i);
            u.count[i] = c;
            u.first[i] = kNobody;
        }
    }

    __device__ __forceinline__ void add(int id, int n) const {
        if (inside(id)) atomicAdd(u.count + id, n);
    }

    // f(j, x[j], y[j]) for the places [from, max(nx, ny)) of two rows, -1 behind the first nx and ny, by `lanes` threads.
    template <typename F>
    __device__ __forceinline__ static void entries(const int32_t* x, int nx, const int32_t* y, int ny, int from, int lane, int lanes,
                                                   F&& f) {
        const int end = max(nx, ny);
        for (int j = from + lane; j < end; j += 8 * lanes) {
            int a[8], b[8];
#pragma unroll
            for (int e = 0; e < 8; ++e) {
                const int i = j + e * lanes;
                a[e] = i < nx ? __ldcg(x + i) : -1;
                b[e] = i < ny ? __ldcg(y + i) : -1;
            }
#pragma unroll
            for (int e = 0; e < 8; ++e)
                if (j + e * lanes < end) f(j + e * lanes, a[e], b[e]);
        }
    }

    // What a slot is to do, in the order in which it becomes known: what the caller says, then pages that its rows name.
    struct Entry {
        int parent, length, keep, grow;
        int last, drops[2];  // the page that ends inside the kept tokens, -1; the first two that a slot which goes on by itself drops
        int4 slot;
        int flags;
    };
    __device__ __forceinline__ Entry ask(int b) const {
        Entry e;
        e.parent = parent(b);
        e.length = __ldcg(p.seq_lens + b);
        e.keep = p.keep ? __ldcg(p.keep + b) : INT32_MAX;
        e.grow = p.grow ? __ldcg(p.grow + b) : 0;
        return e;
    }
    __device__ __forceinline__ void look_up(int b, Entry& e) const {
        const int a = e.parent, cap = p.max_pages << p.page_log2;
        const bool known = slot_exists(a), other = a != b;
        const int old = min(max(e.length, 0), cap), most = known ? other ? length(a) : old : 0;
        const int keeps = min(max(e.keep, 0), most), now = keeps + min(max(e.grow, 0), cap - keeps);
        const int old_n = pages(old), kept_n = pages(keeps);
        // (what a slot that goes on by itself keeps is not written in this call, and can be read from its row at the end)
        const bool staged = other && keeps > 0 && (parent(a) != a || kept(a, most) < keeps);
        const bool ends_inside = keeps & ((1 << p.page_log2) - 1);
        e.last = ends_inside ? __ldcg(row(a) + kept_n - 1) : -1;
#pragma unroll
        for (int j = 0; j < 2; ++j) e.drops[j] = !other && kept_n + j < old_n ? __ldcg(row(b) + kept_n + j) : -1;
        e.slot = make_int4(keeps, now, old_n, e.last);
        e.flags = (other ? kSlotOther : 0) | (staged ? kSlotStaged : 0) | (ends_inside && now > keeps && inside(e.last) ? kSlotWrites : 0);
    }
    __device__ __forceinline__ void enter(int b, const Entry& e) const {
        u.slot[b] = e.slot;
        u.place[b] = make_int4(0, -1, e.flags, e.parent);
        if (e.flags & kSlotWrites) {
            atomicMin(u.first + e.last, order(e.parent, b));
            atomicAdd(u.count + e.last, -1);  // (counted on by move(), or already)
        }
#pragma unroll
        for (int j = 0; j < 2; ++j) add(e.drops[j], -1);
    }
    // Entries of the table that move() and write() read for slot b.
    __device__ __forceinline__ int reads(int b) const {
        const int4 s = get(u.slot + b);
        return get(u.place + b).z & kSlotOther ? max(s.z, pages(s.x)) : s.z - pages(s.x);
    }
    // The rest of what slot b gives up, and what it takes over, by `lanes` threads.  (Pages that it holds in the same place
    // before and after, as when the same prompt is forked again, are left alone.)
    __device__ __forceinline__ void move(int b, int lane, int lanes) const {
        const int4 at = get(u.place + b);
        move(b, get(u.slot + b), at.z, at.w, lane, lanes);
    }
    __device__ __forceinline__ void move(int b, const int4& s, int flags, int from, int lane, int lanes) const {
        const int kept_n = pages(s.x);
        if (!(flags & kSlotOther)) {
            entries(row(b), s.z, nullptr, 0, kept_n + 2, lane, lanes, [&](int, int id, int) { add(id, -1); });
            return;
        }
        int32_t* const to = flags & kSlotStaged ? stage(b) : nullptr;
        entries(row(b), s.z, kept_n > 0 ? row(from) : nullptr, kept_n, 0, lane, lanes, [&](int j, int old, int id) {
            if (old != id) {
                add(old, -1);
                add(id, 1);
            }
            if (to && j < kept_n) to[j] = id;
        });
    }

    // What slot b needs: pages (2^27 at most), and 2^40 if one of them is a copy.
    __device__ __forceinline__ uint64_t needs(int b) const {
        const int4 s = get(u.slot + b), at = get(u.place + b);
        const bool copies = (at.z & kSlotWrites) && (get(u.count + s.w) > 0 || get(u.first + s.w) != order(at.w, b));
        return (uint64_t)(pages(s.y) - pages(s.x) + copies) | (uint64_t)copies << 40;
    }

    // Slot b, by `lanes` threads.
    __device__ __forceinline__ void write(int b, int lane, int lanes) const {
        const int4 s = get(u.slot + b), at = get(u.place + b);
        const int kept_n = pages(s.x), new_n = pages(s.y);
        int32_t* to = row(b);
        int k = at.x;
        int last = s.w;
        if (at.y >= 0) {
            last = get(u.free_ids + k++);
            if (lane == 0)
                *reinterpret_cast<int4*>(p.copies + 4 * (1 + (int64_t)at.y)) = make_int4(s.w, last, s.x & ((1 << p.page_log2) - 1), 0);
        }
        const bool ends_inside = s.x & ((1 << p.page_log2) - 1);
        if (at.z & kSlotOther) {
            const int32_t* from = at.z & kSlotStaged ? stage(b) : slot_exists(at.w) ? row(at.w) : to;
            entries(from, kept_n - ends_inside, nullptr, 0, 0, lane, lanes, [&](int j, int id, int) { to[j] = id; });
        }
        if (lane == 0 && ends_inside && (at.y >= 0 || (at.z & kSlotOther))) to[kept_n - 1] = last;
        for (int j = kept_n + lane; j < new_n; j += lanes) to[j] = get(u.free_ids + k + (j - kept_n));
        for (int j = new_n + lane; j < s.z; j += lanes) to[j] = -1;
        if (lane == 0) p.seq_lens[b] = s.y;
    }

    // The count of page i; the free pages up to `taken` are taken.
    __device__ __forceinline__ void commit(int i, int taken) const {
        const int c = get(u.count + i);
        p.ref[i] = c > 0 ? c : get(u.first + i) != kNobody || i <= taken;
    }

    __device__ __forceinline__ void head(int64_t need, int64_t free_n, int64_t copies, int64_t held) const {
        *reinterpret_cast<int4*>(p.copies) = need <= free_n
                                                 ? make_int4((int)copies, 0, (int)(free_n - need), 0)
                                                 : make_int4(0, (int)min(need - free_n, (int64_t)INT32_MAX), (int)held, 0);
    }
};

// Numbers of a cache of up to kOnePages pages and kOneSeqs slots, by one CTA (a slot to a thread): where the pages that each slot
// gets begin, copies' places in the list, free pages in order, and the list's head.  Returns the pages needed, -1 if they lack.
constexpr int kRounds = kOnePages / kThreads;

template <bool ONE>
__device__ __forceinline__ int64_t number(const Update<ONE>& x, uint32_t (&sums)[3][kWarps], uint64_t (&part)[kWarps]) {
    const PagesUpdateParams& p = x.p;
    const int warp = threadIdx.x / 32, lane = threadIdx.x % 32, b = threadIdx.x;
    // Running sums of what the slots need (a slot's at most 2^15, more than there are pages), of copies, and of free pages: a warp
    // has 32 pages a round, a lane's as bits.
    const uint64_t mine = b < p.n_seqs ? x.needs(b) : 0;
    const int rounds = (p.n_pages + kThreads - 1) / kThreads, w0 = warp * 32 * rounds;
    uint32_t free_bits = 0;
#pragma unroll 4
    for (int r = 0; r < rounds; ++r)
        if (w0 + 32 * r + lane < p.n_pages && x.is_free(w0 + 32 * r + lane)) free_bits |= 1u << r;
    uint32_t need_to = (uint32_t)min(mine & ((1ull << 40) - 1), 1ull << 15), copies_to = (uint32_t)(mine >> 40);
    const uint32_t need_own = need_to, copies_own = copies_to, free_own = __reduce_add_sync(~0u, __popc(free_bits));
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
        const uint32_t n = __shfl_up_sync(~0u, need_to, o), c = __shfl_up_sync(~0u, copies_to, o);
        if (lane >= o) {
            need_to += n;
            copies_to += c;
        }
    }
    if (lane == 31) {
        sums[0][warp] = need_to;
        sums[1][warp] = copies_to;
        sums[2][warp] = free_own;
    }
    __syncthreads();
    const uint32_t v0 = sums[0][lane], v1 = sums[1][lane], v2 = sums[2][lane];
    const uint32_t need = __reduce_add_sync(~0u, v0), copies = __reduce_add_sync(~0u, v1), free_n = __reduce_add_sync(~0u, v2);
    const uint32_t need_at = __reduce_add_sync(~0u, lane < warp ? v0 : 0) + need_to - need_own;
    const uint32_t copies_at = __reduce_add_sync(~0u, lane < warp ? v1 : 0) + copies_to - copies_own;
    uint32_t free_at = __reduce_add_sync(~0u, lane < warp ? v2 : 0);
    if (need > free_n) {
        int held = 0;
        for (int i = threadIdx.x; i < p.n_pages; i += kThreads) held += __ldcg(p.ref + i) <= 0;
        uint64_t all_need, all_held;
        block_scan(mine & ((1ull << 40) - 1), &all_need, part);
        block_scan(held, &all_held, part);
        if (threadIdx.x == 0) x.head(all_need, free_n, copies, all_held);
        return -1;
    }
    if (threadIdx.x == 0) x.head(need, free_n, copies, 0);
    if (b < p.n_seqs) {
        x.u.place[b].x = (int)need_at;
        if (copies_own) x.u.place[b].y = (int)copies_at;
    }
    if (free_at < need) {
        for (int r = 0; r < rounds; ++r) {
            const uint32_t m = __ballot_sync(~0u, free_bits >> r & 1);
            if (free_bits >> r & 1) x.u.free_ids[free_at + __popc(m & ((1u << lane) - 1))] = w0 + 32 * r + lane;
            free_at += __popc(m);
        }
    }
    return need;
}

__global__ void __launch_bounds__(kThreads) pages_update_kernel(const __grid_constant__ PagesUpdateParams p, int32_t* stage) {
    extern __shared__ int4 smem[];
    __shared__ uint64_t part[kWarps];
    __shared__ uint32_t sums[3][kWarps];
    __shared__ uint16_t long_rows[kOneSeqs];  // (in any order: counts are added up, rows written by themselves)
    __shared__ int n_long;
    Books u;
    u.slot = smem;
    u.place = u.slot + p.n_seqs;
    u.count = reinterpret_cast<int32_t*>(u.place + p.n_seqs);
    u.first = reinterpret_cast<uint32_t*>(u.count + p.n_pages);
    u.free_ids = reinterpret_cast<int32_t*>(u.first + p.n_pages);
    u.stage = stage;
    const Update<true> x{p, u};
    using Entry = Update<true>::Entry;
    const int b = threadIdx.x;  // (one slot to a thread: kOneSeqs of them at most)
    begin_kernel(false);
    Entry e;
    if (b < p.n_seqs) e = x.ask(b);
    if (threadIdx.x == 0) n_long = 0;
    {
        int c[kRounds];
#pragma unroll
        for (int r = 0; r < kRounds; ++r) c[r] = b + r * kThreads < p.n_pages ? __ldcg(p.ref + b + r * kThreads) : 0;
        if (b < p.n_seqs) x.look_up(b, e);  // (its loads are under way with the counts')
#pragma unroll
        for (int r = 0; r < kRounds; ++r) {
            const int i = b + r * kThreads;
            if (i >= p.n_pages) break;
            u.count[i] = c[r];
            u.first[i] = kNobody;
        }
    }
    __syncthreads();
    if (b < p.n_seqs) x.enter(b, e);
    __syncthreads();
    // rows are short, or many, or both: each has its share of the threads, but 8; a long one all of them, after the others
    const int lanes = max(8, kThreads >> (32 - __clz(max(p.n_seqs, 1) - 1)));
    const int group = threadIdx.x / lanes, row_lane = threadIdx.x % lanes;
    auto is_long = [&](int s) { return x.reads(s) > 64 * lanes; };
    for (int s = group; s < p.n_seqs; s += kThreads / lanes) {
        if (!is_long(s))
            x.move(s, row_lane, lanes);
        else if (row_lane == 0)
            long_rows[atomicAdd(&n_long, 1)] = (uint16_t)s;
    }
    __syncthreads();
    if (n_long > 0) {
        for (int k = 0; k < n_long; ++k) x.move(long_rows[k], threadIdx.x, kThreads);
        __syncthreads();
    }

    // what lacks changes nothing
    const int64_t need = number<true>(x, sums, part);
    if (need < 0) return;
    __syncthreads();
    const int taken = need > 0 ? u.free_ids[need - 1] : -1;
    for (int i = threadIdx.x; i < p.n_pages; i += kThreads) x.commit(i, taken);
    for (int s = group; s < p.n_seqs; s += kThreads / lanes)
        if (!is_long(s)) x.write(s, row_lane, lanes);
    for (int k = 0; k < n_long; ++k) x.write(long_rows[k], threadIdx.x, kThreads);
}

// The same, a launch for each step, with the books in the workspace.
constexpr int kStepThreads = 256;
constexpr int kStepLanes = 32;  // to a row

__global__ void __launch_bounds__(kStepThreads) pages_init_kernel(const __grid_constant__ PagesUpdateParams p, const Books u) {
    const Update<false> x{p, u};
    begin_kernel(false);
    x.init(blockIdx.x * kStepThreads + threadIdx.x, gridDim.x * kStepThreads);
}

__global__ void __launch_bounds__(kStepThreads) pages_count_kernel(const __grid_constant__ PagesUpdateParams p, const Books u) {
    const Update<false> x{p, u};
    begin_kernel(false);
    const int groups = gridDim.x * (kStepThreads / kStepLanes), group = blockIdx.x * (kStepThreads / kStepLanes) + threadIdx.x / kStepLanes;
    const int lane = threadIdx.x % kStepLanes;
    for (int64_t b = group; b < p.n_seqs; b += groups) {
        Update<false>::Entry e = {};
        if (lane == 0) {
            e = x.ask((int)b);
            x.look_up((int)b, e);
            x.enter((int)b, e);
        }
        int4 slot;
        slot.x = __shfl_sync(~0u, e.slot.x, 0);
        slot.y = __shfl_sync(~0u, e.slot.y, 0);
        slot.z = __shfl_sync(~0u, e.slot.z, 0);
        slot.w = __shfl_sync(~0u, e.slot.w, 0);
        x.move((int)b, slot, __shfl_sync(~0u, e.flags, 0), __shfl_sync(~0u, e.parent, 0), lane, kStepLanes);
    }
}

__global__ void __launch_bounds__(kThreads, 1) pages_number_one_kernel(const __grid_constant__ PagesUpdateParams p, const Books u) {
    __shared__ uint64_t part[kWarps];
    __shared__ uint32_t sums[3][kWarps];
    const Update<false> x{p, u};
    begin_kernel(false);
    const int64_t need = number<false>(x, sums, part);
    if (threadIdx.x == 0) {
        u.totals[0] = max(need, (int64_t)0);
        u.totals[1] = need < 0 ? -1 : need;
    }
}

// One cluster; CTA `rank` has a share of the slots and of the pages.
__global__ void __launch_bounds__(kThreads, 1) pages_number_kernel(const __grid_constant__ PagesUpdateParams p, const Books u) {
    __shared__ uint64_t part[kWarps];
    __shared__ uint64_t said[3];  // to the cluster: what its slots need, their copies, its free pages | those before << 32
    const Update<false> x{p, u};
    const int rank = (int)cluster_rank(), warp = threadIdx.x / 32, lane = threadIdx.x % 32;
    const int s0 = share(0, p.n_seqs, rank, kCtas), s1 = share(0, p.n_seqs, rank + 1, kCtas);
    const int p0 = share(0, p.n_pages, rank, kCtas), p1 = share(0, p.n_pages, rank + 1, kCtas);
    const int w0 = share(p0, p1, warp, kWarps), w1 = share(p0, p1, warp + 1, kWarps);
    begin_kernel(false);
    uint64_t needs = 0, copying = 0;  // of this CTA's slots
    for (int64_t b0 = s0; b0 < s1; b0 += kThreads) {
        const bool some = b0 + threadIdx.x < s1;
        uint64_t sum;
        block_scan(some ? x.needs((int)b0 + threadIdx.x) : 0, &sum, part);
        needs += sum & ((1ull << 40) - 1);
        copying += sum >> 40;
    }
    auto is_free = [&](int i) { return x.is_free(i); };
    int held = 0;
    for (int i = p0 + threadIdx.x; i < p1; i += kThreads) held += __ldcg(p.ref + i) <= 0;
    const int mine = each_of(w0, w1, is_free, [](int, int) {});
    uint64_t sum;
    const int before = (int)(uint32_t)block_scan((lane == 0 ? mine : 0) | (uint64_t)held << 32, &sum, part);
    if (threadIdx.x == 0) {
        said[0] = needs;
        said[1] = copying;
        said[2] = sum;
    }
    cluster_sync();
    // all CTAs' numbers, and those of the ones before this
    uint64_t told[3], earlier[3];
#pragma unroll
    for (int k = 0; k < 3; ++k) {
        told[k] = lane < kCtas ? cluster_read(&said[k], lane) : 0;
        earlier[k] = lane < rank ? told[k] : 0;
    }
#pragma unroll
    for (int o = kCtas / 2; o > 0; o >>= 1)
#pragma unroll
        for (int k = 0; k < 3; ++k) {
            told[k] += __shfl_xor_sync(~0u, told[k], o);
            earlier[k] += __shfl_xor_sync(~0u, earlier[k], o);
        }
#pragma unroll
    for (int k = 0; k < 3; ++k) {
        told[k] = __shfl_sync(~0u, told[k], 0);
        earlier[k] = __shfl_sync(~0u, earlier[k], 0);
    }
    const int64_t need = told[0], copies = told[1], free_n = (uint32_t)told[2], left = told[2] >> 32, free_at = (uint32_t)earlier[2];
    int64_t need_at = earlier[0], copies_at = earlier[1];
    cluster_arrive();  // (waited for at the end: others may still read what this CTA says)
    if (rank == 0 && threadIdx.x == 0) {
        x.head(need, free_n, copies, left);
        u.totals[0] = need;
        u.totals[1] = free_n;
    }
    if (need <= free_n) {
        for (int64_t b0 = s0; b0 < s1; b0 += kThreads) {
            const int b = (int)b0 + threadIdx.x;
            const uint64_t n = b0 + threadIdx.x < s1 ? x.needs(b) : 0;
            uint64_t all;
            const uint64_t at = block_scan(n, &all, part);
            if (b0 + threadIdx.x < s1) {
                u.place[b].x = (int)(need_at + (at & ((1ull << 40) - 1)));
                if (n >> 40) u.place[b].y = (int)(copies_at + (at >> 40));
            }
            need_at += all & ((1ull << 40) - 1);
            copies_at += all >> 40;
        }
        const int64_t at = free_at + __shfl_sync(~0u, before, 0);
        if (at < need) each_of(w0, w1, is_free, [&](int i, int k) { u.free_ids[at + k] = i; });
    }
    cluster_wait();
}

__global__ void __launch_bounds__(kStepThreads, 4) pages_write_kernel(const __grid_constant__ PagesUpdateParams p, const Books u) {
    const Update<false> x{p, u};
    begin_kernel(false);
    const int64_t need = __ldcg(u.totals);
    if (need > __ldcg(u.totals + 1)) return;
    const int groups = gridDim.x * (kStepThreads / kStepLanes), group = blockIdx.x * (kStepThreads / kStepLanes) + threadIdx.x / kStepLanes;
    for (int64_t b = group; b < p.n_seqs; b += groups) x.write((int)b, threadIdx.x % kStepLanes, kStepLanes);
    const int taken = need > 0 ? __ldcg(u.free_ids + need - 1) : -1;
    for (int i = blockIdx.x * kStepThreads + threadIdx.x; i < p.n_pages; i += gridDim.x * kStepThreads) x.commit(i, taken);
}

// Entries of the page table by their pages' new ids (those that name no live page stay): thread `at` of n.
__device__ __forceinline__ void rename(const PagesCompactParams& p, int64_t at, int64_t n) {
    const int64_t entries = (int64_t)p.n_seqs * p.max_pages;
    for (; at < entries; at += 8 * n) {
        int id[8], to[8];
#pragma unroll
        for (int e = 0; e < 8; ++e) id[e] = at + e * n < entries ? __ldcg(p.page_table + at + e * n) : -1;
#pragma unroll
        for (int e = 0; e < 8; ++e) to[e] = id[e] >= 0 && id[e] < p.n_pages ? __ldcg(p.new_id + id[e]) : -1;
#pragma unroll
        for (int e = 0; e < 8; ++e)
            if (at + e * n < entries) p.page_table_out[at + e * n] = to[e] >= 0 ? to[e] : id[e];
    }
}

// Live pages with ids from their number on go, lowest first, to the free ids below it, lowest first.
//
// Up to kOneCompact pages by one CTA, their counts in its shared memory; who moves where is exchanged there, too.  It also renames
// the entries of a small table.  (Loops of as many rounds as there are pages for: written out for all kRounds, the code, run
// through once, came to 9.4 us for 125 pages instead of 2.6.  9104 pages take it 8.9, the cluster below 8.8.)
constexpr int kOneCompact = 8192;

__global__ void __launch_bounds__(kThreads, 1) pages_compact_kernel(const __grid_constant__ PagesCompactParams p) {
    extern __shared__ int32_t counts[];  // [n_pages], then the ids that move and those that they go to, [n_pages / 2]
    uint16_t* const movers = reinterpret_cast<uint16_t*>(counts + p.n_pages);
    uint16_t* const holes = movers + p.n_pages / 2;
    __shared__ uint32_t sums[2][kWarps];
    const int warp = threadIdx.x / 32, lane = threadIdx.x % 32;
    const int rounds = (p.n_pages + kThreads - 1) / kThreads, w0 = warp * 32 * rounds;  // (a warp has 32 pages a round)
    auto page = [&](int r) { return w0 + 32 * r + lane; };
    begin_kernel(false);
    uint32_t live = 0;
#pragma unroll 4
    for (int r = 0; r < rounds; ++r) {
        if (page(r) >= p.n_pages) break;
        const int c = __ldcg(p.ref + page(r));
        counts[page(r)] = c;
        live |= (uint32_t)(c > 0) << r;
    }
    const uint32_t live_here = __reduce_add_sync(~0u, __popc(live));
    if (lane == 0) sums[0][warp] = live_here;
    __syncthreads();
    const int n_live = (int)__reduce_add_sync(~0u, sums[0][lane]);
    uint32_t moves = 0, filled = 0;  // this lane's pages that move, and free ones that are filled
    for (int r = 0; r < rounds; ++r) {
        const int i = page(r);
        const bool alive = live >> r & 1;
        moves |= (uint32_t)(i >= n_live && alive) << r;
        filled |= (uint32_t)(i < n_live && !alive) << r;
    }
    // (as many of the one as of the other, n_pages / 2 at most: both in a word)
    const uint32_t here = __reduce_add_sync(~0u, (uint32_t)__popc(moves) | (uint32_t)__popc(filled) << 16);
    if (lane == 0) sums[1][warp] = here;
    __syncthreads();
    const uint32_t v = sums[1][lane], all = __reduce_add_sync(~0u, v), before = __reduce_add_sync(~0u, lane < warp ? v : 0);
    // f(move's and filling's place in the order, page, whether it moves, whether it is filled) for this lane's pages
    auto each = [&](auto&& f) {
        int at_moves = before & 0xffff, at_holes = before >> 16;
        for (int r = 0; r < rounds; ++r) {
            const bool x = moves >> r & 1, y = filled >> r & 1;
            const uint32_t m = __ballot_sync(~0u, x), h = __ballot_sync(~0u, y), less = (1u << lane) - 1;
            f(at_moves + __popc(m & less), at_holes + __popc(h & less), page(r), x, y);
            at_moves += __popc(m);
            at_holes += __popc(h);
        }
    };
    each([&](int k, int l, int i, bool x, bool y) {
        if (x) movers[k] = (uint16_t)i;
        if (y) holes[l] = (uint16_t)i;
    });
    __syncthreads();
    // (every count has been read: ref_out may be ref)
    int4* rows = reinterpret_cast<int4*>(p.copies) + 1;
    if (threadIdx.x == 0) rows[-1] = make_int4((int)(all & 0xffff), 0, p.n_pages - n_live, 0);
    each([&](int k, int l, int i, bool x, bool y) {
        if (i >= p.n_pages) return;
        const int from = y ? movers[l] : i, c = counts[from];
        if (y) rows[l] = make_int4(from, i, 1 << p.page_log2, 0);
        p.ref_out[i] = x ? 0 : max(c, 0);
        p.new_id[i] = x ? holes[k] : c > 0 && !y ? i : -1;
    });
    if (!p.rename) return;
    __syncthreads();
    rename(p, threadIdx.x, kThreads);
}

// More pages by a cluster, whose CTAs each take a share of them; who is live stays in shared memory, a bit for each page.
__global__ void __launch_bounds__(kThreads) pages_compact_cluster_kernel(const __grid_constant__ PagesCompactParams p) {
    extern __shared__ uint32_t bits[];
    __shared__ uint64_t part[kWarps];
    __shared__ uint64_t said[2];  // to the cluster: its live pages; those that move | free ids that are filled << 32
    const int rank = (int)cluster_rank(), warp = threadIdx.x / 32, lane = threadIdx.x % 32;
    // (shares in whole words of bits)
    const int words = (p.n_pages + 31) / 32;
    const int c0 = share(0, words, rank, kCtas), c1 = share(0, words, rank + 1, kCtas);
    const int v0 = share(c0, c1, warp, kWarps), v1 = share(c0, c1, warp + 1, kWarps);
    const int w0 = 32 * v0, w1 = min(32 * v1, p.n_pages);
    auto tell = [&](int k, uint64_t mine, uint64_t* before) {  // the sum over the CTAs, and over those before this one
        if (threadIdx.x == 0) said[k] = mine;
        cluster_sync();
        uint64_t all = lane < kCtas ? cluster_read(&said[k], lane) : 0, less = lane < rank ? all : 0;
#pragma unroll
        for (int o = 16; o > 0; o >>= 1) {
            all += __shfl_xor_sync(~0u, all, o);
            less += __shfl_xor_sync(~0u, less, o);
        }
        *before = less;
        return all;
    };
    begin_kernel(false);
    int mine = 0;
#pragma unroll 8
    for (int v = v0; v < v1; ++v) {
        const int i = 32 * v + lane;
        const uint32_t m = __ballot_sync(~0u, i < p.n_pages && __ldcg(p.ref + i) > 0);
        if (lane == 0) bits[v - c0] = m;
        mine += __popc(m);
    }
    __syncwarp();
    uint64_t sum, less;
    block_scan(lane == 0 ? mine : 0, &sum, part);
    const int n_live = (int)tell(0, sum, &less);
    auto live = [&](int i) { return bits[i / 32 - c0] >> (i % 32) & 1; };
    auto moves = [&](int i) { return i >= n_live && live(i); };
    auto filled = [&](int i) { return i < n_live && !live(i); };
    const uint64_t movers = each_of(w0, w1, moves, [](int, int) {}), holes = each_of(w0, w1, filled, [](int, int) {});
    uint64_t before = block_scan(lane == 0 ? movers | holes << 32 : 0, &sum, part);
    const uint64_t all = tell(1, sum, &less);
    before = __shfl_sync(~0u, before, 0) + less;
    const int at_moves = (int)(uint32_t)before, at_holes = (int)(before >> 32);
    int4* rows = reinterpret_cast<int4*>(p.copies) + 1;
    if (rank == 0 && threadIdx.x == 0) rows[-1] = make_int4((int)(uint32_t)all, 0, p.n_pages - n_live, 0);
    each_of(w0, w1, moves, [&](int i, int k) { rows[at_moves + k].x = i; });
    // (loads before stores: ref_out may be ref, so the compiler keeps them in order)
    for (int i0 = w0 + lane; i0 < w1; i0 += 8 * 32) {
        int count[8];
#pragma unroll
        for (int e = 0; e < 8; ++e) count[e] = i0 + 32 * e < w1 ? __ldcg(p.ref + i0 + 32 * e) : 0;
#pragma unroll
        for (int e = 0; e < 8; ++e) {
            const int i = i0 + 32 * e;
            if (i >= w1) break;
            if (count[e] <= 0) {
                p.new_id[i] = -1;
                if (i >= n_live) p.ref_out[i] = 0;
            } else if (i < n_live) {
                p.new_id[i] = i;
                p.ref_out[i] = count[e];
            }
        }
    }
    cluster_sync();
    // (from here on counts of pages that move are read, each by the one that then clears it)
    int done = 0;
    for (int i0 = w0; i0 < min(w1, n_live); i0 += 4 * 32) {
        int k[4], from[4], count[4];
#pragma unroll
        for (int e = 0; e < 4; ++e) {
            const int i = i0 + 32 * e + lane;
            const bool x = i < w1 && filled(i);
            const uint32_t m = __ballot_sync(~0u, x);
            k[e] = x ? at_holes + done + __popc(m & ((1u << lane) - 1)) : -1;
            done += __popc(m);
        }
#pragma unroll
        for (int e = 0; e < 4; ++e) from[e] = k[e] >= 0 ? __ldcg(&rows[k[e]].x) : 0;
#pragma unroll
        for (int e = 0; e < 4; ++e) count[e] = k[e] >= 0 ? __ldcg(p.ref + from[e]) : 0;
#pragma unroll
        for (int e = 0; e < 4; ++e) {
            if (k[e] < 0) continue;
            const int i = i0 + 32 * e + lane;
            rows[k[e]] = make_int4(from[e], i, 1 << p.page_log2, 0);
            p.new_id[from[e]] = i;
            p.ref_out[i] = count[e];
            p.ref_out[from[e]] = 0;
        }
    }
}

__global__ void __launch_bounds__(256) pages_rename_kernel(const __grid_constant__ PagesCompactParams p) {
    begin_kernel(false);
    rename(p, blockIdx.x * 256ll + threadIdx.x, gridDim.x * 256ll);
}

// The pages' data.  A page of K, or of V, in pieces of kCopyThreads * AHEAD vectors of 16 bytes; those of tokens that the copy
// leaves out are passed over.  Bound by HBM: 2322 pages of 256 KB (K and V) 181 us, 6.7 TB/s, 0.99 of a copy.  An SM has 64 KB
// under way, in the fewer CTAs the larger a page is: with eight vectors to a thread, one CTA 216 us, two 182, three 199, four 192;
// four vectors 191 to 207, streaming loads and stores 187.
constexpr int kCopyThreads = 256;
__host__ __device__ constexpr int copy_ctas(int ahead) { return ahead > 1 ? 16 / ahead : 8; }  // on an SM

template <int AHEAD>
__global__ void __launch_bounds__(kCopyThreads) pages_copy_kernel(const __grid_constant__ PagesCopyParams p, int head_log2,
                                                                                    int pieces) {
    begin_kernel(false);
    const int n = min(max(__ldcg(p.copies), 0), p.max_copies);
    const int64_t items = (int64_t)n * p.n_layers * 2 * pieces;
    const int head = 1 << head_log2;               // vectors of a page's head
    const int64_t page = (int64_t)p.Hkv << head_log2;
    const int row_log2 = head_log2 - p.page_log2;  // vectors of a token
    for (int64_t item = blockIdx.x; item < items; item += gridDim.x) {
        const int64_t whole = item / pieces, copy = (whole >> 1) / p.n_layers;
        const int layer = (int)((whole >> 1) - copy * p.n_layers);
        const int4 c = __ldcg(reinterpret_cast<const int4*>(p.copies) + 1 + copy);
        if (c.x < 0 || c.x >= p.n_pages || c.y < 0 || c.y >= p.n_pages || c.x == c.y) continue;
        uint4* pool = reinterpret_cast<uint4*>(static_cast<char*>(whole & 1 ? p.v_pages : p.k_pages) + layer * p.layer_bytes);
        const uint4* from = pool + c.x * page;
        uint4* to = pool + c.y * page;
        const int64_t v0 = (item - whole * pieces) * (kCopyThreads * AHEAD) + threadIdx.x;
        auto wanted = [&](int64_t v) { return v < page && (int)(v & (head - 1)) >> row_log2 < c.z; };
        uint4 w[AHEAD];
#pragma unroll
        for (int e = 0; e < AHEAD; ++e)
            if (wanted(v0 + e * kCopyThreads)) w[e] = __ldcg(from + v0 + e * kCopyThreads);
#pragma unroll
        for (int e = 0; e < AHEAD; ++e)
            if (wanted(v0 + e * kCopyThreads)) to[v0 + e * kCopyThreads] = w[e];
    }
}

template <int AHEAD>
cudaError_t launch_copy(const PagesCopyParams& p, int head_log2, cudaStream_t stream) {
    const int64_t per = kCopyThreads * AHEAD, pieces = (((int64_t)p.Hkv << head_log2) + per - 1) / per;
    const int64_t items = (int64_t)p.max_copies * p.n_layers * 2 * pieces;
    return launch_dependent(pages_copy_kernel<AHEAD>, dim3((unsigned)std::min<int64_t>(items, copy_ctas(AHEAD) * 152)), kCopyThreads, 0,
                            stream, p, head_log2, (int)pieces);
}

}  // namespace

size_t pages_update_workspace(int n_seqs, int max_pages, int n_pages) {
    Books u;
    return layout(n_seqs, max_pages, n_pages, nullptr, &u);
}

cudaError_t launch_pages_update(const PagesUpdateParams& p, cudaStream_t stream) {
    Books u;
    layout(p.n_seqs, p.max_pages, p.n_pages, static_cast<char*>(p.ws), &u);
    if (one_cta(p)) {
        cudaError_t e = allow_smem<pages_update_kernel>((int)books_bytes(kOneSeqs, kOnePages));
        if (e != cudaSuccess) return e;
        return launch_dependent(pages_update_kernel, dim3(1), kThreads, books_bytes(p.n_seqs, p.n_pages), stream, p, u.stage);
    }
    const auto ctas = [](int64_t threads) { return dim3((unsigned)std::max<int64_t>(1, std::min<int64_t>((threads + 255) / 256, 8 * 152))); };
    cudaError_t e = launch_dependent(pages_init_kernel, ctas(p.n_pages), kStepThreads, 0, stream, p, u);
    if (e == cudaSuccess) e = launch_dependent(pages_count_kernel, ctas((int64_t)kStepLanes * p.n_seqs), kStepThreads, 0, stream, p, u);
    if (e == cudaSuccess)
        e = p.n_pages <= kOnePages && p.n_seqs <= kOneSeqs
                ? launch_dependent(pages_number_one_kernel, dim3(1), kThreads, 0, stream, p, u)
                : launch_clusters(pages_number_kernel, 1, kCtas, kThreads, 0, stream, p, u);
    const int64_t threads = std::max<int64_t>((int64_t)kStepLanes * p.n_seqs, p.n_pages);
    if (e == cudaSuccess) e = launch_dependent(pages_write_kernel, ctas(threads), kStepThreads, 0, stream, p, u);
    return e;
}

cudaError_t launch_pages_compact(const PagesCompactParams& params, cudaStream_t stream) {
    PagesCompactParams p = params;
    const bool one = p.n_pages <= kOneCompact;
    const int64_t entries = (int64_t)p.n_seqs * p.max_pages;
    p.rename = one && entries <= 8 * kThreads;  // (one round of that CTA; a launch for it 2 us more)
    cudaError_t e;
    if (one) {
        e = allow_smem<pages_compact_kernel>(6 * kOneCompact);
        if (e == cudaSuccess) e = launch_dependent(pages_compact_kernel, dim3(1), kThreads, 6 * (size_t)p.n_pages, stream, p);
    } else {
        const int words = (p.n_pages + 31) / 32;
        e = allow_smem<pages_compact_cluster_kernel>((1 << 23) / 8 / kCtas + 4);
        if (e == cudaSuccess)
            e = launch_clusters(pages_compact_cluster_kernel, 1, kCtas, kThreads, 4 * (size_t)((words + kCtas - 1) / kCtas), stream, p);
    }
    if (e != cudaSuccess || entries == 0 || p.rename) return e;
    return launch_dependent(pages_rename_kernel, dim3((unsigned)std::min<int64_t>((entries + 255) / 256, 8 * 152)), 256, 0, stream, p);
}

cudaError_t launch_pages_copy(const PagesCopyParams& p, cudaStream_t stream) {
    int row_log2 = 0;
    while (16 << row_log2 < p.row_bytes) ++row_log2;
    const int head_log2 = row_log2 + p.page_log2;
    const int64_t page = (int64_t)p.Hkv << head_log2;
    return page <= kCopyThreads       ? launch_copy<1>(p, head_log2, stream)
           : page <= 2 * kCopyThreads ? launch_copy<2>(p, head_log2, stream)
           : page <= 4 * kCopyThreads ? launch_copy<4>(p, head_log2, stream)
                                      : launch_copy<8>(p, head_log2, stream);
}

}  // namespace usp
