// Verification of drafted tokens against the target's probabilities, from given random numbers.
//
// The rows of a sequence are the tokens that the model was given last: one that counts already and its drafts.  Row i holds the
// target's probabilities p_i of the token after it, and for a draft x = tokens[i + 1] the probabilities q_{i + 1} that it was
// drawn from.  Draft by draft x is accepted if u_{i + 1} q_{i + 1}(x) < p_i(x); after the first that is not, the next token is
// drawn from max(p_i - q_{i + 1}, 0), after none from the last row's p: the tokens are distributed as the target's own.
//
// The draw: the weights' running sum in the order of the tokens, the first token at which it exceeds u_0 times the total.
// A float32 sum of 10^5 weights is off by more than most weights are, so the sums are whole numbers of 2^-46, to which the
// probabilities are rounded (float64 would do as well, but its units are scarce); they do not depend on the order either.
//
// Bound by HBM for many sequences (one row of p, and of q where a draft is refused, are read once; 64 of 131072 float32 tokens
// 13.3 us in a captured graph, 5.0 TB/s with the 4 us that a launch, the drafts' dependent loads and the search take, and 15.2
// called from Python, 4.4 TB/s) and by latency for few: a
// cluster of CTAs takes a sequence, each CTA a slice of the vocabulary in tiles, whose sums stay in shared
// memory; the CTA that holds the threshold finds the tile by them and goes over that tile alone again.
#include <algorithm>
#include <type_traits>

#include "cluster.cuh"
#include "paged.cuh"

namespace usp {

namespace {

constexpr int kThreads = 256;
constexpr int kWarps = kThreads / 32;
constexpr int kMaxVocab = 1 << 19;
// A lane's values of a tile: twice as many in vectors of bf16 (200 sequences of 50001 tokens 7 % less time), not in
// general (126 sequences of 5239 8.0 against 7.0).
template <typename T, bool VEC>
constexpr int kEach = VEC && sizeof(T) == 2 ? 16 : 8;
template <typename T, bool VEC>
constexpr int kTile = 32 * kEach<T, VEC>;  // tokens

__device__ __forceinline__ float value(const float* p) { return *p; }
__device__ __forceinline__ float value(const __nv_bfloat16* p) {
    return __uint_as_float((uint32_t) * reinterpret_cast<const uint16_t*>(p) << 16);
}

// A lane's values of a tile, as loaded: whole vectors, or one by one where the tile is not 16-byte aligned and where the row begins
// or ends inside it (EDGE: places [from, to) of it are the row's).  Which lane has which does not matter to a sum.
template <typename T, bool VEC, int E>
struct Loaded {
    float x[E];
    template <bool EDGE>
    __device__ __forceinline__ void load(const T* p, int from, int to, int lane) {
#pragma unroll
        for (int e = 0; e < E; ++e) {
            const int i = lane + 32 * e;
            x[e] = !EDGE || (i >= from && i < to) ? value(p + i) : 0.f;
        }
    }
    __device__ __forceinline__ float at(int e) const { return x[e]; }
};
template <typename T, int E>
struct Loaded<T, true, E> {
    static constexpr int V = E * sizeof(T) / 16;  // vectors
    uint32_t w[4 * V];
    template <bool EDGE>
    __device__ __forceinline__ void load(const T* p, int, int, int lane) {
#pragma unroll
        for (int v = 0; v < V; ++v) {
            const uint4 x = reinterpret_cast<const uint4*>(p)[lane + 32 * v];
            w[4 * v] = x.x;
            w[4 * v + 1] = x.y;
            w[4 * v + 2] = x.z;
            w[4 * v + 3] = x.w;
        }
    }
    __device__ __forceinline__ float at(int e) const {
        if constexpr (sizeof(T) == 4) return __uint_as_float(w[e]);
        return __uint_as_float(e % 2 ? w[e / 2] & 0xffff0000u : w[e / 2] << 16);
    }
};

// Sums of x in [0, 1], each rounded to whole numbers of 2^-46, kept as two digits: added to a power of two a number's last bits
// are the digit, what that leaves is exact and, added to a smaller one, gives the next.  (The powers' own bits, which come with
// every digit, cancel where numbers are subtracted.)  All that is issued, loads and sums of tiles included, is 23 instructions of a
// lane for a pair of p and q in float32 (64 sequences of 131072 tokens) and 15 for p alone in bf16 (200 of 50001); with a third
// digit, to 2^-53, the pair took 27.
struct Digits {
    static constexpr float kOne = 1.f, kTwo = 0x1.8p-23f;  // steps of 2^-23 and 2^-46 (x = 1 is the next power: a step on)
    uint32_t d0 = 0, d1 = 0;
    static __device__ __forceinline__ void of(float x, uint32_t& a, uint32_t& b) {
        const float t = x + kOne;
        a = __float_as_uint(t);
        b = __float_as_uint((x - (t - kOne)) + kTwo);
    }
    __device__ __forceinline__ void add(float x) {
        uint32_t a, b;
        of(x, a, b);
        d0 += a - __float_as_uint(kOne);
        d1 += b - __float_as_uint(kTwo);
    }
    __device__ __forceinline__ void add(float x, float y) {  // x - y, x >= y (a digit of the difference may be negative)
        uint32_t a, b, c, d;
        of(x, a, b);
        of(y, c, d);
        d0 += a - c;
        d1 += b - d;
    }
    __device__ __forceinline__ uint64_t whole() const { return (uint64_t)(((int64_t)(int32_t)d0 << 23) + (int32_t)d1); }
};
// (what is not in [0, 1] is taken as the nearer end, NaN as 0)
__device__ __forceinline__ uint64_t fixed46(float x) {
    Digits d;
    d.add(__saturatef(x));
    return d.whole();
}

// u in [0, 1) in whole numbers of 2^-64; what is not in it (NaN: 0) taken as the nearer end.
__device__ __forceinline__ uint64_t fixed64(float u) {
    const uint32_t bits = __float_as_uint(fminf(fmaxf(u, 0.f), 0x1.fffffep-1f));
    const uint64_t m = (bits & 0x7fffffu) | 0x800000u;
    const int shift = (int)(bits >> 23) - 86;
    return shift >= 0 ? m << shift : m >> min(-shift, 63);
}

// A tile's sum is 2^55 at most, a warp's 2^63, a row's 2^65 (of 2^19 ones; rows need not add up to 1): 128 bits from the CTA's
// on, so that a token does not depend on how many CTAs its sequence has.
using Wide = unsigned __int128;

__device__ __forceinline__ uint64_t warp_scan(uint64_t x, int lane) {  // inclusive
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
        const uint64_t y = __shfl_up_sync(~0u, x, o);
        if (lane >= o) x += y;
    }
    return x;
}
// The sum over the lanes, to all, in pieces that the warp's own addition takes: of numbers of 2^50 at most, or 2^65.
__device__ __forceinline__ uint64_t lanes_total(uint64_t x) {
    const uint32_t a = __reduce_add_sync(~0u, (uint32_t)x & ((1u << 26) - 1));
    return a + ((uint64_t)__reduce_add_sync(~0u, (uint32_t)(x >> 26)) << 26);
}
__device__ __forceinline__ Wide lanes_total_wide(Wide x) {
    constexpr uint32_t kPiece = (1u << 26) - 1;
    const uint64_t low = (uint64_t)x;
    const uint32_t a = __reduce_add_sync(~0u, (uint32_t)low & kPiece), b = __reduce_add_sync(~0u, (uint32_t)(low >> 26) & kPiece);
    const uint32_t c = __reduce_add_sync(~0u, (uint32_t)(x >> 52));
    return a + ((Wide)b << 26) + ((Wide)c << 52);
}

template <int N>
using Const = std::integral_constant<int, N>;

// A sequence's weights: max(p - q, 0) with q a row of the draft, p without one token (`except`), or p.  Places are counted from
// the 16-byte boundary before the row, so that its vectors are aligned: the row has places [from, to).
template <typename T, bool VEC>
struct Weights {
    static constexpr int E = kEach<T, VEC>, kLength = kTile<T, VEC>;
    const T *p, *q;  // q null: none
    int from, to;
    int except;      // its place, -1: none

    // A lane's places in a row, from i on: their values and the sum of their weights.
    __device__ __forceinline__ uint64_t few(int i, float (&x)[E], float (&y)[E]) const {
        Digits d;
#pragma unroll
        for (int e = 0; e < E; ++e) {
            const bool some = i + e >= from && i + e < to && i + e != except;
            x[e] = some ? value(p + i + e) : 0.f;
            y[e] = some && q ? value(q + i + e) : 0.f;
        }
#pragma unroll
        for (int e = 0; e < E; ++e) {
            y[e] = __saturatef(y[e]);
            x[e] = fmaxf(__saturatef(x[e]), y[e]);
            d.add(x[e], y[e]);
        }
        return d.whole();
    }
    // Sums of N tiles from place i on, `step` places apart (loads first), each to all lanes; Q: q is not null; EDGE: the row's
    // first tile or last.
    template <bool Q, bool EDGE, int N>
    __device__ __forceinline__ void tiles(int i, int step, int lane, uint64_t (&sum)[N]) const {
        Loaded<T, VEC && !EDGE, E> a[N], b[Q ? N : 1];
#pragma unroll
        for (int k = 0; k < N; ++k) a[k].template load<EDGE>(p + i + k * step, from - i, to - i, lane);
        if constexpr (Q)
#pragma unroll
            for (int k = 0; k < N; ++k) b[k].template load<EDGE>(q + i + k * step, from - i, to - i, lane);
#pragma unroll
        for (int k = 0; k < N; ++k) {
            Digits d;
#pragma unroll
            for (int e = 0; e < E; ++e) {
                const float x = __saturatef(a[k].at(e));
                if constexpr (Q) {
                    const float y = __saturatef(b[k].at(e));
                    d.add(fmaxf(x, y), y);
                } else {
                    d.add(x);
                }
            }
            sum[k] = lanes_total(d.whole());
            const int j = except - (i + k * step);
            if (!Q && j >= 0 && j < kLength) sum[k] -= fixed46(value(p + except));
        }
    }
    // Sums of the tiles [first, end), taken by the CTA's warps in turn, to `out`; returns the sum of this warp's.
    template <bool Q>
    __device__ __forceinline__ uint64_t slice(int first, int end, int warp, int lane, uint64_t* out) const {
        constexpr int N = VEC && !Q ? 4 : 2;  // tiles at a time (of vectors: 128 bytes of a lane in flight)
        const int whole = min(end, to / kLength);
        uint64_t sum = 0;
        int t = first + warp;
        auto some = [&](auto edge, auto count) {
            uint64_t s[count.value];
            tiles<Q, edge.value>(t * kLength, kWarps * kLength, lane, s);
#pragma unroll
            for (int k = 0; k < count.value; ++k) {
                sum += s[k];
                if (lane == 0) out[t - first + k * kWarps] = s[k];
            }
            t += count.value * kWarps;
        };
        if (t == 0 && from > 0) some(Const<1>(), Const<1>());
        while (t + (N - 1) * kWarps < whole) some(Const<0>(), Const<N>());
        if constexpr (N > 2)
            while (t + kWarps < whole) some(Const<0>(), Const<2>());
        if constexpr (N > 1)
            if (t < whole) some(Const<0>(), Const<1>());
        if (t < end) some(Const<1>(), Const<1>());
        return sum;
    }
};

template <typename T, bool VEC>
__global__ void __launch_bounds__(kThreads, 4) verify_kernel(const VerifyParams p, int size) {
    __shared__ uint64_t tile_sum[kMaxVocab / kTile<T, VEC> + 1];  // (rows begin inside a vector)
    __shared__ uint64_t warp_total[kWarps];
    __shared__ ulonglong2 cta_total[2];   // low and high word (a place for each of two goes)
    constexpr int E = kEach<T, VEC>, kLength = kTile<T, VEC>;
    const int rank = (int)cluster_rank(), b = blockIdx.x / size;
    const int warp = threadIdx.x / 32, lane = threadIdx.x % 32;
    begin_kernel(false);
    const int t0 = min(max(p.q_start[b], 0), p.n_tokens);
    const int n = min(max(p.q_start[b + 1], t0), p.n_tokens) - t0;
    const int len = p.seq_lens ? p.seq_lens[b] : 0;
    if (n == 0) {
        if (rank == 0 && threadIdx.x == 0) {
            p.n_accepted[b] = 0;
            p.next[b] = -1;
            if (p.keep_lens) p.keep_lens[b] = len;
        }
        return;
    }
    const T* target = static_cast<const T*>(p.target) + t0 * p.target_stride;
    const T* draft = p.draft ? static_cast<const T*>(p.draft) + t0 * p.draft_stride : nullptr;
    const float u0 = p.u[t0];

    // drafts accepted, found by every warp for itself
    int a = n - 1;
    for (int i0 = 0; i0 < n - 1; i0 += 32) {
        const int i = i0 + lane;
        bool refused = false;
        if (i < n - 1) {
            const int x = p.tokens[t0 + i + 1];
            refused = true;
            if (x >= 0 && x < p.vocab) {
                const double q = draft ? (double)value(draft + (i + 1) * p.draft_stride + x) : 1.0;
                refused = !((double)p.u[t0 + i + 1] * q < (double)value(target + i * p.target_stride + x));  // (exact)
            }
        }
        const uint32_t r = __ballot_sync(~0u, refused);
        if (r) {
            a = i0 + __ffs(r) - 1;
            break;
        }
    }
    const T* row = target + a * p.target_stride;
    const int skip = VEC ? (int)(reinterpret_cast<uintptr_t>(row) % 16 / sizeof(T)) : 0;
    Weights<T, VEC> w{row - skip, nullptr, skip, skip + p.vocab, -1};
    if (a < n - 1) {
        const int x = p.tokens[t0 + a + 1];
        if (draft)
            w.q = draft + (a + 1) * p.draft_stride - skip;
        else if (x >= 0 && x < p.vocab)
            w.except = skip + x;
    }
    const int all = (w.to + kLength - 1) / kLength;
    const int first = all * rank / size, end = all * (rank + 1) / size;  // this CTA's tiles

    Wide total = 0, mine = 0, before = 0;
    for (int go = 0; go < 2; ++go) {
        const uint64_t sum = w.q ? w.template slice<true>(first, end, warp, lane, tile_sum)
                                 : w.template slice<false>(first, end, warp, lane, tile_sum);
        if (lane == 0) warp_total[warp] = sum;
        __syncthreads();
        mine = lanes_total_wide(lane < kWarps ? warp_total[lane] : 0);
        if (threadIdx.x == 0) cta_total[go] = make_ulonglong2((uint64_t)mine, (uint64_t)(mine >> 64));
        cluster_sync();
        const ulonglong2 said = lane < size ? cluster_read(&cta_total[go], lane) : make_ulonglong2(0, 0);
        const Wide x = (Wide)said.y << 64 | said.x;
        total = lanes_total_wide(x);
        before = lanes_total_wide(lane < rank ? x : 0);
        if (total > 0 || (!w.q && w.except < 0)) break;
        // nothing is left of the row (q >= p throughout, as rounded): drawn from p itself
        w.q = nullptr;
        w.except = -1;
    }
    cluster_arrive();  // (waited for at the end: others may still read this CTA's total)
    if (rank == 0 && threadIdx.x == 0) {
        p.n_accepted[b] = a;
        if (p.keep_lens) p.keep_lens[b] = len - (n - 1 - a);
        if (total == 0) p.next[b] = -1;
    }
    // the first token whose running sum exceeds u0 times the total, rounded down
    const uint64_t at = fixed64(u0);
    Wide rest = (Wide)__umul64hi((uint64_t)total, at) + (uint64_t)(total >> 64) * (Wide)at;
    if (warp == 0 && rest >= before && rest - before < mine) {          // (in one CTA of the cluster)
        rest -= before;
        for (int t = first; t < end; t += 32) {
            const uint64_t to = warp_scan(t + lane < end ? tile_sum[t + lane - first] : 0, lane);  // (32 tiles: 2^60 at most)
            const uint32_t over = __ballot_sync(~0u, to > rest);
            if (!over) {
                rest -= __shfl_sync(~0u, to, 31);
                continue;
            }
            const int k = __ffs(over) - 1;
            const uint64_t less = __shfl_sync(~0u, to, max(k - 1, 0));
            uint64_t left = (uint64_t)rest - (k > 0 ? less : 0);  // (of this tile)
            // the tile again: the lane that holds it, whose values then go to all
            const int i0 = (t + k) * kLength;
            float x[E], y[E];
            const uint64_t upto = warp_scan(w.few(i0 + lane * E, x, y), lane);
            const int l = max(__ffs(__ballot_sync(~0u, upto > left)) - 1, 0);
            const uint64_t less_l = __shfl_sync(~0u, upto, max(l - 1, 0));
            if (l > 0) left -= less_l;
            Digits run;
            int e = 0;
#pragma unroll
            for (int j = 0; j < E; ++j) {
                run.add(__shfl_sync(~0u, x[j], l), __shfl_sync(~0u, y[j], l));
                e += run.whole() <= left;
            }
            if (lane == 0) p.next[b] = i0 + l * E + min(e, E - 1) - skip;
            break;
        }
    }
    cluster_wait();
}

}  // namespace

cudaError_t launch_verify(const VerifyParams& p, cudaStream_t stream) {
    // A cluster's CTAs: as many as the SMs hold at once (four each; of a cluster's size less one may be left over in each of the
    // eight groups that clusters do not cross), but no fewer than 256 tokens for each warp.
    const int most = std::min(8, std::max(1, p.vocab / (256 * kWarps)));
    const int size = std::min(most, std::max(1, (4 * 152 + 8) / (p.n_seqs + 8)));
    // Vectors need a row's and, where a draft's is subtracted, both rows' places aligned alike: any single row is (from its first
    // 16-byte boundary on), two where the strides are.
    const bool vec = !p.draft || (p.target_stride * p.elem % 16 == 0 && p.draft_stride * p.elem % 16 == 0);
    auto kernel = p.elem == 4 ? vec ? verify_kernel<float, true> : verify_kernel<float, false>
                              : vec ? verify_kernel<__nv_bfloat16, true> : verify_kernel<__nv_bfloat16, false>;
    return launch_clusters(kernel, (unsigned)p.n_seqs, (unsigned)size, kThreads, 0, stream, p, size);
}

}  // namespace usp
