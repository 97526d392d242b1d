// Verification of drafted tokens against the target's probabilities, from given random numbers.
//
// The rows of a sequence are the tokens that the model was given last: one that counts already and its drafts.  Row i holds the
// target's probabilities p_i of the token after it, and for a draft x = tokens[i + 1] the probabilities q_{i + 1} that it was
// drawn from.  Draft by draft x is accepted if u_{i + 1} q_{i + 1}(x) < p_i(x); after the first that is not, the next token is
// drawn from max(p_i - q_{i + 1}, 0), after none from the last row's p: the tokens are distributed as the target's own.
//
// The draw: the weights' running sum in the order of the tokens, the first token at which it exceeds u_0 times the total.
// A float32 sum of 10^5 weights is off by more than most weights are, so the sums are whole numbers of 2^-53 (weights are
// cut to that; float64 would do as well, but its units are scarce), which do not depend on the order either.
//
// Bound by HBM for many sequences (one row of p, and of q where a draft is refused, are read once) and by latency for few: a
// cluster of CTAs takes a sequence, each a slice of the vocabulary in registers' sums only; the CTA, then the warp that holds
// the threshold goes over its part again, out of L2.
#include <algorithm>

#include "cluster.cuh"
#include "paged.cuh"

namespace usp {

namespace {

constexpr int kThreads = 512;
constexpr int kWarps = kThreads / 32;

__device__ __forceinline__ float value(const float* p, int64_t i) { return p[i]; }
__device__ __forceinline__ float value(const __nv_bfloat16* p, int64_t i) {
    return __uint_as_float((uint32_t) reinterpret_cast<const uint16_t*>(p)[i] << 16);
}

// x in [0, 1] in whole numbers of 2^-53 (53 > 0: cut off), what is not in it (NaN: 0) taken as the nearer end.
__device__ __forceinline__ uint64_t fixed53(float x) {
    const uint32_t bits = __float_as_uint(fminf(fmaxf(x, 0.f), 1.f));
    const uint32_t m = (bits & 0x7fffffu) | 0x800000u;
    const int shift = (int)(bits >> 23) - 97;                    // x = m 2^(exponent - 150)
    return shift >= 0 ? (uint64_t)m << shift : (uint64_t)(m >> min(-shift, 31));
}
// u in [0, 1) in whole numbers of 2^-64; what is not in it (NaN: 0) taken as the nearer end.
__device__ __forceinline__ uint64_t fixed64(float u) {
    const uint32_t bits = __float_as_uint(fminf(fmaxf(u, 0.f), 0x1.fffffep-1f));
    const uint64_t m = (bits & 0x7fffffu) | 0x800000u;
    const int shift = (int)(bits >> 23) - 86;
    return shift >= 0 ? m << shift : m >> min(-shift, 63);
}

// Sums stop at the largest number, so that rows which are no probabilities (a thousand ones) still lead to a token.
__device__ __forceinline__ uint64_t add(uint64_t x, uint64_t y) { return x + y < x ? ~0ull : x + y; }
__device__ __forceinline__ uint64_t warp_sum(uint64_t x) {
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) x = add(x, __shfl_xor_sync(~0u, x, o));
    return x;
}

// A sequence's weights: max(p - q, 0) with q a row of the draft, one token (`except`), or nothing.
template <typename T>
struct Weights {
    const T *p, *q;  // q null: none
    int except;      // -1: none
    __device__ __forceinline__ uint64_t at(int i) const {
        const uint64_t a = fixed53(value(p, i));
        if (q) {
            const uint64_t b = fixed53(value(q, i));
            return a > b ? a - b : 0;
        }
        return i == except ? 0 : a;
    }
    // this thread's share of the weights of [i0, i1), which a warp takes in turn (at most 1024 of them: no overflow)
    __device__ __forceinline__ uint64_t sum(int i0, int i1, int lane) const {
        uint64_t s = 0;
        int i = i0 + lane;
        if (q) {
            for (; i + 7 * 32 < i1; i += 8 * 32) {
                float a[8], b[8];
#pragma unroll
                for (int e = 0; e < 8; ++e) a[e] = value(p, i + 32 * e);
#pragma unroll
                for (int e = 0; e < 8; ++e) b[e] = value(q, i + 32 * e);
#pragma unroll
                for (int e = 0; e < 8; ++e) {
                    const uint64_t x = fixed53(a[e]), y = fixed53(b[e]);
                    s += x > y ? x - y : 0;
                }
            }
        } else {
            for (; i + 7 * 32 < i1; i += 8 * 32) {
                float a[8];
#pragma unroll
                for (int e = 0; e < 8; ++e) a[e] = value(p, i + 32 * e);
#pragma unroll
                for (int e = 0; e < 8; ++e) s += i + 32 * e == except ? 0 : fixed53(a[e]);
            }
        }
        for (; i < i1; i += 32) s += at(i);
        return s;
    }
};

// Piece k of [i0, i1) cut into n equal ones.
__device__ __forceinline__ int cut(int i0, int i1, int k, int n) { return i0 + (int)((int64_t)(i1 - i0) * k / n); }

// Of n <= 32 sums in order (lane k has the k-th): the one that holds `rest`, which becomes what is left within it.
__device__ __forceinline__ int holder(uint64_t sum, int lane, int n, uint64_t& rest) {
    uint64_t to = lane < n ? sum : 0;
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
        const uint64_t x = __shfl_up_sync(~0u, to, o);
        if (lane >= o) to = add(to, x);
    }
    const uint32_t over = __ballot_sync(~0u, lane < n && to > rest);
    const int k = over ? __ffs(over) - 1 : n - 1;
    const uint64_t before = __shfl_sync(~0u, to, max(k - 1, 0));
    if (k > 0) rest -= min(rest, before);
    return k;
}

template <typename T>
__global__ void __launch_bounds__(kThreads) verify_kernel(const VerifyParams p, int size) {
    __shared__ uint64_t warp_total[kWarps];
    __shared__ uint64_t cta_total[2];   // (a place for each of two goes)
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

    // drafts accepted, found by every warp for itself
    int a = n - 1;
    for (int i0 = 0; i0 < n - 1; i0 += 32) {
        const int i = i0 + lane;
        bool refused = false;
        if (i < n - 1) {
            const int x = p.tokens[t0 + i + 1];
            refused = true;
            if (x >= 0 && x < p.vocab) {
                const double q = draft ? (double)value(draft + (i + 1) * p.draft_stride, x) : 1.0;
                refused = !((double)p.u[t0 + i + 1] * q < (double)value(target + i * p.target_stride, x));  // (exact)
            }
        }
        const uint32_t r = __ballot_sync(~0u, refused);
        if (r) {
            a = i0 + __ffs(r) - 1;
            break;
        }
    }
    Weights<T> w{target + a * p.target_stride, nullptr, -1};
    if (a < n - 1) {
        if (draft)
            w.q = draft + (a + 1) * p.draft_stride;
        else
            w.except = p.tokens[t0 + a + 1];
    }
    const int i0 = cut(0, p.vocab, rank, size), i1 = cut(0, p.vocab, rank + 1, size);

    uint64_t total = 0, mine = 0, before = 0, sum = 0;
    for (int go = 0; go < 2; ++go) {
        sum = warp_sum(w.sum(cut(i0, i1, warp, kWarps), cut(i0, i1, warp + 1, kWarps), lane));
        if (lane == 0) warp_total[warp] = sum;
        __syncthreads();
        sum = lane < kWarps ? warp_total[lane] : 0;
        mine = warp_sum(sum);
        if (threadIdx.x == 0) cta_total[go] = mine;
        cluster_sync();
        const uint64_t x = lane < size ? cluster_read(&cta_total[go], lane) : 0;
        total = warp_sum(x);
        before = warp_sum(lane < rank ? x : 0);
        if (total > 0 || (!w.q && w.except < 0)) break;
        // nothing is left of the row (q >= p throughout, as rounded): drawn from p itself
        w.q = nullptr;
        w.except = -1;
    }
    if (rank == 0 && threadIdx.x == 0) {
        p.n_accepted[b] = a;
        if (p.keep_lens) p.keep_lens[b] = len - (n - 1 - a);
        if (total == 0) p.next[b] = -1;
    }
    uint64_t rest = __umul64hi(total, fixed64(p.u[t0]));  // the first token whose running sum exceeds this
    if (rest >= before && rest - before < mine) {         // (one CTA of the cluster)
        rest -= before;
        const int k = holder(sum, lane, kWarps, rest);    // the warp whose part holds it: gone over by all
        const int j0 = cut(i0, i1, k, kWarps), j1 = cut(i0, i1, k + 1, kWarps);
        sum = warp_sum(w.sum(cut(j0, j1, warp, kWarps), cut(j0, j1, warp + 1, kWarps), lane));
        if (lane == 0) warp_total[warp] = sum;
        __syncthreads();
        sum = lane < kWarps ? warp_total[lane] : 0;
        const int l = holder(sum, lane, kWarps, rest);
        if (warp == 0) {
            const int c0 = cut(j0, j1, l, kWarps), c1 = cut(j0, j1, l + 1, kWarps);
            for (int i = c0; i < c1; i += 32) {
                const uint64_t x = i + lane < c1 ? w.at(i + lane) : 0;
                uint64_t to = x;
#pragma unroll
                for (int o = 1; o < 32; o <<= 1) {
                    const uint64_t y = __shfl_up_sync(~0u, to, o);
                    if (lane >= o) to += y;
                }
                const uint32_t over = __ballot_sync(~0u, to > rest);
                if (over) {
                    if (lane == 0) p.next[b] = i + __ffs(over) - 1;
                    break;
                }
                rest -= __shfl_sync(~0u, to, 31);
            }
        }
    }
    cluster_sync();  // (others may still read this CTA's total)
}

}  // namespace

cudaError_t launch_verify(const VerifyParams& p, cudaStream_t stream) {
    // A cluster's CTAs: as many as the SMs hold at once, but no fewer than 2048 tokens each.
    int size = 1;
    while (size < 8 && (int64_t)p.n_seqs * size * 2 <= 4 * 152 && p.vocab >= 2048 * size * 2) size *= 2;
    auto kernel = p.elem == 4 ? verify_kernel<float> : verify_kernel<__nv_bfloat16>;
    return launch_clusters(kernel, (unsigned)p.n_seqs, (unsigned)size, kThreads, 0, stream, p, size);
}

}  // namespace usp
