// Rotary position embedding with several axes, of the queries and keys of a sequence-sharded batch, and its backward.
//
// Per token, head and i < rot/2 the pair (a, b) of frequency f_i turns by the angle r f_i, r being the token's position on
// the pair's axis (time, height, width ...):
//   a' = a cos(r f_i) - b sin(r f_i),  b' = b cos(r f_i) + a sin(r f_i).
// The backward is the transposed rotation, by -r f_i.  Angles as in kv_append.cu (rotary.cuh).
//
// Bound by HBM: every value is read once and written once.  Work is cut as in kv_append.cu, into items of two 16-byte vectors; a
// CTA takes a few whole tokens and its threads ask for their angles' positions and frequencies first, then for the data, and form the
// cosines and sines (one per pair and token, shared by all heads) while that is under way.  131072 tokens of 32 query and 8 KV
// heads of 128 bf16 values: 394 us in a captured graph, 6.8 TB/s (1.00 of a copy), 396 called from Python; 4097 tokens of 8 heads
// of 64 float32 values 4.2 us in a graph, 4.8 called.
#include <algorithm>

#include "paged.cuh"
#include "rotary.cuh"

namespace usp {

namespace {

constexpr int kMaxTokens = 16;

template <typename T, bool INTERLEAVED, int kThreads, int kAhead>
__global__ void __launch_bounds__(kThreads) rotary_kernel(const __grid_constant__ RotaryParams p, int tokens_per_cta, int item_log2) {
    constexpr int V = Vec<T>::N, kItems = kThreads * kAhead;  // items of a CTA per round
    __shared__ float2 cs[kMaxTokens][64];
    __shared__ int positions[USP_MAX_AXES * kMaxTokens];
    __shared__ Frequency frequencies[64];
    static_assert(USP_MAX_AXES * kMaxTokens <= kThreads, "a position to a thread");
    const int64_t t0 = (int64_t)blockIdx.x * tokens_per_cta;
    const int n_tok = (int)min((int64_t)tokens_per_cta, p.n_tokens - t0);
    const int d = p.d, half = p.rot / 2;
    const int hq = p.q ? p.Hq : 0, heads = hq + (p.k ? p.Hkv : 0), per_token = heads << item_log2;
    const int total = n_tok * per_token;

    struct Item {
        int tok, head, e0, e1;
        bool rotates;
    };
    auto item = [&](int x) {
        Item it;
        it.tok = x / per_token;
        const int y = x - it.tok * per_token;
        it.head = y >> item_log2;
        const int i = (y & ((1 << item_log2) - 1)) * V;  // values of the first vectors before this one
        it.rotates = i < half;
        if (INTERLEAVED || !it.rotates) {
            it.e0 = 2 * i;
            it.e1 = 2 * i + V;
        } else {
            it.e0 = i;
            it.e1 = i + half;
        }
        return it;
    };
    uint4 w[kAhead][2];
    auto fetch = [&](int x0) {
#pragma unroll
        for (int u = 0; u < kAhead; ++u) {
            const int x = x0 + u * kThreads;
            if (x < total) {
                const Item it = item(x);
                const int64_t t = t0 + it.tok;
                const T* src = it.head < hq ? static_cast<const T*>(p.q) + t * p.q_stride + it.head * d
                                            : static_cast<const T*>(p.k) + t * p.k_stride + (it.head - hq) * d;
                w[u][0] = __ldcs(reinterpret_cast<const uint4*>(src + it.e0));
                w[u][1] = __ldcs(reinterpret_cast<const uint4*>(src + it.e1));
            }
        }
    };
    begin_kernel(false);
    // Positions and frequencies are asked for first, then the data.  A few angles of a thread keep theirs in registers; with few
    // heads a CTA has up to 1024 angles of 16 tokens, whose positions go through shared memory (85360 tokens of 6 heads of 64
    // values 31.0 -> 27.3 us; 131072 of 40 heads of 128 would take 402 us so instead of 391).
    constexpr int kEarly = 2;
    const int angles = n_tok * half;
    if (angles <= kEarly * kThreads) {
        int at[kEarly];
        float freq[kEarly];
#pragma unroll
        for (int e = 0; e < kEarly; ++e) {
            const int x = threadIdx.x + e * kThreads, tok = x / max(half, 1), i = x - tok * half;
            if (x < angles) {
                at[e] = p.pos[pair_axis(p.axes, i) * (int64_t)p.n_tokens + t0 + tok];
                freq[e] = p.inv_freq[i];
            }
        }
        asm volatile("" ::: "memory");
        fetch(threadIdx.x);
        asm volatile("" ::: "memory");
#pragma unroll
        for (int e = 0; e < kEarly; ++e) {
            const int x = threadIdx.x + e * kThreads, tok = x / max(half, 1), i = x - tok * half;
            if (x < angles) cs[tok][i] = turn(at[e], frequency(freq[e]));
        }
    } else {
        const int places = p.n_axes * n_tok;
        int at = 0;
        float f = 0.f;
        if (threadIdx.x < places) at = p.pos[threadIdx.x / n_tok * (int64_t)p.n_tokens + t0 + threadIdx.x % n_tok];
        if (threadIdx.x < half) f = p.inv_freq[threadIdx.x];
        asm volatile("" ::: "memory");
        fetch(threadIdx.x);
        asm volatile("" ::: "memory");
        if (threadIdx.x < places) positions[threadIdx.x] = at;
        if (threadIdx.x < half) frequencies[threadIdx.x] = frequency(f);
        __syncthreads();
        for (int x = threadIdx.x; x < angles; x += kThreads) {
            const int tok = x / half, i = x - tok * half;
            cs[tok][i] = turn(positions[pair_axis(p.axes, i) * n_tok + tok], frequencies[i]);
        }
    }
    __syncthreads();
    const float sign = p.inverse ? -1.f : 1.f;
    for (int x0 = threadIdx.x; x0 < total; x0 += kItems) {
        if (x0 != threadIdx.x) fetch(x0);
#pragma unroll
        for (int u = 0; u < kAhead; ++u) {
            const int x = x0 + u * kThreads;
            if (x >= total) break;
            const Item it = item(x);
            if (it.rotates)
                rotate_vectors<T, INTERLEAVED>(w[u][0], w[u][1], cs[it.tok] + (INTERLEAVED ? it.e0 / 2 : it.e0), sign);
            const int64_t t = t0 + it.tok;
            T* dst = it.head < hq ? static_cast<T*>(p.q_out) + t * p.q_out_stride + it.head * d
                                  : static_cast<T*>(p.k_out) + t * p.k_out_stride + (it.head - hq) * d;
            __stcs(reinterpret_cast<uint4*>(dst + it.e0), w[u][0]);
            __stcs(reinterpret_cast<uint4*>(dst + it.e1), w[u][1]);
        }
    }
}

template <typename T, int kThreads, int kAhead>
cudaError_t launch_t(const RotaryParams& p, int items, cudaStream_t s) {
    int item_log2 = 0;  // items per head
    while ((2 * Vec<T>::N << item_log2) < p.d) ++item_log2;
    const int per_token = ((p.q ? p.Hq : 0) + (p.k ? p.Hkv : 0)) << item_log2;
    // few heads: several tokens per CTA, as long as there are CTAs enough for every SM
    int n = std::min(kMaxTokens, std::max(1, items / per_token));
    while (n > 1 && (p.n_tokens + n - 1) / n < 4 * 152) --n;
    const unsigned grid = (unsigned)((p.n_tokens + n - 1) / n);
    return p.interleaved ? launch_dependent(rotary_kernel<T, true, kThreads, kAhead>, dim3(grid), kThreads, 0, s, p, n, item_log2)
                         : launch_dependent(rotary_kernel<T, false, kThreads, kAhead>, dim3(grid), kThreads, 0, s, p, n, item_log2);
}

template <typename T>
cudaError_t launch_sized(const RotaryParams& p, cudaStream_t s) {
    // Little work goes in one round, everything that the SMs hold under way together; more of it streams best through small CTAs of
    // several rounds, many to an SM, and the largest with two rounds' more work to each (tokens of 32 query and 8 KV heads of 128
    // bf16 values, the three ways: 3000 of them 11.8, 12.7 and 18.2 us, 8000 31.8, 29.1 and 30.9, 131072 453, 400 and 391).
    const int64_t items = (int64_t)p.n_tokens * ((p.q ? p.Hq : 0) + (p.k ? p.Hkv : 0)) * p.d / (2 * Vec<T>::N);
    return items <= 3 << 19 ? launch_t<T, 96, 4>(p, 384, s) : launch_t<T, 64, 3>(p, items <= 8 << 20 ? 384 : 640, s);
}

}  // namespace

cudaError_t launch_rotary(const RotaryParams& p, cudaStream_t stream) {
    return p.elem == 4 ? launch_sized<float>(p, stream) : launch_sized<__nv_bfloat16>(p, stream);
}

}  // namespace usp
