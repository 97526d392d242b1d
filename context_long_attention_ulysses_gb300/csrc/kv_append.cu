// Rotary position embedding of new queries and keys, and keys and values written into the paged cache.
//
// Per token, head and i < rot/2 the pair (a, b) of frequency f_i turns by the angle r f_i (r: the token's position):
//   a' = a cos(r f_i) - b sin(r f_i),  b' = b cos(r f_i) + a sin(r f_i).
// With several axes r is the token's position on the pair's axis.
// The angle is formed to 64 bits for |f_i| < 2^24, in float64 beyond (in float32 the angle of position 10^6 is off by up to 0.06
// rad); sine, cosine and the rotation are float32.
//
// Bound by HBM: every value is read once and written once (k twice with k_out).  A head is d / (2 V) items of two 16-byte
// vectors (V values): the two that a rotation pairs up, or two neighbours where pairs are neighbours or pass unchanged.  A
// CTA takes as many tokens as make about kItems items; its threads first load their angles' positions and frequencies, then
// issue the data's loads, find the tokens' slots (two dependent loads) and the tokens' cosines and sines (one per pair, shared by
// all heads), and only then wait for the data.  (Positions on three axes are three lines of memory: asked for behind the
// data, 32768 tokens took 140.5 us, before it 132.4; on one axis 131.5 and 130.5.)  Measured: 32768 tokens of 32 query and 8 KV
// heads of 128 bf16 values, k_out too, 130.5 us (three axes 132.4, 6.6 TB/s, 0.97 of a copy); one token each of eight
// sequences 3.5 us in a graph.
#include <algorithm>
#include <cmath>

#include "paged.cuh"
#include "rotary.cuh"

namespace usp {

namespace {

// (96 threads with four items in flight, measured against 128 x 3, 64 x 3, 64 x 6 and 256 x 3 for a prompt of 32768 tokens:
// 135.6 us against 137.3, 136.7, 147.4 and 154)
constexpr int kThreads = 96;
constexpr int kAhead = 4;                     // items of a thread in flight
constexpr int kItems = kThreads * kAhead;     // items of a CTA per round
constexpr int kMaxTokens = 16;

template <typename T, bool INTERLEAVED>
__global__ void __launch_bounds__(kThreads) kv_append_kernel(const AppendParams p, int tokens_per_cta, int item_log2) {
    constexpr int V = Vec<T>::N;
    __shared__ float2 cs[kMaxTokens][64];
    __shared__ int64_t s_row[kMaxTokens];  // row of head 0 in the pool, -1: padding
    __shared__ int s_pos[USP_MAX_AXES * kMaxTokens];
    __shared__ Frequency s_freq[64];
    static_assert(USP_MAX_AXES * kMaxTokens <= kThreads, "a position to a thread");
    const int t0 = blockIdx.x * tokens_per_cta, n_tok = min(tokens_per_cta, p.n_tokens - t0);
    const int d = p.d, half = p.rot / 2, psize = 1 << p.page_log2;
    const int hq = p.q ? p.Hq : 0, heads = hq + 2 * p.Hkv, per_token = heads << item_log2;
    const int total = n_tok * per_token;

    // an item: token, head (q heads, then k, then v), place of its two vectors within the head
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
        it.rotates = it.head < hq + p.Hkv && i < half;
        if (INTERLEAVED || !it.rotates) {
            it.e0 = 2 * i;
            it.e1 = 2 * i + V;
        } else {
            it.e0 = i;
            it.e1 = i + half;
        }
        return it;
    };
    auto source = [&](const Item& it) {
        const int64_t t = t0 + it.tok;
        return it.head < hq ? static_cast<const T*>(p.q) + t * p.q_stride + it.head * d
               : it.head < hq + p.Hkv ? static_cast<const T*>(p.k) + t * p.k_stride + (it.head - hq) * d
                                      : static_cast<const T*>(p.v) + t * p.v_stride + (it.head - hq - p.Hkv) * d;
    };
    uint4 w[kAhead][2];
    auto fetch = [&](int x0) {
#pragma unroll
        for (int u = 0; u < kAhead; ++u) {
            const int x = x0 + u * kThreads;
            if (x < total) {
                const Item it = item(x);
                const T* src = source(it);
                w[u][0] = __ldcs(reinterpret_cast<const uint4*>(src + it.e0));
                w[u][1] = __ldcs(reinterpret_cast<const uint4*>(src + it.e1));
            }
        }
    };
    begin_kernel(false);
    // Positions and frequencies are asked for before the data: of one angle to a thread in registers, of more (up to 1024 of 16
    // tokens, with few heads) through shared memory.
    const int angles = n_tok * half;
    const bool few = angles <= kThreads;
    const int32_t* positions = p.rot_pos ? p.rot_pos : p.pos;
    int r0 = 0;
    float f0 = 0.f;
    if (few) {
        if (threadIdx.x < angles) {
            const int tok = threadIdx.x / half, i = threadIdx.x - tok * half;
            r0 = positions[pair_axis(p.axes, i) * (int64_t)p.n_tokens + t0 + tok];
            f0 = p.inv_freq[i];
        }
    } else {
        if (threadIdx.x < p.n_axes * n_tok) r0 = positions[threadIdx.x / n_tok * (int64_t)p.n_tokens + t0 + threadIdx.x % n_tok];
        if (threadIdx.x < half) f0 = p.inv_freq[threadIdx.x];
    }
    fetch(threadIdx.x);
    if (threadIdx.x < n_tok) {
        const int t = t0 + threadIdx.x, s = p.seq[t], pos = p.pos[t];
        int64_t row = -1;
        if (s >= 0 && s < p.n_seqs && pos >= 0 && pos >> p.page_log2 < p.max_pages) {
            const int page = p.page_table[(int64_t)s * p.max_pages + (pos >> p.page_log2)];
            if (page >= 0 && page < p.n_pages) row = (((int64_t)page * p.Hkv) << p.page_log2) + (pos & (psize - 1));
        }
        s_row[threadIdx.x] = row;
    }
    // (the angles need not wait for the slots)
    if (few) {
        if (threadIdx.x < angles) {
            const int tok = threadIdx.x / half, i = threadIdx.x - tok * half;
            cs[tok][i] = turn(r0, frequency(f0));
        }
    } else {
        if (threadIdx.x < p.n_axes * n_tok) s_pos[threadIdx.x] = r0;
        if (threadIdx.x < half) s_freq[threadIdx.x] = frequency(f0);
        __syncthreads();
        for (int x = threadIdx.x; x < angles; x += kThreads) {
            const int tok = x / half, i = x - tok * half;
            cs[tok][i] = turn(s_pos[pair_axis(p.axes, i) * n_tok + tok], s_freq[i]);
        }
    }
    __syncthreads();
    for (int x0 = threadIdx.x; x0 < total; x0 += kItems) {
        if (x0 != threadIdx.x) fetch(x0);
#pragma unroll
        for (int u = 0; u < kAhead; ++u) {
            const int x = x0 + u * kThreads;
            if (x >= total) break;
            const Item it = item(x);
            const int64_t row = s_row[it.tok];
            if (row < 0) continue;
            if (it.rotates) {
                rotate_vectors<T, INTERLEAVED>(w[u][0], w[u][1], cs[it.tok] + (INTERLEAVED ? it.e0 / 2 : it.e0));
            }
            auto store = [&](T* dst) {  // (streaming: 141 us against 148)
                __stcs(reinterpret_cast<uint4*>(dst + it.e0), w[u][0]);
                __stcs(reinterpret_cast<uint4*>(dst + it.e1), w[u][1]);
            };
            const int64_t t = t0 + it.tok;
            if (it.head < hq) {
                store(static_cast<T*>(p.q_out) + (t * p.Hq + it.head) * d);
            } else if (it.head < hq + p.Hkv) {
                const int h = it.head - hq;
                store(static_cast<T*>(p.k_pages) + (row + ((int64_t)h << p.page_log2)) * d);
                if (p.k_out) store(static_cast<T*>(p.k_out) + (t * p.Hkv + h) * d);
            } else {
                const int h = it.head - hq - p.Hkv;
                store(static_cast<T*>(p.v_pages) + (row + ((int64_t)h << p.page_log2)) * d);
            }
        }
    }
}

template <typename T>
cudaError_t launch_t(const AppendParams& p, cudaStream_t s) {
    int item_log2 = 0;  // items per head
    while ((2 * Vec<T>::N << item_log2) < p.d) ++item_log2;
    const int per_token = ((p.q ? p.Hq : 0) + 2 * p.Hkv) << item_log2;
    // few heads: several tokens per CTA, as long as there are CTAs enough for every SM
    int n = std::min(kMaxTokens, std::max(1, kItems / per_token));
    while (n > 1 && (p.n_tokens + n - 1) / n < 4 * 152) --n;
    const unsigned grid = (unsigned)((p.n_tokens + n - 1) / n);
    return p.interleaved ? launch_dependent(kv_append_kernel<T, true>, dim3(grid), kThreads, 0, s, p, n, item_log2)
                         : launch_dependent(kv_append_kernel<T, false>, dim3(grid), kThreads, 0, s, p, n, item_log2);
}

}  // namespace

cudaError_t launch_kv_append(const AppendParams& p, cudaStream_t stream) {
    return p.elem == 4 ? launch_t<float>(p, stream) : launch_t<__nv_bfloat16>(p, stream);
}

}  // namespace usp
