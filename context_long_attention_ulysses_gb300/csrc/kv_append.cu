// Rotary position embedding of new queries and keys, and keys and values written into the paged cache.
//
// Per token, head and i < rot/2 the pair (a, b) of frequency f_i turns by the angle r f_i (r: the token's position):
//   a' = a cos(r f_i) - b sin(r f_i),  b' = b cos(r f_i) + a sin(r f_i).
// The angle is formed to 64 bits for |f_i| < 2^24, in float64 beyond (in float32 the angle of position 10^6 is off by up to 0.06
// rad); sine, cosine and the rotation are float32.
//
// Bound by HBM: every value is read once and written once (k twice with k_out).  A head is d / (2 V) items of two 16-byte
// vectors (V values): the two that a rotation pairs up, or two neighbours where pairs are neighbours or pass unchanged.  A
// CTA takes as many tokens as make about kItems items; its threads first issue their loads, then find the tokens' slots
// (two dependent loads) and the tokens' cosines and sines (one per pair, shared by all heads), and only then wait for the
// data.  Measured: 32768 tokens of 32 query and 8 KV heads of 128 bf16 values, k_out too, 134 us, 6.5 TB/s (0.98 of a copy);
// one token each of eight sequences 3.5 us in a graph.
#include <algorithm>
#include <cmath>

#include <cuda_bf16.h>

#include "paged.cuh"

namespace usp {

namespace {

// (96 threads with four items in flight, measured against 128 x 3, 64 x 3, 64 x 6 and 256 x 3 for a prompt of 32768 tokens:
// 135.6 us against 137.3, 136.7, 147.4 and 154)
constexpr int kThreads = 96;
constexpr int kAhead = 4;                     // items of a thread in flight
constexpr int kItems = kThreads * kAhead;     // items of a CTA per round
constexpr int kMaxTokens = 16;

// cos and sin of r * f.  Only the fraction of the turns r f / 2 pi counts, so it is formed in 64-bit fixed point, where whole
// turns fall off the top: f = m 2^-shift with an integer m of 24 bits, the fraction of f / 2 pi is m * (2^64 / 2 pi) >> shift
// to 64 bits: off by f / 2 units of the last bit, as the constant is by a half, and by one of the shift.  Times r, up to 2^31, that
// is less than 2^-30 turns for f up to 8.  (The scarce float64 units took 3.5 of 144 us for a prompt of 32768 tokens; they
// remain for f of 2^24 and more, where r f and its turns are three roundings, 3 2^-53 of themselves; infinities and NaN give NaN.)
__device__ __forceinline__ float2 turn(int r, float f) {
    const uint32_t bits = __float_as_uint(f) & 0x7fffffffu;
    const int exponent = (int)(bits >> 23), shift = 150 - exponent;
    float s, c;
    if (shift >= 0) {
        const uint32_t m = exponent > 0 ? (bits & 0x7fffffu) | 0x800000u : 0u;  // (a subnormal f turns by nothing: 2^-95 turns)
        constexpr uint64_t kPerTurn = 0x28be60db9391054aull;                    // 2^64 / 2 pi
        const uint64_t lo = m * kPerTurn, hi = __umul64hi((uint64_t)m, kPerTurn);
        const uint64_t frac = shift == 0 ? lo : shift < 64 ? (lo >> shift) | (hi << (64 - shift)) : shift < 128 ? hi >> (shift - 64) : 0;
        int64_t turns = (int64_t)((uint64_t)(int64_t)r * frac);
        if (f < 0.f) turns = -turns;
        sincospif((float)(int)(turns >> 32) * 0x1p-31f, &s, &c);
    } else {
        const double turns = (double)r * (double)f * 0.15915494309189535;  // / 2 pi
        sincospif(2.f * (float)(turns - rint(turns)), &s, &c);
    }
    return make_float2(c, s);
}

// The values of a 16-byte vector, and back (one rounding).
template <typename T>
struct Vec;
template <>
struct Vec<float> {
    static constexpr int N = 4;
    static __device__ __forceinline__ void open(const uint4& w, float (&x)[4]) {
        x[0] = __uint_as_float(w.x);
        x[1] = __uint_as_float(w.y);
        x[2] = __uint_as_float(w.z);
        x[3] = __uint_as_float(w.w);
    }
    static __device__ __forceinline__ uint4 close(const float (&x)[4]) {
        return make_uint4(__float_as_uint(x[0]), __float_as_uint(x[1]), __float_as_uint(x[2]), __float_as_uint(x[3]));
    }
};
template <>
struct Vec<__nv_bfloat16> {
    static constexpr int N = 8;
    static __device__ __forceinline__ void open(const uint4& w, float (&x)[8]) {
        const uint32_t u[4] = {w.x, w.y, w.z, w.w};
#pragma unroll
        for (int e = 0; e < 4; ++e) {
            x[2 * e] = __uint_as_float(u[e] << 16);
            x[2 * e + 1] = __uint_as_float(u[e] & 0xffff0000u);
        }
    }
    static __device__ __forceinline__ uint4 close(const float (&x)[8]) {
        uint32_t u[4];
#pragma unroll
        for (int e = 0; e < 4; ++e)
            asm("cvt.rn.bf16x2.f32 %0, %1, %2;" : "=r"(u[e]) : "f"(x[2 * e + 1]), "f"(x[2 * e]));
        return make_uint4(u[0], u[1], u[2], u[3]);
    }
};

template <typename T, bool INTERLEAVED>
__global__ void __launch_bounds__(kThreads) kv_append_kernel(const AppendParams p, int tokens_per_cta, int item_log2) {
    constexpr int V = Vec<T>::N;
    __shared__ float2 cs[kMaxTokens][64];
    __shared__ int64_t s_row[kMaxTokens];  // row of head 0 in the pool, -1: padding
    __shared__ int s_rot[kMaxTokens];
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
    // (not through shared memory: the angles need not wait for the slots)
    for (int x = threadIdx.x; x < n_tok * half; x += kThreads) {
        const int tok = x / half, i = x - tok * half;
        cs[tok][i] = turn(p.rot_pos ? p.rot_pos[t0 + tok] : p.pos[t0 + tok], p.inv_freq[i]);
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
                float a[V], b[V];
                Vec<T>::open(w[u][0], a);
                Vec<T>::open(w[u][1], b);
                if constexpr (INTERLEAVED) {
                    const float2* c = cs[it.tok] + it.e0 / 2;
#pragma unroll
                    for (int e = 0; e < V; e += 2) {
                        const float2 f = c[e / 2], g = c[(V + e) / 2];
                        const float a0 = a[e], a1 = a[e + 1], b0 = b[e], b1 = b[e + 1];
                        a[e] = a0 * f.x - a1 * f.y;
                        a[e + 1] = a1 * f.x + a0 * f.y;
                        b[e] = b0 * g.x - b1 * g.y;
                        b[e + 1] = b1 * g.x + b0 * g.y;
                    }
                } else {
                    const float2* c = cs[it.tok] + it.e0;
#pragma unroll
                    for (int e = 0; e < V; ++e) {
                        const float2 f = c[e];
                        const float a0 = a[e], b0 = b[e];
                        a[e] = a0 * f.x - b0 * f.y;
                        b[e] = b0 * f.x + a0 * f.y;
                    }
                }
                w[u][0] = Vec<T>::close(a);
                w[u][1] = Vec<T>::close(b);
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
