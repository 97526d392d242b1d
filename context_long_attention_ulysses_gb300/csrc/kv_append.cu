// Rotary position embedding of new queries and keys, and keys and values written into the paged cache.
//
// Per token, head and i < rot/2 the pair (a, b) of frequency f_i turns by the angle r f_i (r: the token's position):
//   a' = a cos(r f_i) - b sin(r f_i),  b' = b cos(r f_i) + a sin(r f_i).
// The angle is the float64 product of the position and the float32 frequency, reduced by 2 pi in float64 (in float32
// the angle of position 10^6 is off by up to 0.06 rad); sine, cosine and the rotation are float32.
#include <cmath>

#include <cuda_bf16.h>

#include "kernels.h"

namespace usp {

namespace {

constexpr int kThreads = 128;

// cos and sin of r * f
__device__ __forceinline__ float2 turn(int r, float f) {
    const double turns = (double)r * (double)f * 0.15915494309189535;  // / 2 pi
    float s, c;
    sincospif(2.f * (float)(turns - rint(turns)), &s, &c);
    return make_float2(c, s);
}

__device__ __forceinline__ float ld(const float* p) { return *p; }
__device__ __forceinline__ float ld(const __nv_bfloat16* p) { return __bfloat162float(*p); }
__device__ __forceinline__ void st(float* p, float x) { *p = x; }
__device__ __forceinline__ void st(__nv_bfloat16* p, float x) { *p = __float2bfloat16_rn(x); }

template <typename T>
__global__ void __launch_bounds__(kThreads) kv_append_kernel(const AppendParams p) {
    const int t = blockIdx.x;
    const int s = p.seq[t], pos = p.pos[t];
    if (s < 0 || s >= p.n_seqs || pos < 0 || pos >> p.page_log2 >= p.max_pages) return;
    const int page = p.page_table[(int64_t)s * p.max_pages + (pos >> p.page_log2)];
    if (page < 0 || page >= p.n_pages) return;
    const int r = p.rot_pos ? p.rot_pos[t] : pos;
    __shared__ float2 cs[64];
    for (int i = threadIdx.x; i < p.rot / 2; i += kThreads) cs[i] = turn(r, p.inv_freq[i]);
    __syncthreads();
    const int psize = 1 << p.page_log2, slot = pos & (psize - 1), d = p.d, half = p.rot / 2;
    const T* q = p.q ? static_cast<const T*>(p.q) + t * p.q_stride : nullptr;
    const T* k = static_cast<const T*>(p.k) + t * p.k_stride;
    const T* v = static_cast<const T*>(p.v) + t * p.v_stride;
    T* q_out = static_cast<T*>(p.q_out) + (int64_t)t * p.Hq * d;
    T* k_out = p.k_out ? static_cast<T*>(p.k_out) + (int64_t)t * p.Hkv * d : nullptr;
    T* kp = static_cast<T*>(p.k_pages) + (((int64_t)page * p.Hkv) * psize + slot) * d;
    T* vp = static_cast<T*>(p.v_pages) + (((int64_t)page * p.Hkv) * psize + slot) * d;
    const int64_t hs = (int64_t)psize * d;
    // pairs, then the elements that pass, of each q and k head; a thread handles both of a pair
    const int per = half + (d - p.rot);
    for (int x = threadIdx.x; x < (p.Hq + p.Hkv) * per; x += kThreads) {
        const int h = x / per, i = x % per;
        const bool is_q = h < p.Hq;
        if (is_q && !q) continue;
        const T* src = is_q ? q + h * d : k + (h - p.Hq) * d;
        int e0, e1;
        if (i < half) {
            e0 = p.interleaved ? 2 * i : i;
            e1 = p.interleaved ? 2 * i + 1 : i + half;
        } else {
            e0 = e1 = p.rot + (i - half);
        }
        float a = ld(src + e0), b = ld(src + e1);
        if (i < half) {
            const float2 w = cs[i];
            const float a2 = a * w.x - b * w.y, b2 = b * w.x + a * w.y;
            a = a2;
            b = b2;
        }
        if (is_q) {
            st(q_out + h * d + e0, a);
            st(q_out + h * d + e1, b);
        } else {
            const int hk = h - p.Hq;
            st(kp + hk * hs + e0, a);
            st(kp + hk * hs + e1, b);
            if (k_out) {
                st(k_out + hk * d + e0, a);
                st(k_out + hk * d + e1, b);
            }
        }
    }
    for (int x = threadIdx.x; x < p.Hkv * d; x += kThreads) vp[(x / d) * hs + x % d] = v[x];
}

}  // namespace

cudaError_t launch_kv_append(const AppendParams& p, cudaStream_t stream) {
    if (p.elem == 4)
        kv_append_kernel<float><<<p.n_tokens, kThreads, 0, stream>>>(p);
    else
        kv_append_kernel<__nv_bfloat16><<<p.n_tokens, kThreads, 0, stream>>>(p);
    return cudaGetLastError();
}

}  // namespace usp
