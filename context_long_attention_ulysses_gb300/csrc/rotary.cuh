// What the rotating kernels share: the angle of a position and a frequency, 16-byte vectors of values, the rotation of a
// pair of vectors, and the axes of the pairs.
#pragma once

#include <cstdint>

#include <cuda_bf16.h>
#include <cuda_runtime.h>

#include "kernels.h"

namespace usp {

__device__ __forceinline__ int pair_axis(const PairAxes& x, int i) { return x.w[i >> 4] >> (2 * (i & 15)) & 3; }

// cos and sin of r * f.  Only the fraction of the turns r f / 2 pi counts, so it is formed in 64-bit fixed point, where whole
// turns fall off the top: f = m 2^-shift with an integer m of 24 bits, the fraction of f / 2 pi is m * (2^64 / 2 pi) >> shift
// to 64 bits: off by f / 2 units of the last bit, as the constant is by a half, and by one of the shift.  Times r, up to 2^31, that
// is less than 2^-30 turns for f up to 8.  (The scarce float64 units took 3.5 of 144 us for a prompt of 32768 tokens; they
// remain for f of 2^24 and more, where r f and its turns are three roundings, 3 2^-53 of themselves; infinities and NaN give NaN.)
// What goes into sine and cosine is float32: half turns in [-1, 1), off by 2^-25 at most, an angle by 2^-25 pi (9.4e-8 rad), as much
// as a float32 result's own rounding.
struct Frequency {
    uint64_t turns;  // fraction of the turns of one position, times 2^64
    float f;
    bool far;        // 2^24 and more: by f
};
__device__ __forceinline__ Frequency frequency(float f) {
    const uint32_t bits = __float_as_uint(f) & 0x7fffffffu;
    const int exponent = (int)(bits >> 23), shift = 150 - exponent;
    const uint32_t m = exponent > 0 ? (bits & 0x7fffffu) | 0x800000u : 0u;  // (a subnormal f turns by nothing: 2^-95 turns)
    constexpr uint64_t kPerTurn = 0x28be60db9391054aull;                    // 2^64 / 2 pi
    const uint64_t lo = m * kPerTurn, hi = __umul64hi((uint64_t)m, kPerTurn);
    const uint64_t frac = shift <= 0 ? lo : shift < 64 ? (lo >> shift) | (hi << (64 - shift)) : shift < 128 ? hi >> (shift - 64) : 0;
    return {f < 0.f ? (uint64_t)0 - frac : frac, f, shift < 0};
}
__device__ __forceinline__ float2 turn(int r, const Frequency& q) {
    float s, c;
    if (!q.far) {
        const int64_t turns = (int64_t)((uint64_t)(int64_t)r * q.turns);
        sincospif((float)(int)(turns >> 32) * 0x1p-31f, &s, &c);
    } else {
        const double turns = (double)r * (double)q.f * 0.15915494309189535;  // / 2 pi
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

// Rotates the values of two vectors w0, w1 of a head, c[i] = (cos, sin) of the pairs: INTERLEAVED, both hold neighbouring
// pairs, c that of w0's first; otherwise a value of w0 and one of w1 are a pair, c that of the first.  With `sign` -1 by the
// negative angles, the transposed rotation.
template <typename T, bool INTERLEAVED>
__device__ __forceinline__ void rotate_vectors(uint4& w0, uint4& w1, const float2* c, float sign = 1.f) {
    constexpr int V = Vec<T>::N;
    float a[V], b[V];
    Vec<T>::open(w0, a);
    Vec<T>::open(w1, b);
    if constexpr (INTERLEAVED) {
#pragma unroll
        for (int e = 0; e < V; e += 2) {
            const float2 f = c[e / 2], g = c[(V + e) / 2];
            const float fs = sign * f.y, gs = sign * g.y;
            const float a0 = a[e], a1 = a[e + 1], b0 = b[e], b1 = b[e + 1];
            a[e] = a0 * f.x - a1 * fs;
            a[e + 1] = a1 * f.x + a0 * fs;
            b[e] = b0 * g.x - b1 * gs;
            b[e + 1] = b1 * g.x + b0 * gs;
        }
    } else {
#pragma unroll
        for (int e = 0; e < V; ++e) {
            const float2 f = c[e];
            const float fs = sign * f.y;
            const float a0 = a[e], b0 = b[e];
            a[e] = a0 * f.x - b0 * fs;
            b[e] = b0 * f.x + a0 * fs;
        }
    }
    w0 = Vec<T>::close(a);
    w1 = Vec<T>::close(b);
}

}  // namespace usp
