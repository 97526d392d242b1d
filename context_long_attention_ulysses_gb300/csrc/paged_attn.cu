// Attention over a paged cache (decoding, verification, chunks of prompts) and behind a shared prefix: the choice of
// kernels, the workspace, and the join of partial results.
//
// Per row (token, query head): S_j = scale q.k_j over the keys the row sees, o = softmax(S) V, lse = ln sum exp(S), in one
// pass over the keys with a running maximum and sum.  How the work is cut is explained in paged.cuh.
#include <algorithm>
#include <cmath>

#include <cuda_bf16.h>

#include "paged.cuh"

namespace usp {

namespace {

constexpr int kSms = 152;
constexpr float kLn2 = 0.6931471805599453f;

__device__ __forceinline__ void put(float* p, float x) { *p = x; }
__device__ __forceinline__ void put(__nv_bfloat16* p, float x) { *p = __float2bfloat16_rn(x); }

// ---------------------------------------------------------------- joining partial results
// WPR warps per row: o = sum_c 2^(lse_c - lse) o_c over the row's partial results, the prefix's first, keys in order.
// Bound by latency: the log-sum-exps are read by all lanes at once, the outputs kAhead at a time (one after the other they
// took 15 us for the 38 parts of a row, which is what few rows have; so those have more warps, too).
template <typename T, int D, int WPR>
__global__ void __launch_bounds__(256) paged_merge_kernel(const PagedArgs a) {
    constexpr int V = D / 32, kRows = 8 / WPR, kAhead = 4;
    __shared__ float s_sum[8], s_acc[WPR > 1 ? 8 : 1][D];
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5, w = warp % WPR;
    const int64_t row = (int64_t)blockIdx.x * kRows + warp / WPR;
    const bool in = row < (int64_t)a.n_tokens * a.Hq;
    // the prefix's parts: one per CTA from pc0 on, each the first piece (slot 0) of its CTA, but for the unit's first part
    // where that CTA's share begins in the unit before
    int n_pre = 0;
    int64_t p0 = 0, p1 = 0;
    if (in && a.prefix_len > 0) {
        const int t = (int)(row / a.Hq), hq = (int)(row % a.Hq), h = hq / a.g;
        const int64_t R = (int64_t)t * a.g + (hq - h * a.g);
        const int tiles = (a.prefix_len + a.p_keys - 1) / a.p_keys;
        const int nrt = (int)(((int64_t)a.n_tokens * a.g + a.p_rows - 1) / a.p_rows);
        const int64_t total = (int64_t)a.Hkv * nrt * tiles, base = ((int64_t)h * nrt + R / a.p_rows) * tiles;
        const int r = (int)(R % a.p_rows), c0 = share_owner(base, total, a.p_ctas);
        n_pre = share_owner(base + tiles - 1, total, a.p_ctas) - c0 + 1;
        p0 = ((int64_t)c0 * 2 + (total * c0 / a.p_ctas < base ? 1 : 0)) * a.p_rows + r;
        p1 = ((int64_t)c0 * 2) * a.p_rows + r;
    }
    grid_dependency_wait();  // all above needs nothing that a kernel before this one writes
    const uint2 info = in ? a.row_info[row] : make_uint2(kRowDone, 0);
    const uint32_t kind = info.x & 3u;
    if (WPR == 1 && kind == kRowDone) return;
    if (kind == kRowDone) n_pre = 0;
    const float *oo = a.slot_o, *ol = a.slot_l;
    int n_own = 0;
    int64_t o0 = 0, o1 = 0;  // slot 1 of the unit's first CTA, then slot 0 of those after it
    if (kind == kRowWhole) {
        oo = a.own_o;
        ol = a.own_lse;
        n_own = 1;
        o0 = row;
    } else if (kind == kRowSplit) {
        const int c0 = info.y & 0xffffu, c1 = info.y >> 16, r = info.x >> 2;
        n_own = c1 - c0 + 1;
        o0 = ((int64_t)c0 * 2 + 1) * a.rows + r;
        o1 = ((int64_t)c0 * 2) * a.rows + r;
    }
    const int n = n_pre + n_own;
    auto lse_of = [&](int c) -> float {
        if (c < n_pre) return a.pslot_l[c ? p1 + (int64_t)c * 2 * a.p_rows : p0];
        c -= n_pre;
        return ol[c ? o1 + (int64_t)c * 2 * a.rows : o0];
    };
    auto out_of = [&](int c) -> const float* {
        if (c < n_pre) return a.pslot_o + (c ? p1 + (int64_t)c * 2 * a.p_rows : p0) * D;
        c -= n_pre;
        return oo + (c ? o1 + (int64_t)c * 2 * a.rows : o0) * D;
    };
    float mx = -INFINITY;
    for (int c = lane; c < n; c += 32) mx = fmaxf(mx, lse_of(c));
    for (int o = 16; o; o >>= 1) mx = fmaxf(mx, __shfl_xor_sync(~0u, mx, o));
    const float ms = mx == -INFINITY ? 0.f : mx;
    float acc[V], sum = 0.f;
#pragma unroll
    for (int e = 0; e < V; ++e) acc[e] = 0.f;
    for (int c0 = w; c0 < n; c0 += WPR * kAhead) {
        float x[kAhead][V], f[kAhead];
#pragma unroll
        for (int u = 0; u < kAhead; ++u) {
            const int c = c0 + u * WPR;
            f[u] = c < n ? lse_of(c) : -INFINITY;
            const float* src = out_of(c < n ? c : c0) + lane * V;
#pragma unroll
            for (int e = 0; e < V; ++e) x[u][e] = src[e];
        }
#pragma unroll
        for (int u = 0; u < kAhead; ++u) {
            const float g = exp2f(f[u] - ms);
            sum += g;
#pragma unroll
            for (int e = 0; e < V; ++e) acc[e] = fmaf(g, x[u][e], acc[e]);
        }
    }
    if constexpr (WPR > 1) {
        if (lane == 0) s_sum[warp] = sum;
#pragma unroll
        for (int e = 0; e < V; ++e) s_acc[warp][lane * V + e] = acc[e];
        __syncthreads();
        if (w != 0 || kind == kRowDone) return;
#pragma unroll
        for (int x = 1; x < WPR; ++x) {
            sum += s_sum[warp + x];
#pragma unroll
            for (int e = 0; e < V; ++e) acc[e] += s_acc[warp + x][lane * V + e];
        }
    }
    const float inv = sum > 0.f ? 1.f / sum : 0.f;
    T* out = static_cast<T*>(a.o) + row * D + lane * V;
#pragma unroll
    for (int e = 0; e < V; ++e) put(out + e, acc[e] * inv);
    if (lane == 0) a.lse[row] = sum > 0.f ? (ms + log2f(sum)) * kLn2 : -INFINITY;
}

size_t align256(size_t x) { return (x + 255) & ~(size_t)255; }

}  // namespace

// The kernel for `rows` rows per KV head: rows of a unit, keys of a tile, CTAs that run at a time.
struct Pick {
    int rows, keys, ctas;
};
static Pick pick(const PagedArgs& a, int64_t rows) {
    if (a.elem == 4) return {8, 64, kSms};
    if (rows <= 32) return {rows <= 16 ? 16 : 32, 64, kSms * 2};
    return {rows <= 128 ? 128 : 256, 128, kSms};
}

size_t paged_plan(PagedArgs* a, int max_q, void* ws) {
    const int64_t rows = (int64_t)a->n_tokens * a->Hq;
    const Pick own = pick(*a, (int64_t)max_q * a->g);
    a->rows = own.rows;
    a->ctas = own.ctas;
    a->p_rows = a->p_ctas = a->p_keys = 0;
    if (a->prefix_len > 0) {
        const int64_t batch = (int64_t)a->n_tokens * a->g;
        const Pick pre = pick(*a, batch);
        a->p_rows = pre.rows;
        a->p_keys = pre.keys;
        // no share longer than a unit, so that it touches two units at most: one slot each; none empty; whole waves
        const int64_t units = (batch + pre.rows - 1) / pre.rows * a->Hkv;
        const int64_t tiles = units * ((a->prefix_len + pre.keys - 1) / pre.keys);
        const int64_t waves = (units + pre.ctas - 1) / pre.ctas;
        a->p_ctas = (int)std::min(tiles, waves * pre.ctas);
    }
    size_t at = 0;
    char* w = static_cast<char*>(ws);
    auto take = [&](size_t bytes) {
        char* p = w ? w + at : nullptr;
        at += align256(bytes);
        return p;
    };
    a->row_info = reinterpret_cast<uint2*>(take(rows * sizeof(uint2)));
    a->slot_o = reinterpret_cast<float*>(take((size_t)a->ctas * 2 * a->rows * a->d * 4));
    a->slot_l = reinterpret_cast<float*>(take((size_t)a->ctas * 2 * a->rows * 4));
    a->own_o = a->own_lse = a->pslot_o = a->pslot_l = nullptr;
    if (a->prefix_len > 0) {
        a->own_o = reinterpret_cast<float*>(take((size_t)rows * a->d * 4));
        a->own_lse = reinterpret_cast<float*>(take((size_t)rows * 4));
        a->pslot_o = reinterpret_cast<float*>(take((size_t)a->p_ctas * 2 * a->p_rows * a->d * 4));
        a->pslot_l = reinterpret_cast<float*>(take((size_t)a->p_ctas * 2 * a->p_rows * 4));
    }
    return at;
}

cudaError_t launch_paged_own(const PagedArgs& a, cudaStream_t stream) {
    if (a.elem == 4) return launch_paged_f32(a, false, stream);
    return a.rows <= 32 ? launch_paged_mma(a, false, stream) : launch_paged_tc(a, false, stream);
}

cudaError_t launch_paged_prefix(const PagedArgs& a, cudaStream_t stream) {
    if (a.elem == 4) return launch_paged_f32(a, true, stream);
    return a.p_rows <= 32 ? launch_paged_mma(a, true, stream) : launch_paged_tc(a, true, stream);
}

template <typename T, int D>
static cudaError_t merge_t(const PagedArgs& a, cudaStream_t stream) {
    // few rows have many parts each (a batch of any size is cut into as many shares as there are CTAs)
    const int64_t rows = (int64_t)a.n_tokens * a.Hq;
    if (rows <= 8 * kSms) return launch_dependent(paged_merge_kernel<T, D, 8>, (unsigned)rows, 256, 0, stream, a);
    return launch_dependent(paged_merge_kernel<T, D, 1>, (unsigned)((rows + 7) / 8), 256, 0, stream, a);
}

cudaError_t launch_paged_merge(const PagedArgs& a, cudaStream_t stream) {
    if (a.elem == 4) return a.d == 64 ? merge_t<float, 64>(a, stream) : merge_t<float, 128>(a, stream);
    return a.d == 64 ? merge_t<__nv_bfloat16, 64>(a, stream) : merge_t<__nv_bfloat16, 128>(a, stream);
}

}  // namespace usp
