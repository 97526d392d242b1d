// Attention over a paged cache in float32, on CUDA cores (the tensor cores' tf32 would not keep float32's digits).
//
// With 8 rows per KV head a key costs 4 d 8 flops per 8 d bytes, within what the CUDA cores do at the memory's rate, so
// the kernel is built around the loads as its bf16 sibling is: each of eight warps owns 1024 / d keys of a tile and streams
// them by itself through a ring of shared memory (cp.async, 16 bytes a lane; missing keys are filled with zeros), with a
// running maximum, sum and output of its own; the eight meet only where a piece ends.  (Four warps with twice the keys, one
// per scheduler, left it waiting for its own instructions: 34 us for 16 sequences of up to 16000 tokens.)
//   scores: d/32 lanes per key, 32 values each; a key's row is padded by 16 bytes, so that 8 lanes' 16-byte reads fall into
//           different banks, and the rows of Q are read by all lanes of a part at once
//   output: a lane holds d/32 columns; the probabilities go through shared memory to be read by all lanes
// More rows are more units, each reading K and V again (through L2).
#include <cmath>

#include "paged.cuh"

namespace usp {

namespace {

constexpr int kPieceCost = 2;  // see paged.cuh
constexpr int kWarps = 8, kThreads = 32 * kWarps;
constexpr int kRows = 8;
constexpr float kLn2 = 0.6931471805599453f;

template <int D>
struct Cfg {
    static constexpr int kParts = D / 32;                         // lanes per key in the scores
    static constexpr int kSub = 32 / kParts;                      // keys of a warp in a tile
    static constexpr int kKeyTile = kWarps * kSub;
    static constexpr int kKStride = D + 4;                        // floats per key of K in shared memory
    static constexpr int kStageFloats = kSub * (kKStride + D);    // K, V
    static constexpr int kStages = 3;                             // about 130 KB in flight per SM
    static constexpr int kOffJoin = kWarps * kStages * kStageFloats;
    static constexpr int kOffQ = kOffJoin + kWarps / 2 * kRows * D;
    static constexpr int kOffP = kOffQ + kRows * D;
    static constexpr int kOffStat = kOffP + kWarps * kSub * kRows;
    static constexpr int kFloats = kOffStat + 2 * kWarps * kRows;
};

// 16 bytes global -> shared, zeros where !live
__device__ __forceinline__ void copy16(uint32_t dst, const float* src, bool live) {
    asm volatile("cp.async.cg.shared.global [%0], [%1], 16, %2;" ::"r"(dst), "l"(src), "r"(live ? 16 : 0) : "memory");
}
__device__ __forceinline__ void copies_commit() { asm volatile("cp.async.commit_group;" ::: "memory"); }
template <int N>
__device__ __forceinline__ void copies_wait() { asm volatile("cp.async.wait_group %0;" ::"n"(N) : "memory"); }

template <int D, bool PREFIX>
__global__ void __launch_bounds__(kThreads, 1) paged_f32_kernel(const PagedArgs a) {
    using C = Cfg<D>;
    constexpr int M = kRows, V = D / 32, S = C::kStages, kVecs = D / 4;  // kVecs: 16-byte vectors of a row
    constexpr int kSub = C::kSub, kKeyTile = C::kKeyTile;
    extern __shared__ __align__(16) float smem[];
    __shared__ Share share;
    __shared__ uint32_t s_live[kWarps][S];  // keys of the stage that exist
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5, cta = blockIdx.x;
    let_dependents_start();
    if constexpr (!PREFIX) {
        find_share<M, C::kKeyTile, kPieceCost, kThreads>(a, cta, a.ctas, &share);
        finish_empty_rows<float, M, C::kKeyTile, kThreads>(a, cta, a.ctas);
        __syncthreads();
    }
    float* ring = smem + warp * S * C::kStageFloats;
    const uint32_t ring_addr = static_cast<uint32_t>(__cvta_generic_to_shared(ring));
    float* s_q = smem + C::kOffQ;
    float* s_p = smem + C::kOffP + warp * kSub * M;  // [key][row]
    float* s_m = smem + C::kOffStat;
    float* s_l = s_m + kWarps * M;
    const float* kp = static_cast<const float*>(a.k_pages);
    const float* vp = static_cast<const float*>(a.v_pages);
    constexpr uint32_t kAll = 0xffffffffu >> (32 - kSub);
    const int key = lane % kSub, part = lane / kSub;  // scores: this lane's key and 32 of its values

    auto piece = [&](const Seg& g) {
        const int first = PREFIX ? 0 : a.key_begin, end = seg_key_end<PREFIX>(a, g);
        // ---- rows
        for (int x = threadIdx.x; x < M * D; x += kThreads) {
            const int r = x / D, R = g.row0 + r, i = R / a.g;
            s_q[x] = r < g.n_rows ? static_cast<const float*>(a.q)[((int64_t)(g.t0 + i) * a.Hq + g.h * a.g + (R - i * a.g)) * D +
                                                                   x % D] * a.scale_log2
                                  : 0.f;
        }
        int lim[M], lim_min = INT_MAX;
#pragma unroll
        for (int r = 0; r < M; ++r) {
            lim[r] = r < g.n_rows ? row_limit<PREFIX>(a, g, r) : INT_MAX;
            lim_min = min(lim_min, lim[r]);
        }
        __syncthreads();
        float acc[M][V], m[M], l[M];
#pragma unroll
        for (int r = 0; r < M; ++r) {
            m[r] = -INFINITY;
            l[r] = 0.f;
#pragma unroll
            for (int c = 0; c < V; ++c) acc[r][c] = 0.f;
        }
        // ---- this warp's keys of tile x: where they lie (row of the pool, -1: no key)
        auto locate = [&](int x) -> int64_t {
            const int j = (g.tile0 + x) * kKeyTile + warp * kSub + key;
            if (x >= g.n_tiles || j < first || j >= end) return -1;
            const int page = seg_page<PREFIX>(a, g, j >> a.page_log2);
            if (page < 0) return -1;
            return (((int64_t)page * a.Hkv + g.h) << a.page_log2) + (j & ((1 << a.page_log2) - 1));
        };
        auto issue = [&](int x, int64_t row) {
            if (x < g.n_tiles) {
                const int st = x % S;
                const uint32_t k_dst = ring_addr + st * C::kStageFloats * 4, v_dst = k_dst + kSub * C::kKStride * 4;
                const uint32_t live = __ballot_sync(~0u, row >= 0) & kAll;
                if (lane == 0) s_live[warp][st] = live;
                if (live) {
#pragma unroll
                    for (int i = 0; i < kSub * kVecs / 32; ++i) {
                        const int r = (i * 32 + lane) / kVecs, c = (i * 32 + lane) % kVecs;
                        const int64_t at = __shfl_sync(~0u, row, r);
                        const int64_t off = (at < 0 ? 0 : at) * D + c * 4;
                        copy16(k_dst + (r * C::kKStride + c * 4) * 4, kp + off, at >= 0);
                        copy16(v_dst + (r * D + c * 4) * 4, vp + off, at >= 0);
                    }
                }
            }
            copies_commit();
        };
        int64_t ahead = locate(0);
        for (int x = 0; x < S - 1; ++x) {
            const int64_t now = ahead;
            ahead = locate(x + 1);
            issue(x, now);
        }
        for (int x = 0; x < g.n_tiles; ++x) {
            const int64_t now = ahead;
            ahead = locate(x + S);  // its page is on its way while this tile is worked on
            copies_wait<S - 2>();
            __syncwarp();
            issue(x + S - 1, now);  // into the stage that was read in the iteration before
            const int st = x % S;
            const uint32_t live = s_live[warp][st];
            if (live) {
                const float* ks = ring + st * C::kStageFloats;
                const float* vs = ks + kSub * C::kKStride;
                float s[M];
#pragma unroll
                for (int r = 0; r < M; ++r) s[r] = 0.f;
                const float* kr = ks + key * C::kKStride + part * 32;
                const float* qr = s_q + part * 32;
#pragma unroll 4
                for (int c = 0; c < 8; ++c) {
                    const float4 k4 = *reinterpret_cast<const float4*>(kr + c * 4);
#pragma unroll
                    for (int r = 0; r < M; ++r) {
                        const float4 q4 = *reinterpret_cast<const float4*>(qr + r * D + c * 4);
                        s[r] = fmaf(q4.x, k4.x, s[r]);
                        s[r] = fmaf(q4.y, k4.y, s[r]);
                        s[r] = fmaf(q4.z, k4.z, s[r]);
                        s[r] = fmaf(q4.w, k4.w, s[r]);
                    }
                }
                const int j = (g.tile0 + x) * kKeyTile + warp * kSub + key;
                const bool masked = (live != kAll) || (g.tile0 + x) * kKeyTile + (warp + 1) * kSub > lim_min;
                float al[M];
                bool grew = false;
#pragma unroll
                for (int r = 0; r < M; ++r) {
#pragma unroll
                    for (int o = 16; o >= kSub; o >>= 1) s[r] += __shfl_xor_sync(~0u, s[r], o);
                    if (masked && (j >= lim[r] || !(live >> key & 1u))) s[r] = -INFINITY;
                    float mx = s[r];
#pragma unroll
                    for (int o = kSub / 2; o; o >>= 1) mx = fmaxf(mx, __shfl_xor_sync(~0u, mx, o));
                    const bool up = mx > m[r];
                    al[r] = up ? exp2f(m[r] - mx) : 1.f;
                    if (up) m[r] = mx;
                    grew |= up;
                    s[r] = exp2f(s[r] - (m[r] == -INFINITY ? 0.f : m[r]));
                    l[r] = l[r] * al[r] + s[r];
                }
                if (part == 0) {
#pragma unroll
                    for (int r = 0; r < M; r += 4)
                        *reinterpret_cast<float4*>(s_p + key * M + r) = make_float4(s[r], s[r + 1], s[r + 2], s[r + 3]);
                }
                if (grew) {  // the same for all lanes
#pragma unroll
                    for (int r = 0; r < M; ++r)
#pragma unroll
                        for (int c = 0; c < V; ++c) acc[r][c] *= al[r];
                }
                __syncwarp();
#pragma unroll 4
                for (int k = 0; k < kSub; ++k) {
                    float v[V], p[M];
#pragma unroll
                    for (int c = 0; c < V; ++c) v[c] = vs[k * D + lane * V + c];
#pragma unroll
                    for (int r = 0; r < M; r += 4) *reinterpret_cast<float4*>(p + r) = *reinterpret_cast<const float4*>(s_p + k * M + r);
#pragma unroll
                    for (int r = 0; r < M; ++r)
#pragma unroll
                        for (int c = 0; c < V; ++c) acc[r][c] = fmaf(p[r], v[c], acc[r][c]);
                }
            }
            __syncwarp();
        }
        copies_wait<0>();
        // ---- join the warps (four and four through the same buffer), normalise, store
        float* s_join = smem + C::kOffJoin;
#pragma unroll
        for (int r = 0; r < M; ++r) {
            // the parts of a key hold the same sums: add up one lane per key
            for (int o = kSub / 2; o; o >>= 1) l[r] += __shfl_xor_sync(~0u, l[r], o);
            if (lane == 0) {
                s_m[warp * M + r] = m[r];
                s_l[warp * M + r] = l[r];
            }
            if (warp >= 4)
#pragma unroll
                for (int c = 0; c < V; ++c) s_join[((warp - 4) * M + r) * D + lane * V + c] = acc[r][c];
        }
        __syncthreads();
        if (warp < 4) {
#pragma unroll
            for (int r = 0; r < M; ++r) {
                const float m2 = s_m[(warp + 4) * M + r], mx = fmaxf(m[r], m2), ms = mx == -INFINITY ? 0.f : mx;
                const float f1 = exp2f(m[r] - ms), f2 = exp2f(m2 - ms);
#pragma unroll
                for (int c = 0; c < V; ++c) {
                    float* y = s_join + (warp * M + r) * D + lane * V + c;
                    *y = f1 * acc[r][c] + f2 * *y;
                }
                __syncwarp();
                if (lane == 0) {
                    s_m[warp * M + r] = mx;
                    s_l[warp * M + r] = f1 * l[r] + f2 * s_l[(warp + 4) * M + r];
                }
            }
        }
        __syncthreads();
        for (int x = threadIdx.x; x < g.n_rows * kVecs; x += kThreads) {
            const int r = x / kVecs, c = x % kVecs * 4;
            float mx = -INFINITY;
#pragma unroll
            for (int w = 0; w < 4; ++w) mx = fmaxf(mx, s_m[w * M + r]);
            const float ms = mx == -INFINITY ? 0.f : mx;
            float sum = 0.f;
            float4 o = make_float4(0.f, 0.f, 0.f, 0.f);
#pragma unroll
            for (int w = 0; w < 4; ++w) {
                const float f = exp2f(s_m[w * M + r] - ms);
                const float4 y = *reinterpret_cast<const float4*>(s_join + (w * M + r) * D + c);
                sum += f * s_l[w * M + r];
                o.x = fmaf(f, y.x, o.x);
                o.y = fmaf(f, y.y, o.y);
                o.z = fmaf(f, y.z, o.z);
                o.w = fmaf(f, y.w, o.w);
            }
            const bool has = sum > 0.f;
            o = has ? make_float4(o.x / sum, o.y / sum, o.z / sum, o.w / sum) : make_float4(0.f, 0.f, 0.f, 0.f);
            const float lse2 = has ? ms + log2f(sum) : -INFINITY;
            const RowDst dst = row_dst<M, PREFIX>(a, g, r, cta);
            *reinterpret_cast<float4*>((dst.out ? static_cast<float*>(dst.out) : dst.part) + c) = o;
            if (c == 0) {
                *dst.lse = dst.out ? lse2 * kLn2 : lse2;
                if (!PREFIX && g.ends) note_row<M>(a, g, r, cta);
            }
        }
        __syncthreads();
    };
    if constexpr (PREFIX) {
        piece(prefix_piece<M, kKeyTile>(a, cta));
    } else {
        Seg g;
        OwnWalk<M, kKeyTile, kPieceCost> walk(a, share);
        while (walk.next(g)) piece(g);
        grid_dependency_wait();  // ends after the prefix kernel: the merge after this one sees both
    }
}

template <int D>
cudaError_t launch_d(const PagedArgs& a, bool prefix, cudaStream_t s) {
    constexpr size_t smem = Cfg<D>::kFloats * 4;
    auto set = [](auto kern) {
        return cudaFuncSetAttribute(kern, cudaFuncAttributeMaxDynamicSharedMemorySize, (int)smem);
    };
    if (prefix) {
        const cudaError_t e = set(paged_f32_kernel<D, true>);
        if (e != cudaSuccess) return e;
        paged_f32_kernel<D, true><<<a.p_ctas, kThreads, smem, s>>>(a);
        return cudaGetLastError();
    }
    const cudaError_t e = set(paged_f32_kernel<D, false>);
    return e != cudaSuccess ? e : launch_own(paged_f32_kernel<D, false>, a, kThreads, smem, s, a);
}

}  // namespace

cudaError_t launch_paged_f32(const PagedArgs& a, bool prefix, cudaStream_t s) {
    return a.d == 64 ? launch_d<64>(a, prefix, s) : launch_d<128>(a, prefix, s);
}

}  // namespace usp
