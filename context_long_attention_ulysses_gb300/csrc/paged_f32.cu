// Attention over a paged cache in float32, on CUDA cores (the tensor cores' tf32 would not keep float32's digits).
//
// With 8 rows per KV head a key costs 4 d 8 flops per 8 d bytes, within what the CUDA cores do at the memory's rate, so
// the kernel is built around the loads as its bf16 sibling is: each of eight warps owns 1024 / d keys of a tile and streams
// them by itself through a ring of shared memory (cp.async, 16 bytes a lane; missing keys are filled with zeros), with a
// running maximum, sum and output of its own; the eight meet only where a piece ends.  (Four warps with twice the keys, one
// per scheduler, left it waiting for its own instructions: 34 us for 16 sequences of up to 16000 tokens.)
//   scores: eight lanes per key, d/8 values each, whose part of all 8 rows of Q stays in registers (read from shared memory
//           for every key it was most of that memory's traffic, half of its peak, and the kernel took 28 us); the eight
//           lanes' sums are added such that each ends with the whole score of one row, and does the softmax of that row
//   output: a lane holds d/32 columns; the probabilities go through shared memory to be read by all lanes
// More rows are more units, each reading K and V again (through L2).
// Measured: 16 sequences of 500 to 16000 tokens, 8 query and 2 KV heads of 64 values, 86 MB, in 27.5 us, 3.1 TB/s, the whole call
// or this kernel alone with cold caches.  What bounds it is latency: the SMs are at work for three quarters of that time, and then
// two warps per scheduler wait for their own instructions (1.41 cycles per instruction, for loads 0.72, shared memory 0.47,
// each other 0.39): issue slots are at 39 %, no pipe above 25 %.
#include <cmath>

#include "paged.cuh"
#include "ptx.cuh"

namespace usp {

namespace {

constexpr int kPieceCost = f32_unit(64).piece;
constexpr int kWarps = 8, kThreads = 32 * kWarps;
constexpr int kRows = 8;
constexpr float kLn2 = 0.6931471805599453f;

template <int D>
struct Cfg {
    static constexpr int kSub = 1024 / D;                         // keys of a warp in a tile
    static constexpr int kKeyTile = kWarps * kSub;
    static_assert(f32_unit(D).rows == kRows && f32_unit(D).keys == kKeyTile && f32_unit(D).ctas_per_sm == 1 &&
                  f32_unit(D).piece == kPieceCost, "the unit's shape");
    static constexpr int kStageFloats = kSub * 2 * D;             // K, V
    static constexpr int kStages = 3;                             // about 130 KB in flight per SM
    static constexpr int kOffJoin = kWarps * kStages * kStageFloats;
    static constexpr int kOffP = kOffJoin + kWarps / 2 * kRows * D;
    static constexpr int kOffScale = kOffP + kWarps * kSub * kRows;
    static constexpr int kOffStat = kOffScale + kWarps * kRows;
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
    begin_kernel(PREFIX);
    if constexpr (!PREFIX) {
        find_share<M, C::kKeyTile, kPieceCost, kThreads>(a, cta, a.ctas, &share);
        finish_empty_rows<float, M, C::kKeyTile, kThreads>(a, cta, a.ctas);
        __syncthreads();
    }
    float* ring = smem + warp * S * C::kStageFloats;
    const uint32_t ring_addr = static_cast<uint32_t>(__cvta_generic_to_shared(ring));
    float* s_p = smem + C::kOffP + warp * kSub * M;  // [key][row]
    float* s_al = smem + C::kOffScale + warp * M;
    float* s_m = smem + C::kOffStat;
    float* s_l = s_m + kWarps * M;
    const float* kp = static_cast<const float*>(a.k_pages);
    const float* vp = static_cast<const float*>(a.v_pages);
    constexpr uint32_t kAll = 0xffffffffu >> (32 - kSub);
    const int ckey = lane % kSub;                     // copies: the key this lane looks up
    const int part = lane & 7, kk = lane >> 3;        // scores: values 4 part .. of every 32, of keys kk, kk + 4, ..
    constexpr int NP = kSub / 4, NV = D / 32;         // keys per lane, 16-byte vectors per lane and key
                                                      // softmax: row `part` of the unit, those keys

    // Where this warp's keys of tile x of a piece lie (row of the pool, -1: no key).
    auto locate = [&](const Seg& g, int x) -> int64_t {
        const int j = (g.tile0 + x) * kKeyTile + warp * kSub + ckey;
        if (j < (PREFIX ? 0 : a.key_begin) || j >= seg_key_end<PREFIX>(a, g)) return -1;
        const int page = seg_page<PREFIX>(a, g, j >> a.page_log2);
        if (page < 0) return -1;
        return (((int64_t)page * a.Hkv + g.h) << a.page_log2) + (j & ((1 << a.page_log2) - 1));
    };
    // The copies run on across pieces, up to the end of the next one: `next_row` is where the tile to be issued next lies.
    Seg cur{}, nxt{};
    bool has_nxt = false;
    int it = 0, issued = 0;           // tiles worked on and tiles issued by this CTA so far
    int ahead = 0;                    // tiles of the current piece (and then the next) that were issued
    int64_t next_row = -1;
    auto find_next = [&] {            // `ahead` is the tile to be issued next
        const int y = ahead - cur.n_tiles;
        next_row = y < 0 ? locate(cur, ahead) : has_nxt && y < nxt.n_tiles ? locate(nxt, y) : -1;
    };
    auto issue = [&] {                // one group of copies, if there is a tile
        if (ahead >= cur.n_tiles + (has_nxt ? nxt.n_tiles : 0)) return;
        const int st = issued % S;
        const uint32_t k_dst = ring_addr + st * C::kStageFloats * 4, v_dst = k_dst + kSub * D * 4;
        const uint32_t live = __ballot_sync(~0u, next_row >= 0) & kAll;
        if (lane == 0) s_live[warp][st] = live;
        if (live) {
#pragma unroll
            for (int i = 0; i < kSub * kVecs / 32; ++i) {
                const int r = (i * 32 + lane) / kVecs, c = (i * 32 + lane) % kVecs;
                const int64_t at = __shfl_sync(~0u, next_row, r);
                const int64_t off = (at < 0 ? 0 : at) * D + c * 4;
                copy16(k_dst + (r * D + c * 4) * 4, kp + off, at >= 0);
                copy16(v_dst + (r * D + c * 4) * 4, vp + off, at >= 0);
            }
        }
        copies_commit();
        ++issued;
        ++ahead;
        find_next();  // its page is on its way while the tile before is worked on
    };

    // Works through `cur`; then `nxt` becomes the current piece.
    auto piece = [&] {
        const Seg& g = cur;
        while (issued < it + S - 1 && ahead < cur.n_tiles + (has_nxt ? nxt.n_tiles : 0)) issue();
        // ---- rows
        float4 q[M][NV];
#pragma unroll
        for (int r = 0; r < M; ++r) {
            const bool live = r < g.n_rows;
            const int R = g.row0 + (live ? r : 0), i = R / a.g;
            const float4* src = reinterpret_cast<const float4*>(
                static_cast<const float*>(a.q) + ((int64_t)(g.t0 + i) * a.Hq + g.h * a.g + (R - i * a.g)) * D) + part;
#pragma unroll
            for (int v = 0; v < NV; ++v) {
                const float4 w = live ? *(src + 8 * v) : make_float4(0.f, 0.f, 0.f, 0.f);
                q[r][v] = make_float4(w.x * a.scale_log2, w.y * a.scale_log2, w.z * a.scale_log2, w.w * a.scale_log2);
            }
        }
        const int lim = part < g.n_rows ? row_limit<PREFIX>(a, g, part) : INT_MAX;
        const int lim_min = __reduce_min_sync(~0u, lim);
        // (packed float32: the scores sum two products, the output takes two rows at a time)
        float2 acc[V][M / 2];
        float m = -INFINITY, l = 0.f;
#pragma unroll
        for (int c = 0; c < V; ++c)
#pragma unroll
            for (int r = 0; r < M / 2; ++r) acc[c][r] = make_float2(0.f, 0.f);
        for (int x = 0; x < g.n_tiles; ++x, ++it) {
            if (issued - it >= S - 1) copies_wait<S - 2>(); else copies_wait<0>();
            __syncwarp();
            if (issued < it + S) issue();  // into the stage that was read in the iteration before
            const int st = it % S;
            const uint32_t live = s_live[warp][st];
            if (live) {
                const float* ks = ring + st * C::kStageFloats;
                const float* vs = ks + kSub * D;
                float s[NP];
#pragma unroll
                for (int j = 0; j < NP; ++j) {
                    float2 s2[M];
#pragma unroll
                    for (int r = 0; r < M; ++r) s2[r] = make_float2(0.f, 0.f);
                    const float4* kr = reinterpret_cast<const float4*>(ks + (j * 4 + kk) * D) + part;
#pragma unroll
                    for (int v = 0; v < NV; ++v) {
                        const float4 k4 = kr[8 * v];
#pragma unroll
                        for (int r = 0; r < M; ++r) {
                            s2[r] = fma2(make_float2(q[r][v].x, q[r][v].y), make_float2(k4.x, k4.y), s2[r]);
                            s2[r] = fma2(make_float2(q[r][v].z, q[r][v].w), make_float2(k4.z, k4.w), s2[r]);
                        }
                    }
                    // add the eight lanes up, each step keeping half of the rows
                    float t[M];
#pragma unroll
                    for (int r = 0; r < M; ++r) t[r] = s2[r].x + s2[r].y;
#pragma unroll
                    for (int o = 4; o; o >>= 1) {
                        const bool hi = lane & o;
#pragma unroll
                        for (int r = 0; r < o; ++r)
                            t[r] = (hi ? t[r + o] : t[r]) + __shfl_xor_sync(~0u, hi ? t[r] : t[r + o], o);
                    }
                    s[j] = t[0];
                }
                const int key0 = (g.tile0 + x) * kKeyTile + warp * kSub + kk;
                if (live != kAll || key0 - kk + kSub > lim_min) {
#pragma unroll
                    for (int j = 0; j < NP; ++j)
                        if (key0 + 4 * j >= lim || !(live >> (4 * j + kk) & 1u)) s[j] = -INFINITY;
                }
                float mx = s[0];
#pragma unroll
                for (int j = 1; j < NP; ++j) mx = fmaxf(mx, s[j]);
                mx = fmaxf(mx, __shfl_xor_sync(~0u, mx, 8));
                mx = fmaxf(mx, __shfl_xor_sync(~0u, mx, 16));
                const bool up = mx > m;
                if (__any_sync(~0u, up)) {
                    const float al = up ? exp2f(m - mx) : 1.f;
                    if (up) m = mx;
                    l *= al;
                    if (kk == 0) s_al[part] = al;
                    __syncwarp();
#pragma unroll
                    for (int r = 0; r < M / 2; ++r) {
                        const float2 al2 = *reinterpret_cast<const float2*>(s_al + 2 * r);
#pragma unroll
                        for (int c = 0; c < V; ++c) acc[c][r] = mul2(acc[c][r], al2);
                    }
                }
                const float ms = m == -INFINITY ? 0.f : m;
#pragma unroll
                for (int j = 0; j < NP; ++j) {
                    s[j] = exp2f(s[j] - ms);
                    l += s[j];
                    s_p[(4 * j + kk) * M + part] = s[j];
                }
                __syncwarp();
#pragma unroll 4
                for (int k = 0; k < kSub; ++k) {
                    float v[V];
                    float4 p[M / 4];
#pragma unroll
                    for (int c = 0; c < V; c += 2) *reinterpret_cast<float2*>(v + c) = *reinterpret_cast<const float2*>(vs + k * D + lane * V + c);
#pragma unroll
                    for (int r = 0; r < M / 4; ++r) p[r] = *reinterpret_cast<const float4*>(s_p + k * M + 4 * r);
#pragma unroll
                    for (int c = 0; c < V; ++c) {
                        const float2 vv = make_float2(v[c], v[c]);
#pragma unroll
                        for (int r = 0; r < M / 4; ++r) {
                            acc[c][2 * r] = fma2(make_float2(p[r].x, p[r].y), vv, acc[c][2 * r]);
                            acc[c][2 * r + 1] = fma2(make_float2(p[r].z, p[r].w), vv, acc[c][2 * r + 1]);
                        }
                    }
                }
            }
            __syncwarp();
        }
        // ---- join the warps (four and four through the same buffer), normalise, store
        float* s_join = smem + C::kOffJoin;
        l += __shfl_xor_sync(~0u, l, 8);
        l += __shfl_xor_sync(~0u, l, 16);
        if (kk == 0) {
            s_m[warp * M + part] = m;
            s_l[warp * M + part] = l;
        }
        if (warp >= 4)
#pragma unroll
            for (int r = 0; r < M; ++r)
#pragma unroll
                for (int c = 0; c < V; ++c)
                    s_join[((warp - 4) * M + r) * D + lane * V + c] = r & 1 ? acc[c][r / 2].y : acc[c][r / 2].x;
        __syncthreads();
        if (warp < 4) {
#pragma unroll
            for (int r = 0; r < M; ++r) {
                const float m1 = s_m[warp * M + r], m2 = s_m[(warp + 4) * M + r], mx = fmaxf(m1, m2);
                const float ms = mx == -INFINITY ? 0.f : mx, f1 = exp2f(m1 - ms), f2 = exp2f(m2 - ms);
#pragma unroll
                for (int c = 0; c < V; ++c) {
                    float* y = s_join + (warp * M + r) * D + lane * V + c;
                    *y = f1 * (r & 1 ? acc[c][r / 2].y : acc[c][r / 2].x) + f2 * *y;
                }
                __syncwarp();
                if (lane == 0) {
                    s_m[warp * M + r] = mx;
                    s_l[warp * M + r] = f1 * s_l[warp * M + r] + f2 * s_l[(warp + 4) * M + r];
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
            const bool has = sum != 0.f;  // (NaN, too, which has to show)
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
        cur = prefix_piece<M, kKeyTile>(a, cta);
        find_next();
        piece();
        grid_dependency_wait();  // end after the own kernel
    } else {
        OwnWalk<M, kKeyTile, kPieceCost> walk(a, share);
        if (walk.next(cur)) {
            find_next();
            for (;;) {
                has_nxt = walk.next(nxt);
                if (has_nxt && ahead == cur.n_tiles) find_next();
                piece();
                if (!has_nxt) break;
                ahead -= cur.n_tiles;
                cur = nxt;
            }
        }
    }
}

template <int D>
cudaError_t launch_d(const PagedArgs& a, bool prefix, cudaStream_t s) {
    constexpr size_t smem = Cfg<D>::kFloats * 4;
    const cudaError_t e = prefix ? allow_smem<paged_f32_kernel<D, true>>((int)smem) : allow_smem<paged_f32_kernel<D, false>>((int)smem);
    if (e != cudaSuccess) return e;
    return prefix ? launch_dependent(paged_f32_kernel<D, true>, dim3(a.p_ctas), kThreads, smem, s, a)
                  : launch_dependent(paged_f32_kernel<D, false>, dim3(a.ctas), kThreads, smem, s, a);
}

}  // namespace

cudaError_t launch_paged_f32(const PagedArgs& a, bool prefix, cudaStream_t s) {
    return a.d == 64 ? launch_d<64>(a, prefix, s) : launch_d<128>(a, prefix, s);
}

}  // namespace usp
