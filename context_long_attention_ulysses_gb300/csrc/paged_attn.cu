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

// ---------------------------------------------------------------- joining partial results
// o = sum_c 2^(lse_c - lse) o_c over a row's partial results, the prefix's first, keys in order.  A row's parts:
struct Parts {
    const float *po, *pl;  // prefix part c: log-sum-exp at pl[c * p_step_l], values at po + c * p_step_o
    const float *oo, *ol;  // own part c, likewise (the first part of a cut unit is in slot 1, the others in slot 0)
    int64_t p_step_l, p_step_o, o_step_l, o_step_o, o_fix_l, o_fix_o;
    int n_pre, n;          // prefix parts, all parts
    int p_col, o_col;      // floats between groups of four columns
};

// Row (token t, KV head h, place j in the group); `info` as note_row wrote it.
__device__ __forceinline__ Parts row_parts(const PagedArgs& a, int t, int h, int j, uint2 info) {
    Parts p{};
    const int64_t row = (int64_t)t * a.Hq + h * a.g + j;
    if (a.prefix_len > 0) {
        const int R = t * a.g + j, nrt = (a.n_tokens * a.g + a.p_rows - 1) / a.p_rows, rt = R / a.p_rows;
        const int r = R - rt * a.p_rows;
        const int64_t slot = ((int64_t)h * nrt + rt) * a.p_split;
        const bool groups = a.p_rows >= 128;
        p.n_pre = a.p_split;
        p.pl = a.pslot_l + slot * a.p_rows + r;
        p.po = a.pslot_o + slot * a.p_rows * a.d + (groups ? r * 4 : r * a.d);
        p.p_step_l = a.p_rows;
        p.p_step_o = (int64_t)a.p_rows * a.d;
        p.p_col = groups ? a.p_rows * 4 : 4;
    }
    p.n = p.n_pre;
    p.o_col = 4;
    const uint32_t kind = info.x & 3u;
    // A kernel whose wait gave up has not noted its rows: what the workspace held instead (an earlier call's words, say) leads
    // nowhere outside it.  Without a prefix there is no own_o.
    if (kind == kRowWhole && a.prefix_len == 0) return p;
    if (kind == kRowWhole) {
        p.n += 1;
        p.oo = a.own_o + row * a.d;
        p.ol = a.own_lse + row;
    } else if (kind == kRowSplit) {
        const int c0 = info.y & 0xffffu, c1 = info.y >> 16, r = info.x >> 2;
        if (c0 > c1 || c1 >= a.ctas || r >= a.rows) return p;
        const bool groups = a.rows >= 128;
        p.n += c1 - c0 + 1;
        p.ol = a.slot_l + ((int64_t)c0 * 2 + 1) * a.rows + r;
        p.oo = a.slot_o + ((int64_t)c0 * 2 + 1) * a.rows * a.d + (groups ? r * 4 : r * a.d);
        p.o_step_l = 2 * a.rows;
        p.o_step_o = (int64_t)2 * a.rows * a.d;
        p.o_fix_l = -a.rows;
        p.o_fix_o = -(int64_t)a.rows * a.d;
        p.o_col = groups ? a.rows * 4 : 4;
    }
    return p;
}
__device__ __forceinline__ float part_lse(const Parts& p, int c) {
    if (c < p.n_pre) return __ldcg(p.pl + c * p.p_step_l);
    c -= p.n_pre;
    return __ldcg(p.ol + c * p.o_step_l + (c ? p.o_fix_l : 0));
}
// columns 4 * c4 .. of part c
__device__ __forceinline__ float4 part_cols(const Parts& p, int c, int c4) {
    if (c < p.n_pre) return __ldcg(reinterpret_cast<const float4*>(p.po + c * p.p_step_o + c4 * p.p_col));
    c -= p.n_pre;
    return __ldcg(reinterpret_cast<const float4*>(p.oo + c * p.o_step_o + (c ? p.o_fix_o : 0) + c4 * p.o_col));
}

__device__ __forceinline__ void put4(float* p, const float4& x) { *reinterpret_cast<float4*>(p) = x; }
__device__ __forceinline__ void put4(__nv_bfloat16* p, const float4& x) {
    uint2 w;
    asm("cvt.rn.bf16x2.f32 %0, %1, %2;" : "=r"(w.x) : "f"(x.y), "f"(x.x));
    asm("cvt.rn.bf16x2.f32 %0, %1, %2;" : "=r"(w.y) : "f"(x.w), "f"(x.z));
    *reinterpret_cast<uint2*>(p) = w;
}

// A CTA joins ROWS = 4 or 1 neighbouring rows of a KV head: thread = (row, four columns, every WAYS-th part), with a
// running maximum, four parts' reads in flight.  With four rows the reads of slots kept in column groups are 64 contiguous
// bytes (a row at a time they would be 16; eight rows were 1 us slower for 64 samples behind a prefix).  A call of few rows
// has many parts per row, 38 for one sequence of 128K tokens, and is bound by the latency of the reads, so it takes more
// ways, unless its slots are in column groups: one after the other these took 15 us.  With few parts per row more ways only
// cost: two instead of one, 40 us against 21 for the two parts of 65536 rows, 10 against 9 for five parts of 6400.
template <typename T, int D, int ROWS, int NT>
__global__ void __launch_bounds__(NT) paged_merge_kernel(const PagedArgs a) {
    constexpr int kCols = D / 4, kWays = NT / (kCols * ROWS), kAhead = 4;
    __shared__ float4 s_acc[kWays > 1 ? NT : 1];
    __shared__ float2 s_stat[kWays > 1 ? NT : 1];
    const int r = threadIdx.x % ROWS, c4 = threadIdx.x / ROWS % kCols, way = threadIdx.x / (ROWS * kCols);
    const int h = blockIdx.y, R = blockIdx.x * ROWS + r, t = R / a.g, j = R - t * a.g;
    const bool in = R < a.n_tokens * a.g;
    const int64_t row = (int64_t)t * a.Hq + h * a.g + j;
    begin_kernel(false);
    const uint2 info = in ? __ldcg(a.row_info + row) : make_uint2(kRowDone, 0);
    const bool done = (info.x & 3u) == kRowDone;
    Parts p{};
    if (!done) p = row_parts(a, t, h, j, info);
    float4 acc = make_float4(0.f, 0.f, 0.f, 0.f);
    float sum = 0.f, mx = -INFINITY;
    for (int c0 = way; c0 < p.n; c0 += kWays * kAhead) {
        float4 x[kAhead];
        float f[kAhead], m = mx;
#pragma unroll
        for (int u = 0; u < kAhead; ++u) {
            const int c = c0 + u * kWays;
            f[u] = c < p.n ? part_lse(p, c) : -INFINITY;
            x[u] = c < p.n ? part_cols(p, c, c4) : make_float4(0.f, 0.f, 0.f, 0.f);
        }
#pragma unroll
        for (int u = 0; u < kAhead; ++u) m = fmaxf(m, f[u]);
        const float ms = m == -INFINITY ? 0.f : m, al = exp2f(mx - ms);
        mx = m;
        sum *= al;
        acc = make_float4(acc.x * al, acc.y * al, acc.z * al, acc.w * al);
#pragma unroll
        for (int u = 0; u < kAhead; ++u) {
            const float w = exp2f(f[u] - ms);
            sum += w;
            acc.x = fmaf(w, x[u].x, acc.x);
            acc.y = fmaf(w, x[u].y, acc.y);
            acc.z = fmaf(w, x[u].z, acc.z);
            acc.w = fmaf(w, x[u].w, acc.w);
        }
    }
    if constexpr (kWays > 1) {
        s_acc[threadIdx.x] = acc;
        s_stat[threadIdx.x] = make_float2(mx, sum);
        __syncthreads();
        if (way != 0) return;
#pragma unroll
        for (int w = 1; w < kWays; ++w) mx = fmaxf(mx, s_stat[threadIdx.x + w * ROWS * kCols].x);
        const float ms = mx == -INFINITY ? 0.f : mx;
        sum = 0.f;
        acc = make_float4(0.f, 0.f, 0.f, 0.f);
#pragma unroll
        for (int w = 0; w < kWays; ++w) {
            const float4 y = s_acc[threadIdx.x + w * ROWS * kCols];
            const float2 z = s_stat[threadIdx.x + w * ROWS * kCols];
            const float f = exp2f(z.x - ms);
            sum = fmaf(f, z.y, sum);
            acc.x = fmaf(f, y.x, acc.x);
            acc.y = fmaf(f, y.y, acc.y);
            acc.z = fmaf(f, y.z, acc.z);
            acc.w = fmaf(f, y.w, acc.w);
        }
    }
    if (done) return;
    const float inv = sum != 0.f ? 1.f / sum : 0.f;  // (NaN has to show)
    put4(static_cast<T*>(a.o) + row * D + c4 * 4, make_float4(acc.x * inv, acc.y * inv, acc.z * inv, acc.w * inv));
    if (c4 == 0) a.lse[row] = sum != 0.f ? (mx + log2f(sum)) * kLn2 : -INFINITY;
}

size_t align256(size_t x) { return (x + 255) & ~(size_t)255; }

}  // namespace

// The kernel for `rows` rows per KV head: its unit, and the CTAs that run at a time.
struct Pick {
    int rows, keys, ctas, piece;
    float us;  // time of a tile
    Pick(const UnitShape& u, float tile_us) : rows(u.rows), keys(u.keys), ctas(kSms * u.ctas_per_sm), piece(u.piece), us(tile_us) {}
};
// bf16 by the rows per KV head, 32 query and 8 KV heads of 128 values, 16 sequences of 1000 to 20000 tokens:
//   20 rows: 84.1 us in a unit of 32 (m16n8k16 products), 93.2 in one of 128 (tcgen05); 32 rows: 85.2 and 90.9
//   48 rows: 91.6 in a unit of 128, 162 in two of 32
//   64 rows: 93.1 in one of 128, 108 in one of 256, whose second stream is idle; 96 rows: 97.8 and 112
// and 160 rows of 8 sequences: 59.6 in one of 256, 67.8 in two of 128.
static Pick pick(const PagedArgs& a, int64_t rows) {
    if (a.elem == 4) return {f32_unit(a.d), 1.5f};
    if (rows <= 16) return {mma_unit(a.d, 1), 1.5f};
    if (rows <= 32) return {mma_unit(a.d, 2), a.d == 64 ? 0.8f : 1.5f};
    return rows <= 128 ? Pick{tc_unit(1), 1.1f} : Pick{tc_unit(2), 1.6f};
}

size_t paged_plan(PagedArgs* a, int max_q, void* ws) {
    const int64_t rows = (int64_t)a->n_tokens * a->Hq;
    const Pick own = pick(*a, (int64_t)max_q * a->g);
    a->rows = own.rows;
    a->ctas = own.ctas;
    a->p_rows = a->p_ctas = a->p_split = 0;
    if (a->prefix_len > 0) {
        const int64_t batch = (int64_t)a->n_tokens * a->g;
        // Rows of a unit and its parts: few waves of CTAs, each of few tiles and the cost of a piece, and few partial results,
        // which the merge reads back at about 2 TB/s.  (Units of 256 rows always, and as many parts as CTAs, the partial results
        // left out of the account: 37.6 us for 106 samples behind 1271 tokens against 29.5, 29 requests with one KV head
        // behind 53364 41.6 against 34.4, 200 requests behind 4001 122.9 against 120.5.)
        float best = INFINITY;
        for (const Pick& pre : {pick(*a, batch), pick(*a, std::min<int64_t>(batch, 128))}) {
            const int64_t units = (batch + pre.rows - 1) / pre.rows * a->Hkv, tiles = (a->prefix_len + pre.keys - 1) / pre.keys;
            const float slot = (float)pre.rows * a->d * 4 / 2e6f;
            for (int64_t quarter = 1; quarter <= 16; ++quarter) {  // of a wave
                const int64_t k = std::max<int64_t>(1, std::min(tiles, quarter * pre.ctas / (4 * units)));
                const int64_t waves = (units * k + pre.ctas - 1) / pre.ctas;
                const float cost = (float)(waves * ((tiles + k - 1) / k + pre.piece)) * pre.us + (float)(units * k) * slot;
                if (cost < best) {
                    best = cost;
                    a->p_rows = pre.rows;
                    a->p_split = (int)k;
                    a->p_ctas = (int)(units * k);
                }
            }
        }
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
        a->pslot_o = reinterpret_cast<float*>(take((size_t)a->p_ctas * a->p_rows * a->d * 4));
        a->pslot_l = reinterpret_cast<float*>(take((size_t)a->p_ctas * a->p_rows * 4));
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
    const int batch = a.n_tokens * a.g;
    if ((int64_t)batch * a.Hkv <= 8 * kSms && a.rows < 128 && a.p_rows < 128)
        return launch_dependent(paged_merge_kernel<T, D, 1, 512>, dim3(batch, a.Hkv), 512, 0, stream, a);
    // parts of a row: those of the prefix, and own ones as equal shares give them
    const int64_t units = (int64_t)a.Hkv * std::max(a.n_seqs, (batch + a.rows - 1) / a.rows);
    const dim3 grid((batch + 3) / 4, a.Hkv);
    // (few CTAs with very many parts each: 31.4 us against 34.4 for 29 requests with one KV head behind 53364 tokens)
    if (a.p_split + a.ctas / units > 32 && (int64_t)grid.x * grid.y <= kSms)
        return launch_dependent(paged_merge_kernel<T, D, 4, 1024>, grid, 1024, 0, stream, a);
    if (a.p_split + a.ctas / units > 8)
        return launch_dependent(paged_merge_kernel<T, D, 4, 512>, grid, 512, 0, stream, a);
    return launch_dependent(paged_merge_kernel<T, D, 4, 128>, grid, 128, 0, stream, a);
}

cudaError_t launch_paged_merge(const PagedArgs& a, cudaStream_t stream) {
    if (a.elem == 4) return a.d == 64 ? merge_t<float, 64>(a, stream) : merge_t<float, 128>(a, stream);
    return a.d == 64 ? merge_t<__nv_bfloat16, 64>(a, stream) : merge_t<__nv_bfloat16, 128>(a, stream);
}

}  // namespace usp
