/*
 * usp.h -- C ABI of libusp: Ulysses sequence-parallel attention on one GB300.
 *
 * What the library computes (sources are the web pages on Ulysses sequence
 * parallelism and context parallelism):
 *  - "Million-Token-Kontexte im Training" (bytewire.ai), section "Ulysses: Die
 *    Sequenz als Verteilungseinheit": the sequence is split along tokens over
 *    P devices; for attention, Q, K and V are exchanged by an all-to-all.
 *  - "Ulysses Sequence Parallelism" (topot.news), section "Как работает
 *    Ulysses": equal parts per device; after the all-to-all each device has
 *    the full context for its share of the attention.
 *  - "Context Parallelism" (ultralytics.com glossary), sections "So
 *    funktioniert Kontextparallelitaet" (ring attention: partial attention
 *    per KV block, exact equality with full-sequence attention; token-local
 *    layers on the local shard) and "Praktische Anwendung und Kompromisse"
 *    (B x H x N x d tensors with the sequence at dimension 2, causal scaled
 *    dot product attention, loss mean(out^2) and its backward).
 *
 * The P "ranks" are P slices of device buffers on ONE GPU; the all-to-all is
 * an on-device layout remap.
 *
 * Layouts (row-major, innermost last; every tensor is one contiguous device
 * buffer):
 *   logical          [B][H][N][d]
 *   sequence-sharded [P][B][N/P][H][d]   rank p holds tokens [p*N/P, (p+1)*N/P)
 *   head-sharded     [P][B][H/P][N][d]   rank r holds heads  [r*H/P, (r+1)*H/P)
 *   hybrid (2-D)     [P][B][H/Pu][N/Pr][d] rank g*Pu + u holds heads
 *                    [u*H/Pu, (u+1)*H/Pu) of token chunk g (P = Pu * Pr)
 *   LSE (head-sharded attention)    float32 [P][B][Hq/P][N]
 *   LSE (sequence-sharded ring, all-gather, fused) float32 [P][B][N/P][Hq]
 *   LSE (hybrid)                    float32 [P][B][Hq/Pu][N/Pr]
 * H is Hq for Q, O, dO, dQ and Hkv for K, V, dK, dV.  Query head h attends
 * with KV head h / (Hq/Hkv) (contiguous groups); each rank's query heads then
 * use only that rank's KV heads.
 *
 * Conventions for every entry point:
 *  - Ownership: the caller allocates and owns every buffer.  The library
 *    never allocates, frees or synchronises (except usp_device_status, which
 *    synchronises the given stream to read the status word).
 *  - Streams: all work is enqueued on `stream` (a cudaStream_t; NULL is the
 *    legacy default stream) in call order.  Inputs must stay valid until the
 *    work completes.
 *  - Errors: arguments are validated on the host before anything is
 *    enqueued; a non-OK status means nothing was enqueued.  A launch failure
 *    returns USP_ERR_CUDA.  Device-side waits are bounded; a wait that gives
 *    up records USP_ERR_TIMEOUT in a device status word that
 *    usp_device_status() reads.  No C++ exception crosses this ABI.
 *  - Pointers: device pointers, 16-byte aligned, non-overlapping unless a
 *    function says otherwise.  Empty problems (B == 0 or N == 0) are valid
 *    and enqueue nothing.
 *  - Precision: USP_BF16 tensors are bf16 with float32 accumulation; the
 *    softmax probabilities are rounded to bf16 before the P.V product.
 *    USP_F32 attention runs in true float32 (CUDA cores, forward only).
 */
#ifndef USP_H
#define USP_H

#include <stddef.h>
#include <stdint.h>

#ifdef __cplusplus
extern "C" {
#endif

typedef enum {
    USP_OK = 0,
    USP_ERR_INVALID_ARG = 1, /* null problem, bad sizes or divisibility */
    USP_ERR_UNSUPPORTED = 2, /* valid request the library does not implement (e.g. d not 64/128) */
    USP_ERR_MISALIGNED = 3,  /* a pointer is NULL or not 16-byte aligned */
    USP_ERR_WORKSPACE = 4,   /* workspace too small */
    USP_ERR_CUDA = 5,        /* a CUDA runtime/driver call or launch failed */
    USP_ERR_TIMEOUT = 6      /* a bounded device-side wait gave up */
} usp_status;

typedef enum { USP_F32 = 0, USP_BF16 = 1 } usp_dtype;

/* The problem of the glossary page's example: Q of shape B x Hq x N x d,
 * K and V of shape B x Hkv x N x d, sequence-parallel degree P, causal flag
 * (is_causal), softmax scale (0 selects the default 1/sqrt(d)).
 * Requirements: B, N >= 0; Hq, Hkv, P >= 1; N % P == 0; Hq % Hkv == 0;
 * B * Hq <= 65535; d in {64, 128} for attention.  Every entry point except
 * the ring ones also needs Hq % P == 0 and Hkv % P == 0 (each rank gets whole
 * heads after the all-to-all). */
typedef struct {
    int B;
    int Hq;
    int Hkv;
    int N;
    int d;
    int P;
    int causal;
    float scale;
    int dtype; /* usp_dtype */
} usp_problem;

typedef void* usp_stream; /* cudaStream_t */

/* All-to-all before attention (bytewire.ai "Ulysses: Die Sequenz als
 * Verteilungseinheit"; topot.news "Как работает Ulysses"):
 *   dst[r][b][h'][n][:] = src[n/(N/P)][b][n%(N/P)][r*Hx/P + h'][:]
 * src: sequence-sharded [P][B][N/P][Hx][d]; dst: head-sharded
 * [P][B][Hx/P][N][d]; element type p->dtype.  Hx is the head count of the
 * tensor moved (p->Hq or p->Hkv); Hx % P == 0.  A bit-exact copy.
 * d * element size must be a multiple of 16 bytes.  src and dst must not
 * overlap. */
usp_status usp_a2a_seq2head(const usp_problem* p, int Hx, const void* src, void* dst, usp_stream stream);

/* All-to-all after attention, the inverse of usp_a2a_seq2head (token-local
 * layers then run on the local shard: ultralytics.com "So funktioniert"):
 *   dst[p][b][n'][h][:] = src[h/(Hx/P)][b][h%(Hx/P)][p*N/P + n'][:]
 * src head-sharded, dst sequence-sharded.  Same rules as above. */
usp_status usp_a2a_head2seq(const usp_problem* p, int Hx, const void* src, void* dst, usp_stream stream);

/* Attention forward on head-sharded buffers (every rank, one call):
 *   S_ij = scale * Q_i . K_j ;  causal: keys j > i are masked
 *   O_i  = softmax_j(S_i) V ;   lse_i = ln sum_j exp(S_ij)   (float32)
 * q, o: [P][B][Hq/P][N][d]; k, v: [P][B][Hkv/P][N][d]; lse: [P][B][Hq/P][N].
 * dtype BF16: tensor cores (d = 64 or 128).  dtype F32: float32 CUDA cores.
 * ("Context Parallelism", ultralytics.com: scaled_dot_product_attention with
 * is_causal=True in "Praktische Anwendung und Kompromisse".) */
usp_status usp_attn_fwd(const usp_problem* p, const void* q, const void* k, const void* v, void* o,
                        float* lse, usp_stream stream);

/* Bytes of workspace usp_attn_bwd needs: linear in N, never quadratic: per
 * query row, rows padded to 128-row tiles, 40 bytes (D_i and lse_i*log2(e)
 * as float32, and -lse_i/scale and -D_i each as three bf16 numbers in a
 * 16-byte row) plus the float32 dQ accumulator (4*d bytes).  Returns 0 for an
 * invalid problem. */
size_t usp_attn_bwd_workspace_size(const usp_problem* p);

/* Attention backward on head-sharded buffers (the backward of the glossary
 * page's example, any upstream gradient dO):
 *   P_ij = exp(S_ij - lse_i);  D_i = dO_i . O_i
 *   dV_j = sum_{h in group} sum_i P_ij dO_i
 *   dS_ij = P_ij (dO_i . V_j - D_i)
 *   dQ_i = scale sum_j dS_ij K_j ;  dK_j = scale sum_{h in group} sum_i dS_ij Q_i
 * q, o, dout, dq as q above; k, v, dk, dv as k above; lse from usp_attn_fwd.
 * ws: device workspace of at least usp_attn_bwd_workspace_size(p) bytes,
 * 256-byte aligned; its contents on entry do not matter.  dtype BF16 only
 * (USP_ERR_UNSUPPORTED for F32).
 * One pass over the visible block pairs computes S and dP once per pair: dK
 * and dV accumulate in fixed order (bit-reproducible); each pair's part of
 * dQ is added into a float32 accumulator in the workspace by atomic
 * reductions, whose order varies from run to run, so dQ can differ between
 * runs in its last bf16 bit.  usp_attn_bwd_deterministic gives bit-
 * reproducible results. */
usp_status usp_attn_bwd(const usp_problem* p, const void* q, const void* k, const void* v, const void* o,
                        const float* lse, const void* dout, void* dq, void* dk, void* dv, void* ws,
                        size_t ws_bytes, usp_stream stream);

/* Bytes of workspace usp_attn_bwd_deterministic needs: 40 bytes per query
 * row, rows padded to 128-row tiles (the rows of usp_attn_bwd's workspace,
 * without the dQ accumulator).  Returns 0 for an invalid problem. */
size_t usp_attn_bwd_deterministic_workspace_size(const usp_problem* p);

/* usp_attn_bwd with bit-reproducible results: the same operation, layouts and
 * checks, computed in three passes without atomics (the softmax statistics,
 * then dK and dV per key tile, then dQ per query tile, which computes S and
 * dP a second time).  dK and dV equal usp_attn_bwd's bit for bit; dQ agrees
 * within the rounding of dS to bf16 (the dQ pass forms dS its own way).
 * ws: at least usp_attn_bwd_deterministic_workspace_size(p) bytes, 256-byte
 * aligned. */
usp_status usp_attn_bwd_deterministic(const usp_problem* p, const void* q, const void* k, const void* v,
                                      const void* o, const float* lse, const void* dout, void* dq, void* dk,
                                      void* dv, void* ws, size_t ws_bytes, usp_stream stream);

/* Size of the scratch array built into the library for
 * usp_attn_bwd_noalloc: 64 MiB, enough for B*Hq*roundup(N,128) <= 1.6 Mi
 * query rows at 40 bytes each (e.g. 32 heads of 49 152 tokens): the workspace
 * of usp_attn_bwd_deterministic. */
#define USP_NOALLOC_SCRATCH_BYTES ((size_t)64 << 20)

/* usp_attn_bwd for callers that cannot allocate device memory -- code inside
 * a framework that owns every device allocation, plugins handed no
 * allocator, or code that must not call the allocator once running.  The
 * pages have no counterpart to this entry point; it exists for such callers.
 * Same arguments, layouts and results as usp_attn_bwd_deterministic (whose
 * small workspace suits a fixed array), minus the workspace:
 * the workspace is a file-scope device array of USP_NOALLOC_SCRATCH_BYTES
 * inside the library, held on every GPU that loads it until the process
 * exits.  Nothing is allocated or freed by the call.
 *  - Set-up: the first call on each device looks up the array's device
 *    address (cudaGetSymbolAddress) with that device current; make that first
 *    call before any stream capture.  The address is kept for the life of the
 *    process: after cudaDeviceReset on a device this entry point must not be
 *    called there again (the array may have moved; the same holds for every
 *    entry point, whose device status word is looked up the same way).
 *  - Checks: every argument check of usp_attn_bwd (sizes, d, dtype,
 *    pointers), then the size limit, come before any CUDA call.  Problems
 *    needing more than USP_NOALLOC_SCRATCH_BYTES
 *    (usp_attn_bwd_deterministic_workspace_size) return USP_ERR_WORKSPACE
 *    with nothing enqueued.
 *  - Sharing: every call on a device uses the same array, and the array keeps
 *    the last call's contents (each call rewrites every entry it reads before
 *    reading it).  Calls that can overlap on the GPU -- on different streams,
 *    or from different host threads -- race on the array and must be
 *    serialised by the caller. */
usp_status usp_attn_bwd_noalloc(const usp_problem* p, const void* q, const void* k, const void* v, const void* o,
                                const float* lse, const void* dout, void* dq, void* dk, void* dv,
                                usp_stream stream);

/* Bytes of workspace usp_ring_attn_fwd needs: a float32 running output and a
 * float32 partial output (d values per query row) plus a float32 partial LSE
 * per query row -- linear in N.  The running LSE lives in the caller's lse. */
size_t usp_ring_workspace_size(const usp_problem* p);

/* Ring attention forward on sequence-sharded buffers ("Context
 * Parallelism", ultralytics.com, "So funktioniert Kontextparallelitaet"):
 * for step t = 0..P-1 rank i attends KV block j = (i - t) mod P -- skipped
 * when j > i under the causal mask, masked only when j == i -- and merges the
 * partial into its running result by log-sum-exp (usp_ring_merge).  Passing
 * a KV block to the next rank is an index rotation on one GPU.
 * q, o: [P][B][N/P][Hq][d] bf16; k, v: [P][B][N/P][Hkv][d] bf16;
 * lse: float32 [P][B][N/P][Hq].  ws: at least usp_ring_workspace_size(p)
 * bytes, 256-byte aligned.  dtype BF16, d in {64, 128}. */
usp_status usp_ring_attn_fwd(const usp_problem* p, const void* q, const void* k, const void* v, void* o,
                             float* lse, void* ws, size_t ws_bytes, usp_stream stream);

/* Bytes of workspace usp_ring_attn_bwd needs: 40 bytes per query row of
 * every rank and head (rows padded to 128 per rank: D_i and lse_i*log2(e) as
 * float32, -lse_i/scale and -D_i as three bf16 each), plus float32
 * accumulators for dQ, dK and dV (d values per row) -- linear in N. */
size_t usp_ring_bwd_workspace_size(const usp_problem* p);

/* Ring attention backward on sequence-sharded buffers: the gradients of the
 * causal attention of the whole sequence, computed with the ring schedule of
 * usp_ring_attn_fwd ("Context Parallelism", ultralytics.com, "So funktioniert
 * Kontextparallelitaet": at step t = 0..P-1 rank i holds KV block
 * j = (i - t) mod P, skipped when j > i under the causal mask, masked only
 * when j == i).  Each step adds rank i's partial gradients for the block
 * pair (i, j), taken with the merged LSE of the forward and D_i = dO_i . O_i:
 *   dQ_i += scale sum_j dS_ij K_j   (stays on rank i)
 *   dK_j += scale sum_{h in group} sum_i dS_ij Q_i,  dV_j += sum P_ij dO_i
 *                                   (travel with the KV block)
 * in float32, then rounds once to bf16.  The pages name no ring backward;
 * this is the plain reading that the forward's schedule and the backward of
 * the glossary page's example leave.
 * q, o, dout, dq: [P][B][N/P][Hq][d] bf16; k, v, dk, dv: [P][B][N/P][Hkv][d]
 * bf16; lse: float32 [P][B][N/P][Hq] from usp_ring_attn_fwd.  ws: at least
 * usp_ring_bwd_workspace_size(p) bytes, 256-byte aligned, contents on entry
 * irrelevant.  dtype BF16, d in {64, 128}; Hq % Hkv == 0; N % P == 0. */
usp_status usp_ring_attn_bwd(const usp_problem* p, const void* q, const void* k, const void* v, const void* o,
                             const float* lse, const void* dout, void* dq, void* dk, void* dv, void* ws,
                             size_t ws_bytes, usp_stream stream);

/* ---- all-gather-KV context parallelism ("Context Parallelism",
 * ultralytics.com, "So funktioniert Kontextparallelitaet": the variant in
 * which every rank gathers the whole K and V and attends its own query
 * shard).  On one GPU the gather is one device copy per (rank, batch) chunk
 * into the workspace; the attention of rank i uses global token positions
 * (its queries are tokens i*N/P ..), so causal masking spans shards. */

/* Bytes of workspace usp_allgather_attn_fwd needs: the gathered K and V
 * (bf16, B*N*Hkv*d each) -- linear in N. */
size_t usp_allgather_workspace_size(const usp_problem* p);

/* Forward: o, lse of every rank's query shard against all keys.
 * q, o: [P][B][N/P][Hq][d] bf16; k, v: [P][B][N/P][Hkv][d] bf16; lse: float32
 * [P][B][N/P][Hq].  ws: at least usp_allgather_workspace_size(p) bytes,
 * 256-byte aligned.  dtype BF16, d in {64, 128}; Hq % Hkv == 0; N % P == 0. */
usp_status usp_allgather_attn_fwd(const usp_problem* p, const void* q, const void* k, const void* v, void* o,
                                  float* lse, void* ws, size_t ws_bytes, usp_stream stream);

/* Bytes of workspace usp_allgather_attn_bwd needs: the gathered K and V,
 * 40 bytes per padded query row of every rank and head, and float32 dK, dV
 * accumulators for the whole sequence -- linear in N. */
size_t usp_allgather_bwd_workspace_size(const usp_problem* p);

/* Backward of usp_allgather_attn_fwd: dQ_i from one pass of rank i over the
 * gathered keys; dK and dV as the sum over ranks of each rank's partial over
 * all keys (float32, summed in rank order: the reduce of a reduce-scatter),
 * after which rank j keeps its shard's rows, rounded to bf16 (the scatter).
 * Layouts as in the forward; dout, dq like q; dk, dv like k.  ws: at least
 * usp_allgather_bwd_workspace_size(p) bytes, 256-byte aligned. */
usp_status usp_allgather_attn_bwd(const usp_problem* p, const void* q, const void* k, const void* v, const void* o,
                                  const float* lse, const void* dout, void* dq, void* dk, void* dv, void* ws,
                                  size_t ws_bytes, usp_stream stream);

/* ---- zigzag (load-balanced) ring attention.  Causal ring attention over
 * contiguous shards gives rank i i+1 of the P block pairs; the zigzag layout
 * cuts the sequence into 2P chunks of c = N/(2P) tokens and gives rank r
 * chunks r and 2P-1-r, so that every rank does the same work at every ring
 * step.  The pages describe the ring without a balance; this layout is the
 * plain balanced reading of it.
 * Zigzag-sharded buffers: [P][B][2][c][H][d] -- rank r's shard holds chunk r
 * then chunk 2P-1-r.  Requires N % (2P) == 0 (USP_ERR_INVALID_ARG otherwise). */

/* Contiguous sequence shards ([P][B][N/P][Hx][d], as usp_a2a_seq2head reads)
 * to zigzag shards and back: a permutation of c-token chunks, one device copy
 * each.  dtype gives the element size; src and dst must not overlap. */
usp_status usp_zigzag_shard(const usp_problem* p, int Hx, const void* src, void* dst, usp_stream stream);
usp_status usp_zigzag_unshard(const usp_problem* p, int Hx, const void* src, void* dst, usp_stream stream);

/* Workspace of usp_zigzag_attn_fwd (equal to usp_ring_workspace_size) and of
 * usp_zigzag_attn_bwd (40 bytes per padded query row of every chunk and head,
 * float32 dQ, dK, dV accumulators) -- linear in N; 0 for an invalid problem. */
size_t usp_zigzag_workspace_size(const usp_problem* p);
size_t usp_zigzag_bwd_workspace_size(const usp_problem* p);

/* Zigzag ring forward: at step t = 0..P-1 rank i holds the KV chunks of rank
 * j = (i - t) mod P and attends both of its query chunks to each of them at
 * global positions (pairs wholly in the future are empty), merging every
 * partial by log-sum-exp as usp_ring_attn_fwd does.  q, o, lse, k, v in the
 * zigzag layout (lse: float32 [P][B][2][c][Hq]).  dtype BF16, d in {64, 128}. */
usp_status usp_zigzag_attn_fwd(const usp_problem* p, const void* q, const void* k, const void* v, void* o,
                               float* lse, void* ws, size_t ws_bytes, usp_stream stream);

/* Zigzag ring backward: usp_ring_attn_bwd's accumulation over the same chunk
 * pairs (dK, dV travel with the KV chunks, dQ stays), float32, rounded once
 * to bf16.  Layouts as in the forward. */
usp_status usp_zigzag_attn_bwd(const usp_problem* p, const void* q, const void* k, const void* v, const void* o,
                               const float* lse, const void* dout, void* dq, void* dk, void* dv, void* ws,
                               size_t ws_bytes, usp_stream stream);

/* ---- Ulysses attention with the all-to-all fused into the kernels ("Million-
 * Token-Kontexte im Training", bytewire.ai, "Ulysses: Die Sequenz als
 * Verteilungseinheit": the exchange that gives each rank the whole sequence
 * for its heads).  The attention kernels read Q, K, V and dO and write O, LSE,
 * dQ, dK and dV in place in the sequence-sharded layout: every tile load and
 * every result row addresses token n of a head as row n mod (N/P) of shard
 * n div (N/P), so no remap runs and no head-sharded copy exists.  Results are
 * those of usp_a2a_seq2head -> usp_attn_fwd / usp_attn_bwd -> usp_a2a_head2seq,
 * bit for bit (the same per-head work, tile for tile), except dQ, whose
 * float32 accumulation order varies from run to run in both (see
 * usp_attn_bwd); only the LSE layout differs: float32 [P][B][N/P][Hq], as in
 * ring mode.
 * Preconditions as usp_attn_fwd (Hq % P = Hkv % P = 0, dtype BF16, d in
 * {64, 128}) plus (N/P) % 128 == 0: a 128-row tile never straddles two shards
 * (USP_ERR_UNSUPPORTED otherwise). */
usp_status usp_fused_attn_fwd(const usp_problem* p, const void* q, const void* k, const void* v, void* o,
                              float* lse, usp_stream stream);

/* Bytes of workspace usp_fused_attn_bwd needs (equal to
 * usp_attn_bwd_workspace_size); 0 for an invalid problem. */
size_t usp_fused_attn_bwd_workspace_size(const usp_problem* p);

/* Backward of usp_fused_attn_fwd (the one-pass backward of usp_attn_bwd):
 * q, k, v, o, dout, dq, dk, dv sequence-sharded, lse as the forward wrote it.
 * ws: at least usp_fused_attn_bwd_workspace_size(p) bytes, 256-byte
 * aligned. */
usp_status usp_fused_attn_bwd(const usp_problem* p, const void* q, const void* k, const void* v, const void* o,
                              const float* lse, const void* dout, void* dq, void* dk, void* dv, void* ws,
                              size_t ws_bytes, usp_stream stream);

/* ---- 2-D (hybrid) sequence parallelism: Ulysses inside groups of Pu ranks,
 * ring attention across the Pr = P/Pu groups (the pages name hybrid
 * strategies -- bytewire.ai, "Praktische Implikationen fuer den Einsatz" --
 * and both exchanges: the all-to-all, and the ring of "Context Parallelism",
 * ultralytics.com, "So funktioniert Kontextparallelitaet").
 * Group g holds the contiguous token chunk g of Nc = N/Pr tokens (its ranks
 * g*Pu .. g*Pu + Pu - 1 hold the chunk's Pu shards of N/P tokens).  The
 * all-to-all inside the group gives rank g*Pu + u the heads u*H/Pu ..
 * (u+1)*H/Pu - 1 of the chunk: the hybrid layout [P][B][H/Pu][Nc][d], LSE
 * float32 [P][B][Hq/Pu][Nc].  Pu = P is the Ulysses layout (Pr = 1), Pu = 1
 * per-rank head-major shards of the ring.
 * Every hybrid call: Pu >= 1, P % Pu == 0, Hq % Pu == 0, Hkv % Pu == 0 (else
 * USP_ERR_INVALID_ARG), plus the usp_problem checks without the head split. */

/* Sequence-sharded [P][B][N/P][Hx][d] -> hybrid layout (one Ulysses remap of
 * Nc tokens over Pu ranks per group), and back.  Bit copies, any dtype,
 * d * element size in {64, 128, 256, 512} bytes; src and dst must not
 * overlap. */
usp_status usp_hybrid_seq2head(const usp_problem* p, int Pu, int Hx, const void* src, void* dst, usp_stream stream);
usp_status usp_hybrid_head2seq(const usp_problem* p, int Pu, int Hx, const void* src, void* dst, usp_stream stream);

/* Bytes of workspace usp_hybrid_attn_fwd needs (float32 running and partial
 * outputs and partial LSE, as usp_ring_workspace_size) and usp_hybrid_attn_bwd
 * needs (40 bytes per padded query row of every rank and local head, float32
 * dQ, dK, dV accumulators); 0 for an invalid problem. */
size_t usp_hybrid_workspace_size(const usp_problem* p, int Pu);
size_t usp_hybrid_bwd_workspace_size(const usp_problem* p, int Pu);

/* Hybrid forward on hybrid-layout q, k, v: at ring step t = 0..Pr-1 the ranks
 * of group i attend their heads of chunk i to the same heads' KV of chunk
 * j = (i - t) mod Pr (skipped when j > i under the causal mask), each partial
 * merged by log-sum-exp as usp_ring_attn_fwd does; o (bf16) and lse in the
 * hybrid layout.  dtype BF16, d in {64, 128}; ws 256-byte aligned. */
usp_status usp_hybrid_attn_fwd(const usp_problem* p, int Pu, const void* q, const void* k, const void* v, void* o,
                               float* lse, void* ws, size_t ws_bytes, usp_stream stream);

/* Hybrid backward: usp_ring_attn_bwd's schedule over the groups (dK, dV
 * travel with the KV chunk, dQ stays), float32, rounded once to bf16; every
 * tensor in the hybrid layout, lse as the forward wrote it. */
usp_status usp_hybrid_attn_bwd(const usp_problem* p, int Pu, const void* q, const void* k, const void* v,
                               const void* o, const float* lse, const void* dout, void* dq, void* dk, void* dv,
                               void* ws, size_t ws_bytes, usp_stream stream);

/* Exact merge of two partial attentions over disjoint key sets, float32
 * (the merge step of ring attention):
 *   lse = ln(exp(lse_a) + exp(lse_b))
 *   o   = exp(lse_a - lse) o_a + exp(lse_b - lse) o_b
 * A row with lse = -inf is an empty partial and contributes nothing; two
 * empty rows give lse = -inf and o = 0.
 * o_*: [rows][d]; lse_*: [rows].  o may alias o_a or o_b and lse may alias
 * lse_a or lse_b (element-wise, in place).  d >= 1 and d % 4 == 0. */
usp_status usp_ring_merge(int64_t rows, int d, const float* o_a, const float* lse_a, const float* o_b,
                          const float* lse_b, float* o, float* lse, usp_stream stream);

/* ---- serving: a paged key/value cache, what fills it and what reads it.
 * The paths above attend a whole sequence at once; answering token by token
 * needs the keys and values of the tokens so far.  They are kept in a pool of
 * pages that sequences of any length share, each page page_size tokens of
 * every KV head, head-major:
 *   k_pages, v_pages  [n_pages][Hkv][page_size][d]   (dtype)
 *   page_table        int32 [n_seqs][max_pages]: page j of a sequence holds
 *                     its tokens [j*page_size, (j+1)*page_size)
 * Tokens of a call are rows of ragged batches: q and o are [n_tokens][Hq][d],
 * lse is float32 [n_tokens][Hq] (natural log).  A sequence-sharded tensor
 * [P][B][N/P][H][d] is such a batch of P*B*N/P rows.  Index arrays are int32
 * device arrays, 4-byte aligned; their values are read on the device, so a
 * captured graph replays with new values.  No index value makes a kernel
 * access memory outside the buffers: what an index out of range means is said
 * at each call.
 * Requirements: n_pages, n_seqs, max_pages >= 0; page_size in {16, 32, 64,
 * 128, 256}; Hq, Hkv >= 1 and Hq % Hkv == 0; Hq <= 65535; d in {64, 128};
 * n_seqs and max_pages * page_size <= 2^31 - 1024, n_pages * Hkv < 2^31, and
 * for the attention calls n_seqs <= 2^24 and n_tokens * Hq <= 2^31 - 513, for
 * usp_kv_append n_tokens <= 2^31 - 16. */
typedef struct {
    int n_pages;
    int page_size;
    int n_seqs;
    int max_pages;
    int Hq;
    int Hkv;
    int d;
    int causal;  /* attention: see usp_paged_attn */
    float scale; /* softmax scale, 0: 1/sqrt(d) */
    int dtype;   /* usp_dtype of the pool, q and o */
} usp_cache;

/* Rotary position embedding of q and k, and k and v written into the cache,
 * in one pass.  Token t of sequence s = seq[t], slot p = pos[t], rotation
 * position r = rot_pos[t] (rot_pos NULL: r = p), per head and i < rot/2, with
 * the pair (a, b) = elements (i, i + rot/2), or (2i, 2i+1) if interleaved:
 *   a' = a cos(r f_i) - b sin(r f_i) ;  b' = b cos(r f_i) + a sin(r f_i)
 * with f_i = inv_freq[i] (float32 [rot/2]); elements rot.. pass unchanged.
 * f_i is finite, of either sign.  For |f_i| < 2^24 the angle is off by less
 * than (|f_i| / 2 + 1) |r| 2^-64 turns, then rounded to float32 (a float32
 * product of position 10^6 and f_0 = 1 would be off by up to 0.06 rad); from
 * 2^24 on r f_i and its turns are formed in float64, off by 3 2^-53 of r f_i.
 * The rotation is float32, rounded once.
 *   q_out [n_tokens][Hq][d] = rotated q ;  k_out [n_tokens][Hkv][d] = rotated k
 *   k_pages[page_table[s][p / page_size]][h][p % page_size] = rotated k,
 *   v_pages likewise = v
 * q, k, v: rows of H*d contiguous elements q_stride, k_stride, v_stride
 * elements apart (slices of one projection's output are fine); 16-byte
 * aligned, strides at least the row and a multiple of 16 bytes.
 * q with q_out may both be NULL (no queries), and k_out may be NULL.  q_out
 * may be q and k_out may be k where the stride is the row length (otherwise
 * USP_ERR_INVALID_ARG); no other overlap.  rot: a multiple of 16 with
 * 0 <= rot <= d; 0 rotates nothing (inv_freq may be NULL).
 * A token without a slot -- seq outside [0, n_seqs), pos outside [0,
 * max_pages*page_size), or a page table entry outside [0, n_pages) -- is
 * padding: nothing is written for it, its rows of q_out and k_out stay as
 * they were.  Two tokens of a call must not share a slot (the slot would hold
 * pieces of both). */
usp_status usp_kv_append(const usp_cache* c, int n_tokens, const void* q, int64_t q_stride, const void* k,
                         int64_t k_stride, const void* v, int64_t v_stride, const int32_t* seq, const int32_t* pos,
                         const int32_t* rot_pos, const float* inv_freq, int rot, int interleaved, void* q_out,
                         void* k_out, void* k_pages, void* v_pages, const int32_t* page_table, usp_stream stream);

/* Bytes of workspace usp_paged_attn needs; 0 for an invalid problem. */
size_t usp_paged_attn_workspace_size(const usp_cache* c, int n_tokens, int max_q);

/* Attention of each sequence's newest tokens over its cached keys: decoding
 * (one token each), verification of drafted tokens, further chunks of prompts.
 * Sequence s has n_q = q_start[s+1] - q_start[s] tokens in this call, rows
 * q_start[s] .. of q, and len = seq_lens[s] cached tokens (those of this call
 * included).  Row i of it sees the keys j < vis,
 *   vis = len - n_q + i + 1 (causal)  or  len (not causal: the states of an
 *   encoder, say),
 *   S_j = scale * q . K_j ;  o = softmax_j(S) V ;  lse = ln sum_j exp(S_j)
 * A row that sees no key (len 0, or vis <= 0) gets o = 0 and lse = -inf.
 * q_start: int32 [n_seqs + 1], not decreasing; NULL: one token per sequence
 * (n_tokens == n_seqs).  Rows of no sequence (before q_start[0], from
 * q_start[n_seqs] on) stay as they were.  max_q: the largest n_q (>= 1); it
 * picks the kernel for that many rows, and a wrong value costs speed only.
 * That kernel serves the whole call: sequences with a token each next to one
 * with a long piece of a prompt are faster in a call of their own (32 query
 * and 8 KV heads of 128, 63 sequences of 500 to 8000 tokens and one piece of
 * 512 at 8192: 298 us in one call, 187 and 73 in two).
 * Values out of range: q_start is clamped to [0, n_tokens], seq_lens to [0,
 * max_pages*page_size]; keys of a page table entry outside [0, n_pages) are
 * left out.  What pages hold beyond a sequence's length (NaN, too) never
 * reaches a result (usp_prefix_attn: beyond its length and the prefix).  A
 * value that is not finite in a key or value below len may reach every row of
 * its sequence, masked or not (0 * inf in the product); a NaN in a query makes
 * that row's o and lse NaN.
 * BF16: float32 scores, sums and accumulation, probabilities rounded to bf16
 * for the product with V; F32: float32 throughout, on CUDA cores.  Results do
 * not depend on the run (fixed order of sums).
 * ws: at least usp_paged_attn_workspace_size(c, n_tokens, max_q) bytes,
 * 256-byte aligned, contents on entry irrelevant; calls that can overlap on
 * the GPU need one each. */
usp_status usp_paged_attn(const usp_cache* c, int n_tokens, int max_q, const void* q, const void* k_pages,
                          const void* v_pages, const int32_t* page_table, const int32_t* seq_lens,
                          const int32_t* q_start, void* o, float* lse, void* ws, size_t ws_bytes, usp_stream stream);

/* Bytes of workspace usp_prefix_attn needs; 0 for an invalid problem.  They
 * follow how the prefix is cut and do not grow with n_tokens and prefix_len
 * throughout (bf16, 32 query and 8 KV heads of 128, 32768 shared tokens: 25 MB
 * for 64 tokens, 15 MB for 65): a workspace that is kept for several shapes
 * has the largest of their sizes. */
size_t usp_prefix_attn_workspace_size(const usp_cache* c, int n_tokens, int max_q, int prefix_len);

/* usp_paged_attn for a batch whose sequences share their first prefix_len
 * tokens: those keys and values are read from prefix_pages (int32
 * [ceil(prefix_len/page_size)], pages of the same pool) not once per sequence
 * but once per tile of the batch's rows of a KV head, the tiles side by side,
 * mostly from L2 -- BF16: up to 256 rows, a matrix product on the tensor
 * cores; F32: 8 rows, on CUDA cores -- and joined by log-sum-exp with each
 * sequence's own keys prefix_len .. len-1, which its page table gives as always
 * (entries of whole prefix pages are not read; where the prefix ends inside a
 * page, the sequence's own page holds its tokens from there on).  Masks,
 * lengths (seq_lens counts the prefix), rows and checks as usp_paged_attn,
 * whose results it gives up to rounding; a sequence no longer than the prefix
 * sees that part of it.  The prefix is one piece to all rows of
 * the batch: a value of it that is not finite may reach every row, those of
 * sequences that end before it, too.  0 <= prefix_len <= max_pages*page_size.
 * ws: at least usp_prefix_attn_workspace_size(c, n_tokens, max_q, prefix_len)
 * bytes, 256-byte aligned. */
usp_status usp_prefix_attn(const usp_cache* c, int n_tokens, int max_q, const void* q, const void* k_pages,
                           const void* v_pages, const int32_t* page_table, const int32_t* seq_lens,
                           const int32_t* q_start, const int32_t* prefix_pages, int prefix_len, void* o, float* lse,
                           void* ws, size_t ws_bytes, usp_stream stream);

/* ---- rotary positions with several axes: tokens of an image or a video have a
 * position on each axis (time, height, width), and each pair of a head's
 * elements turns by the position on the pair's own axis. */
#define USP_MAX_AXES 4
typedef struct {
    int n_axes;       /* 1 .. USP_MAX_AXES */
    int rot;          /* rotated elements of a head: a multiple of 16, 0 <= rot <= d */
    int interleaved;  /* pairs are elements (2i, 2i+1), otherwise (i, i + rot/2) */
    uint8_t axis[64]; /* axis of pair i < rot/2, below n_axes (sections one after the other, in turn, any order) */
} usp_rotary;

/* Rotation of the queries and keys of a sequence-sharded batch, in front of any
 * of the attention paths above: token t of the T = B*N of the layout
 * [P][B][N/P], per head and pair i < rot/2 with elements (a, b),
 *   w = pos[axis[i]][t] f_i ;  a' = a cos w - b sin w ;  b' = b cos w + a sin w
 * inverse != 0 turns by -w: the transposed rotation, which is the backward
 * (gradients of the rotated q and k in, those of q and k out).  Angles,
 * frequencies (inv_freq, float32 [rot/2]) and rounding as usp_kv_append;
 * elements rot.. pass unchanged.
 * pos: int32 [n_axes][P][B][N/P].  q, q_out: rows of Hq*d contiguous elements,
 * one per token, q_stride and q_out_stride elements apart; k, k_out likewise
 * of Hkv*d (slices of one projection's output, and of its gradient, are
 * fine); 16-byte aligned, strides at least the row and a multiple of 16
 * bytes.  q with q_out, or k with k_out, may be NULL.  In place (q_out is q,
 * the strides are equal) is fine, no other overlap.  dtype F32 or BF16, d in
 * {64, 128}; B*N <= 2^31 - 16; p->causal, scale and the head split play no part. */
usp_status usp_rotary_embed(const usp_problem* p, const usp_rotary* r, int inverse, const void* q, int64_t q_stride,
                            const void* k, int64_t k_stride, const int32_t* pos, const float* inv_freq, void* q_out,
                            int64_t q_out_stride, void* k_out, int64_t k_out_stride, usp_stream stream);

/* usp_kv_append with several axes: the pairs of token t turn by
 * rot_pos[axis[i]][t] f_i (rot_pos: int32 [n_axes][n_tokens], needed if
 * rot > 0); pos[t] is the token's slot only.  Everything else as there. */
usp_status usp_kv_append_axes(const usp_cache* c, int n_tokens, const void* q, int64_t q_stride, const void* k,
                              int64_t k_stride, const void* v, int64_t v_stride, const int32_t* seq, const int32_t* pos,
                              const int32_t* rot_pos, const float* inv_freq, const usp_rotary* r, void* q_out, void* k_out,
                              void* k_pages, void* v_pages, const int32_t* page_table, usp_stream stream);

/* ---- who holds the pages of a paged cache, and copies of them.
 * The state of a cache is, on the device, the page table, the lengths and
 *   ref  int32 [n_pages]: how many entries of the page table name the page
 *        (entries of a sequence's length), and holds of the caller's own
 * A page whose count is 0 (or below) is free.  Empty: every length and count 0,
 * whatever the table holds.  A caller who adds 1 to a page's count keeps it,
 * unwritten, until that 1 is taken off (pages of a shared prefix, pages that
 * some other cache uses).  Entries outside [0, n_pages) within a length are
 * no pages: they are handed on as they are and not counted.
 * One table serves the pools of all layers: the calls that change it
 * (usp_pages_update, usp_pages_compact) write a list of the copies that are
 * to be made, and usp_pages_copy makes them, in one layer's pools or in many.
 *   copies  int32 [1 + rows][4], 16-byte aligned: row 0 is
 *           {copies, pages lacking, free pages left, 0}, row 1 + i is copy i,
 *           {from, to, tokens, 0}: the first `tokens` tokens of page `from`
 *           to page `to`.  Rows behind the last copy stay as they were.
 * No page of a list is both copied from and copied to.  All index arrays are
 * read on the device (a captured graph replays with new values), results do
 * not depend on the run. */

/* Bytes of workspace usp_pages_update needs (12 per page, 32 per slot and 4 per
 * entry of the table); 0 for an invalid cache. */
size_t usp_pages_update_workspace_size(const usp_cache* c);

/* One step of all slots: forking, reordering, truncating, freeing and growing
 * sequences.  Slot s goes on with the first
 *   kept = min(keep[s], length of a)  tokens of a = parent[s], and has
 *   now  = min(kept + grow[s], max_pages*page_size)  tokens afterwards
 * (parent NULL: a = s; a outside [0, n_seqs): kept = 0; keep NULL: all; grow
 * NULL: 0; negative numbers are 0; lengths are clamped to the table).  All
 * slots begin from the state before the call, so that slots may change places.
 * Whole pages of the kept tokens are shared with every other slot that goes on
 * with them.  A page that ends inside the kept tokens and is about to be
 * written (now > kept) belongs to the slot alone afterwards: if only such slots hold
 * it, the one that held it before (parent[s] == s), otherwise the lowest, keeps
 * it, and every other one gets a page of its own and a copy in the list; if
 * anyone else holds it, all of them do.  New pages -- a slot's copy before its
 * further pages, lower slots first -- are the free ones with the lowest
 * numbers, those that this call frees among them.
 * seq_lens [n_seqs], page_table [n_seqs][max_pages] and ref are updated in
 * place; entries of a slot that are no longer used become -1.  If there are not
 * enough free pages, nothing is changed, no copy is listed, and row 0 of
 * copies tells how many are lacking.  (Pages may then still be shared that an
 * append would write: a caller who does not look, in a captured step say,
 * makes the step's tokens padding where copies[0][1] > 0, seq = -1.)  copies
 * has n_seqs rows after row 0.
 * (Tokens that are appended next have the slots kept .. now - 1; drafts that
 * were refused are dropped by keep, say by usp_verify_drafts' keep_lens.)
 * Between calls seq_lens, page_table and ref are this call's and
 * usp_pages_compact's to change, and ref by the caller's own holds: the pages
 * that a slot gives up are those of its length as the call finds it.
 * ws: at least usp_pages_update_workspace_size(c) bytes, 256-byte aligned,
 * contents on entry irrelevant; calls that can overlap on the GPU need one
 * each.  n_pages <= 2^23. */
usp_status usp_pages_update(const usp_cache* c, const int32_t* parent, const int32_t* keep, const int32_t* grow,
                            int32_t* seq_lens, int32_t* page_table, int32_t* ref, int32_t* copies, void* ws, size_t ws_bytes,
                            usp_stream stream);

/* Brings a pool's n pages in use to its front: pages with numbers from n on, lowest
 * first, are listed to be copied to the free ones below n, lowest first.
 * new_id int32 [n_pages]: a page's number afterwards, -1 if it is free (for
 * numbers that the caller holds elsewhere, as prefix_pages); ref_out the
 * counts afterwards; page_table_out the table with new numbers (entries that
 * name no page in use stay as they are).  page_table_out may be page_table
 * and ref_out may be ref.  copies has n_pages/2 rows after row 0.
 * n_pages <= 2^23. */
usp_status usp_pages_compact(const usp_cache* c, const int32_t* page_table, const int32_t* ref, int32_t* page_table_out,
                             int32_t* ref_out, int32_t* new_id, int32_t* copies, usp_stream stream);

/* Makes the copies of a list of at most max_copies, in k_pages and v_pages of
 * n_layers layers: layer l's pools begin l*layer_stride elements after the
 * pointers (n_layers 1: layer_stride plays no part; more: it is at least a
 * pool's elements and a multiple of 16 bytes).  Rows with a page outside
 * [0, n_pages) are passed over.  What a page holds behind the copied tokens stays as
 * it was. */
usp_status usp_pages_copy(const usp_cache* c, int max_copies, const int32_t* copies, int n_layers, int64_t layer_stride,
                          void* k_pages, void* v_pages, usp_stream stream);

/* Verification of drafted tokens against the target's probabilities, from given
 * random numbers, so that the tokens are distributed as the target's own
 * (speculative sampling).  Sequence s has n = q_start[s+1] - q_start[s] rows t0
 * = q_start[s] .. of the call, the tokens that usp_paged_attn was just given: one that
 * counts already and n - 1 drafts.  Row t of target holds the probabilities of
 * the token after tokens[t]; row t of draft those from which tokens[t] was drawn
 * (rows t0 are not read); draft NULL: drafts that were not drawn (found in the
 * text, say), as if of probability 1.  For t = t0+1, t0+2, ..., x = tokens[t]:
 *   accepted if u[t] * draft[t][x] < target[t-1][x]  (computed exactly; an x
 *   outside [0, vocab) is refused)
 * up to the first draft that is refused, at t = r.  next[s] is drawn from the weights
 *   w_x = max(target[r-1][x] - draft[r][x], 0)  (draft NULL: target[r-1]
 *         without tokens[r]), or target's last row if no draft is refused
 * as the lowest token whose running sum w_0 + .. + w_x exceeds u[t0] sum w.
 * If all w are 0, target's row itself is drawn from; if that is 0 too, next is -1.
 * n_accepted[s]: drafts accepted; keep_lens[s] = seq_lens[s] - (drafts not
 * accepted), the cached tokens that stay (both NULL: not asked for).  A sequence
 * without rows has n_accepted 0, next -1 and keep_lens seq_lens.  keep_lens may
 * be seq_lens where the caller keeps the pages' books; with usp_pages_update it
 * is an array of its own and passed on as keep: that call counts off the pages
 * of the lengths it finds, and those behind a length which something else made
 * shorter would stay counted for ever.
 * For the draw, target and draft are rounded to whole numbers of 2^-46 and summed
 * exactly, in whatever order.  So next can differ from exact arithmetic where
 * u[t0] is within vocab * 2^-47 / sum w of a border between two tokens' shares
 * of sum w (2^-46 where draft is subtracted), half a step of u being 2^-25.
 * "All w are 0" means as rounded: a row below 2^-47 throughout has no token; and
 * where no target[x] is over draft[x] by a step, any token of target's row may
 * come, the refused one among them (rows that add up to 1 and drafts drawn from
 * theirs are refused there with probability vocab * 2^-46 at most).
 * Probabilities are to be in [0, 1] (what lies outside is taken as the nearer
 * end, NaN as 0; NaN refuses a draft), u in [0, 1); rows need not add up to 1.
 * target, draft: [n_tokens] rows of vocab contiguous elements of dtype F32 or
 * BF16, strides in elements, at least vocab.  q_start is clamped to [0,
 * n_tokens].  1 <= vocab <= 2^19; n_seqs <= 2^28 - 1. */
usp_status usp_verify_drafts(int n_seqs, int n_tokens, int vocab, int dtype, const void* target, int64_t target_stride,
                             const void* draft, int64_t draft_stride, const int32_t* tokens, const float* u,
                             const int32_t* q_start, const int32_t* seq_lens, int32_t* n_accepted, int32_t* next,
                             int32_t* keep_lens, usp_stream stream);

/* ---- kernel tracing ----
 * When enabled, every kernel the library launches is bracketed by two CUDA
 * events recorded on the launch's stream (a few microseconds per launch).
 * usp_trace_report() waits for the pending events and accumulates, per
 * kernel name, the launch count and the summed event-to-event milliseconds.
 * Tracing state is process-wide and not meant for concurrent threads. */
typedef struct {
    char name[32];    /* kernel name, e.g. "attn_fwd", "attn_bwd_dkdv", "a2a_seq2head" */
    int64_t launches; /* launches since the last reset */
    double total_ms;  /* summed durations */
} usp_trace_entry;

/* Turn tracing on (on != 0) or off.  Always USP_OK. */
usp_status usp_trace_enable(int on);

/* Drop pending events and accumulated totals.  Always USP_OK. */
usp_status usp_trace_reset(void);

/* Resolve pending events (this synchronises on them) and write up to
 * max_entries totals into out (out may be NULL to query the count).
 * Returns the number of distinct kernel names, or -1 if an event failed. */
int usp_trace_report(usp_trace_entry* out, int max_entries);

/* Synchronises `stream` and reads the device status word that bounded
 * device-side waits write: USP_OK, or USP_ERR_TIMEOUT (the word is then
 * cleared).  USP_ERR_CUDA if the synchronisation itself fails. */
usp_status usp_device_status(usp_stream stream);

/* Failure-detection check, without a fault: enqueues one CTA that waits on a
 * barrier phase nothing completes.  Its bounded wait gives up after the wait
 * limit (2 s), records a timeout in the device status word exactly as a
 * stalled kernel would, and returns.  usp_device_status() then reports
 * USP_ERR_TIMEOUT and clears the word; the context stays usable.  USP_OK once
 * enqueued, USP_ERR_CUDA if the launch fails. */
usp_status usp_diag_wait_timeout(usp_stream stream);

/* Failure-detection check of the attention kernels' abort path, without a
 * fault: enqueues a write of a timeout record into the device status word
 * (if it is clear), as a wait that gave up would.  Every CTA of the kernels
 * enqueued after it then gives up at its first wait that is not already
 * satisfied, waits (bounded) for its own TMA loads and MMAs in flight, frees
 * its TMEM and returns; their outputs are then undefined.
 * usp_device_status() reports USP_ERR_TIMEOUT and clears the word, after
 * which the context runs every path normally.  USP_OK once enqueued,
 * USP_ERR_CUDA if the launch fails. */
usp_status usp_diag_raise_status(usp_stream stream);

/* Static, human-readable name of a status code. */
const char* usp_status_string(usp_status s);

/* Static build description (architecture, version). */
const char* usp_build_info(void);

#ifdef __cplusplus
}
#endif

#endif /* USP_H */
