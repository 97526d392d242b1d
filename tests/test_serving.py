"""The paged key/value cache: appending rotated keys and values, attention over the cache, attention behind a shared
prefix.  Compared with plain float64 evaluations of the definitions (numpy, below), element by element, with bounds
that follow from the roundings:

- one rounding to type t is off by at most u_t = eps_t / 2 of the value (bf16 2^-8, float32 2^-24);
- a score is a float32 sum of d products (the tensor core may truncate: a whole step, 2^-23, per addition), so it is off by
  e <= (d + 4) 2^-23 max_j scale sum_c |q_c k_jc|, which changes a probability by the factor exp(+-2e);
- probabilities are rounded to bf16 for the product with V, and o divides by the sum of the rounded ones:
  o = sum p (1 + x) v / sum p (1 + x), |x| <= u, is off by at most u sum p |v - o| / sum p <= u (sum p|v| + |o|);
- the float32 sums over n keys add (n + 16) 2^-23 of sum p|v|, the result's own rounding u_t |o|.
"""
import math

import numpy as np
import pytest

import context_long_attention_ulysses_gb300 as usp_mod
from context_long_attention_ulysses_gb300 import _lib, build
from tests.guarded import Guarded

U = {"bf16": 2.0 ** -8, "f32": 2.0 ** -24}


# ------------------------------------------------------------------ plain float64 definitions
def ref_rotate(x, r, inv_freq, interleaved):
    """x [T][H][d] float64, r [T], inv_freq float32 [rot/2]; also the sum |a cos| + |b sin| of each element."""
    half = len(inv_freq)
    ang = np.multiply.outer(np.asarray(r, np.float64), inv_freq.astype(np.float64))
    cs, sn = np.cos(ang)[:, None], np.sin(ang)[:, None]
    y, mag = x.copy(), np.abs(x)
    ia = np.arange(0, 2 * half, 2) if interleaved else np.arange(half)
    ib = ia + 1 if interleaved else ia + half
    a, b = x[..., ia], x[..., ib]
    y[..., ia], y[..., ib] = a * cs - b * sn, b * cs + a * sn
    mag[..., ia] = np.abs(a) + np.abs(b)
    mag[..., ib] = mag[..., ia]
    return y, mag


def ref_attention(q, kp, vp, table, lens, q_start, causal, scale, dtype, prefix_pages=None, prefix_len=0):
    """float64 o, lse and their bounds; q [T][Hq][d], pools [n_pages][Hkv][page][d]; rows of no sequence are NaN."""
    T, Hq, d = q.shape
    n_pages, Hkv, page, _ = kp.shape
    g = Hq // Hkv
    cap = table.shape[1] * page
    o, lse = np.full((T, Hq, d), np.nan), np.full((T, Hq), np.nan)
    bo, bl = np.zeros((T, Hq, d)), np.zeros((T, Hq))
    u = U[dtype]
    for s in range(len(lens)):
        t0, t1 = (s, s + 1) if q_start is None else (min(max(int(x), 0), T) for x in q_start[s:s + 2])
        n, ln = t1 - t0, min(max(int(lens[s]), 0), cap)
        if n <= 0:
            continue
        ids = [int(table[s, j // page]) if j >= prefix_len else int(prefix_pages[j // page]) for j in range(ln)]
        ok = np.array([0 <= i < n_pages for i in ids], bool).reshape(-1)
        at = np.array([i if good else 0 for i, good in zip(ids, ok)], np.int64)
        slot = np.arange(ln) % page
        k, v = kp[at, :, slot].astype(np.float64), vp[at, :, slot].astype(np.float64)  # [ln][Hkv][d]
        k[~ok], v[~ok] = 0.0, 0.0
        for i in range(n):
            vis = max(0, ln - n + i + 1) if causal else ln
            see = ok & (np.arange(ln) < vis)
            for h in range(Hq):
                x = scale * (k[:, h // g] @ q[t0 + i, h])
                if not see.any():
                    o[t0 + i, h], lse[t0 + i, h] = 0.0, -np.inf
                    continue
                e = (d + 4) * 2.0 ** -23 * np.max(scale * (np.abs(k[see, h // g]) @ np.abs(q[t0 + i, h])))
                m = x[see].max()
                p = np.where(see, np.exp(np.minimum(x - m, 0.0)), 0.0)
                tot = p.sum()
                o[t0 + i, h] = (p @ v[:, h // g]) / tot
                lse[t0 + i, h] = m + math.log(tot)
                mag = (p @ np.abs(v[:, h // g])) / tot
                up = U["bf16"] if dtype == "bf16" else 0.0
                few = (see.sum() + 16) * 2.0 ** -23
                bo[t0 + i, h] = (up + 2 * e) * (mag + np.abs(o[t0 + i, h])) + few * mag + u * np.abs(o[t0 + i, h])
                bl[t0 + i, h] = 2 * e + few + 2.0 ** -22 * abs(lse[t0 + i, h])
    return o, lse, bo * 1.01, bl * 1.01  # second-order terms


# ------------------------------------------------------------------ inputs
def _np(t):
    return t.detach().float().cpu().numpy().astype(np.float64)


class Batch:
    """A cache with sequences (tokens of this call, cached tokens), unused slots and pages full of NaN."""

    def __init__(self, seqs, Hq, Hkv, d, page, dtype="bf16", causal=True, prefix=0, seed=0, pad=(0, 0), bad=(), spare=3,
                 ragged=None, first_page=0, scale=0.0):
        import torch
        self.torch = torch
        rng = np.random.default_rng(seed)
        gen = torch.Generator().manual_seed(seed)
        self.seqs, self.dtype, self.prefix = seqs, dtype, prefix
        dt = torch.bfloat16 if dtype == "bf16" else torch.float32
        lens = [ln for _, ln in seqs]
        n_prefix = -(-prefix // page)
        mp = max([1, n_prefix] + [-(-ln // page) for ln in lens])
        used = [max(0, -(-ln // page) - prefix // page) for ln in lens]
        n_pages = first_page + sum(used) + n_prefix + spare
        ids = first_page + rng.permutation(n_pages - first_page)
        table = np.full((len(seqs), mp), -1, np.int64)
        at = n_prefix
        live = np.zeros((n_pages - first_page, page), bool)
        for j in range(n_prefix):
            live[ids[j] - first_page, :min(page, prefix - j * page)] = True
        for s, ln in enumerate(lens):
            for j in range(used[s]):
                jj = prefix // page + j
                table[s, jj] = ids[at]
                live[ids[at] - first_page, max(0, prefix - jj * page):max(0, min(page, ln - jj * page))] = True
                at += 1
        for s, j, value in bad:
            table[s, j] = value
        c = dict(n_pages=n_pages, page_size=page, n_seqs=len(seqs), max_pages=mp, Hq=Hq, Hkv=Hkv, d=d, causal=causal,
                 scale=scale, dtype=dtype)
        self.c = usp_mod.Cache(**c)
        body = (n_pages - first_page, Hkv, page, d)
        dead = torch.from_numpy(~live)[:, None, :, None].expand(body)
        self.kp = torch.randn(body, generator=gen).to(dt).masked_fill(dead, float("nan"))
        self.vp = torch.randn(body, generator=gen).to(dt).masked_fill(dead, float("nan"))
        nq = [n for n, _ in seqs]
        T = pad[0] + sum(nq) + pad[1]
        self.T, self.pad = T, pad
        self.q = torch.randn((T, Hq, d), generator=gen).to(dt)
        self.table, self.lens = table.astype(np.int32), np.array(lens, np.int32)
        self.q_start = None
        if ragged if ragged is not None else (any(n != 1 for n in nq) or pad != (0, 0)):
            self.q_start = (pad[0] + np.concatenate([[0], np.cumsum(nq)])).astype(np.int32)
        self.max_q = max([1] + nq)
        self.prefix_pages = ids[:n_prefix].astype(np.int32) if prefix else None
        self.first_page = first_page

    def ref(self):
        kp, vp = _np(self.kp), _np(self.vp)
        off = np.int64(self.first_page)
        table = np.where((self.table >= off) & (self.table < self.c.n_pages), self.table - off, -1)
        pre = None if self.prefix_pages is None else self.prefix_pages - off
        return ref_attention(_np(self.q), np.nan_to_num(kp), np.nan_to_num(vp), table, self.lens, self.q_start,
                             self.c.causal, self.c.softmax_scale, self.dtype, pre, self.prefix)

    def to_gpu(self, usp, guard):
        t = self.torch
        dev = "cuda"

        def put(x):
            y = guard.empty(tuple(x.shape), x.dtype, dev)
            y.copy_(x)
            return y

        def ints(x):
            return None if x is None else put(t.from_numpy(np.ascontiguousarray(x)))

        self.g = dict(q=put(self.q), table=ints(self.table), lens=ints(self.lens), q_start=ints(self.q_start),
                      prefix=ints(self.prefix_pages))
        if self.first_page:
            shape = self.c.pool_shape()
            for name, x in (("kp", self.kp), ("vp", self.vp)):
                pool = t.empty(shape, dtype=x.dtype, device=dev)
                pool[self.first_page:].copy_(x)
                self.g[name] = pool
        else:
            self.g["kp"], self.g["vp"] = put(self.kp), put(self.vp)
        self.g["o"] = guard.empty((self.T, self.c.Hq, self.c.d), self.c.torch_dtype, dev)
        self.g["lse"] = guard.empty((self.T, self.c.Hq), t.float32, dev)
        self.g["o"].fill_(7.0)
        self.g["lse"].fill_(7.0)
        size = usp.usp_prefix_attn_workspace_size(self.c, self.T, self.max_q, self.prefix)
        self.g["ws"] = guard.bytes(size, dev)
        self.g["ws"].fill_(0xFF)  # NaN everywhere: contents on entry do not matter
        return self

    def run(self, usp, stream=None):
        g = self.g
        if self.prefix:
            usp.usp_prefix_attn(self.c, self.T, self.max_q, g["q"], g["kp"], g["vp"], g["table"], g["lens"], g["q_start"],
                                g["prefix"], self.prefix, g["o"], g["lse"], g["ws"], None, stream)
        else:
            usp.usp_paged_attn(self.c, self.T, self.max_q, g["q"], g["kp"], g["vp"], g["table"], g["lens"], g["q_start"],
                               g["o"], g["lse"], g["ws"], None, stream)
        return g["o"], g["lse"]

    def check(self, o=None, lse=None):
        o = _np(self.g["o"] if o is None else o)
        lse = _np(self.g["lse"] if lse is None else lse)
        ro, rl, bo, bl = self.ref()
        rows = ~np.isnan(rl)
        assert (o[~rows] == 7.0).all() and (lse[~rows] == 7.0).all(), "rows of no sequence were written"
        assert np.isfinite(o[rows]).all()
        seen = rows & (rl > -np.inf)
        assert (lse[rows & ~seen] == -np.inf).all() and (o[rows & ~seen] == 0).all()
        err_l = np.abs(lse[seen] - rl[seen]) - bl[seen]
        assert not seen.any() or err_l.max() <= 0, f"lse off by {err_l.max():.3g} over its bound"
        err_o = np.abs(o[seen] - ro[seen]) - bo[seen]
        assert not seen.any() or err_o.max() <= 0, f"o off by {err_o.max():.3g} over its bound"


# ------------------------------------------------------------------ the oracle itself (CPU)
def test_oracle_rotation_is_a_rotation_and_knows_both_pairings():
    rng = np.random.default_rng(0)
    x = rng.standard_normal((3, 2, 64))
    f = (10000.0 ** (-np.arange(16) / 16)).astype(np.float32)
    y, _ = ref_rotate(x, [0, 5, 100000], f, False)
    z, _ = ref_rotate(x, [0, 5, 100000], f, True)
    assert np.array_equal(y[0], x[0]) and np.array_equal(z[0], x[0])
    assert np.array_equal(y[..., 32:], x[..., 32:])
    assert np.allclose(np.hypot(y[..., :16], y[..., 16:32]), np.hypot(x[..., :16], x[..., 16:32]))
    perm = np.concatenate([np.arange(0, 32, 2), np.arange(1, 32, 2), np.arange(32, 64)])
    w, _ = ref_rotate(x[..., perm], [0, 5, 100000], f, False)
    assert np.allclose(w, z[..., perm])


def test_oracle_attention_equals_the_full_sequence_oracle(orc):
    # a prompt of 40 tokens in pages of 16, all its rows in one call, causal: the attention of the whole sequence
    b = Batch([(40, 40)], 4, 2, 64, 16, "f32")
    o, lse, _, _ = b.ref()
    q = np.ascontiguousarray(b.q.numpy().transpose(1, 0, 2))[None]
    k, v = (np.ascontiguousarray(x.numpy()[b.table[0]].transpose(1, 0, 2, 3).reshape(2, -1, 64)[:, :40])[None]
            for x in (b.kp, b.vp))
    want_o, want_l = orc.attn_rows(q, k, v, causal=True)
    assert np.abs(o.transpose(1, 0, 2) - want_o[0]).max() < 1e-12
    assert np.abs(lse.T - want_l[0]).max() < 1e-12


def test_oracle_prefix_equals_tables_that_share_pages():
    b = Batch([(1, 70), (2, 33), (1, 0), (3, 20)], 4, 2, 64, 16, "f32", prefix=32)
    whole = b.table.copy()
    whole[:, :2] = b.prefix_pages
    o1, l1, _, _ = b.ref()
    o2, l2, _, _ = ref_attention(_np(b.q), np.nan_to_num(_np(b.kp)), np.nan_to_num(_np(b.vp)), whole, b.lens, b.q_start,
                                 True, b.c.softmax_scale, "f32")
    assert np.array_equal(o1, o2) and np.array_equal(l1, l2)
    assert np.isneginf(l1[3]).all() and (o1[3] == 0).all()  # the empty slot


# ------------------------------------------------------------------ refusals (no GPU needed)
@pytest.fixture(scope="module")
def lib():
    build.build()
    return _lib.load()


FAKE = 1 << 20


def _c(**kw):
    base = dict(n_pages=10, page_size=16, n_seqs=2, max_pages=4, Hq=4, Hkv=2, d=64)
    base.update(kw)
    return usp_mod.Cache(**base)


def _append(c=None, T=2, q=FAKE, k=FAKE, v=FAKE, seq=FAKE, pos=FAKE, f=FAKE, qo=FAKE, ko=FAKE, kp=FAKE, vp=FAKE, table=FAKE,
            rot=64, **kw):
    usp_mod.usp_kv_append(c or _c(), T, q, k, v, seq, pos, f, qo, ko, kp, vp, table, rot=rot, **kw)


def _paged(c=None, T=2, max_q=1, q=FAKE, kp=FAKE, vp=FAKE, table=FAKE, lens=FAKE, q_start=None, o=FAKE, lse=FAKE, ws=FAKE,
           ws_bytes=1 << 40):
    usp_mod.usp_paged_attn(c or _c(), T, max_q, q, kp, vp, table, lens, q_start, o, lse, ws, ws_bytes)


def _status(call, /, *a, **kw):
    with pytest.raises(usp_mod.UspError) as e:
        call(*a, **kw)
    return e.value.status


@pytest.mark.parametrize("kw,code", [
    (dict(n_pages=-1), 1), (dict(n_seqs=-1), 1), (dict(max_pages=-1), 1), (dict(Hq=0), 1), (dict(Hkv=0), 1),
    (dict(Hq=5), 1), (dict(scale=-1.0), 1), (dict(scale=float("inf")), 1), (dict(scale=float("nan")), 1),
    (dict(page_size=24), 2), (dict(page_size=8), 2), (dict(page_size=512), 2), (dict(d=96), 2),
    (dict(Hq=65536, Hkv=1), 2), (dict(max_pages=1 << 27), 2), (dict(max_pages=(1 << 27) - 63), 2),
    (dict(n_pages=1 << 30, Hkv=4), 2), (dict(n_seqs=(1 << 31) - 1), 2)])
def test_cache_shapes_are_refused(lib, kw, code):
    for f in (_append, _paged):
        assert _status(f, _c(**kw)) == code
    assert usp_mod.usp_paged_attn_workspace_size(_c(**kw), 2, 1) == 0
    assert usp_mod.usp_prefix_attn_workspace_size(_c(**kw), 2, 1, 16) == 0


def test_append_refusals(lib):
    assert lib.usp_kv_append(None, 0, *([None, 0] * 3), None, None, None, None, 0, 0, *([None] * 5), None) == 1
    assert _status(_append, T=-1) == 1
    for rot in (-16, 8, 80):
        assert _status(_append, rot=rot) == 1
    assert _status(_append, q=None) == 1          # q without q_out and the reverse
    assert _status(_append, qo=None) == 1
    for name in ("k", "v", "kp", "vp", "qo", "ko", "q"):
        assert _status(_append, **{name: FAKE + 8}) == 3
    for name in ("k", "v", "kp", "vp", "seq", "pos", "table", "f"):
        assert _status(_append, **{name: 0}) == 3
    for name in ("seq", "pos", "table", "f"):
        assert _status(_append, **{name: FAKE + 2}) == 3
    assert _status(_append, rot_pos=FAKE + 1) == 3
    args = [FAKE, FAKE, None, FAKE, 64, 0, FAKE, FAKE, FAKE, FAKE, FAKE, None]
    cc = _c().c()
    ok = lambda sq, sk, sv: lib.usp_kv_append(cc, 2, FAKE, sq, FAKE, sk, FAKE, sv, *args)  # noqa: E731
    assert ok(255, 128, 128) == 1 and ok(256, 127, 128) == 1 and ok(256, 128, 0) == 1 and ok(256, 132, 128) == 1
    # nothing to do: no token, no sequence, no page
    _append(T=0)
    for kw in (dict(n_seqs=0), dict(n_pages=0), dict(max_pages=0)):
        _append(_c(**kw))


def test_attention_refusals(lib):
    assert lib.usp_paged_attn(None, *([0] * 2), *([None] * 9), 0, None) == 1
    assert _status(_paged, T=-1) == 1 and _status(_paged, max_q=0) == 1
    assert _status(_paged, T=3) == 1                       # one token per sequence, but 3 tokens of 2 sequences
    for name in ("q", "o", "lse", "kp", "vp"):
        assert _status(_paged, **{name: FAKE + 8}) == 3
        assert _status(_paged, **{name: 0}) == 3
    for name in ("table", "lens"):
        assert _status(_paged, **{name: FAKE + 2}) == 3
        assert _status(_paged, **{name: 0}) == 3
    assert _status(_paged, q_start=FAKE + 2) == 3
    assert _status(_paged, ws=FAKE + 128) == 3 and _status(_paged, ws=0) == 3
    size = usp_mod.usp_paged_attn_workspace_size(_c(), 2, 1)
    assert size > 0 and _status(_paged, ws_bytes=size - 1) == 4
    assert _status(_paged, _c(n_seqs=1 << 20, Hq=4096, Hkv=1), T=1 << 20) == 2   # 2^32 rows
    pre = lambda n, pp=FAKE, ws_bytes=1 << 40: usp_mod.usp_prefix_attn(  # noqa: E731
        _c(), 2, 1, FAKE, FAKE, FAKE, FAKE, FAKE, None, pp, n, FAKE, FAKE, FAKE, ws_bytes)
    assert _status(pre, -1) == 1 and _status(pre, 65) == 1 and _status(pre, 64, 0) == 3 and _status(pre, 64, FAKE + 2) == 3
    assert _status(pre, 64, FAKE, usp_mod.usp_prefix_attn_workspace_size(_c(), 2, 1, 64) - 1) == 4
    # nothing to do
    _paged(_c(n_seqs=0), T=0)
    _paged(T=0, q_start=FAKE)
    assert usp_mod.usp_paged_attn_workspace_size(_c(), 0, 1) == 0


def test_helpers_check_tensors():
    import torch
    c = _c()
    with pytest.raises(ValueError):
        usp_mod.paged_attention(c, torch.zeros(2, 4, 64, dtype=torch.bfloat16), None, None, None, None)
    with pytest.raises(ValueError):                      # a float32 tensor where the cache is bf16
        usp_mod._check(c, "q", torch.zeros(2, 4, 64), (2, 4, 64), torch.bfloat16, torch.device("cpu"))
    with pytest.raises(ValueError):
        usp_mod._check(c, "q", torch.zeros(2, 3, 64), (2, 4, 64), torch.float32, torch.device("cpu"))
    with pytest.raises(TypeError):
        usp_mod._check(c, "seq", [0, 1], (2,), torch.int32, torch.device("cpu"))
    assert c.pool_shape() == (10, 2, 16, 64) and c.table_shape() == (2, 4) and c.pages_for(17) == 2
    with pytest.raises(ValueError):
        usp_mod.Cache(1, 16, 1, 1, 1, 1, 64, dtype="fp8").c()


def test_struct_of_a_cache_is_the_callers_own(lib):
    """A changed struct is another cache's: it does not reach the calls of the one it was made from."""
    import copy
    import pickle
    c = _c()
    size = usp_mod.usp_paged_attn_workspace_size(c, 2, 1)
    assert size > 0
    s = c.c()
    s.d, s.causal = 96, 0
    assert usp_mod.usp_paged_attn_workspace_size(s, 2, 1) == 0
    assert usp_mod.usp_paged_attn_workspace_size(c, 2, 1) == size and c.c().d == 64 and c.c().causal == 1
    for other in (copy.copy(c), copy.deepcopy(c), pickle.loads(pickle.dumps(c))):
        assert other == c and usp_mod.usp_paged_attn_workspace_size(other, 2, 1) == size


def test_row_strides_of_a_fused_projection():
    import torch
    x = torch.zeros(5, 8 * 64)
    assert usp_mod._rows(None, 4, 64) == (0, 256)
    with pytest.raises(ValueError):
        usp_mod._rows(x.view(5, 8, 64)[:, :4], 4, 64)    # not a device tensor


# ------------------------------------------------------------------ GPU
@pytest.fixture(scope="module")
def usp():
    import torch
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    build.build()
    return usp_mod


def _done(usp, guard):
    import torch
    torch.cuda.synchronize()
    assert usp.usp_device_status() == 0
    assert guard.damaged() == []


SMALL = [(1, 1), (1, 5), (1, 16), (1, 17), (1, 63), (1, 64), (1, 65), (1, 200), (1, 0), (1, 333)]
APPEND = [("bf16", 4, 2, 64, 64, False), ("bf16", 32, 8, 128, 128, False), ("bf16", 5, 1, 128, 64, True),
          ("f32", 4, 4, 64, 32, True), ("f32", 6, 3, 128, 16, False), ("bf16", 3, 3, 64, 0, False),
          ("f32", 1, 1, 64, 64, False), ("bf16", 12, 4, 128, 112, False), ("bf16", 2, 2, 64, 16, True)]


@pytest.mark.gpu
@pytest.mark.parametrize("dtype,Hq,Hkv,d,rot,inter", APPEND)
@pytest.mark.parametrize("T,page,far", [(1, 16, False), (37, 16, True), (300, 64, False), (2, 256, True)])
def test_append(usp, dtype, Hq, Hkv, d, rot, inter, T, page, far):
    import torch
    rng = np.random.default_rng(T + rot)
    B, mp = 3, 1 + 300 // page
    c = usp.Cache(B * mp + 2, page, B, mp, Hq, Hkv, d, dtype=dtype)
    dt = c.torch_dtype
    guard = Guarded()
    table = rng.permutation(c.n_pages)[:B * mp].reshape(B, mp).astype(np.int32)
    slots = rng.permutation(B * mp * page)[:T]
    seq, pos = (slots // (mp * page)).astype(np.int32), (slots % (mp * page)).astype(np.int32)
    live = np.ones(T, bool)
    if T > 10:  # padding of every kind, and a page that the table does not have
        seq[1], seq[2], pos[3], pos[4], seq[6] = -1, B, -1, mp * page, 1 << 30
        live[[1, 2, 3, 4, 6]] = False
        table[seq[5], pos[5] // page] = c.n_pages
        bad = (seq == seq[5]) & (pos // page == pos[5] // page)
        live &= ~bad
    rpos = (rng.integers(0, 2 ** 31 - 1, T) if far else pos).astype(np.int32)
    gen = torch.Generator().manual_seed(T)
    qkv = torch.randn((T, (Hq + 2 * Hkv) * d), generator=gen).to(dt).cuda()
    q, k, v = (x.view(T, -1, d) for x in qkv.split([Hq * d, Hkv * d, Hkv * d], 1))
    inv = (500000.0 ** (-np.arange(rot // 2) / max(rot // 2, 1))).astype(np.float32)
    dev = lambda x: torch.from_numpy(np.ascontiguousarray(x)).cuda()  # noqa: E731
    kp, vp = (guard.empty(c.pool_shape(), dt, "cuda").fill_(3.0) for _ in range(2))
    qo, ko = guard.empty((T, Hq, d), dt, "cuda").fill_(5.0), guard.empty((T, Hkv, d), dt, "cuda").fill_(5.0)
    usp.usp_kv_append(c, T, q, k, v, dev(seq), dev(pos), dev(inv), qo, ko, kp, vp, dev(table), rot=rot, interleaved=inter,
                      rot_pos=dev(rpos) if far else None)
    _done(usp, guard)
    # float32 cos and sin (a few steps), two products and a sum, one rounding
    for got, x in ((qo, q), (ko, k)):
        want, mag = ref_rotate(_np(x), rpos, inv, inter)
        got = _np(got)
        bound = 8 * 2.0 ** -24 * mag * (rot > 0) + U[dtype] * np.abs(want) * (1 + 2.0 ** -20)
        passed = np.arange(d) >= rot
        bound[..., passed] = 0
        assert (np.abs(got - want)[live] <= bound[live]).all()
        assert (got[~live] == 5.0).all()
    kpn, vpn, kon, vn = _np(kp), _np(vp), _np(ko), _np(v)
    wk, wv = np.full(kpn.shape, 3.0), np.full(vpn.shape, 3.0)
    for t in np.flatnonzero(live):
        at = (table[seq[t], pos[t] // page], slice(None), pos[t] % page)
        wk[at], wv[at] = kon[t], vn[t]
    assert np.array_equal(kpn, wk) and np.array_equal(vpn, wv)
    # without queries and without k_out; in place
    kp2, vp2 = torch.full_like(kp, 3.0), torch.full_like(vp, 3.0)
    usp.usp_kv_append(c, T, None, k, v, dev(seq), dev(pos), dev(inv), None, None, kp2, vp2, dev(table), rot=rot,
                      interleaved=inter, rot_pos=dev(rpos) if far else None)
    q2, k2, v2 = q.contiguous(), k.contiguous(), v.contiguous()
    kp3, vp3 = torch.full_like(kp, 3.0), torch.full_like(vp, 3.0)
    usp.usp_kv_append(c, T, q2, k2, v2, dev(seq), dev(pos), dev(inv), q2, k2, kp3, vp3, dev(table), rot=rot,
                      interleaved=inter, rot_pos=dev(rpos) if far else None)
    _done(usp, guard)
    for a, b in ((kp2, kp), (vp2, vp), (kp3, kp), (vp3, vp)):
        assert torch.equal(a, b)
    m = torch.from_numpy(live).cuda()
    assert torch.equal(q2[m], qo[m]) and torch.equal(k2[m], ko[m])
    assert torch.equal(q2[~m], q[~m]) and torch.equal(k2[~m], k[~m])


def _turns(r, f):
    """r f / 2 pi less whole turns, to the nearest float64: whole-number arithmetic on 400 bits of 1 / 2 pi."""
    bits = 400
    atan_inv = lambda n: sum((-1) ** k * (1 << bits + 64) // ((2 * k + 1) * n ** (2 * k + 1)) for k in range(120))  # noqa: E731
    pi = 16 * atan_inv(5) - 4 * atan_inv(239)                   # Machin's formula, scaled by 2^464
    per_turn = (1 << 2 * bits + 64) // (2 * pi)                 # 1 / 2 pi, scaled by 2^400
    num, den = np.float32(f).item().as_integer_ratio()          # den is a power of two
    x = r * num * per_turn % (den << bits)                      # (Python's %: 0 <= x)
    x = x - (den << bits) if 2 * x >= den << bits else x
    return x / (den << bits)


def test_oracle_turns():
    assert _turns(0, 1.0) == 0.0
    for r, f in ((1, 1.0), (1000, 0.25), (-7, 0.5), (123456, 1e-3), (3, -2.0)):
        t = r * float(np.float32(f)) / (2 * math.pi)
        assert abs(_turns(r, f) - (t - round(t))) < 1e-11
    # the continued fraction of pi: 710 / 113 of 2 pi is 60 times 10^-6 short of whole
    assert abs(_turns(710, 1.0) * 2 * math.pi - (710 - 226 * math.pi)) < 1e-12


FREQ = [1.0, -1.0, 0.0, -0.0, 0.73, 7.9, -7.9, 3.1e-3, 2.0 ** -40, 1.7 * 2.0 ** -41, 1.9 * 2.0 ** -42, 1.1 * 2.0 ** -60,
        -1.3 * 2.0 ** -104, 1.5 * 2.0 ** -106, 2.0 ** -126, 2.0 ** -140, 8.1, 1000.5, -2.0 ** 22 * 1.3, 2.0 ** 23 * 1.9,
        2.0 ** 24, 1.7 * 2.0 ** 24, -1.1 * 2.0 ** 25, 1.3 * 2.0 ** 31]


@pytest.mark.gpu
@pytest.mark.parametrize("inter", [False, True])
def test_append_angles_of_every_size(usp, inter):
    """Frequencies of either sign, zero, subnormal, from far below one to 2^31, at the nearest and the farthest positions:
    cosine and sine themselves, of pairs (1, 0), against angles in whole-number arithmetic."""
    import torch
    r = [0, 1, 2, 3, 710, 1000, 131071, 1 << 20, (1 << 24) + 1, (1 << 30) - 1, (1 << 31) - 1, -1, -710, -(1 << 31)]
    T, half, d = len(r), len(FREQ), 64
    c = usp.Cache(T, 16, T, 1, 1, 1, d, dtype="f32")
    i32 = dict(dtype=torch.int32, device="cuda")
    a = torch.zeros((T, 1, d), device="cuda")
    first = torch.arange(0, 2 * half, 2) if inter else torch.arange(half)
    other = first + 1 if inter else first + half
    a[..., first] = 1.0
    kp, vp = (torch.zeros(c.pool_shape(), device="cuda") for _ in range(2))
    f = np.array(FREQ, np.float32)
    _, k = usp.kv_append(c, None, a, a, torch.arange(T, **i32), torch.zeros(T, **i32), torch.from_numpy(f).cuda(), kp, vp,
                         torch.arange(T, **i32)[:, None].contiguous(), inter, torch.tensor(r, **i32))
    torch.cuda.synchronize()
    k = _np(k)[:, 0]
    turns = np.array([[_turns(ri, fi) for fi in FREQ] for ri in r])
    size, far = np.abs(f.astype(np.float64))[None], np.abs(np.array(r, np.float64))[:, None]
    # the angle, in radians: the fixed-point product or the three roundings in float64; whole 2^-31 half-turns and the rounding of
    # up to one half-turn to float32.  Then sine and cosine, two steps of a value up to 1.
    angle = np.where(size < 2.0 ** 24, 2 * math.pi * (size / 2 + 1) * far * 2.0 ** -64, 3 * 2.0 ** -53 * size * far)
    bound = angle * (1 + 2.0 ** -20) + math.pi * (2.0 ** -31 + 2.0 ** -24) + 2 * 2.0 ** -23
    assert (np.abs(k[:, first] - np.cos(2 * math.pi * turns)) <= bound).all()
    assert (np.abs(k[:, other] - np.sin(2 * math.pi * turns)) <= bound).all()
    assert (k[:, 2 * half:] == 0).all()


PAGED = [  # seqs, Hq, Hkv, d, page, dtype, more
    (SMALL, 4, 4, 64, 16, {}),
    (SMALL, 32, 8, 128, 64, {}),
    (SMALL, 8, 1, 128, 32, {}),
    (SMALL, 5, 1, 64, 128, {}),
    (SMALL, 32, 2, 128, 256, {}),
    (SMALL, 24, 1, 64, 64, {}),                                                     # 24 rows of one token
    (SMALL, 70, 1, 128, 64, {}),
    ([(1, 1)], 1, 1, 64, 16, {}),
    ([(1, 3000)], 8, 2, 128, 64, {}),
    ([(1, 2500)], 4, 4, 64, 16, {}),
    ([(1, 700 + 37 * i) for i in range(40)], 4, 2, 64, 32, {}),
    ([(0, 10), (2, 40), (5, 5), (3, 1), (1, 0), (4, 130), (7, 64)], 8, 2, 128, 32, {}),   # rows that see nothing
    ([(3, 100), (2, 2), (9, 300)], 4, 1, 64, 64, dict(pad=(2, 3))),
    ([(40, 40), (33, 700), (1, 90)], 8, 2, 128, 64, {}),
    ([(150, 400), (3, 20)], 8, 2, 64, 32, dict(pad=(1, 1))),
    ([(70, 70)], 3, 3, 128, 16, {}),
    ([(300, 1000), (0, 5), (260, 260)], 4, 1, 128, 128, {}),
    ([(140, 100), (90, 0)], 6, 2, 64, 256, {}),                                      # more tokens than keys
    ([(20, 300), (100, 90)], 4, 2, 128, 64, dict(causal=False)),
    (SMALL, 8, 2, 128, 64, dict(causal=False)),
    (SMALL, 4, 4, 128, 32, dict(scale=0.3)),
    ([(1, 100), (1, 100), (2, 200)], 4, 2, 64, 16, dict(bad=((0, 2, -1), (1, 0, 1 << 30), (2, 12, -7), (0, 6, 99999)))),
    ([(1, 30), (60, 260)], 8, 2, 128, 64, dict(bad=((0, 0, -1), (1, 1, 1 << 30), (1, 4, -2)))),
]


@pytest.mark.gpu
@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("case", range(len(PAGED)))
def test_paged_attention(usp, case, dtype):
    seqs, Hq, Hkv, d, page, more = PAGED[case]
    guard = Guarded()
    b = Batch(seqs, Hq, Hkv, d, page, dtype, seed=case, **more).to_gpu(usp, guard)
    b.run(usp)
    _done(usp, guard)
    b.check()
    o, lse = b.g["o"].clone(), b.g["lse"].clone()
    b.g["ws"].fill_(0)
    b.run(usp)
    _done(usp, guard)
    assert b.torch.equal(o, b.g["o"]) and b.torch.equal(lse, b.g["lse"])    # the order of sums is fixed


PREFIX = [
    ([(1, 40), (1, 33), (1, 32), (1, 64), (1, 100)], 4, 4, 64, 16, 32, {}),
    ([(1, 1000 + i) for i in range(1, 20)], 32, 8, 128, 64, 1000, {}),               # the prefix ends inside a page
    ([(1, 129), (1, 500)], 8, 2, 128, 64, 128, {}),
    ([(1, 70), (1, 20), (1, 0), (1, 64)], 8, 2, 128, 16, 64, {}),                    # shorter than the prefix, empty slots
    ([(2, 300), (3, 290), (1, 280), (4, 260)], 8, 2, 64, 32, 256, {}),
    ([(2, 300), (0, 290), (9, 201), (4, 203)], 4, 1, 128, 32, 200, dict(pad=(2, 5))),
    ([(1, 400 + i) for i in range(70)], 8, 1, 128, 64, 399, {}),                     # 560 rows of one KV head
    ([(1, 150 + i % 3) for i in range(33)], 4, 1, 64, 128, 150, {}),
    ([(60, 500), (30, 430)], 8, 2, 128, 64, 420, {}),
    ([(60, 500), (200, 430)], 4, 2, 64, 64, 420, {}),                                # rows that see part of the prefix
    ([(2, 90), (3, 80)], 4, 2, 128, 16, 80, dict(causal=False)),
    ([(1, 20)], 1, 1, 64, 16, 17, {}),
    ([(1, 300), (1, 310)], 4, 2, 64, 16, 290, dict(bad=((0, 18, -1), (1, 18, 1 << 29)))),
]


@pytest.mark.gpu
@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("case", range(len(PREFIX)))
def test_prefix_attention(usp, case, dtype):
    seqs, Hq, Hkv, d, page, prefix, more = PREFIX[case]
    guard = Guarded()
    b = Batch(seqs, Hq, Hkv, d, page, dtype, seed=case, prefix=prefix, **more).to_gpu(usp, guard)
    b.run(usp)
    _done(usp, guard)
    b.check()
    o, lse = b.g["o"].clone(), b.g["lse"].clone()
    b.run(usp)
    _done(usp, guard)
    assert b.torch.equal(o, b.g["o"]) and b.torch.equal(lse, b.g["lse"])


@pytest.mark.gpu
@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("d", [64, 128])
@pytest.mark.parametrize("n", [1, 6, 30, 70])
def test_scores_that_grow_along_the_keys(usp, n, d, dtype):
    """Keys that grow with their position: the running maximum keeps rising, and what is summed so far is scaled down
    again and again, tile after tile."""
    import torch
    guard = Guarded()
    b = Batch([(n, 1900), (n, 700), (n, n)], 8, 2, d, 64, dtype, seed=n)
    for s, ln in enumerate(b.lens):
        for j in range(-(-int(ln) // 64)):
            b.kp[int(b.table[s, j])] *= (1 + (torch.arange(64) + 64 * j) / 48).to(b.kp.dtype)[None, :, None]
    b.to_gpu(usp, guard).run(usp)
    _done(usp, guard)
    b.check()


@pytest.mark.gpu
@pytest.mark.parametrize("d", [64, 128])
def test_short_pieces_of_many_rows(usp, d):
    """Pieces of a tile or two, whose values arrive late: nothing may be taken for the product before it.  The memory is
    cold and busy in every second run; all runs have the same bits."""
    import torch
    guard = Guarded()
    b = Batch([(10, 1206), (6, 878), (9, 300), (20, 140)], 128, 8, d, 16, pad=(2, 1)).to_gpu(usp, guard)
    b.run(usp)
    _done(usp, guard)
    b.check()
    o, lse = b.g["o"].clone(), b.g["lse"].clone()
    noise, side = torch.empty(1 << 28, dtype=torch.uint8, device="cuda"), torch.cuda.Stream()
    for i in range(60):
        b.g["o"].fill_(7.0)
        if i % 2:
            side.wait_stream(torch.cuda.current_stream())
            with torch.cuda.stream(side):
                noise.add_(1)
        b.run(usp)
        torch.cuda.current_stream().wait_stream(side)
        assert torch.equal(b.g["o"], o) and torch.equal(b.g["lse"], lse), i
    _done(usp, guard)


@pytest.mark.gpu
@pytest.mark.parametrize("max_q", [1, 4, 1000])
def test_max_q_is_a_hint(usp, max_q):
    """A wrong max_q costs speed, never results."""
    guard = Guarded()
    b = Batch([(5, 300), (1, 70), (30, 40)], 8, 2, 128, 64)
    b.max_q = max_q
    b.to_gpu(usp, guard)
    b.run(usp)
    _done(usp, guard)
    b.check()


@pytest.mark.gpu
@pytest.mark.parametrize("prefix", [0, 100])
def test_lengths_and_starts_out_of_range_stay_inside(usp, prefix):
    """seq_lens and q_start far out of range are clamped; whatever they say, only o, lse and ws are written."""
    import torch
    guard = Guarded()
    b = Batch([(1, 150), (1, 160), (2, 130)], 8, 2, 128, 64, prefix=prefix, ragged=True).to_gpu(usp, guard)
    b.g["lens"].copy_(torch.tensor([1 << 30, -5, 160], dtype=torch.int32))
    b.g["q_start"].copy_(torch.tensor([-100, 1, 2, 1 << 30], dtype=torch.int32))
    b.run(usp)
    _done(usp, guard)
    b.g["q_start"].copy_(torch.tensor([4, 1, 1 << 30, -3], dtype=torch.int32))
    b.run(usp)
    _done(usp, guard)


@pytest.mark.gpu
@pytest.mark.parametrize("dtype", ["bf16", "f32"])
def test_decoding_steps_between_other_work(usp, dtype):
    """A whole decoding step, with tensor operations before, between and after the calls (each call reads what the one
    before it wrote, and the step after overwrites it): eager steps, and one captured step replayed, give the same bits as
    steps that are waited for one by one."""
    import torch
    B, Hq, Hkv, d, page, steps = 5, 8, 2, 64, 16, 12
    c = usp.Cache(B * 8, page, B, 8, Hq, Hkv, d, dtype=dtype)
    i32 = dict(dtype=torch.int32, device="cuda")
    gen = torch.Generator().manual_seed(1)
    table = torch.randperm(c.n_pages, generator=gen).int().view(B, 8).cuda()
    x = torch.randn((steps, B, (Hq + 2 * Hkv) * d), generator=gen).to(c.torch_dtype).cuda()
    inv = (10000.0 ** (-torch.arange(d // 2, dtype=torch.float64) / (d // 2))).float().cuda()
    pre = table[0, :1].contiguous()
    ws = torch.empty(usp.usp_prefix_attn_workspace_size(c, B, 1, page), dtype=torch.uint8, device="cuda")

    class Run:
        def __init__(self):
            self.kp, self.vp = (torch.zeros(c.pool_shape(), dtype=c.torch_dtype, device="cuda") for _ in range(2))
            self.pos, self.seq = torch.full((B,), page + 3, **i32), torch.arange(B, **i32)
            self.x, self.o = torch.zeros_like(x[0]), torch.zeros((B, Hq, d), dtype=c.torch_dtype, device="cuda")
            self.q, self.lse = torch.zeros_like(self.o), torch.zeros((B, Hq), device="cuda")
            self.total = torch.zeros((B, Hq, d), device="cuda")

        def step(self, wait=False):
            sync = torch.cuda.synchronize if wait else lambda: None
            y = self.x + self.o.view(B, -1).repeat(1, 2)[:, :self.x.shape[1]]        # the answer before goes into this token
            sync()
            q, k, v = (t.view(B, -1, d) for t in y.split([Hq * d, Hkv * d, Hkv * d], 1))
            usp.usp_kv_append(c, B, q, k, v, self.seq, self.pos, inv, self.q, None, self.kp, self.vp, table, rot=d)
            sync()
            self.pos += 1
            sync()
            usp.usp_paged_attn(c, B, 1, self.q, self.kp, self.vp, table, self.pos, None, self.o, self.lse, ws)
            sync()
            self.total += self.o.float()
            sync()
            usp.usp_prefix_attn(c, B, 1, self.o, self.kp, self.vp, table, self.pos, None, pre, page, self.q, self.lse, ws)
            usp.usp_paged_attn(c, B, 1, self.q, self.kp, self.vp, table, self.pos, None, self.o, self.lse, ws)
            sync()
            self.total += self.o.float()

    runs = []
    for kind in ("waited", "eager", "graph"):
        r = Run()
        if kind == "graph":
            s = torch.cuda.Stream()
            s.wait_stream(torch.cuda.current_stream())
            warm = Run()
            with torch.cuda.stream(s):
                warm.step()
            s.synchronize()
            g = torch.cuda.CUDAGraph()
            with torch.cuda.graph(g, stream=s):
                r.step()
        for i in range(steps):
            r.x.copy_(x[i])
            g.replay() if kind == "graph" else r.step(kind == "waited")
        torch.cuda.synchronize()
        assert usp.usp_device_status() == 0
        runs.append((r.total, r.kp, r.vp, r.lse))
    assert torch.isfinite(runs[0][0]).all() and runs[0][0].abs().max() > 0
    for other in runs[1:]:
        for a, b in zip(runs[0], other):
            assert torch.equal(a, b)


@pytest.mark.gpu
@pytest.mark.parametrize("prefix", [0, 500])
def test_captured_graph_replays_with_new_lengths(usp, prefix):
    """One capture serves every later step: tables, lengths and starts are read on the device."""
    import torch
    guard = Guarded()
    long = Batch([(1, 600), (1, 650), (1, 520)], 8, 2, 128, 64, prefix=prefix, seed=1).to_gpu(usp, guard)
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(s):
        long.run(usp)
    s.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph, stream=s):
        long.run(usp)
    for lens in ([600, 650, 520], [1, 0, 519], [555, 64, 501], [600, 650, 520]):
        long.lens = np.array(lens, np.int32)
        long.g["lens"].copy_(torch.from_numpy(long.lens))
        long.g["o"].fill_(7.0)
        graph.replay()
        _done(usp, guard)
        long.check()


@pytest.mark.gpu
@pytest.mark.parametrize("prefix", [0, 300])
@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("n", [1, 6, 20, 70])
def test_nan_of_a_query_or_key_shows(usp, n, dtype, prefix):
    """A NaN in a row of q makes that row's output and log-sum-exp NaN, a NaN in a key those of the rows that see it
    (and no other sequence's, nor another KV head's); nothing turns it into zeros.  Other rows keep their bits."""
    import torch
    guard = Guarded()
    b = Batch([(n, 3000), (n, 400), (n, prefix + n)], 8, 2, 128, 64, dtype, prefix=prefix).to_gpu(usp, guard)
    o, lse = (x.clone() for x in b.run(usp))
    _done(usp, guard)
    b.check()
    last = torch.zeros((b.T, 8), dtype=torch.bool, device="cuda")
    last[n - 1, 1] = last[2 * n - 1, 6] = last[3 * n - 1, 0] = True
    b.g["q"][last] = float("nan")
    for y, was in zip(b.run(usp), (o, lse)):
        _done(usp, guard)
        assert torch.isnan(y[last]).all()
        assert torch.equal(y[~last], was[~last])
    b.g["q"].copy_(b.q)
    page, at = b.table[1, 399 // 64], 399 % 64  # the last key of the second sequence, seen by its last token only
    b.g["kp"][int(page), 1, at, 5] = float("nan")
    hit = torch.zeros_like(last)
    hit[2 * n - 1, 4:] = True
    for y, was in zip(b.run(usp), (o, lse)):
        _done(usp, guard)
        assert torch.isnan(y[hit]).all()
        others = torch.ones_like(last)
        others[n:2 * n, 4:] = False
        assert torch.equal(y[others], was[others])


@pytest.mark.gpu
@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("n", [1, 6, 70])
def test_infinite_value_of_a_prefix(usp, n, dtype):
    """An infinity among the prefix's values reaches that column of that KV head only: there the rows that see it, and
    perhaps those of a sequence that ends before it.  Everything else keeps its bits, and what the pages hold beyond
    lengths and prefix (NaN in every test) still reaches nothing."""
    import torch
    guard = Guarded()
    b = Batch([(n, 700), (n, 290), (n, 350), (n, 60 + n)], 8, 2, 128, 64, dtype, prefix=300).to_gpu(usp, guard)
    o, lse = (x.clone() for x in b.run(usp))
    _done(usp, guard)
    b.check()
    key = 295                                                       # the second and the fourth sequence end before it
    b.g["vp"][int(b.prefix_pages[key // 64]), 1, key % 64, 9] = float("inf")
    b.run(usp)
    _done(usp, guard)
    assert torch.equal(b.g["lse"], lse)
    hit = torch.zeros_like(o, dtype=torch.bool)
    hit[:, 4:, 9] = True
    assert torch.equal(b.g["o"][~hit], o[~hit])
    last = b.g["o"][[n - 1, 3 * n - 1], 4:, 9]                      # the newest token of the others sees it
    assert not torch.isfinite(last).any()
    short = b.g["o"][[*range(n, 2 * n), *range(3 * n, 4 * n)], 4:, 9]
    was = o[[*range(n, 2 * n), *range(3 * n, 4 * n)], 4:, 9]
    assert (torch.isnan(short) | (short == was)).all()


@pytest.mark.gpu
def test_captured_fork_and_join(usp):
    """A captured step whose appending runs on a stream of its own beside other work, and whose attention waits for both."""
    import torch
    guard = Guarded()
    b = Batch([(1, 600), (1, 650), (1, 520)], 8, 2, 128, 64, seed=3).to_gpu(usp, guard)
    g, c = b.g, b.c
    k, v = (torch.empty((3, 2, 128), dtype=torch.bfloat16, device="cuda") for _ in range(2))
    pos, seq = g["lens"] - 1, torch.arange(3, dtype=torch.int32, device="cuda")
    for s in range(3):  # the newest key and value of each sequence arrive through the graph
        page, at = int(b.table[s, (b.lens[s] - 1) // 64]), int(b.lens[s] - 1) % 64
        k[s], v[s] = g["kp"][page, :, at], g["vp"][page, :, at]
        g["kp"][page, :, at] = g["vp"][page, :, at] = float("nan")
    q_in = g["q"].clone()
    b.run(usp)  # (before any capture: the library makes its status word with the first call)
    g["q"].zero_()
    main, side = torch.cuda.Stream(), torch.cuda.Stream()
    torch.cuda.synchronize()

    def step():
        side.wait_stream(main)
        usp.usp_kv_append(c, 3, None, k, v, seq, pos, None, None, None, g["kp"], g["vp"], g["table"], stream=side)
        g["q"].copy_(q_in)
        main.wait_stream(side)
        b.run(usp)
        side.wait_stream(main)
        main.wait_stream(side)

    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph, stream=main):
        step()
    for _ in range(3):
        g["o"].fill_(7.0)
        graph.replay()
        _done(usp, guard)
        b.check()


@pytest.mark.gpu
def test_traced_calls_give_the_same_bits(usp):
    """Events between the launches, which then no longer overlap: the same results, and each launch on record."""
    import torch
    guard = Guarded()
    bs = [Batch([(n, 900 + 100 * i) for i in range(5)], 8, 2, 128, 64, seed=n, prefix=p).to_gpu(usp, guard)
          for n, p in ((1, 0), (1, 640), (70, 0))]
    plain = [tuple(x.clone() for x in b.run(usp)) for b in bs]
    _done(usp, guard)
    usp.usp_trace_reset()
    usp.usp_trace_enable(True)
    try:
        for b, (o, lse) in zip(bs, plain):
            b.g["o"].fill_(7.0)
            b.run(usp)
            _done(usp, guard)
            assert torch.equal(b.g["o"], o) and torch.equal(b.g["lse"], lse)
        seen = {name: launches for name, (launches, _) in usp.usp_trace_report().items()}
    finally:
        usp.usp_trace_enable(False)
        usp.usp_trace_reset()
    assert seen == {"paged_own": 3, "paged_prefix": 1, "paged_merge": 3}


@pytest.mark.gpu
def test_two_streams_at_once(usp):
    import torch
    guard = Guarded()
    bs = [Batch([(1, 900 + 100 * i + j) for j in range(5)], 8, 2, 128, 64, seed=i, prefix=p).to_gpu(usp, guard)
          for i, p in enumerate((0, 640, 0, 320))]
    streams = [torch.cuda.Stream() for _ in bs]
    torch.cuda.synchronize()
    for _ in range(20):
        for b, s in zip(bs, streams):
            b.run(usp, s)
    _done(usp, guard)
    for b in bs:
        b.check()


@pytest.mark.gpu
@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("prefix", [0, 16])
def test_without_pages_no_row_sees_a_key(usp, dtype, prefix):
    """A pool, or a page table, of size zero: every row is empty, and no pool pointer is needed."""
    import torch
    i32 = dict(dtype=torch.int32, device="cuda")
    for kw in (dict(n_pages=0, max_pages=4), dict(n_pages=3, max_pages=0)):
        if prefix > kw["max_pages"] * 16:
            continue
        c = usp.Cache(page_size=16, n_seqs=2, Hq=4, Hkv=2, d=64, dtype=dtype, **kw)
        q = torch.ones((2, 4, 64), dtype=c.torch_dtype, device="cuda")
        o, lse = torch.full_like(q, 7.0), torch.full((2, 4), 7.0, device="cuda")
        table = torch.zeros((2, max(kw["max_pages"], 1)), **i32)
        ws = torch.empty(usp.usp_prefix_attn_workspace_size(c, 2, 1, prefix), dtype=torch.uint8, device="cuda")
        usp.usp_prefix_attn(c, 2, 1, q, None, None, table, torch.tensor([30, 1], **i32), None, table, prefix, o, lse, ws)
        torch.cuda.synchronize()
        assert usp.usp_device_status() == 0
        assert (o == 0).all() and (lse == -math.inf).all()


@pytest.mark.gpu
def test_many_sequences_and_many_short_ones(usp):
    """More sequences than a CTA has threads, most of a tile or less, some empty, one long."""
    guard = Guarded()
    rng = np.random.default_rng(5)
    seqs = [(1, int(n)) for n in rng.integers(0, 40, 1000)]
    seqs[617] = (1, 3000)
    for dtype, Hq, Hkv in (("bf16", 4, 4), ("f32", 2, 1)):
        b = Batch(seqs, Hq, Hkv, 64, 16, dtype).to_gpu(usp, guard)
        b.run(usp)
        _done(usp, guard)
        b.check()
    b = Batch([(int(n % 3), int(n)) for n in rng.integers(0, 40, 700)] + [(90, 500)], 4, 2, 64, 16).to_gpu(usp, guard)
    b.run(usp)
    _done(usp, guard)
    b.check()


@pytest.mark.gpu
def test_wide_tables_and_idle_slots(usp):
    """A serving batch keeps rows for sequences that are not there: their table rows may hold anything."""
    import torch
    guard = Guarded()
    b = Batch([(1, 200), (1, 0), (1, 77), (1, 0)], 8, 2, 128, 64)
    wide = np.full((4, 500), 1 << 30, np.int64)
    wide[:, :b.table.shape[1]] = np.where(b.table < 0, 12345678, b.table)
    b.table = wide.astype(np.int32)
    import dataclasses
    b.c = dataclasses.replace(b.c, max_pages=500)
    b.to_gpu(usp, guard)
    b.run(usp)
    _done(usp, guard)
    b.check()


def test_append_in_place_needs_rows_without_gaps(lib):
    cc, far = _c().c(), FAKE + (1 << 16)
    tail = [FAKE, FAKE, None, FAKE, 64, 0]

    def status(T, q, sq, k, sk, qo, ko):
        return lib.usp_kv_append(cc, T, q, sq, k, sk, far, 512, *tail, qo, ko, far, far, FAKE + 2, None)  # (bad table: 3)

    for T in (2, 7):
        assert status(T, FAKE, 512, FAKE, 128, FAKE, far) == 1 and status(T, FAKE, 256, FAKE, 512, far, FAKE) == 1
        assert status(T, FAKE, 256, FAKE, 128, FAKE, FAKE) == 3 and status(T, FAKE, 512, FAKE, 512, far, far) == 3
    assert status(1, FAKE, 512, FAKE, 512, FAKE, FAKE) == 3       # one token: no stride


def test_append_refuses_more_tokens_than_its_grid_can_count(lib):
    for T in ((1 << 31) - 1, (1 << 31) - 15):
        assert _status(_append, T=T) == 2
        assert _status(_append, _c(Hq=64, Hkv=64), T=T) == 2


def test_attention_refuses_more_sequences_than_a_warp_passes_over_in_time(lib):
    c = _c(n_seqs=(1 << 24) + 1)
    assert _status(_paged, c, q_start=FAKE) == 2
    assert usp_mod.usp_paged_attn_workspace_size(c, 2, 1) == 0
    assert usp_mod.usp_prefix_attn_workspace_size(c, 2, 1, 16) == 0
    assert usp_mod.usp_paged_attn_workspace_size(_c(n_seqs=1 << 24), 2, 1) > 0


def _few_live(usp, B, Hq, Hkv, d, dtype, live, ragged, prefix=0):
    """B sequences of which those of `live` (index -> cached tokens) hold something, one token each; the others are idle
    slots (or, ragged, sequences without a token in this call): o and lse of the live ones against the formula."""
    import torch
    page, mp = 16, max(-(-n // 16) for n in live.values())
    n_pages = mp * len(live)
    c = usp.Cache(n_pages, page, B, mp, Hq, Hkv, d, dtype=dtype)
    gen = torch.Generator().manual_seed(B)
    kp, vp = (torch.randn(c.pool_shape(), generator=gen).to(c.torch_dtype).cuda() for _ in range(2))
    i32 = dict(dtype=torch.int32, device="cuda")
    table, lens = torch.full((B, mp), -1, **i32), torch.zeros(B, **i32)
    at = torch.tensor(sorted(live), device="cuda")
    table[at] = torch.randperm(n_pages, generator=gen).int().view(len(live), mp).cuda()
    lens[at] = torch.tensor([live[b] for b in sorted(live)], **i32)
    T, start, rows = B, None, at
    if ragged:
        T, rows = len(live), torch.arange(len(live), device="cuda")
        n = torch.zeros(B, dtype=torch.int64, device="cuda")
        n[at] = 1
        start = torch.cat([torch.zeros(1, **i32), n.cumsum(0).int()])
    qn = torch.randn((len(live), Hq, d), generator=gen).to(c.torch_dtype)
    q = torch.zeros((T, Hq, d), dtype=c.torch_dtype, device="cuda")
    q[rows] = qn.cuda()
    o, lse = torch.full_like(q, 7.0), torch.full((T, Hq), 7.0, device="cuda")
    pre = table[at[0]].contiguous() if prefix else None
    ws = torch.empty(usp.usp_prefix_attn_workspace_size(c, T, 1, prefix), dtype=torch.uint8, device="cuda")
    usp.usp_prefix_attn(c, T, 1, q, kp, vp, table, lens, start, pre, prefix, o, lse, ws)
    torch.cuda.synchronize()
    assert usp.usp_device_status() == 0
    ro, rl, bo, bl = ref_attention(_np(qn), _np(kp), _np(vp), table[at].cpu().numpy(), lens[at].cpu().numpy(), None, True,
                                   c.softmax_scale, dtype, None if pre is None else pre.cpu().numpy(), prefix)
    assert (np.abs(_np(o[rows]) - ro) <= bo).all() and (np.abs(_np(lse[rows]) - rl) <= bl).all()
    if not ragged:
        idle = torch.ones(B, dtype=torch.bool, device="cuda")
        idle[at] = False
        assert not o[idle].any() and (lse[idle] == -math.inf).all()


@pytest.mark.gpu
def test_a_quarter_million_idle_slots(usp):
    """Idle slots between two sequences are passed over in no time: at 0.18 us a slot and KV head, as it was, the gap takes
    3 s, and the warps that wait for a piece give up after 2."""
    _few_live(usp, 1 << 18, 64, 64, 64, "bf16", {0: 700, (1 << 18) - 1: 900}, False)


@pytest.mark.gpu
@pytest.mark.parametrize("dtype", ["bf16", "f32"])
def test_as_many_sequences_as_allowed(usp, dtype):
    B = 1 << 24
    _few_live(usp, B, 8, 2, 64, dtype, {1: 60, 1 << 23: 500, (1 << 23) + 31: 40, B - 1: 300}, True)


@pytest.mark.gpu
@pytest.mark.parametrize("dtype,Hq,Hkv", [("bf16", 8, 2), ("bf16", 40, 1), ("bf16", 4, 4), ("f32", 8, 2)])
@pytest.mark.parametrize("B", [31, 33, 64, 500])
def test_idle_slots_between_sequences(usp, B, dtype, Hq, Hkv):
    for live in ({0: 100, B - 1: 40}, {B // 2: 300}, {B - 1: 1000}, {0: 33, 1: 5, B - 2: 17},
                 {b: 20 + 7 * b for b in range(0, min(B, 100), 3)}):
        _few_live(usp, B, Hq, Hkv, 64, dtype, live, False)
        _few_live(usp, B, Hq, Hkv, 64, dtype, live, True)
    _few_live(usp, B, Hq, Hkv, 64, dtype, {0: 100, B // 2: 44, B - 1: 70}, False, prefix=48)


@pytest.mark.gpu
def test_abort_path_gives_up_fast_and_recovers(usp):
    """With a timeout on record every kernel gives up at its first wait that is not satisfied, drains its loads and
    products and returns; the host reads the timeout once, and the next run is the clean one, bit for bit."""
    import time

    import torch
    guard = Guarded()
    cases = [([(1, 3000), (1, 500)], 8, 2, 128, 0), ([(6, 900)], 8, 2, 128, 0), ([(70, 900), (3, 10)], 8, 2, 128, 0),
             ([(300, 2000)], 4, 1, 64, 0), ([(1, 1000 + i) for i in range(40)], 8, 2, 128, 900),
             ([(1, 1000 + i) for i in range(3)], 8, 2, 64, 900)]
    bs = [Batch(seqs, Hq, Hkv, d, 64, prefix=p).to_gpu(usp, guard) for seqs, Hq, Hkv, d, p in cases]
    clean = []
    for b in bs:
        b.run(usp)
        _done(usp, guard)
        clean.append((b.g["o"].clone(), b.g["lse"].clone()))
    t0 = time.perf_counter()
    usp.usp_diag_raise_status()
    for b in bs:
        b.run(usp)
    assert usp.usp_device_status() == _lib.USP_ERR_TIMEOUT
    assert time.perf_counter() - t0 < 1.5
    assert usp.usp_device_status() == _lib.USP_OK
    for b, (o, lse) in zip(bs, clean):
        b.run(usp)
        _done(usp, guard)
        assert torch.equal(b.g["o"], o) and torch.equal(b.g["lse"], lse)


@pytest.mark.gpu
@pytest.mark.parametrize("fill", [0xFF, 0x03, 0x7F])
def test_abort_with_a_workspace_that_holds_anything(usp, fill):
    """After a kernel that gave up, the merge finds whatever the workspace held where rows should be noted; it stays
    inside the workspace, and the next run is right."""
    guard = Guarded()
    for seqs, Hq, Hkv, d, p in [([(70, 900), (3, 10)], 8, 2, 128, 0), ([(300, 2000)], 4, 1, 64, 300),
                                ([(40, 5000)], 8, 2, 128, 100), ([(1, 3000)], 8, 2, 64, 0)]:
        b = Batch(seqs, Hq, Hkv, d, 64, prefix=p).to_gpu(usp, guard)
        b.g["ws"].fill_(fill)
        usp.usp_diag_raise_status()
        b.run(usp)
        assert usp.usp_device_status() == _lib.USP_ERR_TIMEOUT
        b.run(usp)
        _done(usp, guard)
        b.check()


@pytest.mark.gpu
@pytest.mark.parametrize("fill", [0x01, 0x02, 0xFE, 0x00])
def test_abort_with_every_kind_of_stale_row_word(usp, fill):
    """The same with words of every kind that the merge tells apart, a split whose CTAs and row are in range among them."""
    guard = Guarded()
    for seqs, Hq, Hkv, d, p in [([(70, 900), (3, 10)], 8, 2, 128, 0), ([(300, 2000)], 4, 1, 64, 300),
                                ([(40, 5000)], 8, 2, 128, 100), ([(1, 3000)], 8, 2, 64, 0), ([(6, 900)], 8, 2, 128, 0)]:
        b = Batch(seqs, Hq, Hkv, d, 64, prefix=p).to_gpu(usp, guard)
        words = b.g["ws"][:8 * b.T * Hq]
        fills = [fill]
        if fill == 0:
            fills = [(3, 0, 0, 0, 0, 0, 1, 0), (3 | 5 << 2, 0, 0, 0, 1, 0, 3, 0)]  # row 0 of CTAs 0 and 1, row 5 of 1 to 3
        for f in fills:
            if fill == 0:
                words.view(-1, 8).copy_(b.torch.tensor(f, dtype=b.torch.uint8))
            else:
                b.g["ws"].fill_(f)
            usp.usp_diag_raise_status()
            b.run(usp)
            assert usp.usp_device_status() == _lib.USP_ERR_TIMEOUT
            b.run(usp)
            _done(usp, guard)
            b.check()


@pytest.mark.gpu
@pytest.mark.parametrize("n", [1, 6, 70])
def test_abort_after_a_prefix_call_in_the_same_workspace(usp, n):
    """One workspace for both calls: what a call behind a prefix noted of its rows is there when a call without one gives
    up before it notes its own."""
    guard = Guarded()
    pre = Batch([(n, 700), (n, 500), (n, 900)], 8, 2, 128, 64, prefix=300).to_gpu(usp, guard)
    own = Batch([(n, 700), (n, 500), (n, 900)], 8, 2, 128, 64, seed=1).to_gpu(usp, guard)
    assert own.g["ws"].numel() <= pre.g["ws"].numel()
    own.g["ws"] = pre.g["ws"]
    for _ in range(2):
        pre.run(usp)
        _done(usp, guard)
        pre.check()
        usp.usp_diag_raise_status()
        own.run(usp)
        assert usp.usp_device_status() == _lib.USP_ERR_TIMEOUT
        own.run(usp)
        _done(usp, guard)
        own.check()


@pytest.mark.gpu
@pytest.mark.parametrize("dtype,d,page", [("bf16", 128, 64), ("f32", 64, 16)])
def test_pool_beyond_32_bit_offsets(usp, dtype, d, page):
    """Pages whose elements lie beyond 2^31 of the pool."""
    import torch
    per_page = 8 * page * d
    first = (1 << 31) // per_page + 5
    guard = Guarded()
    b = Batch([(1, 300), (1, 20), (70, 200)], 16, 8, d, page, dtype, first_page=first).to_gpu(usp, guard)
    b.run(usp)
    _done(usp, guard)
    b.check()
    # and append there
    c = b.c
    x = torch.randn(3, 8, d, device="cuda").to(c.torch_dtype)
    i32 = lambda v: torch.tensor(v, dtype=torch.int32, device="cuda")  # noqa: E731
    usp.usp_kv_append(c, 3, None, x, x, i32([0, 1, 2]), i32([299, 19, 199]), None, None, None, b.g["kp"], b.g["vp"],
                      b.g["table"])
    _done(usp, guard)
    for t, p in enumerate((299, 19, 199)):
        at = int(b.table[t, p // page])
        assert torch.equal(b.g["kp"][at, :, p % page], x[t]) and torch.equal(b.g["vp"][at, :, p % page], x[t])
    del b
    torch.cuda.empty_cache()


@pytest.mark.gpu
def test_helpers(usp):
    import torch
    guard = Guarded()
    b = Batch([(1, 200), (1, 190), (1, 129)], 8, 2, 128, 64, prefix=128).to_gpu(usp, guard)
    g = b.g
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    o, lse = usp.prefix_attention(b.c, g["q"], g["kp"], g["vp"], g["table"], g["lens"], g["prefix"], 128, stream=side)
    torch.cuda.synchronize()
    b.check(o, lse)
    whole = b.table.copy()
    whole[:, :2] = b.prefix_pages
    o2, lse2 = usp.paged_attention(b.c, g["q"], g["kp"], g["vp"], torch.from_numpy(whole).cuda(), g["lens"])
    torch.cuda.synchronize()
    b.check(o2, lse2)
    with pytest.raises(ValueError):
        usp.paged_attention(b.c, g["q"], g["kp"], g["vp"], g["table"].long(), g["lens"])
    with pytest.raises(ValueError):
        usp.prefix_attention(b.c, g["q"], g["kp"], g["vp"], g["table"], g["lens"], g["prefix"], 129)
    with pytest.raises(ValueError):
        usp.paged_attention(b.c, g["q"].float(), g["kp"], g["vp"], g["table"], g["lens"])


@pytest.mark.gpu
def test_helpers_on_a_side_stream_leave_freed_memory_alone(usp):
    """Memory that was freed on the current stream is still being written there when a helper makes its outputs for
    another stream; and outputs freed here are not handed out there while this stream reads them."""
    import torch
    guard = Guarded()
    b = Batch([(1, 200), (1, 190), (1, 129)], 8, 2, 128, 64).to_gpu(usp, guard)
    g, c = b.g, b.c
    side = torch.cuda.Stream()
    torch.cuda.synchronize()
    sizes = [b.T * c.Hq * c.d * 2, b.T * c.Hq * 4, usp.usp_paged_attn_workspace_size(c, b.T, 1)]
    for handle in (side, side.cuda_stream):
        xs = [torch.empty(n, dtype=torch.uint8, device="cuda") for n in sizes]
        torch.cuda._sleep(40_000_000)  # some 20 ms
        for x in xs:
            x.fill_(0x7F)
        del x, xs
        o, lse = usp.paged_attention(c, g["q"], g["kp"], g["vp"], g["table"], g["lens"], stream=handle)
        side.synchronize()
        torch.cuda.synchronize()
        b.check(o, lse)
        torch.cuda._sleep(40_000_000)
        late_o, late_l = o + 0, lse + 0
        del o, lse
        usp.paged_attention(c, torch.zeros_like(g["q"]), g["kp"], g["vp"], g["table"], g["lens"], stream=handle)
        torch.cuda.synchronize()
        b.check(late_o, late_l)


@pytest.mark.gpu
@pytest.mark.parametrize("handle", [False, True])
def test_inputs_freed_while_a_side_stream_reads_them(usp, handle):
    """A helper called for another stream may be given tensors that nothing else holds: their memory must not be handed
    out here before that stream has read it."""
    import torch
    guard = Guarded()
    b = Batch([(1, 200), (1, 190), (1, 129)], 8, 2, 128, 64, prefix=128).to_gpu(usp, guard)
    g, c = b.g, b.c
    whole = b.table.copy()
    whole[:, :2] = b.prefix_pages
    whole = torch.from_numpy(whole).cuda()
    side = torch.cuda.Stream()
    stream = side.cuda_stream if handle else side
    gen = torch.Generator(device="cuda").manual_seed(1)
    x = [torch.randn((3, H, 128), generator=gen, device="cuda").bfloat16() for H in (8, 2, 2)]
    inv = (10000.0 ** (-torch.arange(64, device="cuda", dtype=torch.float64) / 64)).float()
    kp, vp = torch.zeros_like(g["kp"]), torch.zeros_like(g["vp"])
    seq = torch.arange(3, dtype=torch.int32, device="cuda")

    def temporary(*ts):
        return [t.clone() for t in ts]

    def reused():  # whatever the allocator has free on this stream is written over
        free = [torch.empty(n, dtype=torch.uint8, device="cuda") for n in (512, 1024, 1536, 2048, 4096, 6144) for _ in range(24)]
        for t in free:
            t.fill_(0x3F)
        torch.cuda.current_stream().synchronize()

    def paged(q, lens):
        return usp.paged_attention(c, q, g["kp"], g["vp"], whole, lens, stream=stream)

    def prefix(q, lens, pages):
        return usp.prefix_attention(c, q, g["kp"], g["vp"], g["table"], lens, pages, 128, stream=stream)

    def append(q, k, v, seq, pos, inv):
        return usp.kv_append(c, q, k, v, seq, pos, inv, kp, vp, whole, stream=stream)

    for call, args in ((paged, (g["q"], g["lens"])), (prefix, (g["q"], g["lens"], g["prefix"])),
                       (append, (*x, seq, g["lens"] - 1, inv))):
        torch.cuda.synchronize()
        want = [t.clone() for t in call(*args)]
        torch.cuda.synchronize()
        ts = temporary(*args)
        torch.cuda.current_stream().synchronize()
        with torch.cuda.stream(side):
            torch.cuda._sleep(100_000_000)  # some 50 ms
        got = call(*ts)
        del ts
        reused()
        side.synchronize()
        assert usp.usp_device_status() == 0
        for a, w in zip(got, want):
            assert torch.equal(a, w), call.__name__


@pytest.mark.gpu
def test_helpers_captured_on_a_forked_stream(usp):
    """The same inside a capture: temporaries and outputs of a forked stream live as long as the graph needs them."""
    import torch
    guard = Guarded()
    b = Batch([(1, 200), (1, 190), (1, 129)], 8, 2, 128, 64, prefix=128).to_gpu(usp, guard)
    g = b.g
    b.run(usp)
    main, side = torch.cuda.Stream(), torch.cuda.Stream()
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    outs = []
    with torch.cuda.graph(graph, stream=main):
        for scale in (1.0, 2.0):
            q = g["q"] * scale
            side.wait_stream(main)
            o, lse = usp.prefix_attention(b.c, q, g["kp"], g["vp"], g["table"], g["lens"], g["prefix"], 128, stream=side)
            del q
            junk = torch.full_like(g["q"], float("nan"))
            main.wait_stream(side)
            outs.append((o + 0, lse + 0))
            del o, lse, junk
    for _ in range(2):
        graph.replay()
        _done(usp, guard)
        b.check(*outs[0])
    b.q = b.q * 2
    b.check(*outs[1])


@pytest.mark.gpu
def test_helpers_on_the_default_stream_from_another(usp):
    """Stream handle 0 is the default stream: outputs and workspace are made there, whatever the current stream is."""
    import torch
    guard = Guarded()
    b = Batch([(1, 200), (1, 190), (1, 129)], 8, 2, 128, 64).to_gpu(usp, guard)
    g = b.g
    torch.cuda.synchronize()
    with torch.cuda.stream(torch.cuda.Stream()):
        o, lse = usp.paged_attention(b.c, g["q"], g["kp"], g["vp"], g["table"], g["lens"], stream=0)
        x, _ = usp.kv_append(b.c, g["q"], *(torch.zeros(3, 2, 128, dtype=torch.bfloat16, device="cuda"),) * 2,
                             torch.full((3,), -1, dtype=torch.int32, device="cuda"), g["lens"], None, g["kp"], g["vp"],
                             g["table"], stream=torch.cuda.default_stream())
        assert x.shape == g["q"].shape
    torch.cuda.synchronize()
    b.check(o, lse)


@pytest.mark.gpu
@pytest.mark.parametrize("P,path", [(2, "ulysses"), (4, "ring")])
def test_prompt_then_answer(usp, orc, P, path):
    """A prompt through the sequence-parallel attention, its keys and values into the cache, then tokens one by one, and
    the last of them again as drafts of two samples that share the prompt: every output is a row of the causal attention
    of the whole sequence."""
    import torch
    B, Hq, Hkv, d, page, N, steps = 2, 8, 2, 128, 32, 512, 9
    L = N + steps
    gen = torch.Generator().manual_seed(3)
    q, k, v = (torch.randn((B, L, H, d), generator=gen).bfloat16().cuda() for H in (Hq, Hkv, Hkv))
    inv = (500000.0 ** (-torch.arange(d // 2, dtype=torch.float64) / (d // 2))).float().cuda()
    mp = -(-L // page)
    c = usp.Cache(B * mp, page, B, mp, Hq, Hkv, d)
    table = torch.randperm(B * mp, generator=gen).int().view(B, mp).cuda()
    kp, vp = (torch.full(c.pool_shape(), float("nan"), dtype=torch.bfloat16, device="cuda") for _ in range(2))
    i32 = dict(dtype=torch.int32, device="cuda")
    # the prompt, sequence-sharded [P][B][N/P][H][d]: a batch of P*B*N/P tokens for the cache
    p = usp.Problem(B=B, Hq=Hq, Hkv=Hkv, N=N, d=d, P=P)
    shard = lambda x: x[:, :N].reshape(B, P, N // P, -1, d).transpose(0, 1).contiguous()  # noqa: E731
    qs, ks, vs = shard(q), shard(k), shard(v)
    seq = torch.arange(B, **i32).view(1, B, 1).expand(P, B, N // P).reshape(-1).contiguous()
    pos = torch.arange(N, **i32).view(P, 1, N // P).expand(P, B, N // P).reshape(-1).contiguous()
    T = B * N
    q_rot, k_rot = usp.kv_append(c, qs.view(T, Hq, d), ks.view(T, Hkv, d), vs.view(T, Hkv, d), seq, pos, inv, kp, vp, table)
    attend = usp.ulysses_attention_fwd if path == "ulysses" else usp.ring_attention_fwd
    o_prompt, _ = attend(p, q_rot.view(p.seq_shape(Hq)), k_rot.view(p.seq_shape(Hkv)), vs)
    unshard = lambda x, H: x.view(P, B, N // P, H, d).transpose(0, 1).reshape(B, N, H, d)  # noqa: E731
    rot_q, rot_k = [unshard(q_rot, Hq)], [unshard(k_rot, Hkv)]
    outs = []
    every = torch.arange(B, **i32)
    for i in range(steps):
        at = torch.full((B,), N + i, **i32)
        q_rot, k_rot = usp.kv_append(c, q[:, N + i], k[:, N + i], v[:, N + i], every, at, inv, kp, vp, table)
        rot_q.append(q_rot[:, None])
        rot_k.append(k_rot[:, None])
        o, _ = usp.paged_attention(c, q_rot, kp, vp, table, at + 1)
        outs.append(o)
    # the last four tokens of sequence 0 at once, behind its prompt as a shared prefix
    q4, _ = usp.kv_append(c, q[0, L - 4:], k[0, L - 4:], v[0, L - 4:], torch.zeros(4, **i32),
                          torch.arange(L - 4, L, **i32), inv, kp, vp, table)
    one = usp.Cache(B * mp, page, 1, mp, Hq, Hkv, d)
    o4, _ = usp.prefix_attention(one, q4, kp, vp, table[:1], torch.tensor([L], **i32), table[0, :N // page].contiguous(), N,
                                 q_start=torch.tensor([0, 4], **i32), max_q=4)
    torch.cuda.synchronize()
    assert usp.usp_device_status() == 0
    from tests.helpers import TOL_BF16_O_MAXABS, TOL_BF16_O_RELFRO, rel_fro
    heads = []  # the rotated values, within the bound of test_append; the attention of exactly these is the reference
    for rotated, x in ((torch.cat(rot_q, 1), q), (torch.cat(rot_k, 1), k)):
        for b in range(B):
            want, mag = ref_rotate(_np(x[b]), np.arange(L), inv.cpu().numpy(), False)
            assert (np.abs(_np(rotated[b]) - want) <= 8 * 2.0 ** -24 * mag + U["bf16"] * np.abs(want) * 1.001).all()
        heads.append(np.ascontiguousarray(_np(rotated).transpose(0, 2, 1, 3)).astype(np.float32))
    want, _ = orc.attn_rows(*heads, np.ascontiguousarray(_np(v).transpose(0, 2, 1, 3)).astype(np.float32), causal=True)
    want = want.transpose(0, 2, 1, 3)                                     # [B][L][Hq][d]
    got_prompt = _np(unshard(o_prompt.reshape(-1), Hq))
    # the library's tolerances for bf16 outputs
    for a, w in ((got_prompt, want[:, :N]), (_np(torch.stack(outs, 1)), want[:, N:]), (_np(o4), want[0, L - 4:])):
        assert rel_fro(a, w) < TOL_BF16_O_RELFRO
        assert np.abs(a - w).max() < TOL_BF16_O_MAXABS
