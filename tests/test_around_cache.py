"""What goes into and comes out of the paged cache: rotary positions with several axes, the pages' bookkeeping and copies,
the verification of drafted tokens.

Rotations are compared with float64 evaluations of the definition, element by element: cosine and sine in float32 are off
by a few steps (8 2^-24 of |a| + |b| with the products' and the sum's roundings), the result is rounded once, to half a step
of its type.  Everything else is whole numbers and copies, and has to be equal: the pages against a model that takes one
slot after the other, the drafts against sums of whole numbers of any size.
"""
import numpy as np
import pytest

import context_long_attention_ulysses_gb300 as usp_mod
from context_long_attention_ulysses_gb300 import _lib, build
from tests.guarded import Guarded

U = {"bf16": 2.0 ** -8, "f32": 2.0 ** -24}
FAKE = 1 << 20


# ------------------------------------------------------------------ plain definitions
def ref_rotate(x, pos, axis, inv_freq, interleaved, inverse=False):
    """x [T][H][d], pos [axes][T]; also |a| + |b| of each rotated element (|x| of the others)."""
    half = len(axis)
    ang = np.stack([pos[a].astype(np.float64) * float(inv_freq[i]) for i, a in enumerate(axis)], -1) if half else \
        np.zeros((x.shape[0], 0))
    cs, sn = np.cos(ang)[:, None], np.sin(ang)[:, None] * (-1 if inverse else 1)
    ia = np.arange(0, 2 * half, 2) if interleaved else np.arange(half)
    ib = ia + 1 if interleaved else ia + half
    y, mag = x.copy(), np.abs(x)
    a, b = x[..., ia], x[..., ib]
    y[..., ia], y[..., ib] = a * cs - b * sn, b * cs + a * sn
    mag[..., ia] = mag[..., ib] = np.abs(a) + np.abs(b)
    return y, mag


def ref_update(page, table, lens, ref, parent, keep, grow):
    """The pages' bookkeeping, one slot after the other: (table, lens, ref, head, copies)."""
    B, mp = table.shape
    n = len(ref)
    cap = mp * page
    rows, count = [list(map(int, r)) for r in table], [int(x) for x in ref]
    pages = lambda t: -(-t // page)  # noqa: E731
    ok = lambda x: 0 <= x < n  # noqa: E731
    L = [min(max(int(x), 0), cap) for x in lens]
    src = [b if parent is None else int(parent[b]) for b in range(B)]
    kept, now, have = [], [], []
    for b, a in enumerate(src):
        k = L[a] if 0 <= a < B else 0
        if keep is not None:
            k = min(max(int(keep[b]), 0), k)
        kept.append(k)
        now.append(k + min(max(int(grow[b]), 0) if grow is not None else 0, cap - k))
        have.append(rows[a][:pages(k)] if 0 <= a < B else [])
    for b in range(B):
        for x in rows[b][:pages(L[b])]:
            if ok(x):
                count[x] -= 1
    for ids in have:
        for x in ids:
            if ok(x):
                count[x] += 1
    writers = {}
    for b in range(B):
        if kept[b] % page and now[b] > kept[b] and ok(have[b][-1]):
            writers.setdefault(have[b][-1], []).append(((src[b] != b), b))
    stays = {x: min(w)[1] for x, w in writers.items() if count[x] == len(w)}
    copies = [b for b in range(B) if kept[b] % page and now[b] > kept[b] and ok(have[b][-1]) and stays.get(have[b][-1]) != b]
    free = [i for i in range(n) if count[i] <= 0]
    need = sum(pages(now[b]) - pages(kept[b]) for b in range(B)) + len(copies)
    if need > len(free):
        return table, lens, ref, (0, need - len(free), sum(int(x) <= 0 for x in ref), 0), []
    count = [max(x, 0) for x in count]
    left, made = iter(free), []
    for b in range(B):
        ids = list(have[b])
        if b in copies:
            to = next(left)
            made.append((ids[-1], to, kept[b] % page, 0))
            count[ids[-1]] -= 1
            count[to] = 1
            ids[-1] = to
        while len(ids) < pages(now[b]):
            to = next(left)
            count[to] = 1
            ids.append(to)
        for j in range(max(len(ids), pages(L[b]))):
            rows[b][j] = ids[j] if j < len(ids) else -1
    return (np.array(rows, np.int32).reshape(B, mp), np.array(now, np.int32), np.array(count, np.int32),
            (len(made), 0, len(free) - need, 0), made)


def ref_verify(target, draft, tokens, u, q_start, seq_lens):
    """target, draft float64 [T][V]; sums of whole numbers of 2^-46, of any size."""
    T, V = target.shape
    out = []
    whole = lambda row: np.rint(np.clip(np.nan_to_num(row, nan=0.0, posinf=1.0, neginf=0.0), 0, 1) * 2.0 ** 46)  # noqa: E731
    for s in range(len(q_start) - 1):
        t0 = min(max(int(q_start[s]), 0), T)
        n = min(max(int(q_start[s + 1]), t0), T) - t0
        ln = int(seq_lens[s])
        if n == 0:
            out.append((0, -1, ln))
            continue
        a = 0
        while a < n - 1:
            t = t0 + a + 1
            x = int(tokens[t])
            if not 0 <= x < V:
                break
            q = draft[t, x] if draft is not None else 1.0
            if not float(u[t]) * q < target[t - 1, x]:     # (24 bits times 24 bits: exact)
                break
            a += 1
        p = whole(target[t0 + a]).astype(np.uint64)
        w = p
        if a < n - 1:
            if draft is not None:
                q = whole(draft[t0 + a + 1]).astype(np.uint64)
                w = np.where(p > q, p - np.minimum(p, q), 0).astype(np.uint64)
            else:
                w = p.copy()
                if 0 <= int(tokens[t0 + a + 1]) < V:
                    w[int(tokens[t0 + a + 1])] = 0
        if not w.any():
            w = p
        run = np.cumsum(w.astype(object)) if int(w.max()) * V >= 1 << 63 else np.cumsum(w)
        total = int(run[-1])
        nxt = -1
        if total:
            num, den = float(min(max(0.0, float(u[t0])), 1 - 2.0 ** -24)).as_integer_ratio()
            thr = min(total, (1 << 64) - 1) * num // den
            nxt = int(np.argmax(run > thr))
        out.append((a, nxt, ln - (n - 1 - a)))
    return np.array(out, np.int64).reshape(-1, 3).T


# ------------------------------------------------------------------ the models themselves (CPU)
def test_model_of_the_axes():
    r = usp_mod.Rotary.sections((2, 3, 3))
    assert r.axis == (0, 0, 1, 1, 1, 2, 2, 2) and r.rot == 16 and r.axes == 3
    assert usp_mod.Rotary.sections((4, 2, 2), cycled=True).axis == (0, 1, 2, 0, 1, 2, 0, 0)
    assert usp_mod.Rotary.sections((24, 20, 20), cycled=True).axis.count(2) == 20
    with pytest.raises(ValueError):
        usp_mod.Rotary.sections((1, 7), cycled=True)          # the second axis has more than its turns
    rng = np.random.default_rng(0)
    x = rng.standard_normal((5, 2, 32))
    f = rng.uniform(0.01, 1, 8)
    pos = rng.integers(0, 50, (3, 5))
    for inter in (False, True):
        y, _ = ref_rotate(x, pos, r.axis, f, inter)
        back, _ = ref_rotate(y, pos, r.axis, f, inter, inverse=True)
        assert np.allclose(back, x) and np.allclose((y ** 2).sum(), (x ** 2).sum())
        # the same position on every axis is one axis
        one, _ = ref_rotate(x, np.stack([pos[0]] * 3), r.axis, f, inter)
        two, _ = ref_rotate(x, pos[:1], (0,) * 8, f, inter)
        assert np.array_equal(one, two)


def test_model_of_the_drafts_gives_the_targets_distribution():
    """Over a fine grid of numbers, what is emitted first after a token is distributed as the target's row."""
    p, q = np.array([0.5, 0.125, 0.25, 0.125]), np.array([0.25, 0.25, 0.5, 0.0])
    V, n = 4, 64
    got = np.zeros(V)
    for x in range(V):
        for i in range(n):
            for j in range(n):
                tgt, drf = np.stack([p, p]), np.stack([q, q])
                a, nxt, _ = ref_verify(tgt, drf, [0, x], [(j + 0.5) / n, (i + 0.5) / n], [0, 2], [5])[:, 0]
                got[x if a else nxt] += q[x] / n / n
    assert np.abs(got - p).max() < 2.0 / n


def test_model_of_the_pages_keeps_its_books():
    rng = np.random.default_rng(3)
    B, mp, page, n = 5, 6, 16, 21
    table, lens, ref = np.full((B, mp), -1, np.int32), np.zeros(B, np.int32), np.zeros(n, np.int32)
    lacking = 0
    for _ in range(200):
        parent = np.where(rng.random(B) < 0.5, np.arange(B), rng.integers(-1, B, B))
        table, lens, ref, head, copies = ref_update(page, table, lens, ref, parent, rng.integers(0, 100, B),
                                                    rng.integers(0, 40, B))
        lacking += head[1] > 0
        used = [x for b in range(B) for x in table[b, :-(-lens[b] // page)]]
        assert (np.bincount(used, minlength=n) == ref).all() and (table[np.arange(mp) >= -(-lens[:, None] // page)] == -1).all()
        assert head[2] == (ref == 0).sum() and not {c[0] for c in copies} & {c[1] for c in copies}
    assert 0 < lacking < 150


# ------------------------------------------------------------------ refusals (no GPU needed)
@pytest.fixture(scope="module")
def lib():
    build.build()
    return _lib.load()


def _status(call, /, *a, **kw):
    with pytest.raises(usp_mod.UspError) as e:
        call(*a, **kw)
    return e.value.status


def _c(**kw):
    base = dict(n_pages=10, page_size=16, n_seqs=2, max_pages=4, Hq=4, Hkv=2, d=64)
    base.update(kw)
    return usp_mod.Cache(**base)


def _p(**kw):
    base = dict(B=1, Hq=4, Hkv=2, N=8, d=64, P=2)
    base.update(kw)
    return usp_mod.Problem(**base)


R3 = usp_mod.Rotary.sections((8, 12, 12))


def _struct(n_axes=3, rot=64, axis=()):
    s = _lib.UspRotary(n_axes, rot, 0)
    for i, a in enumerate(axis):
        s.axis[i] = a
    return s


def test_rotary_refusals(lib):
    def call(p=None, r=R3, q=FAKE, k=FAKE, pos=FAKE, f=FAKE, qo=FAKE, ko=FAKE, **kw):
        usp_mod.usp_rotary_embed(p or _p(), r, q, k, pos, f, qo, ko, **kw)

    assert lib.usp_rotary_embed(None, None, 0, None, 0, None, 0, None, None, None, 0, None, 0, None) == 1
    assert _status(call, r=None) == 1
    for kw in (dict(N=7), dict(B=-1), dict(Hq=3), dict(dtype="bf16", scale=-1.0)):
        assert _status(call, _p(**kw)) == 1
    for s in (_struct(n_axes=0), _struct(n_axes=5), _struct(rot=8), _struct(rot=-16), _struct(rot=80), _struct(axis=[3])):
        assert _status(call, r=s) == 1
    assert _status(call, _p(d=96)) == 2 and _status(call, _p(B=1 << 12, N=1 << 20, Hq=1, Hkv=1)) == 2
    assert _status(call, q=None) == 1 and _status(call, qo=None) == 1 and _status(call, k=None) == 1 and _status(call, ko=0) == 1
    for name in ("q", "k", "qo", "ko"):
        assert _status(call, **{name: FAKE + 8}) == 3
    for name in ("pos", "f"):
        assert _status(call, **{name: 0}) == 3 and _status(call, **{name: FAKE + 2}) == 3
    c = _p().c()
    raw = lambda q, qs, qo, qos: lib.usp_rotary_embed(c, R3.c(), 0, q, qs, None, 0, FAKE, FAKE, qo, qos, None, 0, None)  # noqa: E731
    assert raw(FAKE, 255, FAKE * 2, 256) == 1 and raw(FAKE, 260, FAKE * 2, 256) == 1 and raw(FAKE, 256, FAKE * 2, 0) == 1
    assert raw(FAKE, 512, FAKE, 256) == 1                     # in place, rows would move over others
    call(_p(B=0)), call(q=None, k=None, qo=None, ko=None)     # nothing to do
    for bad in (usp_mod.Rotary((0, 4)), usp_mod.Rotary((0, -1)), usp_mod.Rotary((0,) * 65), usp_mod.Rotary((0, 1), n_axes=1)):
        with pytest.raises(ValueError):
            bad.c()


def test_structs_of_a_rotation_and_a_problem_are_the_callers_own(lib):
    """A changed struct is another's: it does not reach the calls of the one it was made from, nor do copies share it."""
    import copy
    import pickle
    r, p = usp_mod.Rotary.sections((8, 12, 12)), _p()
    call = lambda p_, r_: usp_mod.usp_rotary_embed(p_, r_, FAKE, FAKE, FAKE + 2, FAKE, FAKE, FAKE)  # noqa: E731  (3: pos misaligned)
    assert _status(call, p, r) == 3
    s, q = r.c(), p.c()
    s.n_axes, q.d = 9, 96
    assert _status(call, p, s) == 1 and _status(call, q, r) == 2 and _status(call, p, r) == 3
    for same in (copy.copy, copy.deepcopy, lambda x: pickle.loads(pickle.dumps(x))):
        assert same(r) == r and same(p) == p and _status(call, same(p), same(r)) == 3


def test_structs_of_another_kind_are_refused(lib):
    """A problem is no cache: its struct is shorter, and a call would read behind its end."""
    c, p = _c(), _p()
    calls = {"problem": lambda x: usp_mod.usp_rotary_embed(x, R3, FAKE, None, FAKE, FAKE, FAKE, None),
             "rotary": lambda x: usp_mod.usp_rotary_embed(p, x, FAKE, None, FAKE, FAKE, FAKE, None),
             "append": lambda x: usp_mod.usp_kv_append_axes(x, 0, *([FAKE] * 7), R3, *([FAKE] * 5)),
             "append's rotary": lambda x: usp_mod.usp_kv_append_axes(c, 0, *([FAKE] * 7), x, *([FAKE] * 5)),
             "update": lambda x: usp_mod.usp_pages_update(x, *([FAKE] * 8), 0),
             "compact": lambda x: usp_mod.usp_pages_compact(x, *([FAKE] * 6)),
             "copy": lambda x: usp_mod.usp_pages_copy(x, 0, FAKE, FAKE, FAKE)}
    mine = {"problem": p, "rotary": R3, "append's rotary": R3}
    for name, call in calls.items():
        for x in (c, p, R3, c.c(), p.c(), R3.c()):
            if type(x) not in (type(mine.get(name, c)), type(mine.get(name, c).c())):
                with pytest.raises(TypeError):
                    call(x)
        for x in ((1, 2), "a text", 5, _lib.UspTraceEntry()):
            with pytest.raises(TypeError):
                call(x)


@pytest.mark.parametrize("make", [_c, _p, lambda: usp_mod.Rotary.sections((8, 12, 12))])
def test_two_threads_first_calls_share_a_struct(lib, make, monkeypatch):
    """A struct whose address a call of one thread holds is not replaced by another thread's that makes one meanwhile."""
    import ctypes
    x = make()
    cls, c = type(x), type(x).c
    other = []

    def interrupted(self):
        if not other:
            other.append(None)
            other[0] = usp_mod._struct(self, cls)            # another thread comes in between
        return c(self)

    monkeypatch.setattr(cls, "c", interrupted)
    mine = usp_mod._struct(x, cls)
    assert mine == other[0] == usp_mod._struct(x, cls)
    kept = type(c(x)).from_address(mine)
    assert bytes(kept) == bytes(c(x)) and ctypes.sizeof(kept) == ctypes.sizeof(c(x))


@pytest.mark.parametrize("make", [_c, _p, lambda: usp_mod.Rotary.sections((8, 12, 12))])
def test_attributes_are_the_fields_before_and_after_a_call(lib, make):
    """What a call keeps is not among an object's attributes, and a copy has its own."""
    import copy
    import dataclasses
    import pickle
    x = make()
    fields = {f.name: getattr(x, f.name) for f in dataclasses.fields(x)}
    at = usp_mod._struct(x, type(x))
    assert vars(x) == fields and type(x)(**vars(x)) == x
    for same in (copy.copy, copy.deepcopy, lambda y: pickle.loads(pickle.dumps(y)), dataclasses.replace):
        y = same(x)
        assert y == x and vars(y) == fields and usp_mod._struct(y, type(y)) != at
        assert bytes(y._kept()[0]) == bytes(x._kept()[0])


def test_a_rotation_keeps_its_axes_when_a_list_changes(lib):
    axes = [0, 1, 2, 0, 1, 2, 0, 0]
    r, a = usp_mod.Rotary(axes), usp_mod.Rotary(np.array(axes))
    assert r == a == usp_mod.Rotary(tuple(axes)) and hash(r) == hash(a)
    before = bytes(r._kept()[0])
    axes[0] = 3
    assert r.axes == 3 and bytes(r.c()) == bytes(r._kept()[0]) == before


def test_axes_are_whole_numbers():
    for axes in ((0, 1.7), (0, 1.0), ("0",), (None,)):
        with pytest.raises(TypeError):
            usp_mod.Rotary(axes)


def test_append_axes_refusals(lib):
    def call(c=None, T=2, rot_pos=FAKE, r=R3, **kw):
        a = dict(q=FAKE, k=FAKE, v=FAKE, seq=FAKE, pos=FAKE, f=FAKE, qo=FAKE, ko=FAKE, kp=FAKE, vp=FAKE, table=FAKE)
        a.update(kw)
        usp_mod.usp_kv_append_axes(c or _c(), T, a["q"], a["k"], a["v"], a["seq"], a["pos"], rot_pos, a["f"], r, a["qo"], a["ko"],
                                   a["kp"], a["vp"], a["table"])

    assert lib.usp_kv_append_axes(None, 0, *([None, 0] * 3), None, None, None, None, None, None, None, None, None, None,
                                  None) == 1
    assert _status(call, r=None) == 1 and _status(call, r=_struct(rot=80)) == 1 and _status(call, r=_struct(axis=[0, 3])) == 1
    assert _status(call, rot_pos=None) == 3 and _status(call, rot_pos=FAKE + 2) == 3
    assert _status(call, _c(d=96)) == 2 and _status(call, T=-1) == 1 and _status(call, q=None) == 1
    for name in ("k", "v", "kp", "vp", "qo", "ko", "q"):
        assert _status(call, **{name: FAKE + 8}) == 3
    for name in ("k", "v", "kp", "vp", "seq", "pos", "table", "f"):
        assert _status(call, **{name: 0}) == 3
    call(T=0)
    call(_c(n_pages=0))


def test_pages_refusals(lib):
    def update(c=None, lens=FAKE, table=FAKE, ref=FAKE, copies=FAKE, ws=FAKE, ws_bytes=1 << 40, parent=FAKE, keep=FAKE, grow=FAKE):
        usp_mod.usp_pages_update(c or _c(), parent, keep, grow, lens, table, ref, copies, ws, ws_bytes)

    def compact(c=None, table=FAKE, ref=FAKE, table_out=FAKE, ref_out=FAKE, new_id=FAKE, copies=FAKE):
        usp_mod.usp_pages_compact(c or _c(), table, ref, table_out, ref_out, new_id, copies)

    def copy(c=None, n=2, copies=FAKE, kp=FAKE, vp=FAKE, layers=1, stride=0):
        usp_mod.usp_pages_copy(c or _c(), n, copies, kp, vp, layers, stride)

    assert lib.usp_pages_update(None, *([None] * 8), 0, None) == 1 and lib.usp_pages_compact(None, *([None] * 7)) == 1
    assert lib.usp_pages_copy(None, 0, None, 1, 0, None, None, None) == 1
    for f in (update, compact, copy):
        assert _status(f, _c(n_pages=-1)) == 1 and _status(f, _c(page_size=24)) == 2 and _status(f, _c(d=96)) == 2
        assert _status(f, copies=FAKE + 8) == 3 and _status(f, copies=0) == 3
    for f in (update, compact):
        assert _status(f, _c(n_pages=(1 << 23) + 1, Hq=1, Hkv=1)) == 2
    for name in ("lens", "table", "ref"):
        assert _status(update, **{name: 0}) == 3
    for name in ("lens", "table", "ref", "parent", "keep", "grow"):
        assert _status(update, **{name: FAKE + 2}) == 3
    for name in ("table", "ref", "table_out", "ref_out", "new_id"):
        assert _status(compact, **{name: 0}) == 3 and _status(compact, **{name: FAKE + 2}) == 3
    size = usp_mod.usp_pages_update_workspace_size(_c())
    assert size > 0 and _status(update, ws_bytes=size - 1) == 4 and _status(update, ws=FAKE + 128) == 3 and _status(update, ws=0) == 3
    assert usp_mod.usp_pages_update_workspace_size(_c(page_size=24)) == 0
    assert _status(copy, n=-1) == 1 and _status(copy, layers=-1) == 1 and _status(copy, layers=2, stride=10 * 2 * 16 * 64 - 8) == 1
    assert _status(copy, layers=2, stride=10 * 2 * 16 * 64 + 4) == 1
    assert _status(copy, kp=FAKE + 8) == 3 and _status(copy, vp=0) == 3
    copy(n=0), copy(layers=0), copy(_c(n_pages=0))


def test_verify_refusals(lib):
    def call(n=2, T=4, V=100, target=FAKE, draft=FAKE, tokens=FAKE, u=FAKE, start=FAKE, lens=FAKE, acc=FAKE, nxt=FAKE, left=FAKE):
        usp_mod.usp_verify_drafts(n, T, V, target, draft, tokens, u, start, lens, acc, nxt, left, dtype="f32")

    assert _status(call, n=-1) == 1 and _status(call, T=-1) == 1 and _status(call, V=0) == 1
    assert _status(call, lens=None) == 1 and _status(call, left=None) == 1
    assert _status(call, V=(1 << 19) + 1) == 2 and _status(call, n=1 << 28) == 2
    for name in ("target", "draft"):
        assert _status(call, **{name: FAKE + 8}) == 3
    for name in ("tokens", "u", "start", "lens", "acc", "nxt", "left"):
        assert _status(call, **{name: FAKE + 2}) == 3
    for name in ("target", "tokens", "u", "start", "acc", "nxt"):
        assert _status(call, **{name: 0}) == 3
    raw = lambda dt, ts, ds: lib.usp_verify_drafts(2, 4, 100, dt, FAKE, ts, FAKE, ds, *([FAKE] * 7), None)  # noqa: E731
    assert raw(0, 99, 100) == 1 and raw(0, 100, 99) == 1 and raw(7, 100, 100) == 1
    call(n=0)


def test_helpers_refuse_host_tensors():
    import torch
    c, x = _c(), torch.zeros(10, dtype=torch.int32)
    for call in (lambda: usp_mod.pages_update(c, x[:2], x, x), lambda: usp_mod.pages_compact(c, x, x),
                 lambda: usp_mod.pages_copy(c, x, torch.zeros(1, 1, 1, 1), x),
                 lambda: usp_mod.verify_drafts(torch.zeros(2, 5), None, x, x, x),
                 lambda: usp_mod.rotary_embed(_p(), R3, torch.zeros(1), None, x, x)):
        with pytest.raises(ValueError):
            call()


def test_arguments_that_are_no_buffers_are_refused(lib):
    import torch
    x, i = torch.zeros(4, 100), torch.zeros(4, dtype=torch.int32)
    calls = [lambda y: usp_mod.usp_pages_copy(_c(), 1, y, FAKE, FAKE),
             lambda y: usp_mod.usp_pages_compact(_c(), y, FAKE, FAKE, FAKE, FAKE, FAKE),
             lambda y: usp_mod.usp_pages_update(_c(), y, None, None, FAKE, FAKE, FAKE, FAKE, FAKE),
             lambda y: usp_mod.usp_verify_drafts(1, 4, 100, FAKE, None, y, FAKE, FAKE, None, FAKE, FAKE, None, "f32"),
             lambda y: usp_mod.usp_verify_drafts(1, 4, 100, y, None, FAKE, FAKE, FAKE, None, FAKE, FAKE, None),
             lambda y: usp_mod.usp_rotary_embed(_p(), R3, y, None, FAKE, FAKE, FAKE, None)]
    for call in calls:
        for y, kind in (("a text", TypeError), ([1], TypeError), (1.5, TypeError)):
            with pytest.raises(kind):
                call(y)
        for y in (x, i, torch.zeros(4, 4, 64)):               # host tensors, or of another shape
            with pytest.raises(ValueError):
                call(y)
    with pytest.raises(ValueError):                           # a row of another type
        usp_mod.usp_verify_drafts(1, 4, 100, x.bfloat16(), None, FAKE, FAKE, FAKE, None, FAKE, FAKE, None, "f32")
    for y in (torch.zeros(2, 1, 4, 4, 32), torch.zeros(2, 1, 4, 3, 64), torch.zeros(8, 4, 64)[:, ::2].expand(8, 2, 64),
              torch.zeros(2, 2, 4, 4, 64).transpose(0, 1)[:, :, 1:]):
        with pytest.raises(ValueError):
            usp_mod.usp_rotary_embed(_p(), R3, y, None, FAKE, FAKE, FAKE, None)
    with pytest.raises((OverflowError, TypeError)):
        usp_mod.usp_pages_copy(_c(), 1 << 40, FAKE, FAKE, FAKE)
    with pytest.raises(TypeError):
        usp_mod._binding().pages_copy(0, 1)
    assert _status(lambda: usp_mod.usp_pages_copy(_c(page_size=24), 1, FAKE, FAKE, FAKE)) == 2


def test_tensors_of_another_type_or_too_short_are_refused(lib):
    """Before anything is launched: elements of another type would be misread, and a kernel would go on behind the end of what is
    shorter than the call says.  (Host tensors: what they hold is refused for its type and length before its place.)"""
    import torch
    bf, f32, i32, i64 = torch.bfloat16, torch.float32, torch.int32, torch.int64
    c, p, T = _c(), _p(N=16), 16
    pool = 10 * 2 * 16 * 64
    size = usp_mod.usp_pages_update_workspace_size(c)
    # per call: its tensors' types, shapes and least lengths, and the numbers of elements that may be more
    q, k = ((T, 4, 64), bf), ((T, 2, 64), bf)
    calls = {
        "rotary": (lambda x: usp_mod.usp_rotary_embed(p, R3, x["q"], x["k"], x["pos"], x["f"], x["qo"], x["ko"]),
                   dict(q=q, k=k, pos=((3 * T,), i32), f=((32,), f32), qo=q, ko=k)),
        "append": (lambda x: usp_mod.usp_kv_append_axes(c, T, x["q"], x["k"], x["v"], x["seq"], x["pos"], x["rot"], x["f"], R3, x["qo"],
                                                        x["ko"], x["kp"], x["vp"], x["table"]),
                   dict(q=q, k=k, v=k, seq=((T,), i32), pos=((T,), i32), rot=((3 * T,), i32), f=((32,), f32), qo=q, ko=k,
                        kp=((pool,), bf), vp=((pool,), bf), table=((2, 4), i32))),
        "update": (lambda x: usp_mod.usp_pages_update(c, x["parent"], x["keep"], x["grow"], x["lens"], x["table"], x["ref"], x["copies"],
                                                      x["ws"], size),
                   dict(parent=((2,), i32), keep=((2,), i32), grow=((2,), i32), lens=((2,), i32), table=((2, 4), i32),
                        ref=((10,), i32), copies=((3, 4), i32), ws=((size,), torch.uint8))),
        "compact": (lambda x: usp_mod.usp_pages_compact(c, x["table"], x["ref"], x["table_out"], x["ref_out"], x["new_id"], x["copies"]),
                    dict(table=((2, 4), i32), ref=((10,), i32), table_out=((2, 4), i32), ref_out=((10,), i32), new_id=((10,), i32),
                         copies=((6, 4), i32))),
        "copy": (lambda x: usp_mod.usp_pages_copy(c, 5, x["copies"], x["kp"], x["vp"], 3, pool + 8),
                 dict(copies=((4,), i32), kp=((3 * pool + 16,), bf), vp=((3 * pool + 16,), bf))),
        "verify": (lambda x: usp_mod.usp_verify_drafts(3, T, 50, x["target"], x["draft"], x["tokens"], x["u"], x["start"], x["lens"],
                                                       x["acc"], x["next"], x["keep"], "f32"),
                   dict(target=((T, 50), f32), draft=((T, 50), f32), tokens=((T,), i32), u=((T,), f32), start=((4,), i32),
                        lens=((3,), i32), acc=((3,), i32), next=((3,), i32), keep=((3,), i32))),
    }
    for name, (call, tensors) in calls.items():
        for arg, (shape, dtype) in tensors.items():
            x = {a: FAKE for a in tensors}
            least = torch.empty(shape, dtype=dtype)
            x[arg] = least
            with pytest.raises(ValueError, match="device tensors"):       # what would do, but for its place
                call(x)
            x[arg] = torch.empty((shape[0] + 1, *shape[1:]), dtype=dtype)
            with pytest.raises(ValueError, match="device tensors"):
                call(x)
            x[arg] = least[:-1]
            with pytest.raises(ValueError, match="at least|more bytes"):
                call(x)
            if dtype == torch.uint8:
                continue
            if name == "copy" and arg != "copies":            # (pages are moved as bytes)
                x[arg] = torch.empty(shape, dtype=torch.float16)
                with pytest.raises(ValueError, match="device tensors"):
                    call(x)
                continue
            for other in {i64, i32, bf, f32, torch.float64} - {dtype}:
                x[arg] = torch.empty(shape, dtype=other)
                with pytest.raises(ValueError, match="expected torch"):
                    call(x)
    # nothing is asked of what a call does not read
    none = torch.empty(0, 4, 64)
    usp_mod.usp_rotary_embed(_p(B=0), R3, none, None, torch.empty(0), torch.empty(0), none, None)
    usp_mod.usp_pages_copy(c, 0, torch.empty(0), torch.empty(0), torch.empty(0))


def test_device_pointers_to_probabilities_need_their_type(lib):
    import torch
    call = lambda target, dtype=None, draft=None: usp_mod.usp_verify_drafts(  # noqa: E731
        1, 4, 100, target, draft, FAKE + 2, FAKE, FAKE, None, FAKE, FAKE, None, dtype)
    for target in (FAKE, 0):
        with pytest.raises(ValueError, match="dtype"):
            call(target)
    for dtype in ("f32", "bf16"):                             # (3: tokens misaligned)
        assert _status(call, FAKE, dtype) == 3
    with pytest.raises(KeyError):
        call(FAKE, "f16")
    assert _status(call, None) == 3
    for wrong in (torch.float16, torch.float64, torch.int32):
        with pytest.raises(ValueError, match="expected float32 or bfloat16"):
            call(torch.zeros(4, 100, dtype=wrong))
    with pytest.raises(ValueError, match="expected torch.bfloat16"):     # one type for both
        call(FAKE, "bf16", torch.zeros(4, 100))


# ------------------------------------------------------------------ GPU
@pytest.fixture(scope="module")
def usp():
    import torch
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    build.build()
    return usp_mod


def _np(t):
    return t.detach().float().cpu().numpy().astype(np.float64)


def _dev(x):
    import torch
    return torch.from_numpy(np.ascontiguousarray(x)).cuda()


def _done(usp, guard):
    import torch
    torch.cuda.synchronize()
    assert usp.usp_device_status() == 0
    assert guard.damaged() == []


def _put(guard, x):
    import torch
    x = torch.as_tensor(x)
    y = guard.empty(tuple(x.shape), x.dtype, "cuda")
    y.copy_(x)
    return y


def _freq(half):
    return (500000.0 ** (-np.arange(half) / max(half, 1))).astype(np.float32)


ROTARY = [("bf16", 32, 8, 128, (16, 24, 24), False, False), ("bf16", 4, 2, 64, (12, 10, 10), True, False),
          ("f32", 4, 4, 64, (16, 16), False, True), ("f32", 5, 1, 128, (8, 8, 8, 8), True, False),
          ("bf16", 3, 3, 128, (56,), False, True), ("bf16", 2, 1, 64, (5, 3), False, False), ("f32", 1, 1, 64, (), False, False)]


@pytest.mark.gpu
@pytest.mark.parametrize("dtype,Hq,Hkv,d,sections,cycled,inter", ROTARY)
@pytest.mark.parametrize("B,N,P", [(1, 1, 1), (1, 37, 1), (2, 150, 2), (1, 1202, 2)])
def test_rotary(usp, dtype, Hq, Hkv, d, sections, cycled, inter, B, N, P):
    import torch
    r = usp.Rotary.sections(sections, cycled, inter)
    p = usp.Problem(B, Hq, Hkv, N, d, P, dtype=dtype)
    dt, T, half = p.torch_dtype, B * N, len(r.axis)
    rng = np.random.default_rng(N)
    gen = torch.Generator().manual_seed(N)
    qkv = torch.randn((P, B, N // P, Hq + 2 * Hkv, d), generator=gen).to(dt).cuda()
    q, k = qkv[..., :Hq, :], qkv[..., Hq:Hq + Hkv, :]
    pos = rng.integers(0, 2 ** 31 - 1 if N == 37 else 5000, (max(r.axes, 1), T)).astype(np.int32)
    if N == 37:
        pos[:, :5] *= -1
    guard = Guarded()
    inv, dpos = _freq(half), _put(guard, torch.from_numpy(pos))
    f = _put(guard, torch.from_numpy(inv)) if half else None
    for inverse in (False, True):
        qo, ko = guard.empty(p.seq_shape(Hq), dt, "cuda"), guard.empty(p.seq_shape(Hkv), dt, "cuda")
        usp.usp_rotary_embed(p, r, q, k, dpos, f, qo, ko, inverse)
        # into slices of one gradient, keys alone; in place
        both = guard.empty(tuple(qkv.shape), dt, "cuda").fill_(3.0)
        usp.usp_rotary_embed(p, r, None, k, dpos, f, None, both[..., Hq:Hq + Hkv, :], inverse)
        same = qkv.clone()
        usp.usp_rotary_embed(p, r, same[..., :Hq, :], None, dpos, f, same[..., :Hq, :], None, inverse)
        _done(usp, guard)
        for got, x in ((qo, q), (ko, k)):
            want, mag = ref_rotate(_np(x).reshape(T, -1, d), pos, r.axis, inv, inter, inverse)
            bound = 8 * 2.0 ** -24 * mag + U[dtype] * np.abs(want) * (1 + 2.0 ** -20)
            bound[..., 2 * half:] = 0
            assert (np.abs(_np(got).reshape(want.shape) - want) <= bound).all()
        assert torch.equal(both[..., Hq:Hq + Hkv, :], ko) and (both[..., :Hq, :] == 3).all() and (both[..., Hq + Hkv:, :] == 3).all()
        assert torch.equal(same[..., :Hq, :], qo) and torch.equal(same[..., Hq:, :], qkv[..., Hq:, :])


@pytest.mark.gpu
@pytest.mark.parametrize("inter", [False, True])
def test_rotary_backward_is_the_gradient(usp, inter):
    """Of L = sum g . R x: dL/dx_i against differences (L is linear, so a step of 1 is as good as any), in float32: each of
    the 2 T H d terms of L carries 10 2^-24 of (|a| + |b|) |g|, a difference of two L's twice their sum."""
    import torch
    r = usp.Rotary.sections((10, 11, 11), False, inter)
    p = usp.Problem(1, 2, 1, 6, 64, 1, dtype="f32")
    gen = torch.Generator().manual_seed(0)
    x, g = (torch.randn(p.seq_shape(2), generator=gen).cuda() for _ in range(2))
    pos = torch.randint(0, 9000, (3, 1, 1, 6), generator=gen).int().cuda()
    f = _dev(_freq(32))
    dx, none = usp.rotary_embed(p, r, g, None, pos, f, inverse=True)
    assert none is None
    L = lambda y: float((usp.rotary_embed(p, r, y, None, pos, f)[0].double() * g.double()).sum())  # noqa: E731
    base = L(x)
    bound = 2 * 10 * 2.0 ** -24 * 2 * float((x.abs() + 1).max()) * float(g.abs().sum())
    for i in (0, 1, 17, 33, 63, 64, 200, 500, 767):
        y = x.clone()
        y.view(-1)[i] += 1.0
        step = float(y.view(-1)[i] - x.view(-1)[i])
        assert abs((L(y) - base) - step * float(dx.view(-1)[i])) <= bound


@pytest.mark.gpu
@pytest.mark.parametrize("dtype,Hq,Hkv,d,sections,cycled,inter", ROTARY)
@pytest.mark.parametrize("T,page", [(1, 16), (130, 64)])
def test_append_axes(usp, dtype, Hq, Hkv, d, sections, cycled, inter, T, page):
    import torch
    r = usp.Rotary.sections(sections, cycled, inter)
    rng = np.random.default_rng(T)
    B, mp = 3, 4
    c = usp.Cache(B * mp + 1, page, B, mp, Hq, Hkv, d, dtype=dtype)
    dt = c.torch_dtype
    guard = Guarded()
    table = rng.permutation(c.n_pages)[:B * mp].reshape(B, mp).astype(np.int32)
    slots = rng.permutation(B * mp * page)[:T]
    seq, pos = (slots // (mp * page)).astype(np.int32), (slots % (mp * page)).astype(np.int32)
    live = np.ones(T, bool)
    if T > 3:
        seq[1], pos[2], live[1], live[2] = -1, -1, False, False
    rpos = rng.integers(0, 100000, (max(r.axes, 1), T)).astype(np.int32)
    gen = torch.Generator().manual_seed(T)
    qkv = torch.randn((T, (Hq + 2 * Hkv) * d), generator=gen).to(dt).cuda()
    q, k, v = (x.view(T, -1, d) for x in qkv.split([Hq * d, Hkv * d, Hkv * d], 1))
    inv = _freq(len(r.axis))
    kp, vp = (guard.empty(c.pool_shape(), dt, "cuda").fill_(3.0) for _ in range(2))
    qo, ko = guard.empty((T, Hq, d), dt, "cuda").fill_(5.0), guard.empty((T, Hkv, d), dt, "cuda").fill_(5.0)
    f = _dev(inv) if len(inv) else None
    args = (_dev(seq), _dev(pos))
    usp.usp_kv_append_axes(c, T, q, k, v, *args, _put(guard, rpos), f, r, qo, ko, kp, vp, _dev(table))
    _done(usp, guard)
    for got, x in ((qo, q), (ko, k)):
        want, mag = ref_rotate(_np(x), rpos, r.axis, inv, inter)
        bound = 8 * 2.0 ** -24 * mag + U[dtype] * np.abs(want) * (1 + 2.0 ** -20)
        bound[..., r.rot:] = 0
        assert (np.abs(_np(got) - want)[live] <= bound[live]).all() and (_np(got)[~live] == 5).all()
    wk, wv = np.full(c.pool_shape(), 3.0), np.full(c.pool_shape(), 3.0)
    for t in np.flatnonzero(live):
        at = (table[seq[t], pos[t] // page], slice(None), pos[t] % page)
        wk[at], wv[at] = _np(ko)[t], _np(v)[t]
    assert np.array_equal(_np(kp), wk) and np.array_equal(_np(vp), wv)
    # the same position on every axis: the bits of the call with one
    one = np.stack([rpos[0]] * rpos.shape[0])
    got = []
    for axes in (True, False):
        kp2, vp2 = torch.full_like(kp, 3.0), torch.full_like(vp, 3.0)
        q2 = torch.full_like(qo, 5.0)
        if axes:
            usp.usp_kv_append_axes(c, T, q, k, v, *args, _dev(one), f, r, q2, None, kp2, vp2, _dev(table))
        else:
            usp.usp_kv_append(c, T, q, k, v, *args, f, q2, None, kp2, vp2, _dev(table), r.rot, inter, _dev(rpos[0]))
        got.append((q2, kp2, vp2))
    torch.cuda.synchronize()
    for a, b in zip(*got):
        assert torch.equal(a, b)


class Pool:
    """A cache's state on the GPU beside the model of it."""

    def __init__(self, usp, guard, B, mp, page, n, seed=0, Hkv=1, d=64, dtype="bf16", data=False):
        import torch
        self.usp, self.rng, self.page = usp, np.random.default_rng(seed), page
        self.c = usp.Cache(n, page, B, mp, Hkv, Hkv, d, dtype=dtype)
        self.table, self.lens, self.ref = np.full((B, mp), -1, np.int32), np.zeros(B, np.int32), np.zeros(n, np.int32)
        self.g = [_put(guard, x) for x in (self.lens, self.table, self.ref)]
        self.copies = guard.empty((1 + B, 4), torch.int32, "cuda").fill_(-7)
        size = usp.usp_pages_update_workspace_size(self.c)
        self.ws = guard.bytes(size, "cuda")
        self.ws.fill_(0xFF)
        self.guard = guard
        self.dargs = [guard.empty((B,), torch.int32, "cuda") for _ in range(3)]
        if data:
            self.kv = [torch.full(self.c.pool_shape(), 0.0, dtype=self.c.torch_dtype, device="cuda") for _ in range(2)]

    def put(self):
        import torch
        for x, y in zip(self.g, (self.lens, self.table, self.ref)):
            x.copy_(torch.from_numpy(y))

    def call(self, args, stream=None):
        lens, table, ref = self.g
        self.usp.usp_pages_update(self.c, *args, lens, table, ref, self.copies, self.ws, None, stream)

    def step(self, parent, keep, grow, call=None):
        import torch
        before = self.copies.cpu().numpy().copy()
        args = []
        for x, d in zip((parent, keep, grow), self.dargs):
            if x is not None:
                d.copy_(torch.from_numpy(np.asarray(x, np.int32)))
            args.append(None if x is None else d)
        (call or self.call)(args)
        _done(self.usp, self.guard)
        self.table, self.lens, self.ref, head, made = ref_update(self.page, self.table, self.lens, self.ref, parent, keep, grow)
        for got, want in zip(self.g, (self.lens, self.table, self.ref)):
            assert np.array_equal(got.cpu().numpy(), want)
        got = self.copies.cpu().numpy()
        assert tuple(got[0]) == head
        assert [tuple(x) for x in got[1:1 + len(made)]] == made
        assert np.array_equal(got[1 + len(made):], before[1 + len(made):])
        return head, made


def _any_step(rng, B, cap, most):
    parent = np.where(rng.random(B) < 0.6, np.arange(B), rng.integers(-2, B + 2, B))
    keep = np.where(rng.random(B) < 0.5, rng.integers(-3, cap + 5, B), 1 << 30)
    grow = np.where(rng.random(B) < 0.7, rng.integers(-2, most, B), rng.integers(0, 3, B))
    return [None if rng.random() < 0.15 else x.astype(np.int32) for x in (parent, keep, grow)]


@pytest.mark.gpu
@pytest.mark.parametrize("B,mp,page,n", [(1, 1, 16, 1), (1, 4, 16, 3), (5, 6, 16, 21), (9, 3, 256, 40), (33, 40, 32, 700),
                                         (70, 100, 64, 4097), (1100, 5, 16, 3000), (3, 2000, 16, 20001), (6, 7, 16, 0),
                                         (4, 0, 16, 5), (300, 1000, 16, 9000), (1024, 9, 16, 16384), (2500, 3, 16, 100),
                                         (2500, 4, 16, 6000)])
def test_pages_update(usp, B, mp, page, n):
    guard = Guarded()
    pool = Pool(usp, guard, B, mp, page, n, seed=B)
    rng = pool.rng
    lacking = copies = 0
    for i in range(25):
        head, made = pool.step(*_any_step(rng, B, mp * page, max(3, n * page // (2 * B))))
        lacking += head[1] > 0
        copies += head[0]
        if i == 12 and n > 4 and B > 1 and mp:      # a page held by the caller, an entry that is no page, a length out of range
            pool.ref[rng.integers(n)] += 1
            b = int(rng.integers(B))
            if pool.lens[b] > 0:
                x = pool.table[b, 0]
                pool.ref[x] -= 1
                pool.table[b, 0] = (-5, n, 1 << 30)[i % 3]
                pool.lens[b] = max(1, pool.lens[b])
            empty = np.flatnonzero(pool.lens == 0)
            if len(empty):
                pool.lens[empty[0]] = -9
            pool.put()
    if n and mp:
        assert lacking < 25 and (copies > 0 or B == 1 or n < B)


@pytest.mark.gpu
def test_pages_update_when_pages_lack(usp):
    """Nothing changes, and the call says how many are lacking; with as many as there are it goes through."""
    guard = Guarded()
    pool = Pool(usp, guard, 3, 8, 16, 10)
    assert pool.step(None, None, [40, 40, 17])[0] == (0, 0, 2, 0)
    assert pool.step(None, None, [8, 8, 33])[0] == (0, 0, 0, 0)      # 48, 48 and 50 tokens: two pages more for the third
    assert pool.step(None, None, [9, 0, 31])[0] == (0, 3, 0, 0)      # 57 and 81 tokens: one page and two
    assert pool.step(None, None, [8, 8, 31])[0] == (0, 4, 0, 0)
    assert pool.step([0, 0, 0], [48, 48, 48], [1, 1, 1])[0] == (0, 0, 10 - 3 - 3, 0)     # what is freed is there at once
    assert pool.step([-1, -1, -1], None, None)[0] == (0, 0, 10, 0)
    assert pool.step(None, None, [64, 64, 33])[0] == (0, 1, 10, 0)   # eleven pages of ten
    assert pool.step(None, None, [64, 64, 32])[0] == (0, 0, 0, 0)


@pytest.mark.gpu
def test_nothing_to_keep_books_of(usp):
    """Caches without slots, pages or entries: the list's head is written all the same."""
    import torch
    guard = Guarded()
    for B, mp, n in ((0, 3, 50), (0, 0, 0), (3, 0, 7), (2, 2, 0), (1500, 0, 0), (1500, 2, 0)):
        c = usp.Cache(n, 16, B, mp, 1, 1, 64)
        lens, table, ref = usp.pages_empty(c)
        copies = guard.empty((1 + B, 4), torch.int32, "cuda").fill_(-7)
        ws = guard.bytes(max(usp.usp_pages_update_workspace_size(c), 256), "cuda")
        usp.usp_pages_update(c, None, None, torch.full((B,), 5, dtype=torch.int32, device="cuda"), lens, table, ref, copies, ws)
        _done(usp, guard)
        need = B if mp else 0
        assert copies[0].tolist() == [0, max(0, need - n), n, 0] and (copies[1:] == -7).all() and (lens == 0).all()
        many, new_id = usp.pages_compact(c, table, ref)
        assert many[0].tolist() == [0, 0, n, 0] and (new_id == -1).all()


@pytest.mark.gpu
def test_the_largest_pool(usp):
    """2^23 pages: grown from nothing pages go out from 0 on; half of them given up, the others move to the front."""
    import torch
    n, mp = 1 << 23, 1 << 22
    c = usp.Cache(n, 16, 3, mp, 1, 1, 64)
    lens, table, ref = usp.pages_empty(c)
    i32 = dict(dtype=torch.int32, device="cuda")
    grow = torch.tensor([16 * mp - 1, 16 * 1000, 16 * (mp - 1000)], **i32)
    assert usp.pages_update(c, lens, table, ref, grow=grow)[0].tolist() == [0, 0, 0, 0]
    assert torch.equal(table.view(-1)[:mp], torch.arange(mp, **i32)) and (ref == 1).all()
    assert torch.equal(table[2, :mp - 1000], torch.arange(mp + 1000, 2 * mp, **i32)) and (table[2, mp - 1000:] == -1).all()
    head = usp.pages_update(c, lens, table, ref, parent=torch.tensor([1, -1, 2], **i32))[0].tolist()
    assert head == [0, 0, n - 1000 - (mp - 1000), 0] and lens.tolist() == [16000, 0, 16 * (mp - 1000)]
    before = table.clone()
    copies, new_id = usp.pages_compact(c, table, ref)
    # live: mp .. mp + 999 (slot 0's) and mp + 1000 .. 2 mp - 1 (slot 2's), mp pages, which go to 0 .. mp - 1
    assert copies[0].tolist() == [mp, 0, n - mp, 0] and (ref[:mp] == 1).all() and (ref[mp:] == 0).all()
    assert torch.equal(copies[1:, 0], torch.arange(mp, 2 * mp, **i32)) and torch.equal(copies[1:, 1], torch.arange(mp, **i32))
    assert torch.equal(table, torch.where(before >= 0, before - mp, before))
    assert (new_id[:mp] == -1).all() and torch.equal(new_id[mp:], torch.arange(mp, **i32))


@pytest.mark.gpu
@pytest.mark.parametrize("B", [4, 70, 1000])
def test_pages_update_long_rows_among_short(usp, B):
    """Conversations of thousands of pages among short ones: grown, forked, reordered (rows put aside), truncated, freed."""
    guard = Guarded()
    mp = 8000 if B < 70 else 900
    pool = Pool(usp, guard, B, mp, 16, 16000, seed=B)
    most, own = mp * 16, np.arange(B)
    grow = np.full(B, 20)
    grow[1], grow[3] = most - 5, most // 2 + 3
    assert pool.step(None, None, grow)[0][1] == 0
    parent = own.copy()
    parent[0], parent[2] = 1, 3
    assert pool.step(parent, None, np.ones(B, int))[0][0] == 1 + 1   # (20, most - 5 and most / 2 + 3 tokens all end inside)
    parent[[0, 1, 2, 3]] = [3, 0, 1, 2]                    # all change places
    pool.step(parent, np.full(B, most - 100), np.zeros(B, int))
    pool.step(parent, None, np.full(B, 3))
    pool.step(None, np.where(own % 2, 7, most), np.zeros(B, int))
    pool.step(None, np.zeros(B, int), None)
    assert (pool.ref == 0).all()


@pytest.mark.gpu
@pytest.mark.parametrize("dtype,Hkv,d,page", [("bf16", 2, 64, 16), ("f32", 3, 128, 32), ("bf16", 8, 128, 64)])
def test_sequences_keep_their_tokens(usp, dtype, Hkv, d, page):
    """Forks, reorderings, refused tokens and compactions at random, with their copies, and new tokens written: what each slot
    reads through the table is always what the tokens were."""
    import torch
    guard = Guarded()
    B, mp, n = 7, 9, 60
    pool = Pool(usp, guard, B, mp, page, n, seed=page, Hkv=Hkv, d=d, dtype=dtype, data=True)
    c, (kp, vp), rng = pool.c, pool.kv, pool.rng
    said = [np.zeros(0, np.int64) for _ in range(B)]     # a number for each token of each slot
    clock, moved = 0, 0
    for i in range(40):
        parent = np.where(rng.random(B) < 0.7, np.arange(B), rng.integers(0, B, B)).astype(np.int32)
        keep = np.where(rng.random(B) < 0.3, rng.integers(0, 60, B), 1 << 20).astype(np.int32)
        grow = rng.integers(0, 25, B).astype(np.int32)
        head, _ = pool.step(parent, keep, grow)
        usp.usp_pages_copy(c, B, pool.copies, kp, vp)
        if head[1] == 0:
            kept = [min(int(keep[b]), len(said[parent[b]])) for b in range(B)]
            said = [said[parent[b]][:kept[b]] for b in range(B)]
            seq, pos = [], []
            for b in range(B):
                m = int(pool.lens[b]) - kept[b]
                seq += [b] * m
                pos += range(kept[b], kept[b] + m)
                said[b] = np.concatenate([said[b], clock + np.arange(m)])
                clock += m
            if seq:
                x = torch.cat([torch.from_numpy(s[int(k):]) for s, k in zip(said, kept)]).remainder(251).to(c.torch_dtype)
                x = x.cuda()[:, None, None].expand(-1, Hkv, d).contiguous()
                usp.kv_append(c, None, x, -x, _dev(np.array(seq, np.int32)), _dev(np.array(pos, np.int32)), None, kp, vp, pool.g[1])
        if i % 5 == 4:
            live = int((pool.ref > 0).sum())
            copies, new_id = usp.pages_compact(c, pool.g[1], pool.g[2])
            usp.pages_copy(c, copies, kp, vp)
            torch.cuda.synchronize()
            new = new_id.cpu().numpy()
            assert sorted(new[new >= 0]) == list(range(live)) and ((new < 0) == (pool.ref <= 0)).all()
            assert np.array_equal(pool.g[1].cpu().numpy(), np.where(pool.table >= 0, new[pool.table], pool.table))
            ref = np.zeros_like(pool.ref)
            ref[new[new >= 0]] = pool.ref[new >= 0]
            assert np.array_equal(pool.g[2].cpu().numpy(), ref)
            moved += int(copies[0, 0])
            pool.table, pool.ref = pool.g[1].cpu().numpy(), ref
        k, v = kp.cpu().float().numpy(), vp.cpu().float().numpy()
        for b in range(B):
            assert len(said[b]) == pool.lens[b]
            t = np.arange(len(said[b]))
            got = k[pool.table[b, t // page], :, t % page]
            assert (got == (said[b] % 251)[:, None, None]).all() and (v[pool.table[b, t // page], :, t % page] == -got).all()
    assert moved > 0 and clock > 300


@pytest.mark.gpu
@pytest.mark.parametrize("n,B,mp,live", [(1, 1, 1, 1.0), (2, 1, 2, 0.5), (300, 12, 31, 0.6), (4097, 50, 70, 0.3), (40000, 3, 7, 0.9),
                                         (1000, 4, 4, 0.0), (1000, 300, 3, 1.0), (0, 2, 2, 0.0), (8192, 5, 9, 0.5), (8193, 5, 9, 0.5), (9104, 127, 297, 0.5),
                                         (70001, 9, 50, 0.5), (300000, 2, 9, 0.2)])
@pytest.mark.parametrize("in_place", [False, True])
def test_pages_compact(usp, n, B, mp, live, in_place):
    import torch
    rng = np.random.default_rng(n)
    guard = Guarded()
    c = usp.Cache(n, 16, B, mp, 1, 1, 64)
    ref = (rng.random(n) < live).astype(np.int32) * rng.integers(1, 5, n).astype(np.int32)
    if n > 100:
        ref[rng.integers(0, n, 5)] = -3               # counted too low: free
    table = rng.integers(-2, n + 2, (B, mp)).astype(np.int32)
    g = [_put(guard, x) for x in (table, ref)]
    out = g if in_place else [guard.empty(tuple(x.shape), torch.int32, "cuda") for x in g]
    new_id = guard.empty((n,), torch.int32, "cuda")
    copies = guard.empty((1 + n // 2, 4), torch.int32, "cuda").fill_(-7)
    usp.usp_pages_compact(c, *g, *out, new_id, copies)
    _done(usp, guard)
    m = int((ref > 0).sum())
    holes = [i for i in range(m) if ref[i] <= 0]
    movers = [i for i in range(m, n) if ref[i] > 0]
    new, want = np.where(ref > 0, np.arange(n), -1), np.where(ref > 0, ref, 0)
    for i, to in zip(movers, holes):
        new[i], want[to], want[i] = to, ref[i], 0
    assert np.array_equal(new_id.cpu().numpy(), new) and np.array_equal(out[1].cpu().numpy(), want)
    inside = (table >= 0) & (table < n)
    named = np.where(inside, np.append(new, -1)[np.clip(table, 0, n)], -1)
    assert np.array_equal(out[0].cpu().numpy(), np.where(named >= 0, named, table))
    rows = copies.cpu().numpy()
    assert tuple(rows[0]) == (len(movers), 0, n - m, 0)
    assert [tuple(x) for x in rows[1:1 + len(movers)]] == [(i, to, 16, 0) for i, to in zip(movers, holes)]
    assert (rows[1 + len(movers):] == -7).all()


@pytest.mark.gpu
@pytest.mark.parametrize("dtype,Hkv,d,page,layers", [("bf16", 1, 64, 16, 1), ("bf16", 8, 128, 64, 3), ("f32", 5, 128, 256, 1),
                                                    ("f32", 2, 64, 32, 2)])
def test_pages_copy(usp, dtype, Hkv, d, page, layers):
    import torch
    guard = Guarded()
    n = 24
    c = usp.Cache(n, page, 1, 1, Hkv, Hkv, d, dtype=dtype)
    gen = torch.Generator().manual_seed(page)
    host = [torch.randn((layers, *c.pool_shape()), generator=gen).to(c.torch_dtype) for _ in range(2)]
    g = [_put(guard, x) for x in host]
    order = np.random.default_rng(page).permutation(n)
    rows = [(order[2 * i], order[2 * i + 1], t, 0) for i, t in enumerate([page, 1, 0, page - 1, page // 2 + 1, -4, page + 9, 7])]
    bad = [(-1, order[20], page, 0), (order[21], n, page, 0), (order[22], order[22], page, 0), (1 << 30, order[20], page, 0)]
    after = [(order[17], order[18], page, 0)]
    head = [(len(rows) + len(bad), 0, 0, 0)]
    copies = _put(guard, np.array(head + rows + bad + after, np.int32))
    usp.usp_pages_copy(c, len(copies) - 1, copies, *g, layers, g[0][0].numel())
    _done(usp, guard)
    for x, y in zip(host, g):
        want = x.clone()
        for a, b, t, _ in rows:
            t = min(max(t, 0), page)
            want[:, b, :, :t] = x[:, a, :, :t]
        assert torch.equal(y.cpu(), want)
    # no more than max_copies, whatever the list says; a list that says nothing
    for count, most in ((1000, 2), (-3, 5), (0, 5)):
        g = [_put(guard, x) for x in host]
        copies[0, 0] = count
        usp.pages_copy(c, copies[:1 + most], *(g if layers > 1 else [y[0] for y in g]))
        _done(usp, guard)
        for x, y in zip(host, g):
            want = x.clone()
            for a, b, t, _ in rows[:most] if count > 0 else []:
                want[:, b, :, :min(max(t, 0), page)] = x[:, a, :, :min(max(t, 0), page)]
            assert torch.equal(y.cpu(), want)


@pytest.mark.gpu
def test_pages_copy_beyond_32_bit_offsets(usp):
    import torch
    c = usp.Cache((1 << 31) // (8 * 64 * 128) + 9, 64, 1, 1, 8, 8, 128)
    kp, vp = (torch.empty(c.pool_shape(), dtype=torch.bfloat16, device="cuda") for _ in range(2))
    n = c.n_pages
    for x in (kp, vp):
        x[n - 4:].normal_()
        x[:3].zero_()
    copies = torch.tensor([[2, 0, 0, 0], [n - 1, 1, 64, 0], [n - 2, n - 4, 33, 0]], dtype=torch.int32, device="cuda")
    last = [x[n - 4].clone() for x in (kp, vp)]
    usp.pages_copy(c, copies, kp, vp)
    torch.cuda.synchronize()
    for x, y in zip((kp, vp), last):
        assert torch.equal(x[1], x[n - 1]) and (x[0] == 0).all() and (x[2] == 0).all()
        assert torch.equal(x[n - 4, :, :33], x[n - 2, :, :33]) and torch.equal(x[n - 4, :, 33:], y[:, 33:])
    del kp, vp, x
    torch.cuda.empty_cache()


def _drafts(rng, nq, V, dtype, sharp=2.0, greedy=False, gap=0):
    """Rows of probabilities as float64 of what the type holds, and the same on the GPU, `gap` elements between rows."""
    import torch
    T = sum(nq)
    dt = torch.bfloat16 if dtype == "bf16" else torch.float32
    logits = rng.standard_normal((T, V)) * sharp
    near = np.roll(logits, 1, 0) + rng.standard_normal((T, V)) * 0.3 * sharp
    soft = lambda x: np.exp(x - x.max(1, keepdims=True)) / np.exp(x - x.max(1, keepdims=True)).sum(1, keepdims=True)  # noqa: E731
    target, draft = soft(logits), soft(near)
    tokens = np.array([rng.choice(V, p=row) for row in draft], np.int32) if not greedy else near.argmax(1).astype(np.int32)

    def dev(x):
        y = torch.full((T, V + gap), float("nan"), dtype=dt, device="cuda")
        y[:, :V] = torch.from_numpy(x).to(dt).cuda()
        return y[:, :V]

    tg, dr = dev(target), None if greedy else dev(draft)
    q_start = np.concatenate([[0], np.cumsum(nq)]).astype(np.int32)
    return dict(tg=tg, dr=dr, target=_np(tg), draft=None if greedy else _np(dr), tokens=tokens, q_start=q_start,
                u=rng.random(T).astype(np.float32) * np.float32(1 - 2.0 ** -24), lens=(np.array(nq) + rng.integers(1, 1000, len(nq))).astype(np.int32))


def _verify(usp, x, T=None):
    import torch
    guard = Guarded()
    n = len(x["q_start"]) - 1
    out = [guard.empty((n,), torch.int32, "cuda").fill_(-77) for _ in range(3)]
    ins = [_put(guard, x[k]) for k in ("tokens", "u", "q_start", "lens")]
    usp.usp_verify_drafts(n, x["target"].shape[0], x["target"].shape[1], x["tg"], x["dr"], *ins[:2], ins[2], ins[3], *out)
    _done(usp, guard)
    got = np.stack([o.cpu().numpy() for o in out])
    want = ref_verify(x["target"], x["draft"], x["tokens"], x["u"], x["q_start"], x["lens"])
    assert np.array_equal(got, want), (got[:, (got != want).any(0)][:, :5], want[:, (got != want).any(0)][:, :5])
    return got


@pytest.mark.gpu
@pytest.mark.parametrize("dtype", ["f32", "bf16"])
@pytest.mark.parametrize("greedy", [False, True])
@pytest.mark.parametrize("V", [1, 2, 31, 33, 511, 4096, 4097, 20001])
def test_verify(usp, V, greedy, dtype):
    rng = np.random.default_rng(V)
    for nq, gap in (([1], 0), ([5], 3), ([3, 1, 0, 6, 2, 4, 70, 1], 8), ([2] * 90, 0)):
        if V * sum(nq) < 3_000_000:
            got = _verify(usp, _drafts(rng, nq, V, dtype, greedy=greedy, gap=gap))
            if 4096 > V > 2 and len(nq) > 20:
                assert 0 < got[0].sum() < 90


@pytest.mark.gpu
@pytest.mark.parametrize("dtype", ["f32", "bf16"])
@pytest.mark.parametrize("seqs", [1, 80, 400])
def test_verify_a_large_vocabulary(usp, seqs, dtype):
    """Weights that differ by many orders of magnitude, so that the running sum needs its bits; at the largest vocabulary
    the one sequence is spread over the most CTAs, with many it is one's."""
    rng = np.random.default_rng(seqs)
    V = {1: 1 << 19, 80: 131072, 400: 32768}[seqs]
    T = {1: 3, 80: 160, 400: 800}[seqs]
    import torch
    gen = torch.Generator(device="cuda").manual_seed(seqs)
    dt = torch.bfloat16 if dtype == "bf16" else torch.float32
    tg, dr = (torch.softmax(torch.randn((T, V), generator=gen, device="cuda") * 5, 1).to(dt) for _ in range(2))
    x = dict(tg=tg, dr=dr, target=_np(tg), draft=_np(dr), tokens=rng.integers(0, V, T).astype(np.int32),
             u=rng.random(T).astype(np.float32), q_start=np.linspace(0, T, seqs + 1).astype(np.int32),
             lens=rng.integers(5, 1000, seqs).astype(np.int32))
    x["u"] = np.minimum(x["u"], np.float32(1 - 2.0 ** -24))
    _verify(usp, x)


@pytest.mark.gpu
@pytest.mark.parametrize("dtype", ["f32", "bf16"])
def test_verify_odd_rows(usp, dtype):
    """Drafts and targets that are equal, rows without mass, NaN, infinities, negative numbers and rows of ones, drafts that
    are no tokens, the ends of the random numbers, starts out of range and out of order."""
    import torch
    rng = np.random.default_rng(7)
    V = 5000
    x = _drafts(rng, [3] * 24, V, dtype)
    tg, dr = x["tg"], x["dr"]
    tg[0:3] = dr[0:3].roll(-1, 0)                    # 0: the draft's own rows: every u accepts
    tg[3:6] = 0                                      # 1: nothing at all
    dr[7] = 1.0                                      # 2: q over p everywhere: drawn from p itself
    tg[9, 17] = float("nan")                         # 3: a NaN where the draft is
    x["tokens"][10] = 17
    tg[12:15] = float("nan")                         # 4
    tg[15, 5], tg[15, 6] = float("inf"), -3.0        # 5
    tg[18:21] = 1.0                                  # 6: no probabilities at all
    x["tokens"][22], x["tokens"][25] = -1, V         # 7, 8: no tokens
    dr[28] = float("nan")                            # 9
    x["u"][30:33], x["u"][33:36] = 0.0, 1 - 2.0 ** -24   # 10, 11
    dr[36:39] = 0                                    # 12: a draft of probability 0
    tg[39:42] = 0
    tg[39:42, V - 1] = 1.0                           # 13: all on the last token
    tg[42:45] = 0
    tg[42:45, 0] = 2.0 ** -50                        # 14: less than half a step of mass
    x["u"][45:48] = float("nan")                     # 15
    x["u"][48], x["u"][51] = 1.0, -0.5               # 16, 17
    x["target"], x["draft"] = _np(tg), _np(dr)
    x["u"] = x["u"].astype(np.float32)
    clean = dict(x)
    clean["u"] = np.nan_to_num(x["u"], nan=0.0)
    clean["u"][46:48] = np.inf                       # (a NaN refuses; as the number of a draw it is 0)
    guard = Guarded()
    n = 24
    want = ref_verify(clean["target"], clean["draft"], clean["tokens"], clean["u"], clean["q_start"], clean["lens"])
    assert want[0, 0] == 2 and want[1, 1] == -1 and want[1, 4] == -1 and want[1, 13] == V - 1 and want[1, 14] == -1
    for start in (x["q_start"], np.array([-5, 3, 2, 9, 40, 30, 72, 100, 80], np.int32)):
        m = len(start) - 1
        out = [guard.empty((m,), torch.int32, "cuda").fill_(-77) for _ in range(2)]
        usp.usp_verify_drafts(m, 72, V, tg, dr, _put(guard, x["tokens"]), _put(guard, x["u"]), _put(guard, start), None, *out, None)
        _done(usp, guard)
        if m == n:
            assert np.array_equal(np.stack([o.cpu().numpy() for o in out]), want[:2])
        else:
            alone = ref_verify(clean["target"], clean["draft"], clean["tokens"], clean["u"], start, np.zeros(m))
            assert np.array_equal(np.stack([o.cpu().numpy() for o in out]), alone[:2])


@pytest.mark.gpu
@pytest.mark.parametrize("dtype", ["f32", "bf16"])
@pytest.mark.parametrize("V", [131072, 1 << 19])
def test_verify_rows_of_ones_whatever_the_cut(usp, V, dtype):
    """Rows need not add up to 1: from the largest sums, 2^65 in whole numbers, a sequence draws the same token alone (eight
    CTAs), among 70 (seven) and among 400 (one).  With V equal weights that is the token floor(u V), exactly."""
    import torch
    dt = torch.bfloat16 if dtype == "bf16" else torch.float32
    ends = np.array([0.9, 0.0, 1 - 2.0 ** -24, 0.125, np.nextafter(np.float32(0.125), np.float32(0)), 0.5, 2.0 ** -19, 0.99], np.float32)
    for seqs in (1, 70, 400):
        rng = np.random.default_rng(seqs)
        u = np.concatenate([ends[:seqs], (rng.integers(0, 1 << 24, max(seqs - 8, 0)) * 2.0 ** -24).astype(np.float32)])
        for rows in (1, 2):                               # the last row's p; p - q, each 1/2, behind a draft that is refused
            guard = Guarded()
            target = torch.ones((seqs * rows, V), dtype=dt, device="cuda")
            draft = None if rows == 1 else torch.full((seqs * rows, V), 0.5, dtype=dt, device="cuda")
            numbers = np.repeat(u, rows)
            out = [guard.empty((seqs,), torch.int32, "cuda").fill_(-77) for _ in range(2)]
            usp.usp_verify_drafts(seqs, seqs * rows, V, target, draft, _put(guard, np.full(seqs * rows, -1, np.int32)),
                                  _put(guard, numbers), _put(guard, np.arange(0, seqs * rows + 1, rows, dtype=np.int32)), None, *out, None)
            _done(usp, guard)
            assert (out[0] == 0).all()
            assert np.array_equal(out[1].cpu().numpy(), np.floor(u.astype(np.float64) * V).astype(np.int64)), (seqs, rows)
        del target, draft
        torch.cuda.empty_cache()


@pytest.mark.gpu
@pytest.mark.parametrize("V,close", [(1 << 17, 2.0 ** -19), (1 << 17, 2.0 ** -8), (50001, 2.0 ** -21), (1000, 0.25)])
def test_verify_draws_from_what_little_is_left(usp, V, close):
    """Target and draft that nearly agree, against running sums in 64 bits.  Two roundings of half a step, 2^-47, to a weight: the
    running sum S_x less u times the total W is off by V 2^-46 at most, so u lies within V 2^-46 / W of the token's share
    [S_x-1 / W, S_x / W]; the comparison's own sums are off by V 2^-53 of W."""
    import torch
    rng = np.random.default_rng(V)
    n = 64
    p = rng.random(V) + 0.5
    p = (p / p.sum()).astype(np.float32)
    q = (p * (1 + close * rng.choice([-1.0, 1.0], V))).astype(np.float32)
    x = int(np.argmax(q / p))                             # refused by the largest number
    w = np.maximum(p.astype(np.float64) - q.astype(np.float64), 0)
    S, W = np.cumsum(w), w.sum()
    assert 0 < W < 2 * close and q[x] * (1 - 2.0 ** -24) >= p[x]
    u = np.empty((n, 2), np.float32)
    u[:, 0], u[:, 1] = (rng.integers(0, 1 << 24, n) * 2.0 ** -24), 1 - 2.0 ** -24
    guard = Guarded()
    tg, dr = (torch.from_numpy(y).cuda().repeat(2 * n, 1) for y in (p, q))
    out = [guard.empty((n,), torch.int32, "cuda").fill_(-77) for _ in range(2)]
    usp.usp_verify_drafts(n, 2 * n, V, tg, dr, _put(guard, np.full(2 * n, x, np.int32)), _put(guard, u.reshape(-1)),
                          _put(guard, np.arange(0, 2 * n + 1, 2, dtype=np.int32)), None, *out, None)
    _done(usp, guard)
    got, at = out[1].cpu().numpy(), u[:, 0].astype(np.float64)
    assert (out[0] == 0).all() and (w[got] > 0).all()
    off = V * 2.0 ** -46 / W + V * 2.0 ** -52
    assert (at >= (S[got] - w[got]) / W - off).all() and (at <= S[got] / W + off).all()


@pytest.mark.gpu
def test_captured_calls_replay_with_new_values(usp):
    """A fork with its copies and a verification, captured on a side stream: later steps replay with new numbers; two
    captures with workspaces of their own do not disturb each other."""
    import torch
    guard = Guarded()
    pools = [Pool(usp, guard, 6, 8, 16, 40, seed=s, data=True) for s in (1, 2)]
    x = _drafts(np.random.default_rng(3), [4, 2, 3], 700, "f32")
    ins = {k: _dev(x[k]) for k in ("tokens", "u", "q_start", "lens")}
    out = [torch.zeros(3, dtype=torch.int32, device="cuda") for _ in range(3)]
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())

    def step(pool):
        pool.call(pool.dargs)
        usp.usp_pages_copy(pool.c, 6, pool.copies, *pool.kv)
        usp.usp_verify_drafts(3, 9, 700, x["tg"], x["dr"], ins["tokens"], ins["u"], ins["q_start"], ins["lens"], *out)

    for p in pools:
        for d in p.dargs:
            d.zero_()
    with torch.cuda.stream(side):
        step(pools[0])
    side.synchronize()
    graphs = []
    for p in pools:
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g, stream=side):
            step(p)
        graphs.append(g)
    for p in pools:
        p.copies.fill_(-7)
        p.lens[:], p.table[:], p.ref[:] = 0, -1, 0
        p.put()
    rng = np.random.default_rng(9)
    for i in range(8):
        for p, g in zip(pools, graphs):
            x["u"] = (rng.random(9) * (1 - 2.0 ** -20)).astype(np.float32)
            ins["u"].copy_(torch.from_numpy(x["u"]))
            parent = rng.integers(0, 6, 6)
            p.step(parent, rng.integers(0, 90, 6), rng.integers(0, 20, 6), call=lambda args, g=g: g.replay())
            got = np.stack([o.cpu().numpy() for o in out])
            assert np.array_equal(got, ref_verify(x["target"], x["draft"], x["tokens"], x["u"], x["q_start"], x["lens"]))


@pytest.mark.gpu
def test_helpers_on_side_streams(usp):
    """The helpers with a stream of their own, its handle, and inputs freed at once; two streams at a time give what one does."""
    import torch
    rng = np.random.default_rng(5)
    x = _drafts(rng, [4, 1, 6], 3000, "f32")
    want = ref_verify(x["target"], x["draft"], x["tokens"], x["u"], x["q_start"], x["lens"])
    c = usp.Cache(50, 16, 4, 6, 1, 1, 64)
    streams = [torch.cuda.Stream() for _ in range(2)]
    ins = [_dev(x[k]) for k in ("tokens", "u", "q_start", "lens")]
    state = [usp.pages_empty(c) for _ in streams]
    grow = _dev(np.array([20, 5, 90, 16], np.int32))
    torch.cuda.synchronize()
    got = []
    for i in range(6):
        for s, st in zip(streams, state):
            handle = s if i % 2 else s.cuda_stream
            got.append(usp.verify_drafts(x["tg"], x["dr"], *ins, stream=handle))
            with torch.cuda.stream(s):
                g2 = grow.clone()
            copies = usp.pages_update(c, *st, grow=g2, keep=torch.zeros_like(grow) if i == 99 else None, stream=handle)
            usp.pages_compact(c, st[1], st[2], stream=handle)
            del g2, copies
    torch.cuda.synchronize()
    for y in got:
        assert np.array_equal(np.stack([o.cpu().numpy() for o in y]), want)
    table, lens, ref = np.full((4, 6), -1, np.int32), np.zeros(4, np.int32), np.zeros(50, np.int32)
    for _ in range(6):
        table, lens, ref, _, _ = ref_update(16, table, lens, ref, None, None, grow.cpu().numpy())
    for st in state:
        assert np.array_equal(st[0].cpu().numpy(), lens) and np.array_equal(st[2].cpu().numpy(), ref)
        assert np.array_equal(st[1].cpu().numpy(), table)        # (pages go out lowest first: the pool is compact as it is)


@pytest.mark.gpu
@pytest.mark.parametrize("dtype", ["bf16", "f32"])
def test_speculative_decoding_never_waits_for_the_host(usp, dtype):
    """A prompt with a picture in it, forked into samples, then steps of speculative decoding whose lengths only the device
    knows: pages_update (drops the refused drafts, makes room), pages_copy, kv_append_axes, paged_attention, verify_drafts,
    in one captured step.  The attention of the last step is that of the tokens that were accepted."""
    import torch
    rng = np.random.default_rng(11)
    B, Hq, Hkv, d, page, k, V, steps, n0 = 3, 4, 2, 64, 16, 4, 50, 7, 37
    n, T = k + 1, 3 * (k + 1)
    c = usp.Cache(60, page, B, 12, Hq, Hkv, d, dtype=dtype)
    r = usp.Rotary.sections((12, 10, 10))
    inv = _dev(_freq(32))
    dt, gen = c.torch_dtype, torch.Generator().manual_seed(2)
    emb = torch.randn((V, (Hq + 2 * Hkv) * d), generator=gen).to(dt).cuda()       # a token's q, k and v
    head = (torch.randn((Hq * d, V), generator=gen) * 0.4).cuda()
    i32 = dict(dtype=torch.int32, device="cuda")
    lens, table, ref = usp.pages_empty(c)
    kp, vp = (torch.zeros(c.pool_shape(), dtype=dt, device="cuda") for _ in range(2))
    axes_of = lambda pos: torch.stack([pos, pos // 3, pos % 7]).int()  # noqa: E731

    def feed(tokens, seq, pos):
        q, kk, v = (t.view(len(tokens), -1, d) for t in emb[tokens.long()].split([Hq * d, Hkv * d, Hkv * d], 1))
        return usp.kv_append_axes(c, r, q, kk, v, seq, pos, axes_of(pos), inv, kp, vp, table)[0]

    prompt = torch.randint(0, V, (n0,), generator=gen).int().cuda()
    usp.pages_copy(c, usp.pages_update(c, lens, table, ref, grow=torch.tensor([n0, 0, 0], **i32)), kp, vp)
    feed(prompt, torch.zeros(n0, **i32), torch.arange(n0, **i32))
    usp.pages_copy(c, usp.pages_update(c, lens, table, ref, parent=torch.zeros(B, **i32)), kp, vp)      # two samples more
    assert (ref > 0).sum() == c.pages_for(n0)
    q_start, seq = torch.arange(0, T + 1, n, **i32), torch.arange(B, **i32).repeat_interleave(n)
    grow, step_of = torch.full((B,), n, **i32), torch.arange(n, **i32).repeat(B)
    first, keep = torch.tensor([1, 2, 3], **i32), torch.full((B,), n0, **i32)
    drafts, u, q_probs = torch.zeros((B, k), **i32), torch.zeros(T, device="cuda"), torch.zeros((T, V), device="cuda")
    kept_o, counts, nexts, o_last = None, torch.zeros(B, **i32), torch.zeros(B, **i32), torch.zeros((T, Hq, d), dtype=dt, device="cuda")

    def step():
        usp.pages_copy(c, usp.pages_update(c, lens, table, ref, keep=keep, grow=grow), kp, vp)
        tokens = torch.cat([first[:, None], drafts], 1).view(-1)
        q = feed(tokens, seq, keep.repeat_interleave(n) + step_of)
        o, _ = usp.paged_attention(c, q, kp, vp, table, lens, q_start, n)
        p = torch.softmax(o.float().view(T, -1) @ head, 1)
        a, nxt, left = usp.verify_drafts(p, q_probs, tokens, u, q_start, lens)
        counts.copy_(a)
        nexts.copy_(nxt)
        o_last.copy_(o)
        keep.copy_(left)
        first.copy_(nxt)

    state = [x.clone() for x in (lens, table, ref, kp, vp, first, keep)]
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(s):
        step()
    s.synchronize()
    for x, y in zip((lens, table, ref, kp, vp, first, keep), state):
        x.copy_(y)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph, stream=s):
        step()
    texts = [[int(t) for t in prompt] for _ in range(B)]     # what is in the cache
    heads = first.tolist()
    total = 0
    for i in range(steps):
        qp = torch.softmax(torch.from_numpy(rng.standard_normal((T, V))).float(), 1)
        dr = torch.multinomial(qp, 1, generator=gen)[:, 0].view(B, n)[:, 1:].int()
        drafts.copy_(dr)
        q_probs.copy_(qp)
        u.copy_(torch.from_numpy(rng.random(T) * 0.9999))
        graph.replay()
        torch.cuda.synchronize()
        fed = [texts[b] + [heads[b]] + dr[b].tolist() for b in range(B)]
        a, nx = counts.tolist(), nexts.tolist()
        texts = [fed[b][:len(texts[b]) + 1 + a[b]] for b in range(B)]
        heads = nx
        total += sum(a)
        assert keep.tolist() == [len(t) for t in texts] and lens.tolist() == [len(t) for t in fed]
    assert usp.usp_device_status() == 0 and 0 < total < steps * B * k
    # the last step's attention, from the tokens alone: the same bits out of a cache that was filled in one go
    lens2, table2, ref2 = usp.pages_empty(c)
    kp2, vp2 = (torch.zeros_like(kp) for _ in range(2))
    usp.pages_update(c, lens2, table2, ref2, grow=lens)
    tokens, pos = (torch.cat([torch.tensor(x(t), **i32) for t in fed]) for x in (lambda t: t, lambda t: range(len(t))))
    of = torch.cat([torch.full((len(t),), b, **i32) for b, t in enumerate(fed)])
    q, kk, v = (t.view(len(tokens), -1, d) for t in emb[tokens.long()].split([Hq * d, Hkv * d, Hkv * d], 1))
    q, _ = usp.kv_append_axes(c, r, q, kk, v, of, pos, axes_of(pos), inv, kp2, vp2, table2)
    last = torch.cat([torch.arange(m - n, m) for m in np.cumsum([len(t) for t in fed])]).cuda()
    o, _ = usp.paged_attention(c, q[last].contiguous(), kp2, vp2, table2, lens2, q_start, n)
    torch.cuda.synchronize()
    assert torch.equal(o, o_last) and torch.isfinite(o.float()).all() and o.float().abs().max() > 0


@pytest.mark.gpu
@pytest.mark.parametrize("inter", [False, True])
def test_a_training_step_with_rotation(usp, orc, inter):
    """Rotation, all-to-all, attention, back, its backward and the rotation's: outputs and gradients of the unrotated q and k
    against the float64 oracle, on the rotated values as rounded, to the attention's own tolerances."""
    import torch
    from tests.helpers import f64, from_seq, gen, rel_fro, to_dev, to_host, to_seq
    B, Hq, Hkv, N, d, P = 1, 4, 2, 256, 64, 2
    p = usp.Problem(B=B, Hq=Hq, Hkv=Hkv, N=N, d=d, P=P)
    r = usp.Rotary.sections((12, 10, 10), cycled=True, interleaved=inter)
    q, k, v, dO = gen((B, Hq, N, d), 0), gen((B, Hkv, N, d), 1), gen((B, Hkv, N, d), 2), gen((B, Hq, N, d), 3)
    t = np.arange(N)
    pos = np.stack([t // 64, t // 8 % 8, t % 8]).astype(np.int32)
    dpos = _dev(pos.reshape(3, P, 1, N // P))                # (token n of the sequence: rank n / (N/P), place n % (N/P))
    f = _freq(32)
    qr, kr = usp.rotary_embed(p, r, to_dev(to_seq(q, P)), to_dev(to_seq(k, P)), dpos, _dev(f))
    o, saved = usp.ulysses_attention_fwd(p, qr, kr, to_dev(to_seq(v, P)))
    dqr, dkr, dv = usp.ulysses_attention_bwd(p, saved, to_dev(to_seq(dO, P)))
    dq, dk = usp.rotary_embed(p, r, dqr, dkr, dpos, _dev(f), inverse=True)
    torch.cuda.synchronize()
    assert usp.usp_device_status() == 0
    logical = lambda x: f64(from_seq(to_host(x)))  # noqa: E731
    rows = lambda x, inverse=False: ref_rotate(x[0].transpose(1, 0, 2), pos, r.axis, f, inter, inverse)[0].transpose(1, 0, 2)[None]  # noqa: E731
    assert rel_fro(logical(qr), rows(f64(q))) < 2.0 ** -8 and rel_fro(logical(kr), rows(f64(k))) < 2.0 ** -8
    qh, kh = from_seq(to_host(qr)), from_seq(to_host(kr))
    want_o, _ = orc.attn_rows(qh, kh, v, causal=True)
    wq, wk, wv, _, _ = orc.attn_bwd_full(qh, kh, v, dO, causal=True)
    assert rel_fro(logical(o), want_o) < 1e-2
    for got, want in ((dq, rows(wq, True)), (dk, rows(wk, True)), (dv, wv)):
        assert rel_fro(logical(got), want) < 2e-2


@pytest.mark.gpu
def test_rows_beyond_32_bit_offsets(usp):
    """Probabilities and queries whose elements lie beyond 2^31 of their tensors."""
    import torch
    V, rng = 131072, np.random.default_rng(1)
    far = (1 << 31) // V + 3
    x = _drafts(rng, [4], 600, "bf16")
    tg, dr = (torch.empty((far + 4, V), dtype=torch.bfloat16, device="cuda") for _ in range(2))
    for big, small in ((tg, x["tg"]), (dr, x["dr"])):
        big[far:] = 0
        big[far:, V - 600:] = small
    tokens, u = torch.zeros(far + 4, dtype=torch.int32, device="cuda"), torch.zeros(far + 4, device="cuda")
    tokens[far:], u[far:] = _dev(x["tokens"]) + (V - 600), _dev(x["u"])
    got = usp.verify_drafts(tg, dr, tokens, u, torch.tensor([far, far + 4], dtype=torch.int32, device="cuda"), _dev(x["lens"]))
    torch.cuda.synchronize()
    want = ref_verify(x["target"], x["draft"], x["tokens"], x["u"], x["q_start"], x["lens"])
    want[1] += V - 600
    assert np.array_equal(np.stack([g.cpu().numpy() for g in got]), want)
    del tg, dr
    T, gap = 40, 1 << 26
    big = torch.empty(T * gap, dtype=torch.bfloat16, device="cuda")
    q = big.as_strided((1, 1, T, 2, 64), (0, 0, gap, 64, 1))
    q.copy_(torch.randn((1, 1, T, 2, 64), generator=torch.Generator().manual_seed(0)))
    r, p = usp.Rotary.sections((16, 16)), usp.Problem(1, 2, 1, T, 64, 1)
    pos = torch.arange(2 * T, dtype=torch.int32, device="cuda").view(2, 1, 1, T)
    want, _ = usp.rotary_embed(p, r, q.contiguous(), None, pos, _dev(_freq(32)))
    usp.usp_rotary_embed(p, r, q, None, pos, _dev(_freq(32)), q, None)
    torch.cuda.synchronize()
    assert torch.equal(q.contiguous(), want)
    del big, q
    torch.cuda.empty_cache()


@pytest.mark.gpu
def test_tensors_that_the_calls_cannot_take(usp):
    """Device tensors without the layout that a call needs, and an argument's own stream, handle or object."""
    import torch
    c, p = _c(), _p(N=16)
    i = torch.zeros((9, 4), dtype=torch.int32, device="cuda")
    with pytest.raises(ValueError):
        usp.usp_pages_copy(c, 8, i[:, ::2], i, i)
    with pytest.raises(ValueError):
        usp.usp_verify_drafts(1, 4, 50, torch.zeros(4, 100, device="cuda")[:, ::2], None, i, i, i, None, i, i, None)
    q = torch.zeros((2, 1, 8, 4, 64), dtype=torch.bfloat16, device="cuda")
    f, pos = torch.zeros(32, device="cuda"), torch.zeros((3, 16), dtype=torch.int32, device="cuda")
    for bad in (q.transpose(3, 4), q[..., :3, :], torch.zeros((2, 1, 9, 4, 64), dtype=torch.bfloat16, device="cuda")[:, :, 1:]):
        with pytest.raises(ValueError):
            usp.usp_rotary_embed(p, R3, bad, None, pos, f, q, None)
    side = torch.cuda.Stream()
    for stream in (None, side, side.cuda_stream, 0):
        usp.usp_rotary_embed(p, R3, q, None, pos, f, q, None, stream=stream)
    torch.cuda.synchronize()
    with pytest.raises((TypeError, ValueError)):
        usp.usp_rotary_embed(p, R3, q, None, pos, f, q, None, stream="a text")
    assert usp.usp_device_status() == 0


@pytest.mark.gpu
@pytest.mark.parametrize("dtype", ["f32", "bf16"])
def test_verify_long_runs_and_rows_apart(usp, dtype):
    """Drafts that are all accepted, more than a warp looks at together, and rows of the two distributions at distances of
    their own."""
    import torch
    rng = np.random.default_rng(2)
    x = _drafts(rng, [70, 33, 34, 2], 900, dtype, gap=4)
    x["dr"] = torch.full((139, 916), float("nan"), dtype=x["tg"].dtype, device="cuda")[:, :900]
    x["dr"].copy_(x["tg"].roll(1, 0))                     # row t is what row t - 1 of the target says: nothing is refused
    x["target"], x["draft"] = _np(x["tg"]), _np(x["dr"])
    x["tokens"] = np.array([int(rng.choice(np.flatnonzero(r > 0))) for r in x["draft"]], np.int32)
    got = _verify(usp, x)
    assert got[0].tolist() == [69, 32, 33, 1]
    x["tokens"][1 + 40] = 900                             # the first: its 41st draft is no token
    assert _verify(usp, x)[0].tolist() == [40, 32, 33, 1]


@pytest.mark.gpu
def test_copies_in_layers_apart_and_an_append_without_queries(usp):
    import torch
    c = usp.Cache(6, 16, 2, 3, 4, 2, 64)
    kp, vp = (torch.randn((3, 9, 2, 16, 64), device="cuda").bfloat16() for _ in range(2))   # three pages between the layers' pools
    want = [x.clone() for x in (kp, vp)]
    copies = torch.tensor([[2, 0, 0, 0], [5, 0, 16, 0], [1, 4, 3, 0]], dtype=torch.int32, device="cuda")
    usp.usp_pages_copy(c, 2, copies, kp.data_ptr(), vp.data_ptr(), 3, 9 * 2 * 16 * 64)
    torch.cuda.synchronize()
    for x, y in zip((kp, vp), want):
        y[:, 0], y[:, 4, :, :3] = y[:, 5].clone(), y[:, 1, :, :3].clone()
        assert torch.equal(x, y)
    # keys and values alone, and q and k of one tensor rotated in place together
    r = usp.Rotary.sections((12, 10, 10))
    i32 = dict(dtype=torch.int32, device="cuda")
    T, f = 20, _dev(_freq(32))
    table, seq, pos = torch.arange(6, **i32).view(2, 3), torch.arange(T, **i32) % 2, torch.arange(T, **i32) // 2
    rot = torch.randint(0, 99, (3, T), device="cuda").int()
    qkv = torch.randn((T, 8, 64), device="cuda").bfloat16()
    q, k, v = qkv[:, :4], qkv[:, 4:6], qkv[:, 6:]
    pools = [[torch.zeros(c.pool_shape(), dtype=torch.bfloat16, device="cuda") for _ in range(2)] for _ in range(2)]
    none, k_out = usp.kv_append_axes(c, r, None, k, v, seq, pos, rot, f, *pools[0], table)
    q_out, k_out2 = usp.kv_append_axes(c, r, q, k, v, seq, pos, rot, f, *pools[1], table)
    assert none is None and torch.equal(k_out, k_out2) and all(torch.equal(a, b) for a, b in zip(*pools))
    p = usp.Problem(1, 4, 2, T, 64, 1)
    v0 = v.clone()
    usp.usp_rotary_embed(p, r, q, k, rot, f, q, k)
    torch.cuda.synchronize()
    assert torch.equal(q, q_out) and torch.equal(k, k_out) and torch.equal(v, v0)


@pytest.mark.gpu
def test_tensors_of_a_subclass(usp):
    """Parameters, and a class that has its own of what a call asks, are tensors like others."""
    import torch

    class Counted(torch.Tensor):
        asked = 0

        def data_ptr(self):
            Counted.asked += 1
            return super().data_ptr()

    x = _drafts(np.random.default_rng(5), [3, 1, 2], 400, "f32")
    ins = [_dev(x[k]) for k in ("tokens", "u", "q_start", "lens")]
    results = []
    for cls in (lambda y: y, lambda y: torch.nn.Parameter(y, requires_grad=False), lambda y: y.as_subclass(Counted)):
        out = [torch.zeros(3, dtype=torch.int32, device="cuda") for _ in range(3)]
        usp.usp_verify_drafts(3, 6, 400, cls(x["tg"]), cls(x["dr"]), *[cls(y) for y in ins], *out)
        results.append(torch.stack(out).tolist())
    assert results[0] == results[1] == results[2] == ref_verify(x["target"], x["draft"], x["tokens"], x["u"], x["q_start"], x["lens"]).tolist()
    assert Counted.asked == 6
    with pytest.raises(ValueError, match="expected torch.float32"):
        usp.usp_verify_drafts(3, 6, 400, x["tg"], x["dr"], ins[0], torch.nn.Parameter(ins[1].double()), *ins[2:], *out)


@pytest.mark.gpu
def test_traced_calls_are_on_record(usp):
    import torch
    c = usp.Cache(40, 16, 3, 20, 1, 1, 64)
    kp, vp = (torch.zeros(c.pool_shape(), dtype=torch.bfloat16, device="cuda") for _ in range(2))
    x = _drafts(np.random.default_rng(1), [3, 2], 300, "f32")
    grow = torch.full((3,), 30, dtype=torch.int32, device="cuda")
    results = []
    for on in (False, True):
        usp.usp_trace_enable(on)
        usp.usp_trace_reset()
        lens, table, ref = usp.pages_empty(c)
        for _ in range(2):
            copies = usp.pages_update(c, lens, table, ref, grow=grow)
            usp.pages_copy(c, copies, kp, vp)
        usp.pages_compact(c, table, ref)
        out = usp.verify_drafts(x["tg"], x["dr"], _dev(x["tokens"]), _dev(x["u"]), _dev(x["q_start"]), _dev(x["lens"]))
        torch.cuda.synchronize()
        results.append([t.tolist() for t in (lens, table, ref, *out)])
    report = usp.usp_trace_report()
    usp.usp_trace_enable(False)
    usp.usp_trace_reset()
    assert results[0] == results[1]
    assert {k: n for k, (n, _) in report.items()} == {"pages_update": 2, "pages_copy": 2, "pages_compact": 1, "verify_drafts": 1}
