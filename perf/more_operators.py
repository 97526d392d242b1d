"""Measured cases of the operators around the paged cache: rotary positions with several axes (in front of the training
paths and while appending), the pages' bookkeeping (forking, truncating, growing, compacting) with the copies it asks for,
and the verification of drafted tokens.

`run` computes each operator in its plain form (elementary torch operations; float64 where angles and sums need it) where
`own` is false, and makes the library's calls where it is true.  `exact` evaluates the definitions in float64, the pages'
one slot after the other.

The lengths of a case follow from the case alone (`_lengths`), the values from the seed.
"""
import math
import random

import numpy as np
import torch

own = False

_DT = {"bf16": torch.bfloat16, "f32": torch.float32}
_ROPE_BASE = 500000.0


# ------------------------------------------------------------------ cases
def _rotary(name, dtype, B, N, P, Hq, Hkv, d, sections, cycled, interleaved, inverse):
    return {"name": name, "op": "rotary", "dtype": dtype, "B": B, "N": N, "P": P, "Hq": Hq, "Hkv": Hkv, "d": d,
            "sections": sections, "cycled": cycled, "interleaved": interleaved, "inverse": inverse}


def _append(name, dtype, Hq, Hkv, d, page, seqs, q_lo, q_hi, start_lo, start_hi, sections, cycled, interleaved, k_out,
            lens=1):
    return {"name": name, "op": "append", "dtype": dtype, "Hq": Hq, "Hkv": Hkv, "d": d, "page": page, "seqs": seqs,
            "q_lo": q_lo, "q_hi": q_hi, "start_lo": start_lo, "start_hi": start_hi, "sections": sections,
            "cycled": cycled, "interleaved": interleaved, "k_out": k_out, "lens": lens}


def _verify(name, dtype, seqs, n_lo, n_hi, vocab, sharp, drafts, empty=0, lens=1):
    return {"name": name, "op": "verify", "dtype": dtype, "seqs": seqs, "n_lo": n_lo, "n_hi": n_hi, "vocab": vocab,
            "sharp": sharp, "drafts": drafts, "empty": empty, "lens": lens}


def _update(name, dtype, Hkv, d, page, roots, children, len_lo, len_hi, shared, cut, grow, copy, spare, lens=1):
    return {"name": name, "op": "update", "dtype": dtype, "Hkv": Hkv, "d": d, "page": page, "roots": roots,
            "children": children, "len_lo": len_lo, "len_hi": len_hi, "shared": shared, "cut": cut, "grow": grow,
            "copy": copy, "spare": spare, "lens": lens}


def _compact(name, dtype, Hkv, d, page, seqs, len_lo, len_hi, shared, percent_live, lens=1):
    return {"name": name, "op": "compact", "dtype": dtype, "Hkv": Hkv, "d": d, "page": page, "seqs": seqs,
            "len_lo": len_lo, "len_hi": len_hi, "shared": shared, "percent_live": percent_live, "lens": lens}


def listed():
    return [
        # q and k of the 128K-token training step, a video behind some text, in front of the all-to-all
        _rotary("rotary_131072", "bf16", 1, 131072, 8, 32, 8, 128, "16,24,24", False, False, False),
        # the way back in float32: rows and columns of images, neighbouring pairs, a ragged number of tokens
        _rotary("rotary_back_f32_4097", "f32", 1, 4097, 1, 4, 4, 64, "16,16", False, True, True),
        # a decoding step of eight conversations with images in them: one token each, latency counts
        _append("append_axes_decode_8", "bf16", 32, 8, 128, 64, 8, 1, 1, 100, 131071, "16,24,24", False, False, False),
        # the prompt of the 32K-token configuration with frames in it: axes dealt out in turn
        _append("append_axes_32768", "bf16", 32, 8, 128, 64, 1, 32768, 32768, 0, 0, "24,20,20", True, False, True),
        # one conversation, four drafts: the smallest check
        _verify("verify_1x5", "f32", 1, 5, 5, 32768, 3.0, "sampled"),
        # a serving batch, five drafts each, a large vocabulary
        _verify("verify_64x6", "f32", 64, 6, 6, 131072, 4.0, "sampled"),
        # drafts taken from the text itself (no probabilities), ragged, an odd vocabulary, two idle slots, bf16
        _verify("verify_200_ragged_bf16", "bf16", 200, 1, 8, 50001, 3.0, "text", empty=2),
        # a speculative step's bookkeeping: 64 conversations lose refused drafts and get room for the next ones
        _update("pages_step_64", "bf16", 8, 128, 64, 64, 0, 17, 32768, 0, 5, 6, False, 200),
        # the smallest fork: eight samples of one short prompt, with the copies of its last page
        _update("pages_fork_8", "bf16", 4, 64, 16, 1, 8, 700, 700, 0, 0, 1, True, 20),
        # 256 samples of a 32K-token prompt: tables, counts, and a page copied for each
        _update("pages_fork_256x32768", "bf16", 8, 128, 64, 1, 256, 32741, 32741, 0, 0, 1, True, 300),
        # a pool half empty after long use: its live pages go to the front, tables follow, pages of 256 KB
        _compact("pages_compact_large", "bf16", 8, 128, 64, 127, 17, 20000, 512, 50),
        # a small float32 pool
        _compact("pages_compact_small_f32", "f32", 2, 64, 16, 12, 5, 500, 0, 60),
    ]


def _log_int(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def _cut_in(rng, total, parts):
    """`total` pairs cut into `parts` axes of at least one each."""
    at = sorted(rng.sample(range(1, total), parts - 1))
    return ",".join(str(b - a) for a, b in zip([0] + at, at + [total]))


def draw(rng):
    op = rng.choice(["rotary", "append", "verify", "verify", "update", "update", "compact"])
    dtype = rng.choice(["bf16", "bf16", "bf16", "f32"])
    Hq, Hkv = rng.choice([(32, 8), (32, 8), (4, 4), (8, 2), (16, 16), (12, 4), (5, 1), (32, 2)])
    d = rng.choice([64, 128])
    page = rng.choice([16, 32, 64, 128, 256])
    lens = rng.randrange(1 << 30)
    half = rng.choice([d, d, d // 2, 16, 48]) // 2
    axes = rng.choice([1, 2, 3, 3, 4])
    cycled = rng.random() < 0.4
    if cycled:   # dealt out in turn: as many each, the rest to the first
        each = half // axes
        sections = ",".join(str(x) for x in [half - each * (axes - 1)] + [each] * (axes - 1))
    else:
        sections = _cut_in(rng, half, axes)
    if op == "rotary":
        P = rng.choice([1, 2, 4, 8])
        B = rng.choice([1, 1, 2])
        most = min(131072, (1 << 29 if dtype == "bf16" else 1 << 28) // ((Hq + Hkv) * d))       # tokens
        N = P * _log_int(rng, 1, most // (B * P))
        c = _rotary("", dtype, B, N, P, Hq, Hkv, d, sections, cycled, rng.random() < 0.4,
                    rng.random() < 0.5)
    elif op == "append":
        tokens = _log_int(rng, 1, 30000)
        seqs = rng.randint(1, min(tokens, 100))
        hi = max(1, 2 * tokens // seqs)
        c = _append("", dtype, Hq, Hkv, d, page, seqs, 1, hi, 0, _log_int(rng, 1, 100000), sections, cycled,
                    rng.random() < 0.4, rng.random() < 0.5, lens)
    elif op == "verify":
        vocab = _log_int(rng, 40, 200000)
        n_hi = rng.randint(1, 9)
        seqs = _log_int(rng, 1, max(2, min(300, 40000000 // (vocab * n_hi))))
        c = _verify("", dtype, seqs, rng.randint(1, n_hi), n_hi, vocab, rng.uniform(1.0, 5.0),
                    rng.choice(["sampled", "sampled", "text"]), rng.choice([0, 0, 1]) if seqs > 1 else 0, lens)
    elif op == "update":
        roots = _log_int(rng, 1, 100)
        children = rng.choice([0, 1, 2, _log_int(rng, 1, 200)]) if roots < 20 else rng.choice([0, 0, 1])
        slots = roots * (1 + children)
        hi = _log_int(rng, 20, max(40, min(60000, 400000 // slots)))
        copy = rng.random() < 0.6
        shared = rng.choice([0, 0, hi // 2 // page * page])
        c = _update("", dtype, Hkv, d, page, roots, children, rng.randint(1, hi), hi, shared, rng.choice([0, 0, 4, 40]),
                    rng.choice([0, 1, 1, 6, _log_int(rng, 1, 2000)]), copy, rng.randint(0, 3000), lens)
        if copy:     # a pool of at most a GB
            per = page * Hkv * d
            while per * _pages_of(c) > 1 << 28 and c["spare"] + c["len_hi"] > 40:
                c["spare"] //= 2
                c["len_hi"] = max(20, c["len_hi"] // 2)
                c["len_lo"] = min(c["len_lo"], c["len_hi"])
                c["shared"] = min(c["shared"], c["len_hi"] // 2 // page * page)
                c["grow"] = min(c["grow"], 64)
                if c["len_hi"] == 20 and per * _pages_of(c) > 1 << 28:
                    c["children"] = c["children"] // 2
    else:
        budget = (1 << 28) // (Hkv * d)                                  # tokens of a pool of at most a GB
        seqs = _log_int(rng, 1, 300)
        hi = max(8, min(20000, budget // seqs // 4))
        hi = _log_int(rng, 8, max(9, hi))
        c = _compact("", dtype, Hkv, d, page, seqs, rng.randint(1, hi), hi, rng.choice([0, hi // 3 // page * page]),
                     rng.choice([10, 30, 50, 70, 95]), lens)
        while page * Hkv * d * _pages_of(c) > 1 << 28 and c["seqs"] > 1:
            c["seqs"] //= 2
    del c["name"]
    return c


def _lengths(c):
    """append: tokens and first slots; verify: rows and cached tokens; update: slots (below); compact: lengths."""
    rng = random.Random(c["lens"])
    if c["op"] == "append":
        nq = [rng.randint(c["q_lo"], c["q_hi"]) for _ in range(c["seqs"])]
        return nq, [rng.randint(c["start_lo"], c["start_hi"]) for _ in range(c["seqs"])]
    if c["op"] == "verify":
        nq = [rng.randint(c["n_lo"], c["n_hi"]) for _ in range(c["seqs"])]
        for i in range(c["empty"]):
            nq[(i * 7 + 3) % c["seqs"]] = 0
        return nq, [n + rng.randint(1, 30000) for n in nq]
    lo, hi = c["len_lo"], c["len_hi"]
    one = lambda: min(hi, max(lo, _log_int(rng, lo, hi)))  # noqa: E731
    if c["op"] == "compact":
        return [one() for _ in range(c["seqs"])]
    # update: per slot its parent, its own tokens, the tokens kept, the room it gets.  Roots go on by themselves and lose
    # `cut` tokens at most; children begin as copies of them, in slots that are empty or hold something finished
    B = c["roots"] * (1 + c["children"]) + 1
    places = list(range(B))
    rng.shuffle(places)
    parent, ln, keep, grow = [-1] * B, [0] * B, [0] * B, [0] * B     # (the last place is an idle slot)
    at = 0
    for _ in range(c["roots"]):
        r = places[at]
        at += 1
        parent[r], ln[r] = r, max(one(), c["shared"])
        keep[r] = max(c["shared"], ln[r] - rng.randint(0, c["cut"]))
        grow[r] = c["grow"]
        for _ in range(c["children"]):
            s = places[at]
            at += 1
            parent[s], keep[s], grow[s] = r, keep[r], c["grow"]
            if rng.random() < 0.3:
                ln[s] = rng.randint(1, 1 + hi // 4)
    return parent, ln, keep, grow


def _pages_of(c):
    """Pages of the pool of a case of pages."""
    p, shared = c["page"], c["shared"] // c["page"]
    if c["op"] == "compact":
        used = shared + sum(max(0, -(-n // p) - shared) for n in _lengths(c))
        return max(used + 1, used * 100 // c["percent_live"])
    parent, ln, keep, grow = _lengths(c)
    used = shared + sum(max(0, -(-n // p) - shared) for n in ln)
    new = sum(-(-(k + g) // p) - k // p for k, g in zip(keep, grow))
    return used + new + c["spare"]


# ------------------------------------------------------------------ inputs
def _normal(shape, dtype, g):
    return torch.randn(shape, generator=g, device="cuda", dtype=dtype)


def _i32(x):
    return torch.as_tensor(np.ascontiguousarray(np.asarray(x, dtype=np.int32))).cuda()


def _sections(c):
    return [int(x) for x in c["sections"].split(",")]


def _pair_axis(c):
    """The axis of each pair: sections one after the other, or axes in turn and the pairs that are left to the first."""
    n = _sections(c)
    if not c["cycled"]:
        return [a for a, x in enumerate(n) for _ in range(x)]
    return [i % len(n) if i // len(n) < n[i % len(n)] else 0 for i in range(sum(n))]


def _grid_positions(c, count, g, first):
    """Positions [axes][count] of a video (frames of a grid) behind `first` tokens of text, on every axis."""
    axes = len(_sections(c))
    i = torch.arange(count, device="cuda")
    side = int(torch.randint(6, 40, (1,), generator=g, device="cuda").item())
    text = i < count // 8
    j = i - count // 8
    at = [j // (side * side), j // side % side, j % side, j // 7][:axes] if axes > 1 else [j]
    start = first + count // 8
    return torch.stack([torch.where(text, first + i, start + a) for a in at]).to(torch.int32)


def _frequencies(c):
    half = sum(_sections(c))
    return (_ROPE_BASE ** (-torch.arange(half, dtype=torch.float64) / half)).float().cuda()


def _table(c, s, order, slots, ln):
    """Page table, counts and pool of slots with these lengths; the first `shared` tokens are in pages of all of them."""
    p, n_pages, shared = c["page"], _pages_of(c), c["shared"] // c["page"]
    more = 0 if c["op"] == "compact" else max([0] + [-(-(k + g) // p) for k, g in zip(s["keep_host"], s["grow_host"])])
    mp = max([1, more] + [-(-n // p) for n in ln])
    ids = order.permutation(n_pages)
    table = np.full((slots, mp), -1, np.int32)
    at = shared
    for b, n in enumerate(ln):
        k = -(-n // p)
        table[b, :min(k, shared)] = ids[:min(k, shared)]
        if k > shared:
            table[b, shared:k] = ids[at:at + k - shared]
            at += k - shared
    s["n_pages"], s["max_pages"] = n_pages, mp
    s["table_host"], s["ref_host"] = table, np.bincount(table[table >= 0], minlength=n_pages).astype(np.int32)
    s["page_table"], s["ref"], s["seq_lens"] = _i32(table), _i32(s["ref_host"]), _i32(ln)


def prepare(case, seed):
    c = case
    g = torch.Generator(device="cuda")
    g.manual_seed(seed * 7919 + 17)
    order = np.random.default_rng(seed)
    dt = _DT[c["dtype"]]
    s = {"case": c}
    if c["op"] in ("rotary", "append"):
        s["axis_host"] = _pair_axis(c)
        s["axis"] = _i32(s["axis_host"])
        s["inv_freq"] = _frequencies(c)
        Hq, Hkv, d = c["Hq"], c["Hkv"], c["d"]
    if c["op"] == "rotary":
        T = c["B"] * c["N"]
        # q, k, v as one projection writes them, on the local shards
        qkv = _normal((c["P"], c["B"], c["N"] // c["P"], Hq + 2 * Hkv, d), dt, g)
        s["q"], s["k"] = qkv[..., :Hq, :], qkv[..., Hq:Hq + Hkv, :]
        pos = _grid_positions(c, c["N"], g, 5).view(-1, c["P"], 1, c["N"] // c["P"])
        s["pos"] = pos.expand(-1, -1, c["B"], -1).contiguous().view(-1, T)
        s["q_out"] = torch.empty(qkv.shape[:3] + (Hq, d), dtype=dt, device="cuda")
        s["k_out"] = torch.empty(qkv.shape[:3] + (Hkv, d), dtype=dt, device="cuda")
    elif c["op"] == "append":
        nq, first = _lengths(c)
        T, B, page = sum(nq), c["seqs"], c["page"]
        used = [list(range(a // page, -(-(a + n) // page))) for a, n in zip(first, nq)]
        mp = max(u[-1] + 1 for u in used)
        n_pages = sum(len(u) for u in used) + 3
        ids, at = order.permutation(n_pages), 0
        table = np.full((B, mp), -1, np.int32)
        for b, u in enumerate(used):
            table[b, u] = ids[at:at + len(u)]
            at += len(u)
        s["table_host"], s["page_table"] = table, _i32(table)
        s["k_pages"], s["v_pages"] = (_normal((n_pages, Hkv, page, d), dt, g) for _ in range(2))
        qkv = _normal((T, (Hq + 2 * Hkv) * d), dt, g)
        s["q"] = qkv[:, :Hq * d].view(T, Hq, d)
        s["k"] = qkv[:, Hq * d:(Hq + Hkv) * d].view(T, Hkv, d)
        s["v"] = qkv[:, (Hq + Hkv) * d:].view(T, Hkv, d)
        s["T"] = T
        s["seq"] = _i32(np.repeat(np.arange(B), nq))
        s["pos"] = _i32(np.concatenate([np.arange(a, a + n) for a, n in zip(first, nq)]))
        # a sequence's rotary positions: behind a picture they are smaller than the slots
        s["rot_pos"] = torch.cat([_grid_positions(c, n, g, a // 2) for a, n in zip(first, nq)], 1).contiguous() \
            if B <= 8 else torch.stack([s["pos"] // (1 + a) for a in range(len(_sections(c)))]).contiguous()
        s["q_out"] = torch.empty((T, Hq, d), dtype=dt, device="cuda")
        s["k_out"] = torch.empty((T, Hkv, d), dtype=dt, device="cuda") if c["k_out"] else None
    elif c["op"] == "verify":
        nq, cached = _lengths(c)
        T, B, V = sum(nq), c["seqs"], c["vocab"]
        start = np.concatenate([[0], np.cumsum(nq)])
        logits = torch.randn((T, V), generator=g, device="cuda") * c["sharp"]
        # most rows have a token that stands out, and the draft's model knows it
        best = torch.randint(V, (T, 1), generator=g, device="cuda")
        logits.scatter_add_(1, best, torch.rand((T, 1), generator=g, device="cuda") * (7 * c["sharp"]))
        s["T"] = T
        s["q_start"], s["seq_lens"] = _i32(start), _i32(cached)
        near = logits.roll(1, 0) + torch.randn((T, V), generator=g, device="cuda") * (0.2 * c["sharp"])
        if c["drafts"] == "sampled":     # row t: what token t was drawn from
            q = torch.softmax(near, -1)
            s["tokens"] = torch.multinomial(q, 1, generator=g)[:, 0].to(torch.int32)
            s["draft"] = q.to(dt)
            del q
        else:
            s["tokens"] = near.argmax(-1).to(torch.int32)
            s["draft"] = None
        del near
        s["target"] = torch.softmax(logits, -1).to(dt)
        s["u"] = torch.rand(T, generator=g, device="cuda")
        s["n_accepted"], s["next"], s["keep_lens"] = (torch.empty(B, dtype=torch.int32, device="cuda") for _ in range(3))
        s["max_n"] = max(nq)
    elif c["op"] == "update":
        parent, ln, keep, grow = _lengths(c)
        B = len(ln)
        s["parent_host"], s["len_host"], s["keep_host"], s["grow_host"] = parent, ln, keep, grow
        _table(c, s, order, B, ln)
        s["parent"], s["keep"], s["grow"] = _i32(parent), _i32(keep), _i32(grow)
        s["copies"] = torch.full((1 + B, 4), -1, dtype=torch.int32, device="cuda")
    else:
        ln = _lengths(c)
        _table(c, s, order, len(ln), ln)
        s["page_table_out"], s["ref_out"] = torch.empty_like(s["page_table"]), torch.empty_like(s["ref"])
        s["new_id"] = torch.empty_like(s["ref"])
        s["copies"] = torch.full((1 + s["n_pages"] // 2, 4), -1, dtype=torch.int32, device="cuda")
    if c["op"] == "compact" or c.get("copy"):
        s["k_pages"], s["v_pages"] = (_normal((s["n_pages"], c["Hkv"], c["page"], c["d"]), dt, g) for _ in range(2))
    if own:
        import context_long_attention_ulysses_gb300 as usp
        s["usp"] = usp
        if c["op"] in ("rotary", "append"):
            s["rotary"] = usp.Rotary(tuple(s["axis_host"]), interleaved=c["interleaved"])
        if c["op"] == "rotary":
            s["problem"] = usp.Problem(B=c["B"], Hq=Hq, Hkv=Hkv, N=c["N"], d=d, P=c["P"], dtype=c["dtype"])
        elif c["op"] == "append":
            s["cache"] = usp.Cache(n_pages=n_pages, page_size=page, n_seqs=B, max_pages=mp, Hq=Hq, Hkv=Hkv, d=d,
                                   dtype=c["dtype"])
        elif c["op"] != "verify":
            s["cache"] = usp.Cache(n_pages=s["n_pages"], page_size=c["page"], n_seqs=len(ln), max_pages=s["max_pages"],
                                   Hq=c["Hkv"], Hkv=c["Hkv"], d=c["d"], dtype=c["dtype"])
            if c["op"] == "update":
                size = usp.usp_pages_update_workspace_size(s["cache"])
                s["ws"] = torch.empty(max(size, 256), dtype=torch.uint8, device="cuda")
    return s


# ------------------------------------------------------------------ one pass
def run(state):
    s, c = state, state["case"]
    op = c["op"]
    if own:
        usp = s["usp"]
        if op == "rotary":
            usp.usp_rotary_embed(s["problem"], s["rotary"], s["q"], s["k"], s["pos"], s["inv_freq"], s["q_out"],
                                 s["k_out"], inverse=c["inverse"])
        elif op == "append":
            usp.usp_kv_append_axes(s["cache"], s["T"], s["q"], s["k"], s["v"], s["seq"], s["pos"], s["rot_pos"],
                                   s["inv_freq"], s["rotary"], s["q_out"], s["k_out"], s["k_pages"], s["v_pages"],
                                   s["page_table"])
        elif op == "verify":
            usp.usp_verify_drafts(c["seqs"], s["T"], c["vocab"], s["target"], s["draft"], s["tokens"], s["u"],
                                  s["q_start"], s["seq_lens"], s["n_accepted"], s["next"], s["keep_lens"])
        elif op == "update":
            usp.usp_pages_update(s["cache"], s["parent"], s["keep"], s["grow"], s["seq_lens"], s["page_table"],
                                 s["ref"], s["copies"], s["ws"])
        else:
            usp.usp_pages_compact(s["cache"], s["page_table"], s["ref"], s["page_table_out"], s["ref_out"], s["new_id"],
                                  s["copies"])
        if "k_pages" in s and op != "append":
            usp.usp_pages_copy(s["cache"], s["copies"].shape[0] - 1, s["copies"], s["k_pages"], s["v_pages"])
    else:
        {"rotary": _plain_rotary, "append": _plain_append, "verify": _plain_verify, "update": _plain_update,
         "compact": _plain_compact}[op](s, c)
        if "k_pages" in s and op != "append":
            _plain_copy(s, c)
    names = {"rotary": ("q_out", "k_out"), "append": ("q_out", "k_out", "k_pages", "v_pages"),
             "verify": ("n_accepted", "next", "keep_lens"),
             "update": ("seq_lens", "page_table", "ref", "copies", "k_pages", "v_pages"),
             "compact": ("page_table_out", "ref_out", "new_id", "copies", "k_pages", "v_pages")}[op]
    return {k: s[k] for k in names if s.get(k) is not None}


def _rotate(x, cos, sin, rot, interleaved):
    x = x.float()
    y = x.clone()
    if interleaved:
        a, b = x[..., 0:rot:2], x[..., 1:rot:2]
        y[..., 0:rot:2] = a * cos - b * sin
        y[..., 1:rot:2] = b * cos + a * sin
    else:
        a, b = x[..., :rot // 2], x[..., rot // 2:rot]
        y[..., :rot // 2] = a * cos - b * sin
        y[..., rot // 2:rot] = b * cos + a * sin
    return y


def _turns(s, pos):
    """cos and sin [T][1][half] of the tokens' angles: far positions need 64 bits."""
    angle = pos[s["axis"].long()].T.double() * s["inv_freq"].double()
    return angle.cos().float()[:, None, :], angle.sin().float()[:, None, :]


def _plain_rotary(s, c):
    cos, sin = _turns(s, s["pos"])
    if c["inverse"]:
        sin = -sin
    rot = 2 * s["axis"].numel()
    for x, y in (("q", "q_out"), ("k", "k_out")):
        flat = s[x].flatten(0, 2)
        s[y].view(flat.shape).copy_(_rotate(flat, cos, sin, rot, c["interleaved"]))


def _plain_append(s, c):
    cos, sin = _turns(s, s["rot_pos"])
    rot, page = 2 * s["axis"].numel(), c["page"]
    s["q_out"].copy_(_rotate(s["q"], cos, sin, rot, c["interleaved"]))
    k = _rotate(s["k"], cos, sin, rot, c["interleaved"]).to(_DT[c["dtype"]])
    if c["k_out"]:
        s["k_out"].copy_(k)
    pos = s["pos"].long()
    ids = s["page_table"][s["seq"].long(), pos // page].long()
    s["k_pages"][ids, :, pos % page] = k
    s["v_pages"][ids, :, pos % page] = s["v"]


def _plain_verify(s, c):
    T, V = s["T"], c["vocab"]
    t0, n = s["q_start"][:-1].long(), (s["q_start"][1:] - s["q_start"][:-1]).long()
    tok, u = s["tokens"].long(), s["u"].double()
    rows = torch.arange(1, T, device="cuda")                          # row t judges by row t - 1 of the target
    p = s["target"][rows - 1, tok[1:]].double()
    q = s["draft"][rows, tok[1:]].double() if s["draft"] is not None else torch.ones_like(p)
    good = torch.cat([torch.zeros(1, dtype=torch.bool, device="cuda"), u[1:] * q < p])
    i = torch.arange(1, max(2, s["max_n"]), device="cuda")
    judged = i < n[:, None]
    good = good[(t0[:, None] + i).clamp(max=T - 1)] & judged
    a = good.int().cumprod(1).sum(1)
    row = (t0 + a).clamp(max=T - 1)
    refused = a < n - 1
    w0 = s["target"][row].double()
    nxt = (row + 1).clamp(max=T - 1)
    if s["draft"] is not None:
        less = s["draft"][nxt].double()
    else:
        less = torch.zeros_like(w0).scatter_(1, tok[nxt][:, None], 1.0)
    w = (w0 - torch.where(refused[:, None], less, 0.0)).clamp(min=0)
    w = torch.where(w.sum(1, keepdim=True) > 0, w, w0)
    cum = w.cumsum(1)
    drawn = (cum <= u[t0.clamp(max=T - 1)][:, None] * cum[:, -1:]).sum(1).clamp(max=V - 1)
    live = n > 0
    s["n_accepted"].copy_(torch.where(live, a, 0))
    s["next"].copy_(torch.where(live & (cum[:, -1] > 0), drawn, -1))
    s["keep_lens"].copy_(s["seq_lens"] - torch.where(live, n - 1 - a, 0))


def _counts(ids, valid, n):
    return torch.zeros(n, dtype=torch.int64, device="cuda").scatter_add_(0, ids.clamp(0, n - 1).reshape(-1).long(),
                                                                         valid.reshape(-1).long())


def _plain_update(s, c):
    page, n, mp = c["page"], s["n_pages"], s["max_pages"]
    table, ref = s["page_table"].long(), s["ref"].long()
    B = table.shape[0]
    b, j = torch.arange(B, device="cuda"), torch.arange(mp, device="cuda")
    a, cap = s["parent"].long(), mp * page
    L = s["seq_lens"].long().clamp(0, cap)
    known = (a >= 0) & (a < B)
    a = torch.where(known, a, 0)
    kept = torch.minimum(s["keep"].long().clamp(min=0), torch.where(known, L[a], 0))
    new = (kept + s["grow"].long().clamp(min=0)).clamp(max=cap)
    full, rest = kept // page, kept % page
    old_n, kept_n, new_n = ((x + page - 1) // page for x in (L, kept, new))
    mine = torch.where(j < old_n[:, None], table, -1)                 # what the slots hold
    have = torch.where(j < kept_n[:, None], table[a], -1)             # what they go on with
    count = ref - _counts(mine, (mine >= 0) & (mine < n), n) + _counts(have, (have >= 0) & (have < n), n)
    last = have.gather(1, full.clamp(max=mp - 1)[:, None])[:, 0]      # pages that end inside, and are written
    writes = (rest > 0) & (new > kept) & (last >= 0) & (last < n)
    at = last.clamp(0, n - 1)
    key = torch.where(a == b, b, b + B)                               # who holds the page already, then the lowest
    writers = _counts(last, writes, n)
    first = torch.full((n,), 2 * B, dtype=torch.int64, device="cuda").scatter_reduce_(
        0, at, torch.where(writes, key, 2 * B), "amin")
    copy = writes & ~((count[at] == writers[at]) & (first[at] == key))
    need = new_n - kept_n + copy.long()
    off = need.cumsum(0) - need
    total = need.sum()
    is_free = count <= 0
    free = torch.sort(torch.where(is_free, 0, n) + torch.arange(n, device="cuda")).values   # free pages, lowest first
    enough = total <= is_free.sum()
    take = lambda k: free[k.clamp(0, n - 1)] % n  # noqa: E731
    row = torch.where(j < new_n[:, None], take(off[:, None] + copy[:, None].long() + j - kept_n[:, None]),
                      torch.where(j < old_n[:, None], -1, table))
    row = torch.where(j < kept_n[:, None], have, row)
    to = take(off)
    row = torch.where(copy[:, None] & (j == full[:, None]), to[:, None], row)
    taken = torch.arange(n, device="cuda") < total
    count = count - _counts(last, copy, n)
    count = torch.where(count < 0, 0, count).scatter(0, free % n, torch.where(taken, 1, count[free % n]))
    place = torch.where(copy & enough, copy.long().cumsum(0), B + 1)
    out = torch.cat([s["copies"], s["copies"][:1]])
    out = out.scatter(0, place[:, None].expand(-1, 4), torch.stack([last, to, rest, torch.zeros_like(to)], 1).int())[:-1]
    short = (total - is_free.sum()).clamp(min=0)
    left = torch.where(enough, is_free.sum() - total, (ref <= 0).sum())
    out[0] = torch.stack([torch.where(enough, copy.sum(), 0), short, left, torch.zeros_like(short)]).int()
    s["copies"].copy_(out)
    s["page_table"].copy_(torch.where(enough, row, table))
    s["ref"].copy_(torch.where(enough, count, ref))
    s["seq_lens"].copy_(torch.where(enough, new, s["seq_lens"].long()))


def _plain_compact(s, c):
    n, ref, table = s["n_pages"], s["ref"].long(), s["page_table"].long()
    i = torch.arange(n, device="cuda")
    live = ref > 0
    count = live.sum()
    moves, hole = live & (i >= count), ~live & (i < count)
    to = torch.sort(torch.where(hole, 0, n) + i).values % n            # holes, lowest first
    rank = moves.long().cumsum(0) - 1
    new = torch.where(live, torch.where(moves, to[rank.clamp(min=0)], i), -1)
    s["new_id"].copy_(new)
    inside = (table >= 0) & (table < n)
    mapped = new[table.clamp(0, n - 1)]
    s["page_table_out"].copy_(torch.where(inside & (mapped >= 0), mapped, table))
    ref_out = torch.where(live & ~moves, ref, 0)
    pad = torch.zeros(1, dtype=torch.int64, device="cuda")
    s["ref_out"].copy_(torch.cat([ref_out, pad]).scatter_add(0, torch.where(moves, new, n), ref)[:n])
    m = s["copies"].shape[0]
    out = torch.cat([s["copies"], s["copies"][:1]])
    rows = torch.stack([i, new, torch.full_like(i, c["page"]), torch.zeros_like(i)], 1).int()
    out = out.scatter(0, torch.where(moves, rank + 1, m)[:, None].expand(-1, 4), rows)[:-1]
    out[0] = torch.stack([moves.sum(), pad[0], n - count, pad[0]]).int()
    s["copies"].copy_(out)


def _plain_copy(s, c):
    """The copies of the list; those past its end copy a page to itself."""
    n = s["n_pages"]
    rows = s["copies"][1:].long()
    real = torch.arange(rows.shape[0], device="cuda") < s["copies"][0, 0]
    src, dst = (torch.where(real, rows[:, k], n) for k in (0, 1))
    count = torch.where(real, rows[:, 2], 0)
    m = torch.full((n + 1,), n, dtype=torch.int64, device="cuda").scatter_(0, dst, src)[:n]      # where a page comes from
    tokens = torch.zeros(n + 1, dtype=torch.int64, device="cuda").scatter_(0, dst, count)[:n]
    step = max(1, rows.shape[0])
    for x in (s["k_pages"], s["v_pages"]):
        order = torch.sort(torch.where(m < n, 0, n) + torch.arange(n, device="cuda")).values[:step] % n
        src = torch.where(m[order] < n, m[order], order)
        keep = (torch.arange(c["page"], device="cuda") >= tokens[order][:, None])[:, None, :, None]
        x[order] = torch.where(keep, x[order], x[src])


# ------------------------------------------------------------------ what a pass cannot do without
def work(case):
    c = case
    e = 2 if c["dtype"] == "bf16" else 4
    if c["op"] == "rotary":
        T, H, half = c["B"] * c["N"], c["Hq"] + c["Hkv"], sum(_sections(c))
        return {"bytes": 2 * T * H * c["d"] * e + T * 4 * len(_sections(c)) + 4 * half, "flops": 6 * T * H * half}
    if c["op"] == "append":
        T, half = sum(_lengths(c)[0]), sum(_sections(c))
        values = T * c["d"] * (2 * (c["Hq"] + 2 * c["Hkv"]) + (c["Hkv"] if c["k_out"] else 0))
        return {"bytes": values * e + T * (12 + 4 * len(_sections(c))) + 4 * half,
                "flops": 6 * T * (c["Hq"] + c["Hkv"]) * half}
    if c["op"] == "verify":
        nq = _lengths(c)[0]
        # a row of the target's probabilities for each sequence, one of the draft's where a draft is refused (most are, at
        # some place), and scalars
        some, judged = sum(n > 0 for n in nq), sum(n > 1 for n in nq)
        rows = some + (judged if c["drafts"] == "sampled" else 0)
        return {"bytes": rows * c["vocab"] * e + sum(nq) * (8 + 2 * e) + 20 * len(nq), "flops": 2 * rows * c["vocab"]}
    p, n = c["page"], _pages_of(c)
    if c["op"] == "update":
        parent, ln, keep, grow = _lengths(c)
        entries = copied = 0
        for b, a in enumerate(parent):
            if a >= 0 and a != b:        # a row read and one written, the one there released
                entries += 2 * -(-keep[b] // p) + -(-ln[b] // p)
                copied += keep[b] % p if grow[b] else 0
            entries += 1 + -(-(keep[b] + grow[b]) // p) - -(-keep[b] // p)
        by = 4 * (entries + n) + 20 * len(ln)
        if c["copy"]:
            by += 4 * copied * c["Hkv"] * c["d"] * e
        return {"bytes": by, "flops": entries + n}
    ln = _lengths(c)
    live = c["shared"] // p + sum(max(0, -(-x // p) - c["shared"] // p) for x in ln)
    moved = live * (n - live) // n                                       # live pages behind the first `live` places
    table = len(ln) * max([1] + [-(-x // p) for x in ln])
    return {"bytes": 4 * moved * p * c["Hkv"] * c["d"] * e + 12 * n + 8 * table, "flops": n}


# ------------------------------------------------------------------ the definitions in float64
def _exact_rotate(x, c, s, pos):
    axis, r = s["axis_host"], 2 * len(s["axis_host"])
    ang = torch.stack([pos[a].to(torch.float64) * s["inv_freq"][i].to(torch.float64) for i, a in enumerate(axis)], -1)
    if c.get("inverse"):
        ang = -ang
    turn = torch.polar(torch.ones_like(ang), ang)[:, None, :]                     # e^{i angle}
    y = x.to(torch.float64)
    z = torch.complex(y[..., 0:r:2], y[..., 1:r:2]) if c["interleaved"] else \
        torch.complex(y[..., :r // 2], y[..., r // 2:r])
    z = z * turn
    both = torch.stack([z.real, z.imag], -1) if c["interleaved"] else torch.stack([z.real, z.imag], -2)
    return torch.cat([both.reshape(*both.shape[:-2], r), y[..., r:]], -1)


def exact(case, seed):
    c, s = case, prepare(case, seed)
    if c["op"] == "rotary":
        out = {}
        for x, y in (("q", "q_out"), ("k", "k_out")):
            flat = s[x].flatten(0, 2)
            step = 1 << 14                                                        # tokens in pieces that fit
            out[y] = torch.cat([_exact_rotate(flat[t:t + step], c, s, s["pos"][:, t:t + step])
                                for t in range(0, flat.shape[0], step)]).view(s[y].shape)
        return out
    if c["op"] == "append":
        nq, first = _lengths(c)
        page = c["page"]
        out = {"q_out": _exact_rotate(s["q"], c, s, s["rot_pos"]), "k_pages": s["k_pages"].to(torch.float64),
               "v_pages": s["v_pages"].to(torch.float64)}
        k = _exact_rotate(s["k"], c, s, s["rot_pos"])
        t = 0
        for b, (n, a) in enumerate(zip(nq, first)):
            done = 0
            while done < n:                                                       # one page at a time
                slot = (a + done) % page
                m = min(page - slot, n - done)
                pid = int(s["table_host"][b, (a + done) // page])
                out["k_pages"][pid, :, slot:slot + m] = k[t + done:t + done + m].transpose(0, 1)
                out["v_pages"][pid, :, slot:slot + m] = s["v"][t + done:t + done + m].to(torch.float64).transpose(0, 1)
                done += m
            t += n
        if c["k_out"]:
            out["k_out"] = k
        return out
    if c["op"] == "verify":
        nq, cached = _lengths(c)
        B = len(nq)
        acc, nxt, left = np.zeros(B, np.int32), np.full(B, -1, np.int32), np.array(cached, np.int32)
        tok, u = s["tokens"].tolist(), s["u"].tolist()
        t = 0
        for b, n in enumerate(nq):
            if n:
                a = 0
                while a < n - 1:
                    x = tok[t + a + 1]
                    q = float(s["draft"][t + a + 1, x]) if s["draft"] is not None else 1.0
                    if not u[t + a + 1] * q < float(s["target"][t + a, x]):
                        break
                    a += 1
                w = s["target"][t + a].double().cpu().numpy()
                if a < n - 1:
                    less = np.eye(1, c["vocab"], tok[t + a + 1])[0] if s["draft"] is None else \
                        s["draft"][t + a + 1].double().cpu().numpy()
                    rest = np.maximum(w - less, 0)
                    w = rest if rest.any() else w
                cum = np.cumsum(w.astype(np.longdouble))
                if cum[-1] > 0:
                    nxt[b] = int(np.argmax(cum > u[t] * cum[-1]))
                acc[b], left[b] = a, cached[b] - (n - 1 - a)
            t += n
        return {"n_accepted": _i32(acc), "next": _i32(nxt), "keep_lens": _i32(left)}
    p, n, table, ref = c["page"], s["n_pages"], s["table_host"], s["ref_host"].astype(np.int64)
    copies = s["copies"].cpu().numpy()
    moves = []
    if c["op"] == "compact":
        live = int((ref > 0).sum())
        holes = [i for i in range(live) if ref[i] == 0]
        new = np.where(ref > 0, np.arange(n), -1)
        out_ref = ref.copy()
        for i in range(live, n):
            if ref[i] > 0:
                new[i] = holes.pop(0)
                out_ref[new[i]], out_ref[i] = ref[i], 0
                moves.append((i, int(new[i]), p, 0))
        out = {"new_id": _i32(new), "ref_out": _i32(out_ref),
               "page_table_out": _i32(np.where(table >= 0, new[np.maximum(table, 0)], table))}
        copies[0] = len(moves), 0, n - live, 0
    else:
        rows = [list(r) for r in table]
        have = []
        for b, a in enumerate(s["parent_host"]):                                  # what each slot goes on with
            k = min(s["keep_host"][b], s["len_host"][a]) if a >= 0 else 0
            have.append((k, list(rows[a][:-(-k // p)]) if a >= 0 else []))
        for b, m in enumerate(s["len_host"]):
            for x in rows[b][:-(-m // p)]:
                ref[x] -= 1
        for k, ids in have:
            for x in ids:
                ref[x] += 1
        writers = {}
        for b, (k, ids) in enumerate(have):
            if k % p and s["grow_host"][b]:
                writers.setdefault(ids[-1], []).append((s["parent_host"][b] != b, b))
        stays = {x: min(w)[1] for x, w in writers.items() if ref[x] == len(w)}
        free = [i for i in range(n) if ref[i] == 0]
        lens, used = [], 0
        for b, (k, ids) in enumerate(have):
            new = k + s["grow_host"][b]
            if k % p and s["grow_host"][b] and stays.get(ids[-1]) != b:
                moves.append((int(ids[-1]), free[used], k % p, 0))
                ref[ids[-1]] -= 1
                ids[-1] = free[used]
                ref[free[used]] = 1
                used += 1
            while len(ids) < -(-new // p):
                ids.append(free[used])
                ref[free[used]] = 1
                used += 1
            old = -(-s["len_host"][b] // p)
            for j in range(max(old, len(ids))):
                rows[b][j] = ids[j] if j < len(ids) else -1
            lens.append(new)
        out = {"seq_lens": _i32(lens), "page_table": _i32(rows), "ref": _i32(ref)}
        copies[0] = len(moves), 0, len(free) - used, 0
    if moves:
        copies[1:1 + len(moves)] = moves
    out["copies"] = _i32(copies)
    for x in ("k_pages", "v_pages"):
        if x in s:
            y = s[x].to(torch.float64)
            for i, to, count, _ in moves:
                y[to, :, :count] = y[i, :, :count]
            out[x] = y
    return out
