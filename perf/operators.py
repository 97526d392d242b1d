"""Measured cases of the serving operators: appending rotated keys and values to a paged cache, attention over
that cache for ragged batches, and attention for a batch whose sequences share a long prefix.

`run` computes each operator in its plain form (elementary torch operations in float32) where `own` is false, and
makes the library's calls where it is true.  `exact` evaluates the definitions in float64.

The sequence lengths of a case follow from the case alone (`_lengths`), the values from the seed.
"""
import math
import random

import torch

own = False

_DT = {"bf16": torch.bfloat16, "f32": torch.float32}
_ROPE_BASE = 500000.0


# ------------------------------------------------------------------ cases
def _append(name, dtype, Hq, Hkv, d, page, seqs, q_lo, q_hi, start_lo, start_hi, rot, interleaved, k_out):
    return {"name": name, "op": "append", "dtype": dtype, "Hq": Hq, "Hkv": Hkv, "d": d, "page": page, "seqs": seqs,
            "q_lo": q_lo, "q_hi": q_hi, "start_lo": start_lo, "start_hi": start_hi, "rot": rot,
            "interleaved": interleaved, "k_out": k_out, "lens": 1}


def _attn(name, dtype, Hq, Hkv, d, page, seqs, q_lo, q_hi, len_lo, len_hi, prefix=0, empty=0, causal=True, lens=1):
    return {"name": name, "op": "prefix" if prefix else "paged", "dtype": dtype, "Hq": Hq, "Hkv": Hkv, "d": d,
            "page": page, "seqs": seqs, "q_lo": q_lo, "q_hi": q_hi, "len_lo": len_lo, "len_hi": len_hi,
            "prefix": prefix, "empty": empty, "causal": causal, "lens": lens}


def listed():
    return [
        # a decoding step of eight conversations at positions up to 128K: one token each, latency counts
        _append("append_decode_8", "bf16", 32, 8, 128, 64, 8, 1, 1, 100, 131071, 128, False, False),
        # the prompt of the 32K-token configuration: rotated q and k for the attention, k and v into the cache
        _append("append_prompt_32768", "bf16", 32, 8, 128, 64, 1, 32768, 32768, 0, 0, 128, False, True),
        # float32, interleaved pairs over half of each head, ragged pieces of prompts, small pages
        _append("append_f32_ragged", "f32", 4, 4, 64, 16, 37, 1, 701, 0, 5000, 32, True, True),
        # the smallest decoding step: four short conversations, four heads of 64 values, small pages
        _attn("decode_small", "bf16", 4, 4, 64, 16, 4, 1, 1, 90, 700),
        # one conversation of 128K tokens: a single token against the whole cache
        _attn("decode_1x131072", "bf16", 32, 8, 128, 64, 1, 1, 1, 131072, 131072),
        # a serving batch of very different lengths, two of its slots empty
        _attn("decode_64_ragged", "bf16", 32, 8, 128, 64, 64, 1, 1, 17, 32768, empty=2),
        # verification of five drafted tokens per sequence: 20 rows a KV head
        _attn("verify_5x16", "bf16", 32, 8, 128, 32, 16, 5, 5, 1000, 20000),
        # the next 2048 tokens of a prompt whose first 64K are in the cache
        _attn("chunk_2048_at_65536", "bf16", 32, 8, 128, 128, 1, 2048, 2048, 67584, 67584),
        # the float32 path: decoding on CUDA cores
        _attn("decode_f32_16", "f32", 8, 2, 64, 64, 16, 1, 1, 500, 16000),
        # 64 samples of one 32K-token prompt: the prompt's keys are read once for all
        _attn("prefix_64x32768", "bf16", 32, 8, 128, 64, 64, 1, 1, 32769, 34800, prefix=32768),
        # 200 requests behind one system prompt of 4001 tokens (not whole pages), own parts of up to 1500
        _attn("prefix_200x4001", "bf16", 32, 8, 128, 128, 200, 1, 1, 4002, 5500, prefix=4001),
        # few short answers to one prompt: the smallest call
        _attn("prefix_small", "bf16", 4, 4, 64, 16, 6, 1, 1, 1030, 1200, prefix=1024),
    ]


def _log_int(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    op = rng.choice(["append", "paged", "paged", "paged", "prefix", "prefix"])
    Hq, Hkv = rng.choice([(32, 8), (32, 8), (4, 4), (8, 2), (16, 16), (12, 4), (5, 1), (32, 2)])
    d = rng.choice([64, 128])
    page = rng.choice([16, 32, 64, 128, 256])
    dtype = rng.choice(["bf16", "bf16", "bf16", "bf16", "f32"])
    lens = rng.randrange(1 << 30)
    if op == "append":
        tokens = _log_int(rng, 1, 40000)
        seqs = rng.randint(1, min(tokens, 100))
        hi = max(1, 2 * tokens // seqs)
        rot = rng.choice([d, d, d // 2, 16])
        c = _append("", dtype, Hq, Hkv, d, page, seqs, 1 if hi > 1 else hi, hi, 0, _log_int(rng, 1, 100000), rot,
                    rng.random() < 0.4, rng.random() < 0.5)
        c["lens"] = lens
    elif op == "paged":
        many = rng.random() < 0.3
        q_hi = _log_int(rng, 2, 600) if many else rng.choice([1, 1, 1, 2, 3, 4, 8])
        seqs = _log_int(rng, 1, 8 if many else 160)
        budget = (1 << 28) // (seqs * Hkv * d)          # values of K of the batch
        if many:
            budget = min(budget, (1 << 33) // (seqs * q_hi * Hq))
        if dtype == "f32":
            budget //= 4
        hi = max(40, _log_int(rng, 40, max(41, min(131072, budget))))
        c = _attn("", dtype, Hq, Hkv, d, page, seqs, rng.randint(1, q_hi), q_hi, rng.randint(1, hi), hi,
                  empty=rng.choice([0, 0, 1]) if seqs > 1 else 0, causal=rng.random() < 0.85, lens=lens)
    else:
        seqs = _log_int(rng, 2, 256)
        budget = max(64, min(65536, (1 << 31) // (seqs * Hq * 8)))
        if dtype == "f32":
            budget = max(64, budget // 4)
        prefix = _log_int(rng, 33, budget)
        q_hi = rng.choice([1, 1, 1, 2, 4])
        own_hi = _log_int(rng, 8, 1500)
        c = _attn("", dtype, Hq, Hkv, d, page, seqs, rng.randint(1, q_hi), q_hi, prefix + q_hi, prefix + q_hi + own_hi,
                  prefix=prefix, empty=rng.choice([0, 0, 1]), causal=rng.random() < 0.9, lens=lens)
    del c["name"]
    return c


def _lengths(c):
    """Tokens of this call, and cached tokens (attention) or first slot (append), of each sequence."""
    rng = random.Random(c["lens"])
    nq = [rng.randint(c["q_lo"], c["q_hi"]) for _ in range(c["seqs"])]
    if c["op"] == "append":
        return nq, [rng.randint(c["start_lo"], c["start_hi"]) for _ in range(c["seqs"])]
    lo, hi = c["len_lo"], c["len_hi"]
    ln = [min(hi, max(lo, _log_int(rng, lo, hi))) for _ in range(c["seqs"])]
    for i in range(c["empty"]):          # slots of the batch that hold no sequence at present
        ln[(i * 7 + 3) % c["seqs"]] = 0
    return nq, ln


# ------------------------------------------------------------------ inputs
def _normal(shape, dtype, g):
    return torch.randn(shape, generator=g, device="cuda", dtype=torch.float32 if dtype == torch.float32 else dtype)


def _i32(x):
    return torch.tensor(x, dtype=torch.int32, device="cuda")


def prepare(case, seed):
    c = case
    g = torch.Generator(device="cuda")
    g.manual_seed(seed * 7919 + 17)
    order = random.Random(seed)
    dt = _DT[c["dtype"]]
    Hq, Hkv, d, page, B = c["Hq"], c["Hkv"], c["d"], c["page"], c["seqs"]
    nq, second = _lengths(c)
    T = sum(nq)
    q_start = [0]
    for n in nq:
        q_start.append(q_start[-1] + n)
    s = {"case": c, "nq": nq, "T": T, "q_start_host": q_start}
    if c["op"] == "append":
        ends = [a + n for a, n in zip(second, nq)]
        max_pages = max(-(-e // page) for e in ends)
        used = [list(range(a // page, -(-e // page))) for a, e in zip(second, ends)]
    else:
        s["lens_host"] = second
        max_pages = max(1, max(-(-n // page) for n in second))
        used = [list(range(c["prefix"] // page, -(-n // page))) for n in second]
    n_prefix = -(-c.get("prefix", 0) // page)
    # pages in the order a pool hands them out after long use: none of them neighbours
    n_pages = sum(len(u) for u in used) + n_prefix + 3
    ids = list(range(n_pages))
    order.shuffle(ids)
    at = n_prefix
    table = [[-1] * max_pages for _ in range(B)]
    for b in range(B):
        if c["op"] != "append" and second[b] > 0:
            for j in range(c["prefix"] // page):
                table[b][j] = ids[j]
        for j in used[b]:
            table[b][j] = ids[at]
            at += 1
    s["page_table"] = _i32(table)
    s["k_pages"] = _normal((n_pages, Hkv, page, d), dt, g)
    s["v_pages"] = _normal((n_pages, Hkv, page, d), dt, g)
    if c["op"] == "append":
        # q, k, v as one projection writes them: a row holds the token's q, k and v heads
        qkv = _normal((T, (Hq + 2 * Hkv) * d), dt, g)
        s["q"] = qkv[:, :Hq * d].view(T, Hq, d)
        s["k"] = qkv[:, Hq * d:(Hq + Hkv) * d].view(T, Hkv, d)
        s["v"] = qkv[:, (Hq + Hkv) * d:].view(T, Hkv, d)
        s["seq"] = _i32([b for b in range(B) for _ in range(nq[b])])
        s["pos"] = _i32([second[b] + i for b in range(B) for i in range(nq[b])])
        half = c["rot"] // 2
        s["inv_freq"] = (_ROPE_BASE ** (-torch.arange(half, dtype=torch.float64) / half)).float().cuda()
        s["q_out"] = torch.empty((T, Hq, d), dtype=dt, device="cuda")
        s["k_out"] = torch.empty((T, Hkv, d), dtype=dt, device="cuda") if c["k_out"] else None
    else:
        s["q"] = _normal((T, Hq, d), dt, g)
        s["seq_lens"] = _i32(second)
        s["q_start"] = None if c["q_hi"] == 1 else _i32(q_start)
        s["prefix_pages"] = _i32(ids[:n_prefix]) if c["prefix"] else None
        s["o"] = torch.empty((T, Hq, d), dtype=dt, device="cuda")
        s["lse"] = torch.empty((T, Hq), dtype=torch.float32, device="cuda")
        # the prefix's last, partly filled page: every sequence has its own copy of those tokens
        rest = c["prefix"] % page
        if rest:
            for b in range(B):
                if second[b] > 0:
                    for x in (s["k_pages"], s["v_pages"]):
                        x[table[b][n_prefix - 1], :, :rest] = x[ids[n_prefix - 1], :, :rest]
    if own:
        import context_long_attention_ulysses_gb300 as usp
        cache = usp.Cache(n_pages=n_pages, page_size=page, n_seqs=B, max_pages=max_pages, Hq=Hq, Hkv=Hkv, d=d,
                          causal=c.get("causal", True), dtype=c["dtype"])
        s["cache"], s["usp"] = cache, usp
        if c["op"] != "append":
            size = (usp.usp_prefix_attn_workspace_size(cache, T, c["q_hi"], c["prefix"]) if c["prefix"]
                    else usp.usp_paged_attn_workspace_size(cache, T, c["q_hi"]))
            s["ws"] = torch.empty(max(size, 256), dtype=torch.uint8, device="cuda")
    return s


# ------------------------------------------------------------------ one pass
def run(state):
    s, c = state, state["case"]
    if own:
        usp = s["usp"]
        if c["op"] == "append":
            usp.usp_kv_append(s["cache"], s["T"], s["q"], s["k"], s["v"], s["seq"], s["pos"], s["inv_freq"], s["q_out"],
                              s["k_out"], s["k_pages"], s["v_pages"], s["page_table"], rot=c["rot"],
                              interleaved=c["interleaved"])
        elif c["op"] == "paged":
            usp.usp_paged_attn(s["cache"], s["T"], c["q_hi"], s["q"], s["k_pages"], s["v_pages"], s["page_table"],
                               s["seq_lens"], s["q_start"], s["o"], s["lse"], s["ws"])
        else:
            usp.usp_prefix_attn(s["cache"], s["T"], c["q_hi"], s["q"], s["k_pages"], s["v_pages"], s["page_table"],
                                s["seq_lens"], s["q_start"], s["prefix_pages"], c["prefix"], s["o"], s["lse"], s["ws"])
    elif c["op"] == "append":
        _plain_append(s, c)
    else:
        _plain_attention(s, c)
    if c["op"] == "append":
        out = {"q_out": s["q_out"], "k_pages": s["k_pages"], "v_pages": s["v_pages"]}
        if c["k_out"]:
            out["k_out"] = s["k_out"]
        return out
    return {"o": s["o"], "lse": s["lse"]}


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


def _plain_append(s, c):
    dt, page = _DT[c["dtype"]], c["page"]
    angle = s["pos"].double()[:, None] * s["inv_freq"].double()   # far positions: the angle needs 64 bits
    cos, sin = angle.cos().float()[:, None, :], angle.sin().float()[:, None, :]
    s["q_out"].copy_(_rotate(s["q"], cos, sin, c["rot"], c["interleaved"]).to(dt))
    k = _rotate(s["k"], cos, sin, c["rot"], c["interleaved"]).to(dt)
    if c["k_out"]:
        s["k_out"].copy_(k)
    pos = s["pos"].long()
    ids = s["page_table"][s["seq"].long(), pos // page].long()
    s["k_pages"][ids, :, pos % page] = k
    s["v_pages"][ids, :, pos % page] = s["v"]


def _keys(pages, ids, first, last):
    """Tokens first .. last of the sequence whose pages are `ids`, as float32 [Hkv][last - first][d]."""
    n, Hkv, page, d = pages.shape
    x = pages[ids[first // page:-(-last // page)].long()].float()
    x = x.permute(1, 0, 2, 3).reshape(Hkv, -1, d)
    off = first % page
    return x[:, off:off + last - first]


def _partial(q, k, v, first, limit):
    """Softmax sums of rows q [H][r][d] over keys first .. of which row r sees those below limit[r]: max, sum, sum of p v."""
    x = q @ k.transpose(1, 2)
    if limit is not None:
        x = torch.where(torch.arange(first, first + k.shape[1], device=x.device)[None] < limit[:, None], x, -torch.inf)
    m = x.amax(2)
    x = torch.exp(x - torch.where(m == -torch.inf, torch.zeros_like(m), m)[..., None])
    return m, x.sum(2), x @ v


def _partial_by_heads(q, k, v, first, limit):
    """`_partial`, over as many heads at a time as 2 Gi scores hold."""
    step = max(1, (1 << 31) // max(1, q.shape[1] * k.shape[1]))
    got = [_partial(q[h:h + step], k[h:h + step], v[h:h + step], first, limit) for h in range(0, q.shape[0], step)]
    return got[0] if len(got) == 1 else tuple(torch.cat(x) for x in zip(*got))


def _join(parts):
    m = torch.stack([p[0] for p in parts]).amax(0)
    safe = torch.where(m == -torch.inf, torch.zeros_like(m), m)
    w = [torch.exp(p[0] - safe) for p in parts]
    total = sum(wi * p[1] for wi, p in zip(w, parts))
    o = sum(wi[..., None] * p[2] for wi, p in zip(w, parts))
    some = total > 0
    o = torch.where(some[..., None], o / torch.where(some, total, torch.ones_like(total))[..., None], 0.0)
    return o, torch.where(some, safe + torch.log(total), -torch.inf)


def _plain_attention(s, c):
    Hq, Hkv, d, P = c["Hq"], c["Hkv"], c["d"], c["prefix"]
    g, dt = Hq // Hkv, _DT[c["dtype"]]
    T = s["T"]
    rows = (s["q"].float() * (1.0 / math.sqrt(d))).view(T, Hkv, g, d).transpose(0, 1).reshape(Hkv, T * g, d)
    lim = None
    if P or any(n > 1 for n in s["nq"]):                                     # keys that each row (token, head) sees
        lim = _i32([ln - n + i + 1 if c["causal"] else ln for n, ln in zip(s["nq"], s["lens_host"]) for i in range(n)])
        lim = lim.repeat_interleave(g)
    if P:                                                                    # the prefix, once for the whole batch
        shared = _partial_by_heads(rows, _keys(s["k_pages"], s["prefix_pages"], 0, P),
                                   _keys(s["v_pages"], s["prefix_pages"], 0, P), 0, lim)
    for b, (n, ln) in enumerate(zip(s["nq"], s["lens_host"])):
        t0 = s["q_start_host"][b]
        r = slice(t0 * g, (t0 + n) * g)
        parts = [tuple(x[:, r] for x in shared)] if P else []
        if ln > P:
            ids = s["page_table"][b]
            parts.append(_partial_by_heads(rows[:, r], _keys(s["k_pages"], ids, P, ln),
                                           _keys(s["v_pages"], ids, P, ln), P, lim[r] if lim is not None else None))
        if parts:
            o, lse = _join(parts)
            s["o"][t0:t0 + n] = o.view(Hkv, n, g, d).transpose(0, 1).reshape(n, Hq, d).to(dt)
            s["lse"][t0:t0 + n] = lse.view(Hkv, n, g).transpose(0, 1).reshape(n, Hq)
        else:
            s["o"][t0:t0 + n] = 0
            s["lse"][t0:t0 + n] = -torch.inf


# ------------------------------------------------------------------ what a pass cannot do without
def work(case):
    c = case
    e = 2 if c["dtype"] == "bf16" else 4
    Hq, Hkv, d, page = c["Hq"], c["Hkv"], c["d"], c["page"]
    nq, second = _lengths(c)
    T = sum(nq)
    if c["op"] == "append":
        values = T * d * ((Hq + 2 * Hkv) + (Hq + 2 * Hkv) + (Hkv if c["k_out"] else 0))
        return {"bytes": values * e + 12 * T + 2 * c["rot"], "flops": T * (Hq + Hkv) * c["rot"] * 3}
    P = c["prefix"]
    keys = P + sum(max(0, ln - P) for ln in second)                  # each key and value that some row sees, once
    pairs = 0
    for n, ln in zip(nq, second):
        pairs += sum(max(0, ln - n + i + 1) for i in range(n)) if c["causal"] else n * ln
    by = keys * Hkv * 2 * d * e + 2 * T * Hq * d * e + T * Hq * 4 + 4 * (keys // page + 2 * c["seqs"])
    return {"bytes": by, "flops": 4 * d * Hq * pairs}


# ------------------------------------------------------------------ the definitions in float64
def exact(case, seed):
    c, s = case, prepare(case, seed)
    Hq, Hkv, d, page = c["Hq"], c["Hkv"], c["d"], c["page"]
    g = Hq // Hkv
    nq, second = _lengths(c)
    table = s["page_table"].tolist()
    if c["op"] == "append":
        r = c["rot"]
        ang = torch.outer(s["pos"].to(torch.float64), s["inv_freq"].to(torch.float64))
        turn = torch.polar(torch.ones_like(ang), ang)[:, None, :]                 # e^{i angle}

        def rotated(x):
            y = x.to(torch.float64)
            z = torch.complex(y[..., 0:r:2], y[..., 1:r:2]) if c["interleaved"] else \
                torch.complex(y[..., :r // 2], y[..., r // 2:r])
            z = z * turn
            both = torch.stack([z.real, z.imag], -1) if c["interleaved"] else torch.stack([z.real, z.imag], -2)
            return torch.cat([both.reshape(*both.shape[:-2], r), y[..., r:]], -1)

        q, k = rotated(s["q"]), rotated(s["k"])
        kp, vp = s["k_pages"].to(torch.float64), s["v_pages"].to(torch.float64)
        t = 0
        for b, (n, a) in enumerate(zip(nq, second)):
            done = 0
            while done < n:                                                       # one page at a time
                slot = (a + done) % page
                m = min(page - slot, n - done)
                pid = table[b][(a + done) // page]
                kp[pid, :, slot:slot + m] = k[t + done:t + done + m].transpose(0, 1)
                vp[pid, :, slot:slot + m] = s["v"][t + done:t + done + m].to(torch.float64).transpose(0, 1)
                done += m
            t += n
        out = {"q_out": q, "k_pages": kp, "v_pages": vp}
        if c["k_out"]:
            out["k_out"] = k
        return out
    o = torch.zeros((s["T"], Hq, d), dtype=torch.float64, device="cuda")
    lse = torch.full((s["T"], Hq), -math.inf, dtype=torch.float64, device="cuda")
    head = s["prefix_pages"].tolist() if c["prefix"] else []
    t = 0
    for b, (n, ln) in enumerate(zip(nq, second)):
        if ln > 0:
            ids = torch.tensor((head[:c["prefix"] // page] + table[b][c["prefix"] // page:])[:-(-ln // page)],
                               device="cuda")
            for h in range(Hkv):
                k = s["k_pages"][ids, h].reshape(-1, d)[:ln].to(torch.float64)
                v = s["v_pages"][ids, h].reshape(-1, d)[:ln].to(torch.float64)
                for i0 in range(0, n, 256):                                       # rows in pieces that fit
                    i1 = min(n, i0 + 256)
                    x = torch.einsum("ngd,kd->ngk", s["q"][t + i0:t + i1, h * g:(h + 1) * g].to(torch.float64), k)
                    x = x / math.sqrt(d)
                    if c["causal"]:
                        last = torch.arange(i0, i1, device="cuda") + (ln - n)
                        hide = torch.arange(ln, device="cuda")[None, :] > last[:, None]
                        x = x.masked_fill(hide[:, None, :], -math.inf)
                    z = torch.logsumexp(x, -1)
                    w = torch.exp(x - torch.where(z.isinf(), torch.zeros_like(z), z)[..., None])
                    o[t + i0:t + i1, h * g:(h + 1) * g] = torch.einsum("ngk,kd->ngd", w, v)
                    lse[t + i0:t + i1, h * g:(h + 1) * g] = z
        t += n
    return {"o": o, "lse": lse}
