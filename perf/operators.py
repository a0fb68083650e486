"""Measured cases of the serving operators: packed prompt attention, accumulated key weights, and a paged
key-value cache that is filled, attended by single tokens and shrunk by accumulated attention weight.

Notation: q [T, Hq, D] and k, v [T, Hkv, D] hold S sequences one behind the other (rows cu[i] .. cu[i+1] - 1
are sequence i); query head h reads KV head h // (Hq // Hkv); a page holds `page` tokens of every KV head
([pages, page, Hkv, D], weights [pages, Hkv, page]); table[b, j] is the page of slots j * page ... of
sequence b. D is 128.
"""
import math
import random

import numpy as np
import torch

own = False
D = 128
SCALE = 1.0 / math.sqrt(D)
DTYPES = {"bf16": torch.bfloat16, "fp16": torch.float16}


# ---------------------------------------------------------------------------
# Cases
# ---------------------------------------------------------------------------
def listed():
    return [
        # one short prompt of a small layer: launch and latency
        dict(name="attn_prompt_2k", op="attn", dtype="bf16", Hq=8, Hkv=2, S=1, lo=2048, hi=2048, window=0, mix=1),
        # a batch of prompts of mixed lengths through streaming heads (causal sliding window)
        dict(name="attn_packed_window", op="attn", dtype="fp16", Hq=32, Hkv=4, S=16, lo=64, hi=8190, window=1024,
             mix=2),
        # one long prompt, every head over all of it
        dict(name="attn_prompt_32k", op="attn", dtype="bf16", Hq=32, Hkv=4, S=1, lo=32768, hi=32768, window=0, mix=3),
        # after a prefill: what the last 64 queries of each prompt paid attention to
        dict(name="weights_last64", op="weights", dtype="bf16", Hq=32, Hkv=4, S=4, lo=1000, hi=32767, window=0,
             obs=64, mix=4),
        # the same over every query of a batch of prompts
        dict(name="weights_all_rows", op="weights", dtype="fp16", Hq=32, Hkv=4, S=6, lo=100, hi=8192, window=0,
             obs=0, mix=5),
        # a decode step's new tokens, one for each of 32 sequences
        dict(name="append_decode_b32", op="append", dtype="fp16", Hkv=4, S=32, lo=1, hi=1, start=3000, page=64,
             weights=0, mix=6),
        # a batch of prompts moves into the cache with its accumulated weights
        dict(name="append_prompts", op="append", dtype="bf16", Hkv=4, S=7, lo=100, hi=20001, start=0, page=64,
             weights=1, mix=7),
        # a single conversation over a few thousand tokens, streaming heads with a sink: latency
        dict(name="decode_b1_window", op="decode", dtype="bf16", Hq=8, Hkv=2, S=1, lo=4099, hi=4099, window=1024,
             sink=4, page=16, weights=0, mix=8),
        # the long-context batch: every head over the whole cache
        dict(name="decode_b8_128k", op="decode", dtype="bf16", Hq=32, Hkv=4, S=8, lo=131072, hi=131072, window=0,
             sink=0, page=64, weights=0, mix=9),
        # many sequences of mixed lengths that also gather the weights for a later eviction
        dict(name="decode_b32_weights", op="decode", dtype="fp16", Hq=32, Hkv=4, S=32, lo=1, hi=16385, window=0,
             sink=0, page=32, weights=1, mix=10),
        # one sequence of a small layer cut to 512 tokens
        dict(name="evict_b1", op="evict", dtype="bf16", Hkv=2, S=1, lo=2500, hi=2500, budget=512, sink=4, recent=64,
             page=16, mix=11),
        # a batch of long prompts cut to 8192 tokens each
        dict(name="evict_b8_32k", op="evict", dtype="fp16", Hkv=4, S=8, lo=5000, hi=32768, budget=8192, sink=1,
             recent=2048, page=64, mix=12),
    ]


def _log(rng, lo, hi):
    return min(hi, max(lo, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))))


def draw(rng):
    while True:
        op = rng.choice(["attn", "attn", "weights", "append", "decode", "decode", "evict"])
        hkv, group = rng.choice([(1, 8), (2, 4), (4, 8), (4, 1), (8, 4), (3, 5), (16, 1), (2, 16)])
        c = dict(op=op, dtype=rng.choice(["bf16", "fp16"]), Hq=hkv * group, Hkv=hkv, mix=rng.randrange(1 << 20))
        page = rng.choice([1, 16, 32, 64, 128, 256])
        if op == "attn":
            hi = _log(rng, 16, 32768)
            c.update(S=_log(rng, 1, 48), lo=rng.choice([0, 1, hi // 4, hi]), hi=hi, window=rng.choice([0, 0, _log(rng, 1, 8192)]))
        elif op == "weights":
            hi = _log(rng, 16, 32768)
            c.update(S=_log(rng, 1, 24), lo=rng.choice([0, 1, hi // 4, hi]), hi=hi, window=rng.choice([0, 0, _log(rng, 1, 8192)]),
                     obs=rng.choice([0, 1, 64, _log(rng, 1, 2048)]))
        elif op == "append":
            hi = rng.choice([1, _log(rng, 16, 32768), _log(rng, 16, 32768)])
            c.update(S=_log(rng, 1, 64), lo=rng.choice([0, 1, hi // 4, hi]), hi=hi, start=rng.choice([0, _log(rng, 1, 4096)]),
                     page=page, weights=rng.randrange(2))
            del c["Hq"]
        elif op == "decode":
            hi = _log(rng, 64, 131072)
            c.update(S=_log(rng, 1, 64), lo=rng.choice([0, 1, hi // 4, hi]), hi=hi, window=rng.choice([0, 0, _log(rng, 1, 8192)]),
                     sink=rng.choice([0, 1, 4, 64, 100]), page=page, weights=rng.randrange(2))
            if c["window"] == 0:
                c["sink"] = 0
        else:
            hi = _log(rng, 64, 131072)
            budget = _log(rng, 16, 16384)
            sink = rng.choice([0, 1, min(4, budget), budget // 4])
            c.update(S=_log(rng, 1, 32), lo=rng.choice([0, 1, hi // 4, hi]), hi=hi, budget=budget, sink=sink,
                     recent=rng.choice([0, min(64, budget - sink), (budget - sink) // 2, budget - sink]), page=page)
            del c["Hq"]
        if _fits(c):
            return c


def _fits(c):
    """No dearer than the largest listed case of its kind, and within a quarter of the card."""
    lens = _lens(c)
    tokens = sum(lens) + c.get("start", 0) * c["S"]
    most = {"attn": 40000, "weights": 50000, "append": 100000, "decode": 1 << 20, "evict": 1 << 18}[c["op"]]
    if tokens > most or tokens * c["Hkv"] > 4 * most or max(lens) * c["S"] * c["Hkv"] > 16 * most:
        return False
    limit = {"attn": 8.9e12, "weights": 3.0e12}.get(c["op"])
    return limit is None or work(c)["flops"] <= limit


def _lens(c):
    """The sequences' lengths: one of `hi` tokens, the others spread over the logarithm of lo .. hi, shuffled."""
    rng = random.Random(c["mix"])
    lens = [c["hi"]] + [rng.choice([0, 1]) if c["lo"] == 0 and rng.random() < 0.2 else _log(rng, max(1, c["lo"]), c["hi"])
                        for _ in range(c["S"] - 1)]
    rng.shuffle(lens)
    return lens


def _pairs(n, window, obs=0):
    """(query, key) pairs of one sequence of n tokens: the last `obs` queries (0: all), each with its last `window` keys."""
    w = min(window, n) if window else n
    o = min(obs, n) if obs else n
    first = n - o + 1                     # keys that the first observed query sees, before the window
    below = max(0, min(n, w) - first)     # queries that see fewer than w keys
    return below * first + below * (below - 1) // 2 + (o - below) * w


def work(c):
    lens = _lens(c)
    T, hkv = sum(lens), c["Hkv"]
    if c["op"] == "attn":
        pairs = sum(_pairs(n, c["window"]) for n in lens)
        return {"bytes": T * ((2 * c["Hq"] + 2 * hkv) * D * 2 + 4 * c["Hq"]), "flops": 4 * D * pairs * c["Hq"]}
    if c["op"] == "weights":
        rows = sum(min(c["obs"] or n, n) for n in lens)
        seen = sum(min(n, min(c["obs"] or n, n) + (c["window"] or n) - 1) if n else 0 for n in lens)
        pairs = sum(_pairs(n, c["window"], c["obs"]) for n in lens)
        return {"bytes": rows * c["Hq"] * (D * 2 + 4) + seen * hkv * D * 2 + T * hkv * 4,
                "flops": 2 * D * pairs * c["Hq"]}
    if c["op"] == "append":
        return {"bytes": T * hkv * (4 * D * 2 + (8 if c["weights"] else 4)), "flops": 0}
    if c["op"] == "decode":
        att = sum(_attended(n, c) for n in lens)
        extra = T * hkv * 8 if c["weights"] else 0
        return {"bytes": att * hkv * 2 * D * 2 + 2 * c["S"] * c["Hq"] * D * 2 + extra, "flops": 4 * D * att * c["Hq"]}
    kept = sum(min(n, c["budget"]) for n in lens)
    return {"bytes": hkv * (sum(n for n in lens if n > c["budget"]) * 4 + kept * (4 * D * 2 + 8 + 4)), "flops": 0}


def _attended(n, c):
    return n if not c["window"] else min(n, min(c["sink"], max(0, n - c["window"])) + c["window"])


# ---------------------------------------------------------------------------
# Inputs
# ---------------------------------------------------------------------------
def prepare(case, seed):
    c = dict(case)
    dev, dt = torch.device("cuda"), DTYPES[c["dtype"]]
    gen = torch.Generator(device=dev).manual_seed(1000 + seed)
    lens = _lens(c)
    T, S, hkv, op = sum(lens), c["S"], c["Hkv"], c["op"]

    def normal(*shape):
        return torch.randn(*shape, device=dev, generator=gen, dtype=dt)

    def clustered(rows, heads):   # rows about one of 64 directions of length 3, as keys and queries of a trained layer
        centres = torch.nn.functional.normalize(torch.randn(64, D, device=dev, generator=gen), dim=-1) * 3
        pick = torch.randint(0, 64, (rows, heads), device=dev, generator=gen)
        return centres.to(dt)[pick] + normal(rows, heads, D)

    st = {"case": c, "lens_host": lens, "cu_host": [sum(lens[:i]) for i in range(S + 1)]}
    st["cu"] = torch.tensor(st["cu_host"], dtype=torch.int32, device=dev)
    if op in ("attn", "weights"):
        hq = c["Hq"]
        st["q"], st["k"] = clustered(T, hq), clustered(T, hkv)
        st["heads"] = list(range(hq))
        if op == "attn":
            st["v"] = normal(T, hkv, D)
            st["o"] = torch.zeros(T, hq, D, device=dev, dtype=dt)
            st["lse"] = torch.zeros(hq, T, device=dev)
        else:
            st["lse"] = _row_lse(st)
            st["w"] = torch.zeros(hkv, T, device=dev)
        return st

    # the cache: pages in random order, each sequence's table as long as the longest needs
    page, start = c["page"], c.get("start", 0)
    need = [(n + start + page - 1) // page for n in lens]
    width, total = max(1, max(need)), max(1, sum(need))
    order = torch.randperm(total, generator=gen, device=dev).to(torch.int32)
    table = torch.zeros(S, width, dtype=torch.int32, device=dev)
    at = 0
    for b in range(S):
        table[b, :need[b]] = order[at:at + need[b]]
        at += need[b]
    st["table"] = table
    st["lens"] = torch.tensor(lens, dtype=torch.int32, device=dev)
    if op == "append":
        st["k"], st["v"] = clustered(T, hkv), normal(T, hkv, D)
        st["pos"] = torch.full((S,), start, dtype=torch.int32, device=dev)
        st["w"] = torch.rand(hkv, T, device=dev, generator=gen) * 4 if c["weights"] else None
        st["kp"] = torch.zeros(total, page, hkv, D, device=dev, dtype=dt)
        st["vp"], st["wp"] = torch.zeros_like(st["kp"]), torch.zeros(total, hkv, page, device=dev)
        return st
    st["kp"] = clustered(total * page, hkv).view(total, page, hkv, D)
    st["vp"] = normal(total, page, hkv, D)
    # accumulated weights fall over many orders; a fifth of the tokens never got any
    st["wp"] = torch.exp(2 * torch.randn(total, hkv, page, device=dev, generator=gen) - 3)
    st["wp"] *= torch.rand(total, hkv, page, device=dev, generator=gen) > 0.2
    if op == "decode":
        st["q"] = clustered(S, c["Hq"])
        st["heads"] = list(range(c["Hq"]))
        st["o"] = torch.zeros(S, c["Hq"], D, device=dev, dtype=dt)
        st["w_out"] = torch.zeros_like(st["wp"]) if c["weights"] else None
        return st
    kept = [(min(n, c["budget"]) + page - 1) // page for n in lens]
    wide, most = max(1, max(kept)), max(1, sum(kept))
    order = torch.randperm(most, generator=gen, device=dev).to(torch.int32)
    to = torch.zeros(S, wide, dtype=torch.int32, device=dev)
    at = 0
    for b in range(S):
        to[b, :kept[b]] = order[at:at + kept[b]]
        at += kept[b]
    st["to_table"] = to
    st["to_k"] = torch.zeros(most, page, hkv, D, device=dev, dtype=dt)
    st["to_v"], st["to_w"] = torch.zeros_like(st["to_k"]), torch.zeros(most, hkv, page, device=dev)
    st["idx"] = torch.zeros(S, hkv, c["budget"], dtype=torch.int32, device=dev)
    st["new_lens"] = torch.zeros(S, dtype=torch.int32, device=dev)
    return st


def _visible(rows, keys, window):
    """rows [r], keys [u] positions of one sequence -> [r, u]: which keys a query attends."""
    ok = keys[None, :] <= rows[:, None]
    return ok & (keys[None, :] > rows[:, None] - window) if window else ok


def _chunks(c, n, first=0):
    """Row ranges of first .. n - 1 whose score rows fit about 2 GB; under a window no longer than it, as their keys are."""
    step = max(16, int(5e8 / max(1, n * c["Hq"])))
    step = min(step, max(256, c["window"])) if c["window"] else step
    return [(a, min(n, a + step)) for a in range(first, n, step)]


def _scores(st, i, a, b, keys=None):
    """fp32 scores [Hkv, G, b - a, keys] of rows a .. b - 1 of sequence i, -inf where not attended, and the first key."""
    c, lo = st["case"], st["cu_host"][i]
    u0 = max(0, a - c["window"] + 1) if c["window"] else 0
    q, k = st["q"][lo + a:lo + b].float(), st["k"][lo + u0:lo + b].float()
    q = q.view(b - a, c["Hkv"], -1, D).permute(1, 2, 0, 3)
    s = torch.matmul(q, k.permute(1, 2, 0)[:, None]) * SCALE
    ok = _visible(torch.arange(a, b, device=q.device), torch.arange(u0, b, device=q.device), c["window"])
    return s.masked_fill_(~ok, -math.inf), u0


def _row_lse(st):
    """ln of the sum of exp of each observed row's scores: what the prompt's attention left behind."""
    c = st["case"]
    lse = torch.zeros(c["Hq"], st["q"].shape[0], device="cuda")
    for i, n in enumerate(st["lens_host"]):
        lo = st["cu_host"][i]
        for a, b in _chunks(c, n, n - min(c["obs"] or n, n)):
            s, _ = _scores(st, i, a, b)
            lse[:, lo + a:lo + b] = torch.logsumexp(s.double(), -1).flatten(0, 1).float()
    return lse


# ---------------------------------------------------------------------------
# The operators
# ---------------------------------------------------------------------------
def run(st):
    return (_run_own if own else _run_plain)(st)


def _run_own(st):
    import long_context_hybrid_b200 as rtp
    c = st["case"]
    window = c.get("window") or None
    if c["op"] == "attn":
        rtp.attn_packed(st["q"], st["k"], st["v"], st["o"], st["heads"], st["cu"], window=window, lse=st["lse"])
        return {"o": st["o"], "lse": st["lse"]}
    if c["op"] == "weights":
        rtp.attn_key_weights(st["q"], st["k"], st["lse"], st["w"], st["heads"], st["cu"], n_obs=c["obs"] or None,
                             window=window)
        return {"w": st["w"]}
    cache = rtp.PagedCache(st["kp"], st["vp"], st["table"], st["wp"])
    if c["op"] == "append":
        rtp.paged_append(cache, st["k"], st["v"], st["cu"], st["pos"], weights=st["w"])
        return {"k": st["kp"], "v": st["vp"], "w": st["wp"]}
    if c["op"] == "decode":
        rtp.paged_attn_decode(st["q"], cache, st["lens"], st["o"], st["heads"], window=window, sink=c["sink"],
                              weights_out=st["w_out"])
        return {"o": st["o"]} if st["w_out"] is None else {"o": st["o"], "w": st["w_out"]}
    to = rtp.PagedCache(st["to_k"], st["to_v"], st["to_table"], st["to_w"])
    rtp.cache_evict(cache, st["lens"], c["budget"], sink=c["sink"], recent=c["recent"], out=to, idx=st["idx"],
                    new_lens=st["new_lens"])
    return {"idx": st["idx"], "lens": st["new_lens"], "k": to.k, "v": to.v, "w": to.weights}


def _run_plain(st):
    return {"attn": _plain_attn, "weights": _plain_weights, "append": _plain_append, "decode": _plain_decode,
            "evict": _plain_evict}[st["case"]["op"]](st)


def _plain_attn(st):
    c = st["case"]
    o, lse = torch.zeros_like(st["o"]), torch.zeros_like(st["lse"])
    for i, n in enumerate(st["lens_host"]):
        lo = st["cu_host"][i]
        for a, b in _chunks(c, n):
            s, u0 = _scores(st, i, a, b)
            top = s.amax(-1, keepdim=True)
            p = s.sub_(top).exp_()
            total = p.sum(-1, keepdim=True)
            v = st["v"][lo + u0:lo + b].float().permute(1, 0, 2)[:, None]
            x = torch.matmul(p, v) / total
            o[lo + a:lo + b] = x.permute(2, 0, 1, 3).reshape(b - a, c["Hq"], D).to(o.dtype)
            lse[:, lo + a:lo + b] = (top + total.log()).flatten(0, 1).squeeze(-1)
    return {"o": o, "lse": lse}


def _plain_weights(st):
    c = st["case"]
    w = torch.zeros_like(st["w"])
    for i, n in enumerate(st["lens_host"]):
        lo = st["cu_host"][i]
        for a, b in _chunks(c, n, n - min(c["obs"] or n, n)):
            s, u0 = _scores(st, i, a, b)
            p = s.sub_(st["lse"][:, lo + a:lo + b].view(c["Hkv"], -1, b - a, 1)).exp_()
            w[:, lo + u0:lo + b] += p.sum((1, 2))
    return {"w": w}


def _plain_append(st):
    c, T = st["case"], st["k"].shape[0]
    t = torch.arange(T, device="cuda", dtype=torch.int32)
    i = torch.searchsorted(st["cu"], t, right=True) - 1
    slot = st["pos"][i] + t - st["cu"][i]
    page, off = st["table"][i, slot // c["page"]], slot % c["page"]
    st["kp"][page, off] = st["k"]
    st["vp"][page, off] = st["v"]
    st["wp"][page, :, off] = st["w"].t() if st["w"] is not None else 0.0
    return {"k": st["kp"], "v": st["vp"], "w": st["wp"]}


def _plain_decode(st):
    c = st["case"]
    S, hkv, table, lens = c["S"], c["Hkv"], st["table"].long(), st["lens"]
    u = torch.arange(table.shape[1] * c["page"], device="cuda")
    ok = u[None, :] < lens[:, None]
    inside = ok
    if c["window"]:
        ok = ok & ((u[None, :] >= lens[:, None] - c["window"]) | (u[None, :] < c["sink"]))
    q = st["q"].float().view(S, hkv, -1, D)
    k = st["kp"][table].flatten(1, 2).float().permute(0, 2, 3, 1)              # [S, Hkv, D, tokens]
    s = (torch.matmul(q, k) * SCALE).masked_fill_(~ok[:, None, None], -math.inf)
    del k
    top = s.amax(-1, keepdim=True)
    p = (s - top.masked_fill(top == -math.inf, 0)).exp()
    total = p.sum(-1, keepdim=True)
    p /= total.masked_fill(total == 0, 1)                                      # a sequence of length 0 attends nothing
    v = st["vp"][table].flatten(1, 2).float().permute(0, 2, 1, 3)
    o = {"o": torch.matmul(p, v).reshape(S, -1, D).to(st["o"].dtype)}
    if st["w_out"] is not None:
        w = torch.zeros_like(st["w_out"])
        b, at = inside.nonzero(as_tuple=True)
        page, off = table[b, at // c["page"]], at % c["page"]
        w[page, :, off] = st["wp"][page, :, off] + p.sum(2)[b, :, at]
        o["w"] = w
    return o


def _plain_evict(st):
    c = st["case"]
    S, hkv, budget, page, lens = c["S"], c["Hkv"], c["budget"], c["page"], st["lens"]
    table = st["table"].long()
    n = table.shape[1] * page
    u = torch.arange(n, device="cuda")
    w = st["wp"][table].permute(0, 2, 1, 3).reshape(S, hkv, n)
    fixed = (u[None, :] < c["sink"]) | (u[None, :] >= lens[:, None] - c["recent"])
    key = w.masked_fill(fixed[:, None], math.inf).masked_fill((u[None, :] >= lens[:, None])[:, None], -math.inf)
    order = torch.sort(key, dim=-1, descending=True, stable=True).indices[..., :budget]
    keep = torch.minimum(lens, torch.full_like(lens, budget))
    j = torch.arange(order.shape[-1], device="cuda")
    real = (j[None, :] < keep[:, None])[:, None].expand_as(order)
    order = torch.sort(order.masked_fill(~real, n), dim=-1).values
    idx = torch.full((S, hkv, budget), -1, dtype=torch.int32, device="cuda")
    idx[..., :order.shape[-1]] = order.masked_fill(~real, -1).to(torch.int32)
    out = {"idx": idx, "lens": keep.to(torch.int32)}
    b, g, at = real.nonzero(as_tuple=True)
    src = order[b, g, at]
    sp, so = table[b, src // page], src % page
    dp, do = st["to_table"].long()[b, at // page], at % page
    out["k"], out["v"], out["w"] = torch.zeros_like(st["to_k"]), torch.zeros_like(st["to_v"]), torch.zeros_like(st["to_w"])
    out["k"][dp, do, g] = st["kp"][sp, so, g]
    out["v"][dp, do, g] = st["vp"][sp, so, g]
    out["w"][dp, g, do] = st["wp"][sp, g, so]
    return out


# ---------------------------------------------------------------------------
# The same from the definitions, in 64 bits: one sequence and head at a time
# ---------------------------------------------------------------------------
def exact(case, seed):
    st = prepare(case, seed)
    return {"attn": _exact_attn, "weights": _exact_weights, "append": _exact_append, "decode": _exact_decode,
            "evict": _exact_evict}[case["op"]](st)


def _exact_head(st, i, h, a, b):
    """Scores of head h, rows a .. b - 1 of sequence i against all its keys, in 64 bits, and which are attended."""
    c, lo, hi = st["case"], st["cu_host"][i], st["cu_host"][i + 1]
    s = st["q"][lo + a:lo + b, h].double() @ st["k"][lo:hi, h * c["Hkv"] // c["Hq"]].double().T / math.sqrt(D)
    gap = torch.arange(a, b, device="cuda")[:, None] - torch.arange(hi - lo, device="cuda")[None, :]
    return s, (gap >= 0) & (gap < (c["window"] or hi - lo + 1))


def _exact_attn(st):
    c = st["case"]
    o = torch.zeros(st["o"].shape, dtype=torch.float64, device="cuda")
    lse = torch.zeros(st["lse"].shape, dtype=torch.float64, device="cuda")
    for i, n in enumerate(st["lens_host"]):
        lo, hi = st["cu_host"][i], st["cu_host"][i + 1]
        for h in range(c["Hq"]):
            v = st["v"][lo:hi, h * c["Hkv"] // c["Hq"]].double()
            for a in range(0, n, 4096):
                b = min(n, a + 4096)
                s, ok = _exact_head(st, i, h, a, b)
                lse[h, lo + a:lo + b] = torch.logsumexp(torch.where(ok, s, -math.inf), 1)
                o[lo + a:lo + b, h] = torch.where(ok, torch.exp(s - lse[h, lo + a:lo + b, None]), 0.0) @ v
    return {"o": o, "lse": lse}


def _exact_weights(st):
    c = st["case"]
    w = torch.zeros(st["w"].shape, dtype=torch.float64, device="cuda")
    for i, n in enumerate(st["lens_host"]):
        lo, hi = st["cu_host"][i], st["cu_host"][i + 1]
        for h in range(c["Hq"]):
            for a in range(max(0, n - c["obs"]) if c["obs"] else 0, n, 4096):
                b = min(n, a + 4096)
                s, ok = _exact_head(st, i, h, a, b)
                p = torch.where(ok, torch.exp(s - st["lse"][h, lo + a:lo + b, None].double()), 0.0)
                w[h * c["Hkv"] // c["Hq"], lo:hi] += p.sum(0)
    return {"w": w}


def _exact_append(st):
    c = st["case"]
    k, v, w = st["kp"].double(), st["vp"].double(), st["wp"].double()
    table = st["table"].cpu().numpy()
    for i, n in enumerate(st["lens_host"]):
        slots = np.arange(c["start"], c["start"] + n)
        page = torch.from_numpy(table[i, slots // c["page"]].astype(np.int64)).cuda()
        off = torch.from_numpy(slots % c["page"]).cuda()
        rows = slice(st["cu_host"][i], st["cu_host"][i + 1])
        k[page, off], v[page, off] = st["k"][rows].double(), st["v"][rows].double()
        w[page, :, off] = st["w"][:, rows].T.double() if st["w"] is not None else 0.0
    return {"k": k, "v": v, "w": w}


def _slots(st, b, n, table):
    u = torch.arange(n, device="cuda")
    return table[b, u // st["case"]["page"]].long(), u % st["case"]["page"], u


def _exact_decode(st):
    c = st["case"]
    o = torch.zeros(st["o"].shape, dtype=torch.float64, device="cuda")
    w = torch.zeros(st["wp"].shape, dtype=torch.float64, device="cuda")
    for b, n in enumerate(st["lens_host"]):
        page, off, u = _slots(st, b, n, st["table"])
        w[page, :, off] = st["wp"][page, :, off].double()
        seen = u[(u < c["sink"]) | (u >= n - c["window"])] if c["window"] else u
        pg, of = page[seen], off[seen]
        for h in range(c["Hq"] if n else 0):
            g = h * c["Hkv"] // c["Hq"]
            p = torch.softmax(st["kp"][pg, of, g].double() @ st["q"][b, h].double() / math.sqrt(D), 0)
            o[b, h] = p @ st["vp"][pg, of, g].double()
            w[pg, g, of] += p
    return {"o": o} if st["w_out"] is None else {"o": o, "w": w}


def _exact_evict(st):
    c = st["case"]
    idx = np.full(tuple(st["idx"].shape), -1, np.int32)
    out = {n: torch.zeros(st["to_" + n].shape, dtype=torch.float64, device="cuda") for n in ("k", "v", "w")}
    for b, n in enumerate(st["lens_host"]):
        page, off, _ = _slots(st, b, n, st["table"])
        keep = min(n, c["budget"])
        dp, do, _ = _slots(st, b, keep, st["to_table"])
        for g in range(c["Hkv"]):
            w = st["wp"][page, g, off].cpu().numpy().astype(np.float64)
            always = [s for s in range(n) if n <= c["budget"] or s < c["sink"] or s >= n - c["recent"]]
            rest = np.setdiff1d(np.arange(n), always)
            best = rest[np.lexsort((rest, -w[rest]))][:keep - len(always)]
            kept = np.sort(np.concatenate([always, best])).astype(np.int64)
            idx[b, g, :keep] = kept
            at = torch.from_numpy(kept).cuda()
            out["k"][dp, do, g] = st["kp"][page[at], off[at], g].double()
            out["v"][dp, do, g] = st["vp"][page[at], off[at], g].double()
            out["w"][dp, g, do] = st["wp"][page[at], g, off[at]].double()
    lens = np.minimum(np.array(st["lens_host"]), c["budget"]).astype(np.int32)
    return {"idx": torch.from_numpy(idx), "lens": torch.from_numpy(lens), **out}
