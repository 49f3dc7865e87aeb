"""Cases of the operators beside the verify matmul: rotary positions with the
append to the paged cache, attention of a chunk of new tokens over that cache,
and sampling from the head's logits.

``run`` computes a case in plain torch operations (32 bits, rounded once at
the end), or with ``own`` set through the framework's entry points.  ``exact``
gives the same outputs in 64 bits from the definitions.

Shapes: 6144-wide queries with 1024-wide keys and values are 48 query and 8
key/value heads of 128; 151936 is the output head's vocabulary.
"""
import math
import random

import numpy as np
import torch

own = False

DTYPES = {"f32": torch.float32, "f16": torch.float16, "bf16": torch.bfloat16}
TURN = 40                      # fraction bits of an angle in turns


# --- the cases -----------------------------------------------------------------

def _rope(name, requests, q, kv, heads, kv_heads, dim, rot, layout, scaling, src, dtype, page):
    return {"name": name, "op": "rope", "requests": requests, "q_min": q[0], "q_max": q[1],
            "kv_min": kv[0], "kv_max": kv[1], "heads": heads, "kv_heads": kv_heads, "dim": dim,
            "rot": rot, "layout": layout, "scaling": scaling, "src": src, "dtype": dtype,
            "page": page, "cache": "token", "lens": 1}


def _attend(name, requests, q, kv, heads, kv_heads, dim, dtype, page, cache="token", window=0,
            tree=False):
    return {"name": name, "op": "attend", "requests": requests, "q_min": q[0], "q_max": q[1],
            "kv_min": kv[0], "kv_max": kv[1], "heads": heads, "kv_heads": kv_heads, "dim": dim,
            "dtype": dtype, "page": page, "cache": cache, "window": window, "tree": tree, "lens": 1}


def _sample(name, rows, vocab, dtype, rule, mask=False, last=False, spread=2.5):
    return {"name": name, "op": "sample", "rows": rows, "vocab": vocab, "dtype": dtype,
            "rule": rule, "mask": mask, "last": last, "spread": spread}


def listed():
    return [
        # the 8 drafted rows of one request, straight from the fp32 q/k/v projections
        _rope("rope_verify8", 1, (8, 8), (4099, 4099), 48, 8, 128, 128, "half", "none", "f32",
              "f16", 64),
        # a batch of requests with 1 to 8 drafted rows each; half of each head rotates
        _rope("rope_batch", 64, (1, 8), (300, 30000), 32, 8, 128, 64, "interleaved", "linear",
              "bf16", "bf16", 16),
        # a prompt's chunk in a long context (frequencies scaled by parts)
        _rope("rope_prompt", 1, (8191, 8191), (100000, 100000), 48, 8, 128, 128, "half",
              "by_parts", "f32", "bf16", 128),
        # plain decoding of one request: latency
        _attend("attend_decode1", 1, (1, 1), (2011, 2011), 48, 8, 128, "f16", 16),
        # one request's tree of 8 drafted tokens after a long context
        _attend("attend_tree8", 1, (8, 8), (32779, 32779), 48, 8, 128, "bf16", 64, tree=True),
        # ordinary batched decoding, ragged contexts
        _attend("attend_decode64", 64, (1, 1), (500, 16384), 48, 8, 128, "f16", 64),
        # batched verify calls of a sliding-window layer with small heads
        _attend("attend_verify32", 32, (1, 8), (900, 20000), 32, 8, 64, "bf16", 32,
                cache="head", window=4096),
        # short prompts and drafts together in one batch
        _attend("attend_mixed", 16, (1, 600), (700, 4096), 48, 8, 128, "bf16", 64),
        # a prompt's chunk of 2048 tokens at the end of a 16k context
        _attend("attend_prompt", 1, (2048, 2048), (16384, 16384), 48, 8, 128, "bf16", 64),
        # one row: latency
        _sample("sample_one", 1, 151936, "f32", "top_k_top_p"),
        # the 8 rows of a verify call, a mask of allowed tokens, temperature after the filters
        _sample("sample_verify8", 8, 151936, "f32", "top_p_min_p", mask=True, last=True),
        # a large batch, every row with its own parameters
        _sample("sample_batch", 256, 151936, "f32", "mixed"),
    ]


def _log(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def _draw_one(rng):
    op = rng.choice(["rope", "attend", "attend", "sample"])
    lens = rng.randrange(1, 1 << 20)
    heads, kv_heads = rng.choice([(48, 8), (32, 8), (28, 4), (16, 2), (8, 8), (20, 4)])
    dim = 128 if heads == 48 else rng.choice([64, 64, 128])
    dtype = rng.choice(["f16", "bf16"])
    page = rng.choice([16, 32, 64, 128])
    cache = rng.choice(["token", "head"])
    if op == "rope":
        b = _log(rng, 1, 64)
        q = rng.choice([(1, 1), (1, 8), (8, 8), (1, _log(rng, 16, 8192))])
        kv = _log(rng, max(64, q[1]), 120000)
        c = _rope(None, b, q, (max(q[1], kv // 3), kv), heads, kv_heads, dim,
                  rng.choice([dim, dim // 2]), rng.choice(["half", "interleaved"]),
                  rng.choice(["none", "linear", "by_parts"]), rng.choice(["f32", "f16", "bf16"]),
                  dtype, page)
        c["cache"] = cache
    elif op == "attend":
        kind = rng.choice(["decode", "verify", "prompt"])
        if kind == "decode":
            b, q, kv = _log(rng, 1, 128), (1, 1), _log(rng, 64, 65536)
        elif kind == "verify":
            b, q, kv = _log(rng, 1, 64), (rng.randrange(1, 5), 8), _log(rng, 64, 65536)
        else:
            b, n = _log(rng, 1, 8), _log(rng, 16, 2048)
            q, kv = (max(1, n // 3), n), _log(rng, n, 16384)
        c = _attend(None, b, q, (max(q[1], kv // 3), kv), heads, kv_heads, dim, dtype, page, cache,
                    rng.choice([0, 0, _log(rng, 128, 8192)]), kind == "verify" and rng.random() < .5)
    else:
        c = _sample(None, _log(rng, 1, 256), _log(rng, 2000, 151936),
                    rng.choice(["f32", "f32", "bf16", "f16"]),
                    rng.choice(["top_k_top_p", "top_p_min_p", "none", "mixed"]),
                    rng.random() < .3, rng.random() < .5, rng.choice([1.5, 2.5, 4.0]))
    c["lens"] = lens
    del c["name"]
    return c


def _memory(c):
    """Bytes that the padded scores and caches of the plain form take."""
    if c["op"] != "attend":
        return 0
    return c["requests"] * c["kv_max"] * (c["heads"] * c["q_max"] + 4 * c["kv_heads"] * c["dim"]) * 4


def draw(rng):
    most = {op: max(_cost(c) for c in listed() if c["op"] == op) for op in ("rope", "attend", "sample")}
    while True:
        c = _draw_one(rng)
        if _cost(c) <= most[c["op"]] and _memory(c) <= 8e9:
            return c


def _cost(c):
    w = work(c)
    return max(w["bytes"], w["flops"] / 280)


# --- lengths and frequencies -----------------------------------------------------

def _lengths(c):
    """New tokens and context (the new tokens included) of each request."""
    rng = random.Random(c["lens"] * 7919 + c["requests"])
    q = [_log(rng, c["q_min"], c["q_max"]) for _ in range(c["requests"])]
    kv = [max(n, _log(rng, c["kv_min"], c["kv_max"])) for n in q]
    if c["requests"] > 1:       # both ends of the range are there
        q[0], kv[0], kv[-1] = c["q_max"], max(c["q_max"], c["kv_max"]), max(q[-1], c["kv_min"])
    return q, kv


def _frequencies(c):
    """Radians per position of each rotated pair, and the factor on cos and sin."""
    f = 10000.0 ** (-2.0 * np.arange(c["rot"] // 2) / c["rot"])
    if c["scaling"] == "linear":
        return f / 4.0, 1.0
    if c["scaling"] == "by_parts":      # Peng et al. 2023: a ramp over the turns in the trained length
        turns = 4096 * f / (2 * np.pi)
        keep = np.clip((turns - 1.0) / (32.0 - 1.0), 0.0, 1.0)
        return f * ((1.0 - keep) / 32.0 + keep), 0.1 * math.log(32.0) + 1.0
    return f, 1.0


def _visible(n, kv, window):
    """(query, key) pairs of one request, and its keys that some query sees."""
    first = kv - n
    lo = np.arange(first, kv)
    lo = np.maximum(lo - window + 1, 0) if window else np.zeros(n, np.int64)
    return int((np.arange(first, kv) - lo + 1).sum()), int(kv - lo[0]) if n else 0


def work(case):
    c = case
    if c["op"] == "sample":
        n = c["rows"] * c["vocab"]
        size = 4 if c["dtype"] == "f32" else 2
        return {"bytes": n * size + (n // 8 if c["mask"] else 0) + c["rows"] * 28, "flops": 3 * n}
    q, kv = _lengths(c)
    if c["op"] == "rope":
        per = (c["heads"] + 2 * c["kv_heads"]) * c["dim"]
        src = 4 if c["src"] == "f32" else 2
        turned = (c["heads"] + c["kv_heads"]) * c["rot"]
        return {"bytes": sum(q) * per * (src + 2), "flops": sum(q) * 3 * turned}
    seen = [_visible(n, k, c["window"]) for n, k in zip(q, kv)]
    pairs, keys = sum(s[0] for s in seen), sum(s[1] for s in seen)
    return {"bytes": keys * c["kv_heads"] * c["dim"] * 4 + sum(q) * c["heads"] * (c["dim"] * 4 + 4),
            "flops": 4 * pairs * c["heads"] * c["dim"]}


# --- what a program has in hand ----------------------------------------------------

def _paged(c, g):
    """Batch metadata and a cache whose pages are in no order, with spare ones."""
    q, kv = _lengths(c)
    page, b = c["page"], c["requests"]
    need = [-(-k // page) for k in kv]
    pages = sum(need) + 3
    order = torch.randperm(pages, generator=g, device="cuda").to(torch.int32)
    table = torch.full((b, max(need)), -1, dtype=torch.int32, device="cuda")
    at = 0
    for r, k in enumerate(need):
        table[r, :k] = order[at:at + k]
        at += k
    start = torch.tensor([0] + list(np.cumsum(q)), dtype=torch.int32, device="cuda")
    length = torch.tensor(kv, dtype=torch.int32, device="cuda")
    dt = DTYPES[c["dtype"]]

    def fill():
        shape = (pages, page, c["kv_heads"], c["dim"])
        if c["cache"] == "head":
            shape = (pages, c["kv_heads"], page, c["dim"])
        t = torch.randn(shape, generator=g, device="cuda", dtype=dt)
        return t.transpose(1, 2) if c["cache"] == "head" else t

    return {"tokens": sum(q), "new": max(q), "start": start, "length": length, "table": table,
            "k": fill(), "v": fill()}


def _tree(q, seed):
    """Each drafted token's parent is an earlier one of its request, or the context."""
    rng, words = random.Random(seed), []
    for n in q:
        own_words = []
        for i in range(n):
            parent = rng.randrange(-1, i) if i else -1
            own_words.append((own_words[parent] if parent >= 0 else 0) | (1 << i))
        words += own_words
    return torch.tensor(words, dtype=torch.int64, device="cuda")


def prepare(case, seed):
    c = case
    g = torch.Generator(device="cuda")
    g.manual_seed(seed)
    if c["op"] == "sample":
        return _prepare_sample(c, g)
    s = {"case": c, **_paged(c, g)}
    t, dim = s["tokens"], c["dim"]
    if c["op"] == "rope":
        src = DTYPES[c["src"]]
        # one row of the joint projection: queries, keys, values
        row = torch.randn((t, c["heads"] + 2 * c["kv_heads"], dim), generator=g, device="cuda")
        s["q"], s["new_k"], s["new_v"] = row.to(src).split([c["heads"], c["kv_heads"], c["kv_heads"]], 1)
        s["out"] = torch.empty((t, c["heads"], dim), dtype=DTYPES[c["dtype"]], device="cuda")
        freqs, s["factor"] = _frequencies(c)
        s["turns"] = torch.tensor(np.rint(freqs / (2 * np.pi) * 2.0 ** TURN).astype(np.int64),
                                  device="cuda")
    else:
        s["q"] = 2 * torch.randn((t, c["heads"], dim), generator=g, device="cuda",
                                 dtype=DTYPES[c["dtype"]])
        s["out"] = torch.empty_like(s["q"])
        s["lse"] = torch.empty((t, c["heads"]), dtype=torch.float32, device="cuda")
        s["scale"] = dim ** -0.5
        s["tree"] = _tree(_lengths(c)[0], seed) if c["tree"] else None
    if own:     # the handles that a program keeps
        import few_row_packed_gb300 as lbv
        s["cache"] = lbv.KVCache(s["k"], s["v"])
        s["batch"] = lbv.Batch(s["start"], s["length"], s["table"], t)
        if c["op"] == "rope":
            layout = lbv.ROPE_HALF if c["layout"] == "half" else lbv.ROPE_INTERLEAVED
            s["rope"] = lbv.Rope(freqs, layout, s["factor"])
        else:
            s["work"] = torch.zeros(lbv.attend_workspace_bytes(s["cache"], s["batch"], c["heads"]),
                                    dtype=torch.uint8, device="cuda")
    return s


def _prepare_sample(c, g):
    m, v = c["rows"], c["vocab"]
    # a broad body and a few tokens well above it, as a head's logits have them
    logits = torch.randn((m, v), generator=g, device="cuda").mul_(c["spread"])
    top = torch.randint(0, v, (m, 40), generator=g, device="cuda")
    high = 6 + 3 * c["spread"] * torch.rand((m, 40), generator=g, device="cuda")
    logits.scatter_reduce_(1, top, high, "amax")        # a token may come twice
    s = {"case": c, "logits": logits.to(DTYPES[c["dtype"]])}
    s["u"] = torch.rand(m, generator=g, device="cuda")

    def spread(lo, hi):
        return lo + (hi - lo) * torch.rand(m, generator=g, device="cuda")

    s["temperature"] = spread(0.5, 1.3)
    s["top_k"] = s["top_p"] = s["min_p"] = s["mask"] = None
    rule = c["rule"]
    if rule in ("top_k_top_p", "mixed"):
        s["top_k"] = torch.randint(5, 200, (m,), generator=g, device="cuda", dtype=torch.int32)
    if rule in ("top_k_top_p", "top_p_min_p", "mixed"):
        s["top_p"] = spread(0.5, 0.99)
    if rule in ("top_p_min_p", "mixed"):
        s["min_p"] = spread(0.0, 0.1)
    if rule == "mixed":         # rows that switch a filter off, and greedy rows
        off = torch.randint(0, 5, (m,), generator=g, device="cuda")
        s["top_k"] = torch.where(off == 0, 0, s["top_k"])
        s["top_p"] = torch.where(off == 1, 1.0, s["top_p"])
        s["min_p"] = torch.where(off == 2, 0.0, s["min_p"])
        s["temperature"] = torch.where(off == 3, 0.0, s["temperature"])
    if c["mask"]:
        words = [torch.randint(-2 ** 31, 2 ** 31, (m, -(-v // 32)), generator=g, device="cuda",
                               dtype=torch.int64).to(torch.int32) for _ in range(2)]
        s["mask"] = words[0] | words[1]         # three tokens in four are allowed
    s["token"] = torch.empty(m, dtype=torch.int32, device="cuda")
    s["prob"] = torch.empty(m, dtype=torch.float32, device="cuda")
    return s


# --- one pass ------------------------------------------------------------------------

def run(state):
    op = state["case"]["op"]
    if own:
        return {"rope": _own_rope, "attend": _own_attend, "sample": _own_sample}[op](state)
    return {"rope": _plain_rope, "attend": _plain_attend, "sample": _plain_sample}[op](state)


def _own_rope(s):
    import few_row_packed_gb300 as lbv
    lbv.rope_append(s["rope"], s["batch"], s["cache"], s["q"], s["new_k"], s["new_v"], s["out"])
    return {"q": s["out"], "k": s["k"], "v": s["v"]}


def _own_attend(s):
    import few_row_packed_gb300 as lbv
    lbv.attend(s["cache"], s["batch"], s["q"], s["out"], s["scale"], window=s["case"]["window"],
               tree=s["tree"], lse=s["lse"], workspace=s["work"])
    return {"out": s["out"], "lse": s["lse"]}


def _own_sample(s):
    import few_row_packed_gb300 as lbv
    lbv.sample(s["logits"], s["u"], s["token"], prob=s["prob"], temperature=s["temperature"],
               top_k=s["top_k"], top_p=s["top_p"], min_p=s["min_p"], mask=s["mask"],
               temperature_last=s["case"]["last"])
    return {"token": s["token"], "prob": s["prob"]}


def _places(s):
    """Request and position of every new token."""
    at = torch.arange(s["tokens"], device="cuda", dtype=torch.int32)
    request = torch.bucketize(at, s["start"][1:], right=True)
    position = s["length"][request] - s["start"][1:][request] + at
    return request, position.long()


def _plain_rope(s):
    c = s["case"]
    request, position = _places(s)
    turn = (position[:, None] * s["turns"]) & ((1 << TURN) - 1)
    angle = (turn.float() * (2 * math.pi / 2 ** TURN))[:, None]
    cos, sin = angle.cos() * s["factor"], angle.sin() * s["factor"]
    half = c["rot"] // 2

    def rotate(x):
        x = x.float()
        if c["layout"] == "half":
            a, b = x[..., :half], x[..., half:2 * half]
            turned = torch.cat((a * cos - b * sin, b * cos + a * sin), -1)
        else:
            a, b = x[..., 0:2 * half:2], x[..., 1:2 * half:2]
            turned = torch.stack((a * cos - b * sin, b * cos + a * sin), -1).flatten(-2)
        return torch.cat((turned, x[..., 2 * half:]), -1)

    s["out"].copy_(rotate(s["q"]))
    page = s["table"][request, position // c["page"]].long()
    slot = position % c["page"]
    s["k"][page, slot] = rotate(s["new_k"]).to(s["k"].dtype)
    s["v"][page, slot] = s["new_v"].to(s["v"].dtype)
    return {"q": s["out"], "k": s["k"], "v": s["v"]}


def _scores_mask(s, count):
    """Which of `count` key positions each of a request's queries sees: [B, new, count]."""
    new = s["start"][1:] - s["start"][:-1]
    first = (s["length"] - new)[:, None, None].long()
    at = torch.arange(s["new"], device="cuda")[None, :, None]
    key = torch.arange(count, device="cuda")[None, None, :]
    mine = first + at
    if s["tree"] is None:
        sees = key <= mine
    else:
        word = s["tree"][(s["start"][:-1, None].long() + at[..., 0]).clamp(max=s["tokens"] - 1)]
        bit = (word[..., None] >> (key - first).clamp(0, 63)) & 1
        sees = (key < first) | ((key - first < 64) & (bit == 1))
    sees = sees & (key < s["length"][:, None, None])
    if s["case"]["window"]:
        sees = sees & (key > mine - s["case"]["window"])
    return sees


def _attention(s, wide):
    """The formula in `wide` (32 or 64 bits), rounded nowhere."""
    c = s["case"]
    b, hkv, dim = c["requests"], c["kv_heads"], c["dim"]
    group, new = c["heads"] // hkv, s["new"]
    request, position = _places(s)
    row = torch.arange(s["tokens"], device="cuda") - s["start"][request]
    q = torch.zeros((b, new, c["heads"], dim), dtype=wide, device="cuda")
    q[request, row] = s["q"].to(wide)
    q = q.view(b, new, hkv, group, dim).permute(0, 2, 3, 1, 4).reshape(b, hkv, group * new, dim)
    pages = s["table"].long().clamp(min=0)
    count = pages.shape[1] * c["page"]
    k = s["k"][pages].reshape(b, count, hkv, dim).permute(0, 2, 3, 1).to(wide)
    score = (q @ k).mul_(s["scale"]).view(b, hkv, group, new, count)
    del k
    score.masked_fill_(~_scores_mask(s, count)[:, None, None], -math.inf)
    top = score.amax(-1, keepdim=True)
    top = torch.where(top == -math.inf, 0, top)
    score.sub_(top).exp_()
    total = score.sum(-1, keepdim=True)
    v = s["v"][pages].reshape(b, count, hkv, dim).permute(0, 2, 1, 3).to(wide)
    unused = torch.arange(count, device="cuda")[None, :] >= s["length"][:, None]
    v = v.masked_fill(unused[:, None, :, None], 0)
    out = (score.view(b, hkv, group * new, count) @ v).view(b, hkv, group, new, dim)
    out = torch.where(total > 0, out / total, 0)
    lse = (top + total.log())[..., 0]
    out = out.permute(0, 3, 1, 2, 4).reshape(b, new, c["heads"], dim)[request, row]
    lse = lse.permute(0, 3, 1, 2).reshape(b, new, c["heads"])[request, row]
    return out, lse


def _plain_attend(s):
    out, lse = _attention(s, torch.float32)
    s["out"].copy_(out)
    s["lse"].copy_(lse)
    return {"out": s["out"], "lse": s["lse"]}


def _allowed(s):
    """Logits in 32 bits, with those that cannot be drawn at -inf."""
    x = s["logits"].float()
    x = torch.where(x.isnan(), -math.inf, x)
    if s["mask"] is not None:
        at = torch.arange(x.shape[1], device="cuda")
        x = torch.where((s["mask"][:, at // 32] >> (at % 32)) & 1 == 1, x, -math.inf)
    return x


def _fraction(p):
    """floor(p * 2^24) of a fraction, as whole numbers."""
    return (p.float() * 2.0 ** 24).clamp(0, 2 ** 24).long()


def _part(fraction, total):
    """floor(fraction * total / 2^24) in whole numbers of at most 63 bits."""
    return fraction * (total >> 32) * 256 + ((fraction * (total & 0xFFFFFFFF)) >> 24)


def _plain_sample(s):
    # Weights are whole numbers, floor(2^40 exp((l - max) / T)): their sums do
    # not depend on the order, so that equal inputs give equal tokens.
    x = _allowed(s)
    m = x.shape[0]
    cold = ~(s["temperature"] > 0)[:, None]
    inverse = torch.where(cold, 1.0, 1.0 / torch.where(cold, 1.0, s["temperature"][:, None]))
    top = x.amax(-1, keepdim=True)
    below = torch.where(x == top, 0.0, x - top)

    def weights(rate):
        w = (below * rate).exp()
        w = torch.where(x == -math.inf, 0.0, w)
        return w, (w * 2.0 ** 40).long()

    drawn = weights(inverse)[1]
    w, whole = weights(1.0 if s["case"]["last"] else inverse)
    order = torch.sort(x, dim=-1, descending=True, stable=True).indices
    ranked = whole.gather(1, order)
    rank = torch.arange(x.shape[1], device="cuda")[None, :]
    count = (x != -math.inf).sum(-1, keepdim=True)
    most = count
    if s["top_k"] is not None:
        k = s["top_k"][:, None].long()
        most = torch.where(k > 0, torch.minimum(k, most), most)
    most = torch.where(cold, torch.minimum(most, torch.ones_like(most)), most)
    ranked = torch.where(rank < most, ranked, 0)
    before = ranked.cumsum(-1) - ranked
    keep = rank < most
    if s["top_p"] is not None:
        p = s["top_p"][:, None]
        limit = _part(_fraction(p), ranked.sum(-1, keepdim=True))
        keep = keep & ((rank == 0) | (before < limit) | (p >= 1))
    if s["min_p"] is not None:
        keep = keep & ((rank == 0) | (w.gather(1, order) >= s["min_p"][:, None]))
    keep = torch.zeros_like(keep).scatter_(1, order, keep)
    drawn = torch.where(keep, drawn, 0)
    upto = drawn.cumsum(-1)
    total = upto[:, -1:]
    target = _part(_fraction(s["u"][:, None]).clamp(max=2 ** 24 - 1), total)
    token = (upto <= target).sum(-1, keepdim=True)
    none = total[:, 0] == 0
    token = torch.where(none[:, None], 0, token)
    prob = drawn.gather(1, token).float() / total.float()
    s["token"].copy_(torch.where(none, -1, token[:, 0]))
    s["prob"].copy_(torch.where(none, 0.0, prob[:, 0]))
    return {"token": s["token"], "prob": s["prob"]}


# --- the definitions in 64 bits ---------------------------------------------------------

def exact(case, seed):
    if work(case)["flops"] > 2e12 or 2 * _memory(case) > 60e9:
        return None
    with torch.no_grad():
        s = prepare(case, seed)
        return {"rope": _exact_rope, "attend": _exact_attend, "sample": _exact_sample}[case["op"]](s)


def _exact_rope(s):
    c = s["case"]
    freqs, factor = _frequencies(c)
    q_len, kv_len = _lengths(c)
    position = torch.cat([torch.arange(k - n, k) for n, k in zip(q_len, kv_len)]).cuda()
    request = torch.repeat_interleave(torch.arange(len(q_len)), torch.tensor(q_len)).cuda()
    angle = position.double()[:, None, None] * torch.from_numpy(freqs).cuda()
    unit = torch.polar(torch.full_like(angle, factor), angle)       # a pair is a complex number

    def rotate(x):
        x, half = x.double(), c["rot"] // 2
        rows, heads = x.shape[:2]
        if c["layout"] == "half":
            pair = x[..., :c["rot"]].reshape(rows, heads, 2, half).transpose(2, 3)
        else:
            pair = x[..., :c["rot"]].reshape(rows, heads, half, 2)
        pair = torch.view_as_real(torch.view_as_complex(pair.contiguous()) * unit)
        if c["layout"] == "half":
            pair = pair.transpose(2, 3)
        y = x.clone()
        y[..., :c["rot"]] = pair.reshape(rows, heads, c["rot"])
        return y

    k, v = s["k"].double(), s["v"].double()
    where = s["table"][request, position // c["page"]].long(), position % c["page"]
    k[where], v[where] = rotate(s["new_k"]), s["new_v"].double()
    return {"q": rotate(s["q"]), "k": k, "v": v}


def _exact_attend(s):
    """Request by request, over the gathered context."""
    c = s["case"]
    group = c["heads"] // c["kv_heads"]
    outs, sums, at = [], [], 0
    for r, (n, kv) in enumerate(zip(*_lengths(c))):
        pages = s["table"][r, :-(-kv // c["page"])].long()
        k, v = (t[pages].reshape(-1, c["kv_heads"], c["dim"])[:kv].double() for t in (s["k"], s["v"]))
        mine = torch.arange(kv - n, kv, device="cuda")[:, None]
        key = torch.arange(kv, device="cuda")[None, :]
        hidden = key > mine
        if s["tree"] is not None:
            bits = (s["tree"][at:at + n, None] >> torch.arange(min(n, 64), device="cuda")) & 1
            hidden = torch.zeros((n, kv), dtype=torch.bool, device="cuda")
            hidden[:, kv - n:] = True
            hidden[:, kv - n:kv - n + bits.shape[1]] = bits == 0
        if c["window"]:
            hidden = hidden | (mine - key >= c["window"])
        out = torch.empty((n, c["heads"], c["dim"]), dtype=torch.float64, device="cuda")
        total = torch.empty((n, c["heads"]), dtype=torch.float64, device="cuda")
        for h in range(c["heads"]):
            score = s["q"][at:at + n, h].double() @ k[:, h // group].T * s["scale"]
            score.masked_fill_(hidden, -math.inf)
            total[:, h] = torch.logsumexp(score, -1)
            out[:, h] = torch.softmax(score, -1) @ v[:, h // group]
        outs.append(out)
        sums.append(total)
        at += n
    return {"out": torch.cat(outs), "lse": torch.cat(sums)}


def _exact_sample(s):
    rows = []
    for i in range(s["case"]["rows"]):
        rows.append(_exact_row({k: (v[i:i + 1] if isinstance(v, torch.Tensor) else v)
                                for k, v in s.items()}))
    return {"token": None, "prob": torch.tensor(rows, dtype=torch.float64)}


def _exact_row(s):
    """Probability of the token drawn for one row."""
    x = _allowed(s)[0].double()
    t = float(s["temperature"])
    value, order = torch.sort(x, descending=True, stable=True)
    n = int((value > -math.inf).sum())
    if n == 0:
        return 0.0
    value, order = value[:n], order[:n]
    if not t > 0:
        return 1.0
    p = torch.softmax(value if s["case"]["last"] else value / t, 0)
    if s["top_k"] is not None and int(s["top_k"]) > 0:
        n = min(n, int(s["top_k"]))
    p = p[:n] / p[:n].sum()
    keep = torch.ones(n, dtype=torch.bool, device="cuda")
    if s["top_p"] is not None and float(s["top_p"]) < 1:
        keep &= p.cumsum(0) - p < float(s["top_p"])
    if s["min_p"] is not None:
        keep &= p >= float(s["min_p"]) * p[0]
    keep[0] = True
    place, by = torch.sort(order[:n][keep])
    p = torch.softmax(value[:n][keep] / t, 0)[by]
    return float(p[min(int((p.cumsum(0) <= float(s["u"])).sum()), len(p) - 1)])
