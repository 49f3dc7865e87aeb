"""Cases of the operators on the cache itself: the append to a cache held in 4
bits with the tokens read back, attention over that cache, attention with a
sliding window whose first tokens stay visible, and moves of tokens and pages.

``run`` computes a case in plain torch operations (32 bits, rounded once at
the end), or with ``own`` set through the framework's entry points.  ``exact``
gives the same outputs in 64 bits from the definitions.

Shapes: 6144-wide queries with 1024-wide keys and values are 48 query and 8
key/value heads of 128.
"""
import math
import random

import numpy as np
import torch

own = False

DTYPES = {"f32": torch.float32, "f16": torch.float16, "bf16": torch.bfloat16}
TURN = 40                      # fraction bits of an angle in turns
GROUP = 64                     # elements of a head that share a scale and a bias


# --- the cases -----------------------------------------------------------------

def _append(name, requests, q, kv, heads, kv_heads, dim, rot, layout, src, dtype, page):
    return {"name": name, "op": "append", "bits": 4, "requests": requests, "q_min": q[0], "q_max": q[1],
            "kv_min": kv[0], "kv_max": kv[1], "heads": heads, "kv_heads": kv_heads, "dim": dim,
            "rot": rot, "layout": layout, "src": src, "dtype": dtype, "page": page, "lens": 1}


def _attend(name, bits, requests, q, kv, heads, kv_heads, dim, dtype, page, window=0, sinks=0, tree=False):
    return {"name": name, "op": "attend", "bits": bits, "requests": requests, "q_min": q[0],
            "q_max": q[1], "kv_min": kv[0], "kv_max": kv[1], "heads": heads, "kv_heads": kv_heads,
            "dim": dim, "dtype": dtype, "page": page, "window": window, "sinks": sinks, "tree": tree,
            "lens": 1}


def _keep(name, bits, requests, q, kv, kv_heads, dim, dtype, page):
    return {"name": name, "op": "keep", "bits": bits, "requests": requests, "q_min": q[0], "q_max": q[1],
            "kv_min": kv[0], "kv_max": kv[1], "kv_heads": kv_heads, "dim": dim, "dtype": dtype,
            "page": page, "lens": 1}


def _copy(name, bits, pages, count, kv_heads, dim, dtype, page):
    return {"name": name, "op": "copy", "bits": bits, "pages": pages, "count": count,
            "kv_heads": kv_heads, "dim": dim, "dtype": dtype, "page": page}


def listed():
    return [
        # the 8 drafted rows of one request, from the fp32 projections: latency
        _append("append4_verify8", 1, (8, 8), (4099, 4099), 48, 8, 128, 128, "half", "f32", "f16", 64),
        # a prompt's chunk in a long context
        _append("append4_prompt", 1, (8191, 8191), (100000, 100000), 48, 8, 128, 128, "half", "f32",
                "bf16", 128),
        # plain decoding of one request: latency
        _attend("attend4_decode1", 4, 1, (1, 1), (2011, 2011), 48, 8, 128, "f16", 16),
        # a few drafted tokens after one very long context
        _attend("attend4_long", 4, 1, (4, 4), (200003, 200003), 32, 8, 128, "bf16", 64),
        # ordinary batched decoding, ragged contexts
        _attend("attend4_decode64", 4, 64, (1, 1), (500, 16384), 48, 8, 128, "f16", 64),
        # batched verify calls of trees of drafted tokens
        _attend("attend4_verify32", 4, 32, (1, 8), (900, 20000), 48, 8, 128, "bf16", 32, tree=True),
        # a prompt's chunk of 2048 tokens at the end of a 16k context
        _attend("attend4_prompt", 4, 1, (2048, 2048), (16384, 16384), 48, 8, 128, "bf16", 64),
        # batched decoding of a layer with a window and sinks, 16-bit cache with small heads
        _attend("sinks_decode32", 16, 32, (1, 8), (700, 60000), 32, 8, 64, "bf16", 32, 4096, 4),
        # a prompt's chunk in such a layer
        _attend("sinks_prompt", 16, 1, (2048, 2048), (16384, 16384), 48, 8, 128, "bf16", 64, 1024, 16),
        # decoding of such a layer over a cache in 4 bits
        _attend("sinks4_decode32", 4, 32, (1, 1), (500, 30000), 48, 8, 128, "f16", 64, 2048, 4),
        # the accepted ones of 64 requests' trees of drafted tokens close up
        _keep("keep_batch64", 16, 64, (8, 64), (300, 4000), 8, 128, "f16", 16),
        # pages of forked requests get copies of their own
        _copy("copy_pages", 16, 600, 256, 8, 128, "bf16", 64),
    ]


def _log(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def _draw_one(rng):
    op = rng.choice(["append", "attend4", "attend4", "sinks", "sinks", "keep", "copy"])
    lens = rng.randrange(1, 1 << 20)
    heads, kv_heads = rng.choice([(48, 8), (32, 8), (28, 4), (16, 2), (8, 8), (20, 4)])
    dim = 128 if heads == 48 else rng.choice([64, 64, 128])
    dtype = rng.choice(["f16", "bf16"])
    page = rng.choice([16, 32, 64, 128])
    if op == "append":
        b = _log(rng, 1, 64)
        q = rng.choice([(1, 1), (1, 8), (8, 8), (1, _log(rng, 16, 8192))])
        kv = _log(rng, max(64, q[1]), 120000)
        c = _append(None, b, q, (max(q[1], kv // 3), kv), heads, kv_heads, dim, rng.choice([dim, dim // 2]),
                    rng.choice(["half", "interleaved"]), rng.choice(["f32", "f16", "bf16"]), dtype, page)
    elif op in ("attend4", "sinks"):
        kind = rng.choice(["decode", "verify", "prompt"])
        if kind == "decode":
            b, q, kv = _log(rng, 1, 128), (1, 1), _log(rng, 64, 65536)
        elif kind == "verify":
            b, q, kv = _log(rng, 1, 64), (rng.randrange(1, 5), 8), _log(rng, 64, 65536)
        else:
            b, n = _log(rng, 1, 8), _log(rng, 16, 2048)
            q, kv = (max(1, n // 3), n), _log(rng, n, 16384)
        masked = op == "sinks" or rng.random() < 0.3
        c = _attend(None, 4 if op == "attend4" else rng.choice([4, 16, 16]), b, q, (max(q[1], kv // 3), kv),
                    heads, kv_heads, dim, dtype, page, _log(rng, 100, 8192) if masked else 0,
                    _log(rng, 1, 130) if masked else 0, kind == "verify" and rng.random() < .5)
    elif op == "keep":
        c = _keep(None, rng.choice([4, 16]), _log(rng, 1, 256), rng.choice([(1, 8), (8, 8), (10, 64)]),
                  (64, _log(rng, 100, 8000)), kv_heads, dim, dtype, page)
    else:
        count = _log(rng, 1, 256)
        c = _copy(None, rng.choice([4, 16]), 2 * count + rng.randrange(1, 90), count, kv_heads, dim, dtype, page)
    if op != "copy":
        c["lens"] = lens
    del c["name"]
    return c


def _memory(c):
    """Bytes that the padded scores and caches of the plain form take."""
    if c["op"] != "attend":
        return 0
    return c["requests"] * c["kv_max"] * (c["heads"] * c["q_max"] + 4 * c["kv_heads"] * c["dim"]) * 4


def draw(rng):
    most = {op: max(_cost(c) for c in listed() if c["op"] == op) for op in ("append", "attend", "keep", "copy")}
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
    kv = [max(n, _log(rng, c["kv_min"], max(c["kv_min"], c["kv_max"]))) for n in q]
    if c["requests"] > 1:       # both ends of the range are there
        q[0], kv[0], kv[-1] = c["q_max"], max(c["q_max"], c["kv_max"]), max(q[-1], c["kv_min"])
    return q, kv


def _kept(c):
    """A word for each request: the path of accepted ones among its new tokens."""
    rng = random.Random(c["lens"] * 104729 + 17)
    return [sum(1 << b for b in range(n) if rng.random() < 0.45) for n in _lengths(c)[0]]


def _frequencies(c):
    """Radians per position of each rotated pair."""
    return 10000.0 ** (-2.0 * np.arange(c["rot"] // 2) / c["rot"])


def _visible(n, kv, window, sinks):
    """(query, key) pairs of one request, and its keys that some query sees."""
    pos = np.arange(kv - n, kv)
    if not window:
        return int((pos + 1).sum()), kv
    lo = np.maximum(pos - window + 1, 0)
    return int((pos + 1 - lo + np.minimum(lo, sinks)).sum()), int(kv - lo[0] + min(int(lo[0]), sinks))


def _token_bytes(c):
    """Bytes of a token's keys and values in one head."""
    return c["dim"] // GROUP * 72 if c["bits"] == 4 else 4 * c["dim"]


def work(case):
    c = case
    if c["op"] == "copy":
        return {"bytes": 2 * c["count"] * c["page"] * c["kv_heads"] * _token_bytes(c), "flops": 0}
    q, kv = _lengths(c)
    if c["op"] == "keep":
        # a kept token behind a dropped one moves; a word and three lengths a request
        moved = sum(sum(1 for b in range(64) if w >> b & 1 and (w & ((1 << b) - 1)) != (1 << b) - 1)
                    for w in _kept(c))
        return {"bytes": 2 * moved * c["kv_heads"] * _token_bytes(c) + 20 * c["requests"], "flops": 0}
    if c["op"] == "append":
        src = 4 if c["src"] == "f32" else 2
        rows = c["heads"] * (src + 2) + 2 * c["kv_heads"] * (src + 2)       # queries; keys and values read back
        return {"bytes": sum(q) * (rows * c["dim"] + 2 * c["kv_heads"] * _token_bytes(c)),
                "flops": sum(q) * (3 * (c["heads"] + c["kv_heads"]) * c["rot"] + 12 * c["kv_heads"] * c["dim"])}
    seen = [_visible(n, k, c["window"], c["sinks"]) for n, k in zip(q, kv)]
    pairs, keys = sum(s[0] for s in seen), sum(s[1] for s in seen)
    return {"bytes": keys * c["kv_heads"] * _token_bytes(c) + sum(q) * c["heads"] * (c["dim"] * 4 + 4),
            "flops": 4 * pairs * c["heads"] * c["dim"]}


# --- a cache in 4 bits ---------------------------------------------------------------
#
# Bytes [pages][heads][chunks of C = min(page, 64) slots][K codes, V codes, scales]: codes are
# [dim / 64][C][32] bytes, in each 32-bit word the even ones of 8 elements in the low half and
# the odd ones in the high half, from the lowest bits on; scales [K, V][dim / 64][C] are pairs
# (scale, bias) of the cache's 16-bit type.  An element is code * scale + bias, rounded to
# that type.

def _page_bytes(c):
    return c["page"] * c["kv_heads"] * (c["dim"] // GROUP) * 72


def _parts(data, c):
    """Codes [pages, heads, chunks, 2, dim / 64, C, 32] and scales [..., C, 2] of the bytes."""
    size, parts = min(c["page"], 64), c["dim"] // GROUP
    chunk = data.view(data.shape[0], c["kv_heads"], c["page"] // size, 72 * parts * size)
    codes = chunk[..., :64 * parts * size].unflatten(-1, (2, parts, size, 32))
    scales = chunk.view(DTYPES[c["dtype"]])[..., 32 * parts * size:].unflatten(-1, (2, parts, size, 2))
    return codes, scales


def _places4(c, slot):
    """Chunk of a page's slot, and its place there."""
    size = min(c["page"], 64)
    return slot // size, slot % size


def _values4(codes, scales, wide):
    """Elements (one more dimension in place of the bytes) in `wide`."""
    code = torch.stack((codes & 15, codes >> 4), -1).unflatten(-2, (8, 2, 2))      # word, odd, byte, half
    code = code.movedim(-3, -1).flatten(-4)
    x = code.to(wide) * scales[..., 0, None].to(wide) + scales[..., 1, None].to(wide)
    return x.to(scales.dtype).to(wide)


# --- what a program has in hand ----------------------------------------------------

def _fill(c, pages, g):
    """The cache's tensors with values in every slot."""
    dt = DTYPES[c["dtype"]]
    if c["bits"] == 16:
        shape = (pages, c["page"], c["kv_heads"], c["dim"])
        return {n: torch.randn(shape, generator=g, device="cuda", dtype=dt) for n in ("k", "v")}
    data = torch.empty((pages, _page_bytes(c)), dtype=torch.uint8, device="cuda")
    codes, scales = _parts(data, c)

    def half():         # codes as groups of normal values have them
        x = torch.randn(codes.shape, generator=g, device="cuda", dtype=torch.float16)
        return x.mul_(3.3).add_(7.5).round_().clamp_(0, 15).to(torch.uint8)

    codes.copy_(half() | half() << 4)
    step = 0.25 + 0.1 * torch.rand(scales.shape[:-1], generator=g, device="cuda")
    low = -7.5 * step + 0.2 * torch.randn(step.shape, generator=g, device="cuda")
    scales[..., 0], scales[..., 1] = step, low
    return {"data": data}


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
    return {"tokens": sum(q), "new": max(q), "start": start, "length": length, "table": table,
            **_fill(c, pages, g)}


def _tree(q, seed):
    """Each drafted token's parent is an earlier one of its request, or the context."""
    rng, words = random.Random(seed), []
    for n in q:
        own_words = []
        for i in range(n):
            parent = rng.randrange(-1, i) if i else -1
            own_words.append((own_words[parent] if parent >= 0 else 0) | (1 << i))
        words += own_words
    return _signed(words)


def _signed(words):
    """64-bit words on the device."""
    return torch.tensor([w - (1 << 64) if w >> 63 else w for w in words], dtype=torch.int64, device="cuda")


def prepare(case, seed):
    c = case
    g = torch.Generator(device="cuda")
    g.manual_seed(seed)
    dt = DTYPES[c["dtype"]]
    if c["op"] == "copy":
        s = {"case": c, **_fill(c, c["pages"], g)}
        order = torch.randperm(c["pages"], generator=g, device="cuda").to(torch.int32)
        s["src"], s["dst"] = order[:c["count"]].clone(), order[c["count"]:2 * c["count"]].clone()
    else:
        s = {"case": c, **_paged(c, g)}
        t, dim = s["tokens"], c["dim"]
    if c["op"] == "append":
        # one row of the joint projection: queries, keys, values
        row = torch.randn((t, c["heads"] + 2 * c["kv_heads"], dim), generator=g, device="cuda")
        s["q"], s["new_k"], s["new_v"] = row.to(DTYPES[c["src"]]).split(
            [c["heads"], c["kv_heads"], c["kv_heads"]], 1)
        s["out"] = torch.empty((t, c["heads"], dim), dtype=dt, device="cuda")
        s["back_k"], s["back_v"] = (torch.empty((t, c["kv_heads"], dim), dtype=dt, device="cuda") for _ in "kv")
        s["turns"] = torch.tensor(np.rint(_frequencies(c) / (2 * np.pi) * 2.0 ** TURN).astype(np.int64),
                                  device="cuda")
    elif c["op"] == "attend":
        s["q"] = 2 * torch.randn((t, c["heads"], dim), generator=g, device="cuda", dtype=dt)
        s["out"] = torch.empty_like(s["q"])
        s["lse"] = torch.empty((t, c["heads"]), dtype=torch.float32, device="cuda")
        s["scale"] = dim ** -0.5
        s["tree"] = _tree(_lengths(c)[0], seed) if c["tree"] else None
    elif c["op"] == "keep":
        s["kept"] = _signed(_kept(c))
        s["left"] = torch.empty(c["requests"], dtype=torch.int32, device="cuda")
    if own:     # the handles that a program keeps
        import few_row_packed_gb300 as lbv
        s["cache"] = (lbv.KVCache(s["k"], s["v"]) if c["bits"] == 16 else
                      lbv.KVCache4(s["data"], c["page"], c["kv_heads"], c["dim"], dt))
        if c["op"] != "copy":
            s["batch"] = lbv.Batch(s["start"], s["length"], s["table"], t)
        if c["op"] == "append":
            # the frequencies that the plain form turns by: whole numbers of 2^-TURN turns
            s["rope"] = lbv.Rope(s["turns"].cpu().numpy() * (2 * np.pi / 2 ** TURN),
                                 lbv.ROPE_HALF if c["layout"] == "half" else lbv.ROPE_INTERLEAVED)
        if c["op"] == "attend":
            s["work"] = torch.zeros(lbv.attend_workspace_bytes(s["cache"], s["batch"], c["heads"]),
                                    dtype=torch.uint8, device="cuda")
    return s


# --- one pass ------------------------------------------------------------------------

def run(state):
    op = state["case"]["op"]
    if own:
        return {"append": _own_append, "attend": _own_attend, "keep": _own_keep, "copy": _own_copy}[op](state)
    return {"append": _plain_append, "attend": _plain_attend, "keep": _plain_keep, "copy": _plain_copy}[op](state)


def _held(s):
    """The whole cache as it is held."""
    return {"data": s["data"]} if s["case"]["bits"] == 4 else {"k": s["k"], "v": s["v"]}


def _own_append(s):
    import few_row_packed_gb300 as lbv
    lbv.rope_append(s["rope"], s["batch"], s["cache"], s["q"], s["new_k"], s["new_v"], s["out"])
    lbv.kv_read(s["batch"], s["cache"], s["back_k"], s["back_v"])
    return {"q": s["out"], "k": s["back_k"], "v": s["back_v"]}


def _own_attend(s):
    import few_row_packed_gb300 as lbv
    lbv.attend(s["cache"], s["batch"], s["q"], s["out"], s["scale"], window=s["case"]["window"],
               sinks=s["case"]["sinks"], tree=s["tree"], lse=s["lse"], workspace=s["work"])
    return {"out": s["out"], "lse": s["lse"]}


def _own_keep(s):
    import few_row_packed_gb300 as lbv
    lbv.kv_keep(s["batch"], s["cache"], s["kept"], s["left"])
    return {"left": s["left"], **_held(s)}


def _own_copy(s):
    import few_row_packed_gb300 as lbv
    lbv.kv_copy_pages(s["cache"], s["src"], s["dst"])
    return _held(s)


def _places(s):
    """Request and position of every new token."""
    at = torch.arange(s["tokens"], device="cuda", dtype=torch.int32)
    request = torch.bucketize(at, s["start"][1:], right=True)
    position = s["length"][request] - s["start"][1:][request] + at
    return request, position.long()


def _quantised(x, dt):
    """Codes (two in a byte) and (scale, bias) of groups of 64 fp32 values."""
    x = x.unflatten(-1, (-1, GROUP))
    low, high = x.amin(-1), x.amax(-1)
    scale, bias = ((high - low) / 15).to(dt), low.to(dt)
    step = scale.float()[..., None]
    code = (x - bias.float()[..., None]) * torch.where(step > 0, 1 / step, 0)
    code = code.round().clamp(0, 15).to(torch.uint8)
    code = code.unflatten(-1, (8, 2, 2, 2)).movedim(-1, -3)                         # word, odd, byte, half
    return (code[..., 0] | code[..., 1] << 4).flatten(-3), torch.stack((scale, bias), -1)


def _plain_append(s):
    c = s["case"]
    request, position = _places(s)
    turn = (position[:, None] * s["turns"]) & ((1 << TURN) - 1)
    angle = (turn.float() * (2 * math.pi / 2 ** TURN))[:, None]
    cos, sin = angle.cos(), angle.sin()
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
    new = torch.stack((rotate(s["new_k"]), s["new_v"].float()), 2)      # [tokens, heads, 2, dim]
    new_codes, new_scales = _quantised(new, DTYPES[c["dtype"]])
    codes, scales = _parts(s["data"], c)
    page = s["table"][request, position // c["page"]].long()
    chunk, slot = _places4(c, position % c["page"])
    codes[page, :, chunk, :, :, slot] = new_codes
    scales[page, :, chunk, :, :, slot] = new_scales
    back = _values4(codes[page, :, chunk, :, :, slot], scales[page, :, chunk, :, :, slot], torch.float32)
    back = back.flatten(-2)
    s["back_k"].copy_(back[:, :, 0])
    s["back_v"].copy_(back[:, :, 1])
    return {"q": s["out"], "k": s["back_k"], "v": s["back_v"]}


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
        sees = sees & ((key > mine - s["case"]["window"]) | (key < s["case"]["sinks"]))
    return sees


def _context(s, wide):
    """Keys and values of every request's pages: [B, count, heads, dim]."""
    c = s["case"]
    pages = s["table"].long().clamp(min=0)
    count = pages.shape[1] * c["page"]
    shape = (c["requests"], count, c["kv_heads"], c["dim"])
    if c["bits"] == 16:
        return tuple(s[n][pages].reshape(shape).to(wide) for n in ("k", "v"))
    codes, scales = _parts(s["data"], c)

    def values(which):          # [B, pages, heads, chunks, dim / 64, C, 64], slots before heads
        x = _values4(codes[pages, :, :, which], scales[pages, :, :, which], wide)
        return x.permute(0, 1, 3, 5, 2, 4, 6).reshape(shape)

    return values(0), values(1)


def _plain_attend(s):
    c = s["case"]
    b, hkv, dim = c["requests"], c["kv_heads"], c["dim"]
    group, new = c["heads"] // hkv, s["new"]
    request, position = _places(s)
    row = torch.arange(s["tokens"], device="cuda") - s["start"][request]
    q = torch.zeros((b, new, c["heads"], dim), device="cuda")
    q[request, row] = s["q"].float()
    q = q.view(b, new, hkv, group, dim).permute(0, 2, 3, 1, 4).reshape(b, hkv, group * new, dim)
    k, v = _context(s, torch.float32)
    count = k.shape[1]
    score = (q @ k.permute(0, 2, 3, 1)).mul_(s["scale"]).view(b, hkv, group, new, count)
    del k
    score.masked_fill_(~_scores_mask(s, count)[:, None, None], -math.inf)
    top = score.amax(-1, keepdim=True)
    top = torch.where(top == -math.inf, 0, top)
    score.sub_(top).exp_()
    total = score.sum(-1, keepdim=True)
    unused = torch.arange(count, device="cuda")[None, :] >= s["length"][:, None]
    v = v.masked_fill(unused[:, :, None, None], 0).permute(0, 2, 1, 3)
    out = (score.view(b, hkv, group * new, count) @ v).view(b, hkv, group, new, dim)
    out = torch.where(total > 0, out / total, 0)
    lse = (top + total.log())[..., 0]
    s["out"].copy_(out.permute(0, 3, 1, 2, 4).reshape(b, new, c["heads"], dim)[request, row])
    s["lse"].copy_(lse.permute(0, 3, 1, 2).reshape(b, new, c["heads"])[request, row])
    return {"out": s["out"], "lse": s["lse"]}


def _plain_keep(s):
    c = s["case"]
    new = s["start"][1:] - s["start"][:-1]
    at = torch.arange(64, device="cuda")
    kept = ((s["kept"][:, None] >> at) & 1 == 1) & (at < new[:, None])
    first = (s["length"] - new).long()[:, None]
    rank = kept.cumsum(1) - 1
    request, token = kept.nonzero(as_tuple=True)
    source, target = (first + at)[request, token], (first + rank)[request, token]

    def place(position):
        return s["table"][request, position // c["page"]].long(), position % c["page"]

    (page0, slot0), (page1, slot1) = place(source), place(target)
    if c["bits"] == 16:
        for t in (s["k"], s["v"]):
            t[page1, slot1] = t[page0, slot0]
    else:
        (chunk0, at0), (chunk1, at1) = _places4(c, slot0), _places4(c, slot1)
        for t in _parts(s["data"], c):
            t[page1, :, chunk1, :, :, at1] = t[page0, :, chunk0, :, :, at0]
    s["left"].copy_(first[:, 0] + kept.sum(1))
    return {"left": s["left"], **_held(s)}


def _plain_copy(s):
    for t in _held(s).values():
        t[s["dst"].long()] = t[s["src"].long()]
    return _held(s)


# --- the definitions in 64 bits ---------------------------------------------------------

def exact(case, seed):
    if case["op"] in ("keep", "copy"):          # moves: no computed numbers
        return None
    if work(case)["flops"] > 2e12 or 2 * _memory(case) > 60e9:
        return None
    with torch.no_grad():
        s = prepare(case, seed)
        return {"append": _exact_append, "attend": _exact_attend}[case["op"]](s)


def _exact_append(s):
    c = s["case"]
    dt = DTYPES[c["dtype"]]
    q_len, kv_len = _lengths(c)
    position = torch.cat([torch.arange(k - n, k) for n, k in zip(q_len, kv_len)]).cuda()
    angle = position.double()[:, None, None] * torch.from_numpy(_frequencies(c)).cuda()
    unit = torch.polar(torch.ones_like(angle), angle)       # a pair is a complex number

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

    def held(x):        # the nearest of 16 levels of each group
        x = x.double().reshape(*x.shape[:2], c["dim"] // GROUP, GROUP)
        low = x.min(-1, keepdim=True).values
        step = ((x.max(-1, keepdim=True).values - low) / 15).to(dt).double()
        low = low.to(dt).double()
        level = torch.where(step > 0, ((x - low) / step).nan_to_num().round().clamp(0, 15), 0)
        return (level * step + low).to(dt).double().reshape(*x.shape[:2], c["dim"])

    return {"q": rotate(s["q"]), "k": held(rotate(s["new_k"])), "v": held(s["new_v"])}


def _exact_rows(s, r, kv):
    """Keys and values of request r in 64 bits: [kv, heads, dim]."""
    c = s["case"]
    pages = s["table"][r, :-(-kv // c["page"])].long()
    if c["bits"] == 16:
        return tuple(t[pages].reshape(-1, c["kv_heads"], c["dim"])[:kv].double() for t in (s["k"], s["v"]))
    size, parts = min(c["page"], 64), c["dim"] // GROUP
    raw = s["data"][pages].reshape(-1, c["kv_heads"], c["page"] // size, 72 * parts * size)
    raw = raw.transpose(1, 2).reshape(-1, c["kv_heads"], 72 * parts * size)     # chunks in order
    out, plane = [], 32 * size
    for which in range(2):
        cols = []
        for part in range(parts):
            p = which * parts + part
            word = raw[:, :, p * plane:(p + 1) * plane].contiguous().view(torch.int32)
            word = word.reshape(-1, c["kv_heads"], size, 8, 1).long() & 0xFFFFFFFF
            at = 2 * parts * plane + 4 * size * p
            pair = raw[:, :, at:at + 4 * size].contiguous().view(DTYPES[c["dtype"]])
            pair = pair.reshape(-1, c["kv_heads"], size, 2).double()
            bits = torch.tensor([4 * (i // 2) + 16 * (i % 2) for i in range(8)], device="cuda")
            both = (word >> bits & 15).reshape(-1, c["kv_heads"], size, GROUP).double()
            cols.append((both * pair[..., :1] + pair[..., 1:]).to(DTYPES[c["dtype"]]).double())
        x = torch.cat(cols, -1).transpose(1, 2)
        out.append(x.reshape(-1, c["kv_heads"], c["dim"])[:kv])
    return out


def _exact_attend(s):
    """Request by request, over the gathered context."""
    c = s["case"]
    group = c["heads"] // c["kv_heads"]
    outs, sums, at = [], [], 0
    for r, (n, kv) in enumerate(zip(*_lengths(c))):
        k, v = _exact_rows(s, r, kv)
        mine = torch.arange(kv - n, kv, device="cuda")[:, None]
        key = torch.arange(kv, device="cuda")[None, :]
        hidden = key > mine
        if s["tree"] is not None:
            bits = (s["tree"][at:at + n, None] >> torch.arange(min(n, 64), device="cuda")) & 1
            hidden = torch.zeros((n, kv), dtype=torch.bool, device="cuda")
            hidden[:, kv - n:] = True
            hidden[:, kv - n:kv - n + bits.shape[1]] = bits == 0
        if c["window"]:
            hidden = hidden | ((mine - key >= c["window"]) & (key >= c["sinks"]))
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
