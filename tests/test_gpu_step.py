"""GPU tests of the rotary append, the attention over the paged cache and the
sampler against the fp64 oracles, at the sizes, masks and layouts where they
can go wrong."""
import numpy as np
import pytest

import few_row_packed_gb300 as lbv
from oracle import step

torch = pytest.importorskip("torch")
pytestmark = pytest.mark.gpu

DT = {"f16": torch.float16, "bf16": torch.bfloat16, "f32": torch.float32}
UNIT = {"f16": 2.0 ** -11, "bf16": 2.0 ** -8}       # half an ulp, relative
TINY = {"f16": 2.0 ** -25, "bf16": 2.0 ** -134}     # half a subnormal step


@pytest.fixture(scope="module", autouse=True)
def built():
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    lbv.build()


def f64(t):
    return t.double().cpu().numpy()


class Setup:
    """A batch over a cache whose pages are in no order; unused slots hold NaN."""

    def __init__(self, q_len, kv_len, kv_heads=2, dim=128, dtype="f16", page=16, order="token",
                 seed=0, pad=0, unmapped=()):
        g = torch.Generator().manual_seed(seed)
        self.g, self.dtype, self.dim = g, dtype, dim
        need = [max(0, -(-k // page)) for k in kv_len]
        pages = sum(need) + 2
        perm = torch.randperm(pages, generator=g).to(torch.int32)
        width = max(max(need), 1) + 1
        table = torch.full((len(q_len), width), -1, dtype=torch.int32)
        at = 0
        for r, n in enumerate(need):
            table[r, :n] = perm[at:at + n]
            at += n
        self.table = table.numpy()
        self.start = np.concatenate([[0], np.cumsum(q_len)]).astype(np.int32)
        self.kv_len = np.array(kv_len, np.int32)
        self.tokens = int(self.start[-1]) + pad
        nan = float("nan")

        def fill():
            shape = {"token": (pages, page, kv_heads, dim), "head": (pages, kv_heads, page, dim),
                     "gap": (pages, page, kv_heads, dim + 8)}[order]
            t = torch.full(shape, nan).to(DT[dtype]).cuda()
            return t.transpose(1, 2) if order == "head" else t[..., :dim]

        self.k, self.v = fill(), fill()
        for r in range(len(q_len)):
            for j in range(max(kv_len[r], 0)):
                for t in (self.k, self.v):
                    t[int(table[r, j // page]), j % page] = torch.randn((kv_heads, dim), generator=g).to(DT[dtype]).cuda()
        self.cache = lbv.KVCache(self.k, self.v)
        self.batch = lbv.Batch(torch.from_numpy(self.start).cuda(), torch.from_numpy(self.kv_len).cuda(),
                               table.cuda(), self.tokens)

    def rows(self, heads, dtype=None, scale=1.0, layout="plain"):
        x = (scale * torch.randn((self.tokens, heads, self.dim), generator=self.g)).to(DT[dtype or self.dtype]).cuda()
        return lay_out(x, layout)


def lay_out(x, layout):
    """The same values with other strides and alignments."""
    t, h, d = x.shape
    if layout == "fused":               # columns of a wider row
        wide = torch.zeros((t, h + 3, d), dtype=x.dtype, device=x.device)
        wide[:, 1:1 + h] = x
        return wide[:, 1:1 + h]
    if layout == "odd":                 # odd strides, one element off
        flat = torch.zeros(t * (h * (d + 1) + 1) + 1, dtype=x.dtype, device=x.device)
        y = flat[1:].as_strided((t, h, d), (h * (d + 1) + 1, d + 1, 1))
        y.copy_(x)
        return y
    if layout == "heads":               # heads outermost
        return x.transpose(0, 1).contiguous().transpose(0, 1)
    return x


# --- rotary append -----------------------------------------------------------------

@pytest.mark.parametrize("src, dtype, dim, rot, interleaved, order, layout, page", [
    ("f32", "f16", 128, 128, False, "token", "plain", 16),
    ("f32", "bf16", 128, 64, True, "head", "fused", 8),
    ("bf16", "bf16", 64, 64, True, "token", "heads", 64),
    ("f16", "f16", 64, 32, False, "gap", "odd", 32),
    ("f32", "f16", 128, 8, True, "head", "odd", 1024),
    ("f16", "bf16", 128, 128, False, "token", "fused", 128),
])
@pytest.mark.parametrize("q_len, kv_len", [
    ([1], [1]), ([3, 0, 8, 1], [3, 5, 70, 33]), ([5, 40], [2, 41]),
])
def test_rope_append(src, dtype, dim, rot, interleaved, order, layout, page, q_len, kv_len):
    s = Setup(q_len, kv_len, dim=dim, dtype=dtype, page=page, order=order, pad=2)
    freqs = lbv.rope_frequencies(rot, 500.0)
    factor = 1.25
    rope = lbv.Rope(freqs, lbv.ROPE_INTERLEAVED if interleaved else lbv.ROPE_HALF, factor)
    q, k, v = (s.rows(h, src, layout=layout) for h in (6, 2, 2))
    out = lay_out(torch.full((s.tokens, 6, dim), 7.0, device="cuda").to(DT[dtype]), layout)
    before = f64(s.k), f64(s.v)
    lbv.rope_append(rope, s.batch, s.cache, q, k, v, out)
    torch.cuda.synchronize()
    req, pos = step.positions(s.start, s.kv_len)
    n = len(req)

    def close(got, x):
        want, size = step.rotate(f64(x)[:n], pos, freqs, interleaved, factor)
        # one rounding; fp32 sums of two products; the angle to 2^-24 half turns
        tol = UNIT[dtype] * np.abs(want) + 2.0 ** -20 * factor * size + TINY[dtype]
        assert np.all(np.abs(got - want) <= tol)

    close(f64(out)[:n], q)
    assert np.all(f64(out)[n:] == 7.0)                  # rows of no request
    rows = [i for i in range(n) if pos[i] >= 0]
    got_k, got_v = f64(s.k), f64(s.v)
    page_of = [int(s.table[req[i], pos[i] // page]) for i in rows]
    slot = [int(pos[i] % page) for i in rows]
    kk = np.zeros((n, 2, dim))
    kk[rows] = got_k[page_of, slot]
    want_k, size = step.rotate(f64(k)[:n], pos, freqs, interleaved, factor)
    tol = UNIT[dtype] * np.abs(want_k) + 2.0 ** -20 * factor * size + TINY[dtype]
    assert np.all(np.abs(kk - want_k)[rows] <= tol[rows])
    vv = v.to(DT[dtype])
    assert np.array_equal(got_v[page_of, slot], f64(vv)[rows])
    for got, was in ((got_k, before[0]), (got_v, before[1])):       # nothing else moved
        got[page_of, slot] = was[page_of, slot] = 0
        assert np.array_equal(got, was, equal_nan=True)


def test_rope_positions_and_missing_slots():
    """Given positions turn the angle only; far positions stay exact; slots that
    do not exist are left out; keys and values go without queries."""
    s = Setup([4], [20], page=8)
    s.table[0, 2] = 99                                   # slots 16..19: outside the cache
    s.batch.block_table.copy_(torch.from_numpy(s.table))
    freqs = lbv.rope_frequencies(128, 10000.0)
    rope = lbv.Rope(freqs)
    where = np.array([1_000_003, -5, 0, 2**31 - 1], np.int32)
    q, k, v = s.rows(2, "f32"), s.rows(2, "f32"), s.rows(2, "f32")
    out = torch.zeros_like(q, dtype=torch.float16)
    before = f64(s.k)
    lbv.rope_append(rope, s.batch, s.cache, q, k, v, out, positions=torch.from_numpy(where).cuda())
    want, size = step.rotate(f64(q), where.astype(np.int64), freqs, False, 1.0)
    # the oracle's own angle carries |position| 2^-53 relative, the kernel's
    # frequency 2^-54 turns per position
    tol = UNIT["f16"] * np.abs(want) + (2.0 ** -20 + 2.0 ** -20) * size + TINY["f16"]
    assert np.all(np.abs(f64(out) - want) <= tol)
    assert np.array_equal(f64(s.k), before, equal_nan=True)
    s.table[0, 2] = [p for p in range(s.cache.pages) if p not in s.table[0, :2]][0]
    s.batch.block_table.copy_(torch.from_numpy(s.table))
    lbv.rope_append(rope, s.batch, s.cache, None, k, v, None)
    assert np.array_equal(f64(s.v)[s.table[0, 2], :4], f64(v.half()))


def test_rope_in_place_equals_out_of_place():
    s = Setup([9, 2], [9, 30], dtype="bf16")
    rope = lbv.Rope(lbv.rope_frequencies(64), lbv.ROPE_HALF)
    q, k, v = s.rows(4), s.rows(2), s.rows(2)
    out = torch.empty_like(q)
    lbv.rope_append(rope, s.batch, s.cache, q, k, v, out)
    lbv.rope_append(rope, s.batch, s.cache, q, k, v, q)
    assert torch.equal(out, q)


# --- attention -----------------------------------------------------------------------

def run_attend(s, q, out=None, scale=None, window=0, tree=None, ws=None):
    scale = s.dim ** -0.5 if scale is None else scale
    out = torch.full((s.tokens, q.shape[1], s.dim), 7.0, device="cuda").to(DT[s.dtype]) if out is None else out
    lse = torch.full((s.tokens, q.shape[1]), 7.0, device="cuda")
    if ws is None:
        ws = torch.zeros(lbv.attend_workspace_bytes(s.cache, s.batch, q.shape[1]), dtype=torch.uint8, device="cuda")
    words = None if tree is None else torch.tensor(np.array(tree, np.uint64).view(np.int64)).cuda()
    lbv.attend(s.cache, s.batch, q, out, scale, window=window, tree=words, lse=lse, workspace=ws)
    lbv.attend_status(ws)
    return out, lse, ws


def check_attend(s, q, out, lse, scale=None, window=0, tree=None):
    scale = s.dim ** -0.5 if scale is None else scale
    n = int(s.start[-1])
    want, ref, A, V, S = step.attend(f64(q)[:n], np.nan_to_num(f64(s.k)), np.nan_to_num(f64(s.v)), s.start,
                                     s.kv_len, s.table, scale, window, tree)
    u = UNIT[s.dtype]
    # scores: an fp32 dot product of dim terms, its scaling and the exponential
    e = (s.dim + 8) * 2.0 ** -24 * S + 2.0 ** -20
    tol = u * np.abs(want) + (u + 2 * e[..., None]) * A + TINY[s.dtype] * (1 + V)
    got = f64(out)
    assert np.all(np.abs(got[:n] - want) <= tol), np.abs(got[:n] - want).max()
    g, none = lse.double().cpu().numpy(), np.isneginf(ref)
    assert np.array_equal(np.isneginf(g[:n]), none)
    assert np.all(got[:n][none] == 0)
    assert np.all(np.abs(g[:n] - ref)[~none] <= (e + 2.0 ** -22 * np.abs(ref))[~none])
    assert np.all(got[n:] == 7.0) and np.all(g[n:] == 7.0)      # rows of no request


LENGTHS = [
    ([1], [1]),                                 # one token, one key
    ([1], [63]), ([1], [64]), ([1], [65]),      # around a block's end
    ([1, 1, 1], [130, 1, 257]),
    ([8], [8]), ([8, 3, 1], [200, 3, 65]),      # drafts, some without a context
    ([0, 5, 0], [40, 77, 0]),                   # requests without new tokens
    ([6, 2], [3, 0]),                           # more new tokens than context: empty rows
    ([70], [70]), ([33, 1], [150, 290]),        # several row tiles
]


@pytest.mark.parametrize("q_len, kv_len", LENGTHS)
@pytest.mark.parametrize("heads, kv_heads, dim, dtype, page, order", [
    (12, 2, 128, "f16", 16, "token"), (7, 1, 64, "bf16", 8, "head"), (2, 2, 128, "bf16", 128, "gap"),
])
def test_attend_lengths(q_len, kv_len, heads, kv_heads, dim, dtype, page, order):
    s = Setup(q_len, kv_len, kv_heads=kv_heads, dim=dim, dtype=dtype, page=page, order=order, pad=1)
    q = s.rows(heads, scale=2.0)
    out, lse, _ = run_attend(s, q)
    check_attend(s, q, out, lse)


@pytest.mark.parametrize("window", [1, 5, 64, 100])
@pytest.mark.parametrize("q_len, kv_len", [([1, 4], [300, 131]), ([50], [90])])
def test_attend_window(window, q_len, kv_len):
    s = Setup(q_len, kv_len, kv_heads=1, dim=64, dtype="bf16", page=32)
    q = s.rows(5, scale=2.0)
    out, lse, _ = run_attend(s, q, window=window)
    check_attend(s, q, out, lse, window=window)
    # pages wholly below every window may be gone
    table = s.batch.block_table.clone()
    for r in range(len(q_len)):
        low = max(0, kv_len[r] - q_len[r] - window + 1)
        s.batch.block_table[r, :low // 32] = -1
    again, _, _ = run_attend(s, q, window=window)
    assert torch.equal(out, again)
    s.batch.block_table.copy_(table)


@pytest.mark.parametrize("window", [0, 6])
@pytest.mark.parametrize("heads, kv_heads, dim, dtype", [(6, 1, 128, "bf16"), (8, 2, 64, "f16")])
def test_attend_tree(heads, kv_heads, dim, dtype, window):
    rng = np.random.default_rng(3)
    s = Setup([8, 1, 70, 5], [75, 1, 70, 5], kv_heads=kv_heads, dim=dim, dtype=dtype, page=16)
    tree = [int(rng.integers(0, 2**63)) for _ in range(s.tokens)]
    tree[0], tree[8], tree[79], tree[80] = 1, 0, 0, 2**64 - 1   # two rows of no context see nothing
    q = s.rows(heads, scale=2.0)
    out, lse, _ = run_attend(s, q, tree=tree, window=window)
    check_attend(s, q, out, lse, tree=tree, window=window)
    assert np.isneginf(lse[8].cpu().numpy()).all()


@pytest.mark.parametrize("layout", ["fused", "odd", "heads"])
@pytest.mark.parametrize("q_len, kv_len", [([3, 1], [80, 17]), ([140], [150])])
def test_attend_strides(layout, q_len, kv_len):
    s = Setup(q_len, kv_len, kv_heads=2, dtype="f16", order="head", page=16)
    q = s.rows(8)
    plain, lse, _ = run_attend(s, q)
    out = lay_out(torch.full_like(q, 7.0), layout)
    strided, lse2, _ = run_attend(s, lay_out(q, layout), out)
    assert torch.equal(plain, strided) and torch.equal(lse, lse2)
    check_attend(s, q, plain, lse)


@pytest.mark.parametrize("scale", [0.0, -0.3, 4.0])
def test_attend_scale(scale):
    """Flat scores, a negative scale, and scores of a hundred: one key wins."""
    s = Setup([2], [190], kv_heads=1, dim=128, dtype="bf16")
    q = s.rows(3, scale=3.0)
    out, lse, _ = run_attend(s, q, scale=scale)
    check_attend(s, q, out, lse, scale=scale)


@pytest.mark.parametrize("dim, dtype, window, scale, wide", [
    (128, "bf16", 0, None, True), (128, "f16", 100, -0.05, True), (64, "bf16", 0, None, False),
])
def test_attend_many_items(dim, dtype, window, scale, wide):
    """More row tiles than SMs, of one to two hundred rows and more: every CTA goes
    from item to item of different kinds."""
    g = np.random.default_rng(dim)
    q_len = [int(n) for n in g.choice([1, 2, 40, 63, 64, 65, 127, 128, 129, 150], 48)]
    kv_len = [n + int(g.integers(0, 300)) for n in q_len]
    s = Setup(q_len, kv_len, kv_heads=8, dim=dim, dtype=dtype, page=16)
    q = s.rows(16, scale=2.0)
    if not wide:                                        # rows at odd strides
        room = torch.empty((q.shape[0], 16, dim + 1), dtype=q.dtype, device="cuda")
        room[..., :dim] = q
        q = room[..., :dim]
    out, lse, _ = run_attend(s, q, scale=scale, window=window)
    check_attend(s, q, out, lse, scale=scale, window=window)


def test_attend_growing_maximum():
    """Scores that rise along the context, so that the reference keeps moving."""
    s = Setup([1], [400], kv_heads=1, dim=64, dtype="f16", page=16)
    flat = s.k.view(-1, 64)
    for j in range(400):
        flat[int(s.table[0, j // 16]) * 16 + j % 16] = j / 40.0
    q = torch.ones((1, 2, 64), device="cuda", dtype=torch.float16)
    q[0, 1] = -1
    out, lse, _ = run_attend(s, q, scale=0.25)
    check_attend(s, q, out, lse, scale=0.25)


def test_attend_repeats_and_batches_alike():
    """The same call twice gives the same bits, with one workspace, and on a
    stream of its own."""
    s = Setup([4, 1, 2], [900, 64, 333], kv_heads=2, dtype="bf16", page=64)
    q = s.rows(12)
    out, lse, ws = run_attend(s, q)
    again, lse2, _ = run_attend(s, q, ws=ws)
    assert torch.equal(out, again) and torch.equal(lse, lse2)
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        third = torch.empty_like(out)
        lbv.attend(s.cache, s.batch, q, third, s.dim ** -0.5, workspace=ws)
    side.synchronize()
    assert torch.equal(out, third)


def test_attend_long_context():
    """A long context over many pages and CTAs: keys that match the query stand
    at known places, all others are orthogonal to it."""
    n, page = 70001, 64
    pages = -(-n // page)
    k = torch.zeros((pages, page, 1, 64), dtype=torch.float16, device="cuda")
    v = torch.randn((pages, page, 1, 64), device="cuda").half()
    table = torch.randperm(pages, device="cuda").to(torch.int32)[None].contiguous()
    where = [0, 4097, 69999, 70000]
    for j in where:
        k[int(table[0, j // page]), j % page, 0, 0] = 1.0
    q = torch.zeros((1, 4, 64), dtype=torch.float16, device="cuda")
    q[..., 0] = 100.0
    cache = lbv.KVCache(k, v)
    batch = lbv.Batch(torch.tensor([0, 1], dtype=torch.int32, device="cuda"),
                      torch.tensor([n], dtype=torch.int32, device="cuda"), table, 1)
    ws = torch.zeros(lbv.attend_workspace_bytes(cache, batch, 4), dtype=torch.uint8, device="cuda")
    out = torch.empty_like(q)
    lbv.attend(cache, batch, q, out, 1.0, workspace=ws)
    want = sum(v[int(table[0, j // page]), j % page, 0].double() for j in where) / 4
    assert torch.all((out[0].double() - want).abs() <= 2.0 ** -11 * want.abs() + 2.0 ** -20)


def test_offsets_past_32_bits():
    """A cache of more than 2^32 elements: the last pages are written and read."""
    pages, page, heads, dim = 2 ** 32 // (64 * 8 * 128) + 3, 64, 8, 128
    free = torch.cuda.mem_get_info()[0]
    if free < 2 * pages * page * heads * dim * 2 + (4 << 30):
        pytest.skip("not enough device memory")
    k = torch.empty((pages, page, heads, dim), dtype=torch.bfloat16, device="cuda")
    v = torch.empty_like(k)
    cache = lbv.KVCache(k, v)
    i32 = dict(dtype=torch.int32, device="cuda")
    table = torch.tensor([[pages - 1, 0]], **i32)
    batch = lbv.Batch(torch.tensor([0, 65], **i32), torch.tensor([65], **i32), table, 65)
    rows = torch.randn((65, 8, 128), device="cuda")
    q = torch.empty((65, 8, 128), dtype=torch.bfloat16, device="cuda")
    rope = lbv.Rope(np.zeros(64))                       # no rotation: a copy
    lbv.rope_append(rope, batch, cache, rows, rows, rows, q)
    bits = rows.bfloat16()
    assert torch.equal(q, bits) and torch.equal(k[pages - 1], bits[:64]) and torch.equal(v[0, 0], bits[64])
    ws = torch.zeros(lbv.attend_workspace_bytes(cache, batch, 8), dtype=torch.uint8, device="cuda")
    out = torch.empty_like(q)
    lbv.attend(cache, batch, q, out, 0.0, workspace=ws)          # flat: the mean of the values so far
    count = torch.arange(1, 66, device="cuda", dtype=torch.float64)[:, None, None]
    want = bits.double().cumsum(0) / count
    size = bits.double().abs().cumsum(0) / count
    assert torch.all((out.double() - want).abs() <= 2.0 ** -8 * want.abs() + (2.0 ** -8 + 2.0 ** -20) * size)


def test_attend_refusals():
    s = Setup([1], [8])
    q = s.rows(2)
    ws = torch.zeros(lbv.attend_workspace_bytes(s.cache, s.batch, 2), dtype=torch.uint8, device="cuda")

    def call(q=q, out=None, scale=1.0, window=0, tree=None, lse=None, ws=ws):
        lbv.attend(s.cache, s.batch, q, torch.empty_like(q) if out is None else out, scale,
                   window=window, tree=tree, lse=lse, workspace=ws)

    call()
    for kw, status in ((dict(ws=None), lbv.ERR_WORKSPACE), (dict(ws=ws[:-256]), lbv.ERR_WORKSPACE),
                       (dict(ws=ws[1:]), lbv.ERR_WORKSPACE), (dict(window=-1), lbv.ERR_INVALID_ARG),
                       (dict(scale=float("nan")), lbv.ERR_INVALID_ARG),
                       (dict(q=s.rows(3)), lbv.ERR_INVALID_ARG),
                       (dict(q=s.rows(2, "bf16")), lbv.ERR_INVALID_ARG),
                       (dict(out=s.rows(4)), lbv.ERR_INVALID_ARG),
                       (dict(out=q[..., :64]), lbv.ERR_INVALID_ARG),
                       (dict(tree=torch.zeros(1, device="cuda")), lbv.ERR_INVALID_ARG),
                       (dict(lse=torch.zeros(1, device="cuda")), lbv.ERR_INVALID_ARG)):
        with pytest.raises(lbv.LbvError) as e:
            call(**kw)
        assert e.value.status == status, kw
    with pytest.raises(lbv.LbvError):
        lbv.KVCache(s.k, s.v[..., :64])
    with pytest.raises(lbv.LbvError):
        lbv.Batch(s.batch.q_start, s.batch.kv_len.long(), s.batch.block_table, 1)


# --- sampling --------------------------------------------------------------------------

def draw(x, u, last=False, mask=None, **rules):
    m = x.shape[0]
    token = torch.full((m,), -9, dtype=torch.int32, device="cuda")
    prob = torch.full((m,), -9.0, device="cuda")
    args = {k: torch.as_tensor(v, dtype=torch.int32 if k == "top_k" else torch.float32).cuda()
            for k, v in rules.items()}
    lbv.sample(x, torch.as_tensor(u, dtype=torch.float32).cuda(), token, prob=prob, mask=mask,
               temperature_last=last, **args)
    return token.cpu().numpy(), prob.cpu().numpy().astype(np.float64)


def check_sample(x, u, token, prob, last=False, **rules):
    """The token is one that the definition can give for logits and sums
    within fp32 rounding (a weight is off by at most (|z| + 4) 2^-24)."""
    eps = 1e-5
    for i in range(x.shape[0]):
        r = {k: v[i] for k, v in rules.items()}
        t = r.pop("temperature", 1.0)
        sets = [step.sample_sets(x[i], t, last=last, slack=s, **r) for s in (-eps, 0.0, eps)]
        if sets[1][0].size == 0:
            assert token[i] == -1 and prob[i] == 0
            continue
        assert token[i] in sets[2][0]
        ok = False
        for kept, w in sets:
            by = np.argsort(kept)
            kept, w = kept[by], w[by] / w.sum()
            at = np.searchsorted(kept, token[i])
            if at < kept.size and kept[at] == token[i]:
                upto = np.cumsum(w)[at]
                near = abs(prob[i] - w[at]) <= 2 * eps * w[at] + eps * (w[at] < 1e-6)
                ok |= upto - w[at] - eps <= u[i] + 2.0 ** -24 and u[i] <= upto + eps and near
        assert ok, (i, token[i], prob[i])


RULES = {
    "none": {}, "temperature": dict(temperature=[.2, .7, 1., 2., 30., 0.]),
    "top_k": dict(top_k=[1, 2, 7, 50, 0, -3]), "top_p": dict(top_p=[.1, .5, .9, .999, 1., 0.]),
    "min_p": dict(min_p=[.5, .1, .001, 1., 0., 1e-6]),
    "all": dict(temperature=[.5, .8, 1., 1.2, 1.5, 3.], top_k=[3, 20, 100, 500, 1000, 0],
                top_p=[.9, .95, .8, .99, .3, .7], min_p=[.05, .02, 0., .001, 1e-4, .01]),
}


@pytest.mark.parametrize("last", [False, True])
@pytest.mark.parametrize("rule", list(RULES))
@pytest.mark.parametrize("n, dtype", [(1, "f32"), (37, "f32"), (5001, "f16"), (33333, "f32"), (151936, "bf16")])
def test_sample(n, dtype, rule, last):
    g = torch.Generator(device="cuda").manual_seed(n)
    x = (2.5 * torch.randn((6, n), generator=g, device="cuda")).to(DT[dtype])
    u = torch.rand(6, generator=g, device="cuda").cpu().numpy()
    token, prob = draw(x, u, last, **RULES[rule])
    check_sample(f64(x), u, token, prob, last, **RULES[rule])


@pytest.mark.parametrize("last", [False, True])
@pytest.mark.parametrize("grid", [0.0, 2.0 ** -6, 0.5])
def test_sample_many_candidates(grid, last):
    """Rows of which thousands of tokens are kept, without and with many equal logits."""
    rules = dict(temperature=[1., 1., .9, 1.3, 1.2, 2., 1.5, 2.5],
                 top_k=[1500, 3000, 20000, 60000, 0, 0, 0, 5000],
                 top_p=[1., 1., 1., .9, .95, .999, 1., .6],
                 min_p=[0., 0., 1e-3, 0., 0., 1e-4, 1e-5, 0.])
    g = torch.Generator(device="cuda").manual_seed(17)
    x = 2.5 * torch.randn((8, 151936), generator=g, device="cuda")
    if grid:
        x = (x / grid).round() * grid
    for m in (8, 24):                                   # rows to both cluster sizes
        u = torch.rand(m, generator=g, device="cuda").cpu().numpy()
        many = {k: v * (m // 8) for k, v in rules.items()}
        rows = x.repeat(m // 8, 1)
        token, prob = draw(rows, u, last, **many)
        check_sample(f64(rows), u, token, prob, last, **many)


@pytest.mark.parametrize("n", [64, 4000, 40001, 151936])
def test_sample_equal_logits(n):
    """All logits equal: every count is exact, ties go by index."""
    x = torch.full((5, n), -3.25, device="cuda")
    u = np.array([0.0, 0.25, 0.5, 0.75, 1 - 2.0 ** -24], np.float32)
    f = np.floor(u.astype(np.float64) * 2 ** 24).astype(np.int64)
    token, prob = draw(x, u)
    assert np.array_equal(token, f * n // 2 ** 24) and np.allclose(prob, 1 / n, rtol=1e-6)
    k = n // 2 + 1
    token, _ = draw(x, u, top_k=[k] * 5)
    assert np.array_equal(token, f * k // 2 ** 24)
    kept = -(-n // 4)                                   # the first tokens until a quarter is reached
    token, _ = draw(x, u, top_p=[0.25] * 5)
    assert np.array_equal(token, f * kept // 2 ** 24)
    token, prob = draw(x, u, temperature=[0.0] * 5)
    assert np.array_equal(token, [0] * 5) and np.array_equal(prob, [1] * 5)


def test_sample_masks_and_specials():
    n = 3000
    inf, nan = float("inf"), float("nan")
    x = torch.randn((8, n), device="cuda")
    x[0] = -inf                                         # nothing to draw
    x[1] = nan
    x[2] = -inf
    x[2, 1234] = -3.4e38                                # one token, the lowest finite value
    x[3, 77] = inf                                      # infinite logits share all weight
    x[3, 2990] = inf
    x[4, 5] = nan
    x[4, 6] = 50.0
    x[5] = -3.4e38                                      # a row of lowest values
    x[6, 0] = 0.0
    x[7] = 0.0
    x[7, 1] = -0.0
    u = np.array([.5, .5, .99, .6, .3, .5, .0, .0004], np.float32)
    for rules in ({}, dict(top_p=[.9] * 8), dict(top_k=[2] * 8), dict(top_k=[2] * 8, top_p=[.99] * 8)):
        token, prob = draw(x, u, **rules)
        assert token[0] == -1 and token[1] == -1 and prob[0] == 0 and prob[1] == 0
        assert token[2] == 1234 and prob[2] == 1
        assert token[3] == 2990 and prob[3] == .5
        assert token[4] == 6
        if rules.get("top_k") is None:
            assert token[5] == (1500 if not rules else 1350)
            assert token[7] == 1                        # -0 and +0 are equal: by index
        else:
            assert token[5] == 1
    words = torch.zeros((8, 94), dtype=torch.int32, device="cuda")
    words[:, 3] = 1 << 4                                # only token 100 allowed
    words[5] = 0
    token, prob = draw(torch.randn((8, n), device="cuda"), u, mask=words)
    assert np.array_equal(token, [100] * 5 + [-1] + [100] * 2)
    words = torch.full((8, 94), -1, dtype=torch.int32, device="cuda")
    a = draw(x, u, mask=words)
    b = draw(x, u)
    assert np.array_equal(a[0], b[0]) and np.array_equal(a[1], b[1])


@pytest.mark.parametrize("dtype", ["f32", "bf16"])
def test_sample_rows_do_not_depend_on_the_batch(dtype):
    """The cluster's size changes with the number of rows, the tokens do not;
    rows at odd strides and offsets included."""
    n, m = 20011, 40
    g = torch.Generator(device="cuda").manual_seed(5)
    wide = torch.randn((m, n + 5), generator=g, device="cuda").mul_(3).to(DT[dtype])
    x = wide[:, 3:3 + n]
    u = torch.rand(m, generator=g, device="cuda").cpu().numpy()
    rules = dict(temperature=[.7 + .01 * i for i in range(m)], top_p=[.5 + .01 * i for i in range(m)])
    token, prob = draw(x, u, **rules)
    whole = draw(x.contiguous(), u, **rules)
    assert np.array_equal(token, whole[0]) and np.array_equal(prob, whole[1])
    for i in (0, 17, 39):
        one = draw(x[i:i + 1], u[i:i + 1], **{k: v[i:i + 1] for k, v in rules.items()})
        assert one[0][0] == token[i] and one[1][0] == prob[i]
    check_sample(f64(x), u, token, prob, **rules)


def test_sample_largest_row():
    n = 700_001
    x = torch.zeros((1, n), device="cuda")
    x[0, n - 1] = 30.0
    token, prob = draw(x, [.5], top_p=[.9])
    assert token[0] == n - 1
    token, _ = draw(x[:, :-1], [.5])
    assert token[0] == 350_000


def test_sample_frequencies():
    """Drawn shares over evenly spaced u equal the softmax."""
    p = np.array([.1, .2, .05, .4, .25])
    m = 4096
    x = torch.tensor(np.log(p), dtype=torch.float32).cuda().expand(m, 5).contiguous()
    u = (np.arange(m) + .5) / m
    token, _ = draw(x, u.astype(np.float32))
    assert np.all(np.abs(np.bincount(token, minlength=5) / m - p) <= 1 / m)
    assert np.all(np.diff(token) >= 0)
