"""GPU tests of the paged cache held in 4 bits: the append that rounds to it, the
tokens read back, and attention over it, against fp64 oracles."""
import numpy as np
import pytest

import few_row_packed_gb300 as lbv
from kv4_setup import DT, TINY, UNIT, Setup4, f64, round16, values, words16
from oracle import kv4, step
from test_gpu_step import LENGTHS, check_attend, lay_out, run_attend

torch = pytest.importorskip("torch")
pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def built():
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    lbv.build()


# --- read ------------------------------------------------------------------------------

@pytest.mark.parametrize("layout", ["plain", "fused", "odd", "heads"])
@pytest.mark.parametrize("dim, dtype, page", [(128, "f16", 8), (64, "bf16", 16), (128, "bf16", 256)])
def test_read(dim, dtype, page, layout):
    """Every code, scale and bias of the new tokens, at any strides; rows of no request stay."""
    s = Setup4([3, 0, 40], [70, 5, 41], dim=dim, dtype=dtype, page=page, pad=2)
    k, v = (lay_out(torch.full((s.tokens, 2, dim), 7.0).to(DT[dtype]).cuda(), layout) for _ in "kv")
    lbv.kv_read(s.batch, s.cache, k, v)
    want = s.values()
    req, pos = step.positions(s.start, s.kv_len)
    for got, held in ((k, want[0]), (v, want[1])):
        rows = np.stack([held[s.table[r, p // page], p % page] for r, p in zip(req, pos)])
        assert np.array_equal(f64(got)[:len(req)], rows)
        assert np.all(f64(got)[len(req):] == 7.0)
    only = torch.zeros_like(v)
    lbv.kv_read(s.batch, s.cache, None, only)
    assert torch.equal(only[:len(req)], v[:len(req)])


@pytest.mark.parametrize("order", ["token", "head", "gap"])
def test_read_of_16_bits(order):
    from test_gpu_step import Setup
    s = Setup([3, 9], [40, 9], dim=64, dtype="bf16", page=8, order=order, pad=1)
    s.table[0, 4] = 99                                  # slots 32..39: outside the cache
    s.batch.block_table.copy_(torch.from_numpy(s.table))
    k, v = (torch.full((s.tokens, 2, 64), 7.0, dtype=torch.bfloat16, device="cuda") for _ in "kv")
    lbv.kv_read(s.batch, s.cache, k, v)
    for got, held in ((k, s.k), (v, s.v)):
        assert torch.all(got[:3] == 0) and torch.all(got[12:] == 7.0)
        for i in range(9):
            assert torch.equal(got[3 + i], held[int(s.table[1, i // 8]), i % 8])


# --- append ----------------------------------------------------------------------------

@pytest.mark.parametrize("src, dtype, dim, rot, interleaved, layout, page", [
    ("f32", "f16", 128, 128, False, "plain", 16),
    ("f32", "bf16", 128, 64, True, "fused", 8),
    ("bf16", "bf16", 64, 64, True, "heads", 64),
    ("f16", "f16", 64, 32, False, "odd", 32),
    ("f32", "f16", 128, 8, False, "odd", 1024),     # partners four elements apart
    ("f16", "bf16", 128, 128, False, "fused", 128),
    ("f32", "bf16", 64, 24, False, "plain", 16),
])
@pytest.mark.parametrize("q_len, kv_len", [([1], [1]), ([3, 0, 8, 1], [3, 5, 70, 33]), ([5, 40], [2, 41])])
def test_append(src, dtype, dim, rot, interleaved, layout, page, q_len, kv_len):
    s = Setup4(q_len, kv_len, dim=dim, dtype=dtype, page=page, pad=2)
    freqs, factor = lbv.rope_frequencies(rot, 500.0), 1.25
    rope = lbv.Rope(freqs, lbv.ROPE_INTERLEAVED if interleaved else lbv.ROPE_HALF, factor)
    q, k, v = (lay_out(s.rows(h, src), layout) for h in (7, 2, 2))
    out = lay_out(torch.full((s.tokens, 7, dim), 7.0, device="cuda").to(DT[dtype]), layout)
    before = s.data.cpu().numpy()
    lbv.rope_append(rope, s.batch, s.cache, q, k, v, out)
    after = s.data.cpu().numpy()
    held = values(after, page, 2, dim, dtype)
    req, pos = step.positions(s.start, s.kv_len)
    n, u = len(req), UNIT[dtype]
    want, size = step.rotate(f64(q)[:n], pos, freqs, interleaved, factor)
    # one rounding; fp32 sums of two products; the angle to 2^-24 half turns
    assert np.all(np.abs(f64(out)[:n] - want) <= u * np.abs(want) + 2.0 ** -20 * factor * size + TINY[dtype])
    assert np.all(f64(out)[n:] == 7.0)
    keys, size = step.rotate(f64(k)[:n], pos, freqs, interleaved, factor)
    slots = np.zeros((s.pages, before.shape[1]), bool)
    for i in range(n):
        if pos[i] < 0:
            continue
        at, slot = int(s.table[req[i], pos[i] // page]), int(pos[i] % page)
        for h in range(2):
            for which, x, e in ((0, keys[i, h], 2.0 ** -20 * factor * size[i, h]), (1, f64(v)[i, h], np.zeros(dim))):
                for part in range(dim // 64):
                    a, b = kv4.offsets(page, 2, dim, h, slot, which, part)
                    slots[at, a:a + 32] = slots[at, b:b + 4] = True
                    g = slice(part * 64, (part + 1) * 64)
                    scale, bias = torch.from_numpy(after[at, b:b + 4].copy()).view(DT[dtype]).double().tolist()
                    lo, hi, err = x[g].min(), x[g].max(), e[g].max()
                    assert abs(bias - lo) <= u * abs(lo) + 2 * err + TINY[dtype]
                    assert abs(scale - (hi - lo) / 15) <= (u + 2.0 ** -22) * (hi - lo) / 15 + err + TINY[dtype]
                    # Half a step from the nearest code (the reciprocal, the difference and the product are
                    # fp32 of numbers below 16 steps).  Below bias it is code 0, off by the rounding of bias;
                    # above the last code by the roundings of bias and of 15 scales (15 u < 1/2).
                    got = held[which, at, slot, h, g]
                    tol = scale * (.5 + 2.0 ** -18) + u * (abs(lo) + np.abs(got)) + 3 * err + 17 * TINY[dtype]
                    assert np.all(np.abs(got - x[g]) <= tol)
                    if which == 1:                      # not rotated: the same codes
                        codes, s32, b32 = kv4.quantise(x[g].astype(np.float32), lambda t: round16(t, dtype))
                        assert (scale, bias) == (float(s32), float(b32))
                        assert np.array_equal(kv4.unpack(after[at, a:a + 32]), codes)
    assert np.array_equal(after[~slots], before[~slots])            # nothing else moved


def group_values(kind, dtype, g):
    x = g.standard_normal(64)
    return {"flat": np.full(64, 3.0), "zero": np.zeros(64), "low": x * 1e-30, "tiny": x * 1e-7,
            "far": 100 + x * 1e-3, "one": np.where(np.arange(64) == 9, 1000.0, 0.0),
            "largest": np.where(np.arange(64) % 2, 32768.0, -32768.0),
            "nan": np.where(np.arange(64) == 63, np.nan, x), "inf": np.where(np.arange(64) == 5, -np.inf, x),
            "beyond": np.where(np.arange(64) == 5, 32769.0 if dtype == "f16" else 2.0 ** 126 * 1.01, x),
            "bound": np.where(np.arange(64) == 5, 32768.0 if dtype == "f16" else 2.0 ** 126, x)}[kind]


@pytest.mark.parametrize("dtype", ["f16", "bf16"])
@pytest.mark.parametrize("kind", ["flat", "zero", "low", "tiny", "far", "one", "largest", "nan", "inf", "beyond",
                                  "bound"])
def test_append_of_odd_groups(kind, dtype):
    """Groups without a range, of subnormals, far from 0, at the bounds, and past them; their
    neighbours in the head and in the warp are as ever."""
    s = Setup4([3], [5], kv_heads=2, dim=128, dtype=dtype, page=8)
    rope = lbv.Rope(np.zeros(8), lbv.ROPE_HALF)         # turns by nothing
    k, v = s.rows(2, "f32"), s.rows(2, "f32")
    x = group_values(kind, dtype, np.random.default_rng(5)).astype(np.float32)
    v[1, 1, :64] = torch.from_numpy(x).cuda()
    lbv.rope_append(rope, s.batch, s.cache, None, k, v, None)
    after = s.data.cpu().numpy()
    back_k, back_v = (torch.zeros((3, 2, 128), dtype=DT[dtype], device="cuda") for _ in "kv")
    lbv.kv_read(s.batch, s.cache, back_k, back_v)
    for i in range(3):
        at, slot = int(s.table[0, (2 + i) // 8]), (2 + i) % 8
        for h in range(2):
            for which, src in ((0, k), (1, v)):
                for part in range(2):
                    a, b = kv4.offsets(8, 2, 128, h, slot, which, part)
                    g = src[i, h, part * 64:(part + 1) * 64].cpu().numpy()
                    read = (back_v if which else back_k)[i, h, part * 64:(part + 1) * 64]
                    if which and (i, h, part) == (1, 1, 0) and kind in ("nan", "inf", "beyond"):
                        assert torch.isnan(read).all()
                        continue
                    codes, scale, bias = kv4.quantise(g, lambda t: round16(t, dtype))
                    assert torch.from_numpy(after[at, b:b + 4].copy()).view(DT[dtype]).tolist() == [scale, bias]
                    assert np.array_equal(kv4.unpack(after[at, a:a + 32]), codes)
                    assert torch.isfinite(read).all()
                    assert np.array_equal(f64(read), round16(codes * float(scale) + float(bias), dtype))


def test_append_in_place_equals_out_of_place():
    """q_out is q itself, with heads enough for several pieces a thread."""
    s = Setup4([9, 2, 300], [9, 30, 300], dtype="bf16")
    rope = lbv.Rope(lbv.rope_frequencies(128), lbv.ROPE_HALF)
    q, k, v = s.rows(70), s.rows(2), s.rows(2)
    out = torch.empty_like(q)
    lbv.rope_append(rope, s.batch, s.cache, q, k, v, out)
    held = s.data.clone()
    lbv.rope_append(rope, s.batch, s.cache, q, k, v, q)
    assert torch.equal(out, q) and torch.equal(held, s.data)


def test_append_leaves_missing_slots():
    s = Setup4([4], [20], page=8)
    s.table[0, 2] = 99                                   # slots 16..19: outside the cache
    s.batch.block_table.copy_(torch.from_numpy(s.table))
    rope = lbv.Rope(lbv.rope_frequencies(128))
    before = s.data.clone()
    q, k, v = s.rows(2, "f32"), s.rows(2, "f32"), s.rows(2, "f32")
    out = torch.zeros_like(q, dtype=torch.float16)
    where = torch.tensor([7, -5, 0, 2**31 - 1], dtype=torch.int32, device="cuda")
    lbv.rope_append(rope, s.batch, s.cache, q, k, v, out, positions=where)
    assert torch.equal(before, s.data)
    want, size = step.rotate(f64(q), where.cpu().numpy().astype(np.int64), lbv.rope_frequencies(128), False, 1.0)
    assert np.all(np.abs(f64(out) - want) <= UNIT["f16"] * np.abs(want) + 2.0 ** -19 * size + TINY["f16"])


# --- attention -------------------------------------------------------------------------

class Held:
    """What the checks of the 16-bit cache look at, for one of 4 bits."""

    def __init__(self, s):
        v = s.values()
        self.k, self.v = (torch.from_numpy(x) for x in v)
        self.start, self.kv_len, self.table, self.dtype, self.dim = s.start, s.kv_len, s.table, s.dtype, s.dim


@pytest.mark.parametrize("q_len, kv_len", LENGTHS)
@pytest.mark.parametrize("heads, kv_heads, dim, dtype, page", [
    (12, 2, 128, "f16", 16), (7, 1, 64, "bf16", 8), (2, 2, 128, "bf16", 128), (4, 4, 64, "f16", 64),
])
def test_attend_lengths(q_len, kv_len, heads, kv_heads, dim, dtype, page):
    s = Setup4(q_len, kv_len, kv_heads=kv_heads, dim=dim, dtype=dtype, page=page, pad=1)
    q = s.rows(heads, scale=2.0)
    out, lse, _ = run_attend(s, q)
    check_attend(Held(s), q, out, lse)


@pytest.mark.parametrize("window", [1, 5, 64, 100])
@pytest.mark.parametrize("q_len, kv_len", [([1, 4], [300, 131]), ([50], [90])])
def test_attend_window(window, q_len, kv_len):
    s = Setup4(q_len, kv_len, kv_heads=1, dim=64, dtype="bf16", page=32)
    q = s.rows(5, scale=2.0)
    out, lse, _ = run_attend(s, q, window=window)
    check_attend(Held(s), q, out, lse, window=window)
    for r in range(len(q_len)):                         # pages wholly below every window may be gone
        low = max(0, kv_len[r] - q_len[r] - window + 1)
        s.batch.block_table[r, :low // 32] = -1
    again, _, _ = run_attend(s, q, window=window)
    assert torch.equal(out, again)


@pytest.mark.parametrize("window", [0, 6])
@pytest.mark.parametrize("heads, kv_heads, dim, dtype", [(6, 1, 128, "bf16"), (8, 2, 64, "f16"), (2, 1, 128, "f16")])
def test_attend_tree(heads, kv_heads, dim, dtype, window):
    rng = np.random.default_rng(3)
    s = Setup4([8, 1, 70, 5], [75, 1, 70, 5], kv_heads=kv_heads, dim=dim, dtype=dtype, page=16)
    tree = [int(rng.integers(0, 2**63)) for _ in range(s.tokens)]
    tree[0], tree[8], tree[79], tree[80] = 1, 0, 0, 2**64 - 1
    q = s.rows(heads, scale=2.0)
    out, lse, _ = run_attend(s, q, tree=tree, window=window)
    check_attend(Held(s), q, out, lse, tree=tree, window=window)
    assert np.isneginf(lse[8].cpu().numpy()).all()


@pytest.mark.parametrize("layout", ["fused", "odd", "heads"])
@pytest.mark.parametrize("q_len, kv_len", [([3, 1], [80, 17]), ([1, 1], [80, 17]), ([140], [150])])
def test_attend_strides(layout, q_len, kv_len):
    s = Setup4(q_len, kv_len, kv_heads=2, dtype="f16", page=16)
    q = s.rows(8)
    plain, lse, _ = run_attend(s, q)
    out = lay_out(torch.full_like(q, 7.0), layout)
    strided, lse2, _ = run_attend(s, lay_out(q, layout), out)
    assert torch.equal(plain, strided) and torch.equal(lse, lse2)
    check_attend(Held(s), q, plain, lse)


@pytest.mark.parametrize("scale", [0.0, -0.3, 4.0])
@pytest.mark.parametrize("heads", [3, 12])
def test_attend_scale(scale, heads):
    """Flat scores, a negative scale, and scores of a hundred: one key wins."""
    s = Setup4([2], [190], kv_heads=1, dim=128, dtype="bf16")
    q = s.rows(heads, scale=3.0)
    out, lse, _ = run_attend(s, q, scale=scale)
    check_attend(Held(s), q, out, lse, scale=scale)


@pytest.mark.parametrize("q_len, heads", [([2, 1], 2), ([4, 2], 12), ([40, 3], 12)])
def test_attend_scores_of_any_size(q_len, heads):
    """Constant keys of -2^(70 + e) against queries of 2^32 (64 exact products): every score is
    below -10^30, and only the keys of the smallest visible e count, equally."""
    s = Setup4(q_len, [190, 70], kv_heads=2, dim=64, dtype="bf16", page=16, seed=5)
    held = s.data.view(torch.uint8).cpu().numpy()
    e = np.random.default_rng(1).integers(0, 8, (s.pages, 16))
    for slot in range(16):
        for h in range(2):
            _, at = kv4.offsets(16, 2, 64, h, slot, 0, 0)
            pair = np.stack((words16(np.zeros(s.pages), "bf16"), words16(-2.0 ** (70 + e[:, slot]), "bf16")), -1)
            held[:, at:at + 4] = pair.astype("<u2").view(np.uint8)
    s.data.copy_(torch.from_numpy(held))
    q = torch.full((s.tokens, heads, 64), 2.0 ** 32, dtype=torch.bfloat16, device="cuda")
    out, lse, _ = run_attend(s, q, scale=1.0)
    v = s.values()[1]
    req, pos = step.positions(s.start, s.kv_len)
    for t, (r, p) in enumerate(zip(req, pos)):
        at = [(s.table[r, j // 16], j % 16) for j in range(p + 1)]
        low = min(e[x] for x in at)
        rows = np.stack([v[x] for x in at if e[x] == low])                    # [keys, kv heads, dim]
        want = np.repeat(rows.mean(0), heads // 2, 0)
        # probabilities of 1; sums and the division in fp32, rounded once
        tol = UNIT["bf16"] * np.abs(want) + 2.0 ** -16 * np.abs(rows).max()
        assert np.all(np.abs(f64(out)[t] - want) <= tol)
        # the score, exact, times log2 e and back: three roundings of 2^-24 and two constants'
        assert np.all(np.abs(f64(lse)[t] / -2.0 ** (108 + low) - 1) <= 2.0 ** -21)


@pytest.mark.parametrize("dim, dtype, window, scale, heads", [
    (128, "bf16", 0, None, 16), (128, "f16", 100, -0.05, 16), (64, "bf16", 0, None, 16), (128, "f16", 0, None, 8),
])
def test_attend_many_items(dim, dtype, window, scale, heads):
    """More row tiles than SMs: every CTA goes from item to item of different kinds."""
    g = np.random.default_rng(dim)
    few = heads == 8                                    # one query head a group, few new tokens: few rows
    q_len = [int(n) for n in g.choice([1, 1, 2, 3, 8, 9] if few else [1, 2, 40, 63, 64, 65, 127, 128, 129, 150], 48)]
    kv_len = [n + int(g.integers(0, 300)) for n in q_len]
    s = Setup4(q_len, kv_len, kv_heads=8, dim=dim, dtype=dtype, page=16)
    q = s.rows(heads, scale=2.0)
    out, lse, _ = run_attend(s, q, scale=scale, window=window)
    check_attend(Held(s), q, out, lse, scale=scale, window=window)


@pytest.mark.parametrize("q_len, heads", [([4, 1, 2], 12), ([1, 1, 1], 4)])
def test_attend_repeats_and_batches_alike(q_len, heads):
    s = Setup4(q_len, [900, 64, 333], kv_heads=2, dtype="bf16", page=64)
    q = s.rows(heads)
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


@pytest.mark.parametrize("q_len, heads", [([1], 12), ([2], 2)])
def test_attend_pages_outside_the_cache(q_len, heads):
    """A mapped page that does not exist reads as zeros, a missing one below the context too."""
    s = Setup4(q_len, [150], kv_heads=2, page=16)
    s.table[0, 3], s.table[0, 5] = 10 ** 6, -1
    s.batch.block_table.copy_(torch.from_numpy(s.table))
    q = s.rows(heads)
    out, lse, _ = run_attend(s, q)
    check_attend(Held(s), q, out, lse)


@pytest.mark.parametrize("copies", [0, 1, 4])
@pytest.mark.parametrize("q_len, kv_len, heads", [([40, 150, 3] * 20, [400, 420, 90] * 20, 16), ([16], [30011], 48),
                                                  ([1] * 200, [900] * 200, 8), ([1], [100001], 8)])
def test_waits_that_run_out(q_len, kv_len, heads, copies):
    """The first CTA stops filling its ring: the call ends, reports it once, and the next is exact."""
    g = torch.Generator(device="cuda").manual_seed(1)
    page, hk, dim = 64, 8, 128
    need = [-(-k // page) for k in kv_len]
    data = torch.randint(0, 256, (sum(need), kv4.page_bytes(page, hk, dim)), generator=g, device="cuda",
                         dtype=torch.uint8)
    scales = data.view(torch.float16).view(sum(need), hk, -1)[..., 64 * 64:]
    scales.copy_(torch.randn(scales.shape, generator=g, device="cuda") * 0.1)
    table = torch.full((len(q_len), max(need)), -1, dtype=torch.int32)
    at = 0
    for r, n in enumerate(need):
        table[r, :n] = torch.arange(at, at + n, dtype=torch.int32)
        at += n
    start = torch.tensor(np.concatenate([[0], np.cumsum(q_len)]), dtype=torch.int32, device="cuda")
    cache = lbv.KVCache4(data, page, hk, dim, torch.float16)
    batch = lbv.Batch(start, torch.tensor(kv_len, dtype=torch.int32, device="cuda"), table.cuda(), sum(q_len))
    q = torch.randn((sum(q_len), heads, dim), generator=g, device="cuda").half()
    ws = torch.zeros(lbv.attend_workspace_bytes(cache, batch, heads), dtype=torch.uint8, device="cuda")
    want, out = torch.empty_like(q), torch.full_like(q, 7.0)
    lbv.attend(cache, batch, q, want, 0.1, workspace=ws)
    lbv.attend_status(ws)
    lbv.attend_test_wait(cache, batch, q, out, 0.1, ws, copies)
    with pytest.raises(lbv.LbvError) as e:
        lbv.attend_status(ws)
    assert e.value.status == lbv.ERR_TIMEOUT
    lbv.attend_status(ws)
    assert torch.equal(out[-1, -1], want[-1, -1])       # the last item is not the first CTA's
    lbv.attend(cache, batch, q, out, 0.1, workspace=ws)
    assert torch.equal(out, want)
