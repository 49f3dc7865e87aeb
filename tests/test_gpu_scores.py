"""GPU tests of attention at scores of any size, over caches of 16 and of 4 bits: the largest
visible score has weight 1, also where an fp32 number's last bit is worth thousands."""
import numpy as np
import pytest

import few_row_packed_gb300 as lbv
from kv4_setup import DT, UNIT, Setup4, f64, words16
from oracle import kv4, step
from test_gpu_step import Setup, run_attend

torch = pytest.importorskip("torch")
pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def built():
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    lbv.build()


def constant_keys(s, bits, level):
    """Every element of a slot's key is level[page, slot]."""
    if bits == 16:
        s.k.copy_(torch.from_numpy(level)[..., None, None].expand(s.k.shape))
        return f64(s.v)
    held = s.data.cpu().numpy()
    none = words16(np.zeros(s.pages), s.dtype)
    for slot in range(s.page):
        for h in range(s.heads):
            for part in range(s.dim // 64):
                _, at = kv4.offsets(s.page, s.heads, s.dim, h, slot, 0, part)
                pair = np.stack((none, words16(level[:, slot], s.dtype)), -1)
                held[:, at:at + 4] = pair.astype("<u2").view(np.uint8)
    s.data.copy_(torch.from_numpy(held))
    return s.values()[1]


KINDS = [
    (4, [2, 1], 2),             # few rows over 4 bits: a tile of 8 rows,
    (4, [2, 2], 10),            # of 16,
    (4, [4, 2], 12),            # and of 24
    (4, [20, 3], 12),           # many rows over 4 bits: one tile of 128,
    (4, [40, 30], 10),          # two,
    (16, [20, 3], 12),          # over 16 bits,
    (16, [40, 30], 10),
    (16, [2, 1], 2),            # and few rows there
    (16, [2, 2], 14),
]


@pytest.mark.parametrize("bits, q_len, heads", KINDS)
@pytest.mark.parametrize("dtype", ["f16", "bf16"])
@pytest.mark.parametrize("power", [24, 28, 32, 36])
@pytest.mark.parametrize("sign, scale", [(1, 0.3), (-1, 0.3), (1, -0.7)])
def test_one_score_wins(bits, q_len, heads, dtype, power, sign, scale):
    """Constant keys of (1 + r / 128) 2^a against constant queries of (1 + n / 128) 2^b: a score is 64
    equal products of 16 bits, exact in fp32, and scores that differ do so by 2^-8 of them or
    more: only the keys of the largest count, equally."""
    make, many = Setup if bits == 16 else Setup4, sum(q_len) > 20
    s = make(q_len, [190, 300], kv_heads=2, dim=64, dtype=dtype, page=16, seed=power)
    g = np.random.default_rng(power)
    a, b = (power - 6) // 2, power - 6 - (power - 6) // 2
    pages = s.cache.pages
    level = ((128 + g.integers(0, 128, (pages, 16))) / 128 * 2.0 ** a).astype(np.float32)
    v = constant_keys(s, bits, level)
    query = sign * (128 + g.integers(0, 128, (s.tokens, heads))) / 128 * 2.0 ** b
    q = torch.from_numpy(query)[..., None].expand(-1, -1, 64).to(DT[dtype]).cuda()
    assert np.array_equal(f64(q)[..., 0], query)
    out, lse, _ = run_attend(s, q, scale=scale)
    got, got_lse, toward = f64(out), f64(lse), np.sign(sign * scale)
    req, pos = step.positions(s.start, s.kv_len)
    for t, (r, p) in enumerate(zip(req, pos)):
        at = [(s.table[r, j // 16], j % 16) for j in range(p + 1)]
        best = toward * max(toward * level[x] for x in at)
        rows = np.stack([v[x] for x in at if level[x] == best])              # [keys, kv heads, dim]
        want = np.repeat(rows.mean(0), heads // 2, 0)
        # Few rows: probabilities of 1.  Many: all of 2^r, where r, 1/2 at most, is what was rounded off
        # the reference; in 16 bits they are off by half a step, and the sum that divides adds the
        # unrounded ones where no key has half of it.  Sums and the division in fp32, rounded once.
        tol = (2 if many else 1) * UNIT[dtype] * np.abs(want) + 2.0 ** -16 * np.abs(rows).max()
        assert np.all(np.abs(got[t] - want) <= tol), (t, np.abs(got[t] - want).max())
        # the score, exact, times the scale, log2 e and back: five roundings of 2^-24 at most
        ref = 64 * query[t] * float(best) * float(np.float32(scale)) + np.log(len(rows))
        assert np.all(np.abs(got_lse[t] / ref - 1) <= 2.0 ** -21)


@pytest.mark.parametrize("bits", [16, 4])
@pytest.mark.parametrize("dtype", ["f16", "bf16"])
@pytest.mark.parametrize("heads", [1, 12])
def test_a_maximum_that_grows_by_one_unit(bits, dtype, heads):
    """Scores of 2^27 + 16 and then 2^27 + 32, one unit of fp32's last place more: the first keys'
    weight is 2^-16 of the others'.  (2^27 + 16 and 8 round to 2^27 + 32.)  200 requests over the
    same pages, so that most are not divided."""
    requests, page, dim, count = 200, 64, 128, 300
    g = torch.Generator().manual_seed(3)
    level = torch.where(torch.arange(5 * page) < 256, 4.0, 8.0).view(5, page, 1)
    k = torch.empty((5, page, 1, dim))
    k[..., :64], k[..., 64:] = 2.0 ** 14, level[..., None].expand(-1, -1, -1, 64)
    v = torch.randn((5, page, 1, dim), generator=g)
    if bits == 16:
        k, v = k.to(DT[dtype]).cuda(), v.to(DT[dtype]).cuda()
        cache, held = lbv.KVCache(k, v), f64(v)
    else:
        data = torch.zeros((5, kv4.page_bytes(page, 1, dim)), dtype=torch.uint8, device="cuda")
        cache = lbv.KVCache4(data, page, 1, dim, DT[dtype])
        whole = lbv.Batch(*(torch.tensor(x, dtype=torch.int32, device="cuda") for x in ([0, 320], [320], [[0, 1, 2, 3, 4]])), 320)
        still = lbv.Rope(np.zeros(8), lbv.ROPE_HALF)        # turns by nothing
        lbv.rope_append(still, whole, cache, None, k.view(320, 1, dim).cuda(), v.view(320, 1, dim).cuda(), None)
        back = [torch.empty((320, 1, dim), dtype=DT[dtype], device="cuda") for _ in "kv"]
        lbv.kv_read(whole, cache, *back)
        assert torch.equal(back[0].float().cpu(), k.view(320, 1, dim))
        held = f64(back[1])
    table = torch.arange(5, dtype=torch.int32).expand(requests, 5).contiguous().cuda()
    batch = lbv.Batch(torch.arange(requests + 1, dtype=torch.int32, device="cuda"),
                      torch.full((requests,), count, dtype=torch.int32, device="cuda"), table, requests)
    q = torch.zeros((requests, heads, dim), dtype=DT[dtype], device="cuda")
    q[..., 0], q[..., 64] = 2.0 ** 13, 4.0
    out = torch.empty_like(q)
    lse = torch.empty((requests, heads), device="cuda")
    ws = torch.zeros(lbv.attend_workspace_bytes(cache, batch, heads), dtype=torch.uint8, device="cuda")
    scale = float(np.float32(0.6931472))                    # times log2 e, in fp32: 1
    assert np.float32(scale) * np.float32(1.44269504088896341) == 1
    lbv.attend(cache, batch, q, out, scale, lse=lse, workspace=ws)
    lbv.attend_status(ws)
    p = 2.0 ** np.where(np.arange(count) < 256, -16.0, 0.0)
    rows = held.reshape(-1, dim)[:count]
    want, size = p @ rows / p.sum(), p @ np.abs(rows) / p.sum()
    # the probabilities are powers of two; sums and the division in fp32, rounded once
    assert np.all(np.abs(f64(out) - want) <= UNIT[dtype] * np.abs(want) + 2.0 ** -15 * size)
    assert np.all(np.abs(f64(lse) / ((2.0 ** 27 + 32 + np.log2(p.sum())) * np.log(2)) - 1) <= 2.0 ** -21)
