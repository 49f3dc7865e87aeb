"""GPU tests of the append to 4 bits against the definition in elementary fp32 operations,
each rounded by itself: rotated keys, values and queries bit for bit."""
import numpy as np
import pytest

import few_row_packed_gb300 as lbv
from kv4_setup import DT, Setup4
from oracle import kv4, step
from test_gpu_step import lay_out

torch = pytest.importorskip("torch")
pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def built():
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    lbv.build()


def turned(x, places, freqs, interleaved, factor):
    """Rows x [tokens, heads, dim] in fp32, rotated as lbv.h defines it for a cache of 4 bits."""
    part = np.asarray(freqs) / (2 * np.pi)
    whole = [int((t - np.floor(t)) * 2.0 ** 64) for t in part]                          # 2^-64 turns
    cut = np.array([[(int(p) * f % 2 ** 64) >> 24 for f in whole] for p in places], np.uint64)
    angle = torch.from_numpy(cut.astype(np.float32)).cuda() * float(np.float32(2 * np.pi) * np.float32(2.0 ** -40))
    cos, sin = (torch.cos(angle) * factor)[:, None], (torch.sin(angle) * factor)[:, None]
    half = len(freqs)
    y = x.float().clone()
    one, two = (slice(0, 2 * half, 2), slice(1, 2 * half, 2)) if interleaved else (slice(0, half), slice(half, 2 * half))
    a, b = y[..., one].clone(), y[..., two].clone()
    ac, bs, bc, as_ = a * cos, b * sin, b * cos, a * sin
    y[..., one], y[..., two] = ac - bs, bc + as_
    return y


def held(x, dtype):
    """Codes [..., 64], and scale and bias, of groups of 64 along the last dimension."""
    x = x.unflatten(-1, (-1, 64))
    lo, hi = x.amin(-1), x.amax(-1)
    bias, scale = lo.to(DT[dtype]), ((hi - lo) * float(np.float32(1) / np.float32(15))).to(DT[dtype])
    s = scale.float()
    s = torch.where(s >= 2.0 ** -126, s, torch.zeros_like(s))
    inverse = torch.where(s > 0, torch.ones_like(s) / s, torch.zeros_like(s))
    code = ((x - bias.float()[..., None]) * inverse[..., None]).round().clamp(0, 15)
    return code.cpu().numpy().astype(np.int64), s.cpu().numpy(), bias.float().cpu().numpy()


@pytest.mark.parametrize("interleaved", [False, True])
@pytest.mark.parametrize("src, dtype, dim, rot, layout, page", [
    ("f32", "f16", 128, 128, "plain", 16), ("f32", "bf16", 128, 64, "fused", 8), ("bf16", "bf16", 64, 64, "heads", 64),
    ("f16", "f16", 64, 24, "odd", 32), ("f32", "f16", 128, 8, "odd", 128), ("f16", "bf16", 64, 32, "plain", 16),
])
@pytest.mark.parametrize("factor", [1.0, 1.25])
def test_the_definition_bit_for_bit(src, dtype, dim, rot, layout, page, interleaved, factor):
    q_len, kv_len = [30, 5, 1], [100, 5, 60]
    s = Setup4(q_len, kv_len, dim=dim, dtype=dtype, page=page, seed=rot)
    req, pos = step.positions(s.start, s.kv_len)
    freqs = lbv.rope_frequencies(rot, 10000.0)
    rope = lbv.Rope(freqs, lbv.ROPE_INTERLEAVED if interleaved else lbv.ROPE_HALF, factor)
    places = np.array([int(p) for p in pos], np.int64)
    places[:4] = [0, 1_000_003, -7, 2 ** 31 - 1]
    q, k, v = (lay_out(s.rows(h, src), layout) for h in (6, 2, 2))
    out = torch.zeros((s.tokens, 6, dim), dtype=DT[dtype], device="cuda")
    lbv.rope_append(rope, s.batch, s.cache, q, k, v, out, positions=torch.from_numpy(places.astype(np.int32)).cuda())
    assert torch.equal(out, turned(q, places, freqs, interleaved, factor).to(DT[dtype]))
    data = s.data.cpu().numpy()
    for which, rows in ((0, turned(k, places, freqs, interleaved, factor)), (1, v.float())):
        code, scale, bias = held(rows, dtype)
        for i, (r, p) in enumerate(zip(req, pos)):
            at, slot = int(s.table[r, p // page]), int(p % page)
            for h in range(2):
                for part in range(dim // 64):
                    a, b = kv4.offsets(page, 2, dim, h, slot, which, part)
                    assert np.array_equal(kv4.unpack(data[at, a:a + 32]), code[i, h, part]), (which, i, h, part)
                    pair = torch.from_numpy(data[at, b:b + 4].copy()).view(DT[dtype]).tolist()
                    assert pair == [scale[i, h, part], bias[i, h, part]], (which, i, h, part)


def small(bits):
    if bits == 4:
        data = torch.zeros((4, lbv.kv_cache4_page_bytes(16, 2, 64)), dtype=torch.uint8, device="cuda")
        return lbv.KVCache4(data, 16, 2, 64, torch.float16), [data]
    k, v = (torch.zeros((4, 16, 2, 64), dtype=torch.float16, device="cuda") for _ in "kv")
    return lbv.KVCache(k, v), [k, v]


@pytest.mark.parametrize("bits", [16, 4])
def test_keep_refuses_lengths_that_overlap_an_input(bits):
    cache, _ = small(bits)
    room = torch.zeros(64, dtype=torch.int32, device="cuda")
    start, length, table, kept = room[:3], room[8:10], room[16:24].view(2, 4), room[32:36].view(torch.int64)
    start.copy_(torch.tensor([0, 1, 2]))
    length.copy_(torch.tensor([3, 4]))
    batch = lbv.Batch(start, length, table, 2)
    for bad in (start, start[1:], length, room[7:9], room[9:11], table.view(-1), room[23:25], room[32:34], room[35:37],
                room[31:33]):
        with pytest.raises(lbv.LbvError) as e:
            lbv.kv_keep(batch, cache, kept, bad)
        assert e.value.status == lbv.ERR_INVALID_ARG and "left" in str(e.value)
    for good in (room[3:5], room[6:8], room[10:12], room[24:26], room[36:38]):
        lbv.kv_keep(batch, cache, kept, good)
        assert good.tolist() == [2, 3]


@pytest.mark.parametrize("bits", [16, 4])
def test_copy_refuses_more_pairs_than_pages(bits):
    cache, held_by = small(bits)
    pair = torch.full((5,), -1, dtype=torch.int32, device="cuda")
    with pytest.raises(lbv.LbvError) as e:
        lbv.kv_copy_pages(cache, pair, pair)
    assert e.value.status == lbv.ERR_INVALID_ARG and "count" in str(e.value)
    lbv.kv_copy_pages(cache, pair[:4], pair[:4])            # pairs outside the cache are left out
    assert all(not t.any() for t in held_by)
