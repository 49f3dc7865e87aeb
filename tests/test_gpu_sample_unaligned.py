"""GPU tests of the sampler on rows that begin off a 16-byte boundary (odd
vocabularies, odd strides, views): rules that keep thousands of tokens at high
temperatures, where the tokens that the rules drop would weigh as much as those
they keep."""
import numpy as np
import pytest

import few_row_packed_gb300 as lbv
from test_gpu_step import DT, check_sample, draw, f64

torch = pytest.importorskip("torch")
pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def built():
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    lbv.build()


RULES = {
    "top_k": dict(top_k=5000),
    "top_k and top_p": dict(top_k=9000, top_p=0.7),
    "top_p": dict(top_p=0.9),
    "top_k and min_p": dict(top_k=6000, min_p=0.05),
    "none": {},
}


def off_boundary(x, dtype, shift):
    """The values of x in rows of an odd stride, `shift` elements off a boundary."""
    m, n = x.shape
    ld = n + 8 - (n + 8) % 2 + 1
    flat = torch.zeros(m * ld + 16, dtype=DT[dtype], device="cuda")
    view = flat[shift:].as_strided((m, n), (ld, 1))
    view.copy_(x)
    return view


def aligned(x):
    """The values of x in rows that all begin on a 16-byte boundary."""
    room = torch.zeros((x.shape[0], -(-x.shape[1] // 8) * 8), dtype=x.dtype, device="cuda")
    room[:, :x.shape[1]] = x
    return room[:, :x.shape[1]]


@pytest.mark.parametrize("rule", list(RULES))
@pytest.mark.parametrize("dtype, shift", [("f32", 1), ("f32", 3), ("f16", 1), ("f16", 7), ("bf16", 5)])
@pytest.mark.parametrize("temperature, last", [(3.0, False), (8.0, False), (8.0, True)])
def test_unaligned_rows_draw_as_aligned_ones(rule, dtype, shift, temperature, last):
    m, n = 40, 20011
    g = torch.Generator(device="cuda").manual_seed(shift)
    x = off_boundary((2.5 * torch.randn((m, n), generator=g, device="cuda")).to(DT[dtype]), dtype, shift)
    assert any(x[i].data_ptr() % 16 for i in range(m))
    u = (torch.arange(m, device="cuda") + torch.rand(m, generator=g, device="cuda")).div(m).cpu().numpy()
    rules = {"temperature": [temperature] * m, **{k: [v] * m for k, v in RULES[rule].items()}}
    want = draw(aligned(x), u, last, **rules)
    check_sample(f64(x), u, *want, last=last, **rules)
    for rows in (40, 8, 1):                             # both cluster sizes
        for first in range(0, m, max(rows, 8)):
            part = slice(first, first + rows)
            token, prob = draw(x[part], u[part], last, **{k: v[part] for k, v in rules.items()})
            assert np.array_equal(token, want[0][part]) and np.array_equal(prob, want[1][part])


@pytest.mark.parametrize("n", [50257, 4099, 33])
def test_odd_vocabulary(n):
    """Contiguous rows of an odd vocabulary: every alignment, and the tokens over
    evenly spaced u."""
    m = 64
    g = torch.Generator(device="cuda").manual_seed(n)
    x = (2.5 * torch.randn((1, n), generator=g, device="cuda")).expand(m, n).contiguous()
    u = ((np.arange(m) + .5) / m).astype(np.float32)
    k = max(2, n // 3)
    rules = dict(temperature=[5.0] * m, top_k=[k] * m)
    token, prob = draw(x, u, **rules)
    check_sample(f64(x), u, token, prob, **rules)
    assert np.all(np.diff(token) >= 0)                  # one row, so ascending in u
    again = draw(aligned(x), u, **rules)
    assert np.array_equal(token, again[0]) and np.array_equal(prob, again[1])
