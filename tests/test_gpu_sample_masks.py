"""GPU tests of the sampler where a mask leaves few tokens: fewer than top-k
keeps, fewer than a CTA's slices, one, none."""
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


@pytest.mark.parametrize("last", [False, True])
@pytest.mark.parametrize("dtype", ["f32", "bf16"])
@pytest.mark.parametrize("rules", [
    dict(top_k=50), dict(top_k=50, top_p=0.8), dict(top_p=0.8), dict(top_k=50, min_p=0.02), {},
    dict(top_k=3, top_p=0.9), dict(top_k=1),
], ids=str)
def test_few_allowed_tokens(rules, dtype, last):
    m, n = 10, 40009
    g = torch.Generator(device="cuda").manual_seed(4)
    x = (2.5 * torch.randn((m, n), generator=g, device="cuda")).to(DT[dtype])
    allowed = torch.zeros((m, -(-n // 32) * 32), dtype=torch.bool, device="cuda")
    for i, count in enumerate((0, 1, 2, 3, 7, 12, 49, 50, 51, 300)):
        allowed[i, torch.randperm(n, generator=g, device="cuda")[:count]] = True
    bits = allowed.view(m, -1, 32).long() << torch.arange(32, device="cuda")
    words = bits.sum(-1).to(torch.int32)                # the low 32 bits
    hidden = x.masked_fill(~allowed[:, :n], float("-inf"))
    u = torch.rand(m, generator=g, device="cuda").cpu().numpy()
    many = {"temperature": [1.3] * m, **{k: [v] * m for k, v in rules.items()}}
    for rows in (10, 5):                                # both cluster sizes
        token, prob = draw(x[:rows], u[:rows], last, mask=words[:rows],
                           **{k: v[:rows] for k, v in many.items()})
        assert token[0] == -1 and prob[0] == 0 and np.all(token[1:] >= 0)
        check_sample(f64(hidden)[:rows], u[:rows], token, prob, last,
                     **{k: v[:rows] for k, v in many.items()})
        assert all(bool(allowed[i, int(t)]) for i, t in enumerate(token) if t >= 0)
        same = draw(hidden[:rows], u[:rows], last, **{k: v[:rows] for k, v in many.items()})
        assert np.array_equal(token, same[0]) and np.array_equal(prob, same[1])
