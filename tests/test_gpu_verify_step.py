"""GPU test of the verify step as a whole (examples/verify_step.py): drafted rows
that go through it together give what the same tokens give one by one."""
import importlib.util
import os

import pytest

import few_row_packed_gb300 as lbv

torch = pytest.importorskip("torch")
pytestmark = pytest.mark.gpu
PATH = os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))), "examples",
                    "verify_step.py")


@pytest.fixture(scope="module")
def example():
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    lbv.build()
    spec = importlib.util.spec_from_file_location("verify_step", PATH)
    m = importlib.util.module_from_spec(spec)
    spec.loader.exec_module(m)
    return m


def test_rows_together_equal_rows_one_by_one(example):
    tokens = [(37 * i * i + 11) % 2000 for i in range(45)]
    one, many = example.Layer(), example.Layer()
    single = torch.cat([one.logits([t], i) for i, t in enumerate(tokens)])
    chunks, at = [], 0
    for n in (1, 8, 3, 8, 2, 8, 7, 8):
        chunks.append(many.logits(tokens[at:at + n], at))
        at += n
    together = torch.cat(chunks)
    assert at == len(tokens)
    # the cache holds the same rows but for the one-row and few-row kernels'
    # different sums (fp32, then one rounding to fp16): a unit in the last place
    for a, b in ((one.cache.k, many.cache.k), (one.cache.v, many.cache.v)):
        assert torch.all((a - b).abs() <= 2.0 ** -10 * a.abs() + 2.0 ** -14)
    # logits: an activation may differ by a unit in the last place (2^-10) at each of
    # the two fp16 roundings, over 512 of them of size 1 with weights of 0.02
    err, size = (single - together).abs().max(), single.abs().max()
    assert err <= 2 * 2.0 ** -10 * 512 ** 0.5 * size, (err, size)
    assert float((single.argmax(-1) == together.argmax(-1)).float().mean()) > 0.9
    lbv.attend_status(many.workspace)


def test_verify_settles_what_single_steps_sample(example):
    """With peaked rules the accepted tokens are those that sampling one token
    at a time gives, whatever was drafted."""
    layer = example.Layer(seed=3)
    u = torch.full((8,), 0.4, device="cuda")
    greedy = {"temperature": torch.zeros(8, device="cuda")}
    tokens = [5]
    for _ in range(12):
        tokens += layer.verify(tokens[-1], [], len(tokens) - 1, u, **greedy)
    layer = example.Layer(seed=3)
    again, wrong = [5], 0
    while len(again) < len(tokens):
        at = len(again) - 1
        drafts = list(tokens[at + 1:at + 6])
        if len(drafts) > 2:
            drafts[2] = (drafts[2] + 1) % 2000          # a draft that is not accepted
            wrong += 1
        again += layer.verify(again[-1], drafts, at, u, **greedy)
    assert again[:len(tokens)] == tokens and wrong


def test_example_runs(example, capsys):
    example.main()
    assert "tokens in" in capsys.readouterr().out
