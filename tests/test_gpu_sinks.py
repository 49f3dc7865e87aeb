"""GPU tests of attention with a sliding window whose first tokens stay visible,
over caches of 16 and of 4 bits, against the fp64 oracle."""
import numpy as np
import pytest

import few_row_packed_gb300 as lbv
from kv4_setup import Setup4, f64
from oracle import step
from test_gpu_kv4 import Held
from test_gpu_step import TINY, UNIT, Setup

torch = pytest.importorskip("torch")
pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def built():
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    lbv.build()


def run(s, q, window, sinks, tree=None):
    out = torch.full_like(q, 7.0)
    lse = torch.full(q.shape[:2], 7.0, device="cuda")
    ws = torch.zeros(lbv.attend_workspace_bytes(s.cache, s.batch, q.shape[1]), dtype=torch.uint8, device="cuda")
    words = None if tree is None else torch.tensor(np.array(tree, np.uint64).view(np.int64)).cuda()
    lbv.attend(s.cache, s.batch, q, out, s.dim ** -0.5, window=window, sinks=sinks, tree=words, lse=lse, workspace=ws)
    lbv.attend_status(ws)
    return out, lse


def check(s, q, out, lse, window, sinks, tree=None):
    n = int(s.start[-1])
    want, ref, A, V, S = step.attend(f64(q)[:n], np.nan_to_num(f64(s.k)), np.nan_to_num(f64(s.v)), s.start, s.kv_len,
                                     s.table, s.dim ** -0.5, window, tree, sinks)
    u = UNIT[s.dtype]
    # scores: an fp32 dot product of dim terms, its scaling and the exponential; the
    # probabilities and the output are rounded once each
    e = (s.dim + 8) * 2.0 ** -24 * S + 2.0 ** -20
    tol = u * np.abs(want) + (u + 2 * e[..., None]) * A + TINY[s.dtype] * (1 + V)
    got, g, none = f64(out), f64(lse), np.isneginf(ref)
    assert np.all(np.abs(got[:n] - want) <= tol), np.abs(got[:n] - want).max()
    assert np.array_equal(np.isneginf(g[:n]), none) and np.all(got[:n][none] == 0)
    assert np.all(np.abs(g[:n] - ref)[~none] <= (e + 2.0 ** -22 * np.abs(ref))[~none])
    assert np.all(got[n:] == 7.0) and np.all(g[n:] == 7.0)


def make(bits, q_len, kv_len, kv_heads, dim, dtype, page):
    if bits == 16:
        s = Setup(q_len, kv_len, kv_heads=kv_heads, dim=dim, dtype=dtype, page=page, pad=1)
        return s, s
    s = Setup4(q_len, kv_len, kv_heads=kv_heads, dim=dim, dtype=dtype, page=page, pad=1)
    return s, Held(s)


@pytest.mark.parametrize("bits", [16, 4])
@pytest.mark.parametrize("heads, kv_heads, dim, dtype, page", [(4, 2, 128, "f16", 16), (12, 1, 64, "bf16", 8)])
@pytest.mark.parametrize("window, sinks", [
    (1, 1), (5, 4), (64, 1), (64, 64), (30, 65), (100, 130),
    (40, 0),                    # a window alone
    (40, 10 ** 6),              # every key is a sink
    (10 ** 6, 4),               # the window reaches over all
])
@pytest.mark.parametrize("q_len, kv_len", [([1, 2, 0, 1], [700, 131, 9, 3]), ([150, 1], [500, 260])])
def test_lengths(bits, heads, kv_heads, dim, dtype, page, window, sinks, q_len, kv_len):
    """Few rows and many; sinks and windows in one block, in neighbours and far apart."""
    s, held = make(bits, q_len, kv_len, kv_heads, dim, dtype, page)
    q = s.rows(heads, scale=2.0)
    out, lse = run(s, q, window, sinks)
    check(held, q, out, lse, window, sinks)
    # pages wholly between the sinks and every window may be gone
    for r in range(len(q_len)):
        low = max(0, kv_len[r] - q_len[r] - window + 1) // page
        s.batch.block_table[r, min(low, -(-sinks // page)):low] = -1
    again, lse2 = run(s, q, window, sinks)
    assert torch.equal(out, again) and torch.equal(lse, lse2)


@pytest.mark.parametrize("bits", [16, 4])
@pytest.mark.parametrize("heads, dim, dtype", [(2, 128, "bf16"), (9, 64, "f16")])
@pytest.mark.parametrize("window, sinks", [(6, 3), (90, 20)])
def test_tree(bits, heads, dim, dtype, window, sinks):
    rng = np.random.default_rng(3)
    s, held = make(bits, [8, 1, 70, 5], [400, 1, 70, 5], 1, dim, dtype, 16)
    tree = [int(rng.integers(0, 2**63)) for _ in range(s.tokens)]
    tree[0], tree[8], tree[79] = 1, 0, 0
    q = s.rows(heads, scale=2.0)
    out, lse = run(s, q, window, sinks, tree)
    check(held, q, out, lse, window, sinks, tree)


@pytest.mark.parametrize("q_len", [[1], [40]])
def test_without_a_window_sinks_change_nothing(q_len):
    s, _ = make(16, q_len, [300], 2, 128, "f16", 32)
    q = s.rows(4)
    a, b = run(s, q, 0, 0), run(s, q, 0, 17)
    assert torch.equal(a[0], b[0]) and torch.equal(a[1], b[1])


@pytest.mark.parametrize("bits", [16, 4])
def test_many_items(bits):
    """Ragged requests whose shares begin among the sinks, among the window's blocks and between."""
    g = np.random.default_rng(8)
    q_len = [int(n) for n in g.choice([1, 2, 5, 40, 130], 40)]
    kv_len = [n + int(g.integers(0, 900)) for n in q_len]
    s, held = make(bits, q_len, kv_len, 8, 64, "bf16", 16)
    q = s.rows(8, scale=2.0)
    out, lse = run(s, q, 150, 140)
    check(held, q, out, lse, 150, 140)


@pytest.mark.parametrize("q_len", [[1, 1, 1], [70, 3]])
def test_a_share_that_begins_in_the_gap(q_len):
    """Long contexts, divided over the CTAs: most of the keys are left out."""
    kv_len = [5000, 4000, 3500][:len(q_len)]
    s, held = make(16, q_len, kv_len, 2, 64, "f16", 64)
    q = s.rows(4, scale=2.0)
    out, lse = run(s, q, 1000, 300)
    check(held, q, out, lse, 1000, 300)
