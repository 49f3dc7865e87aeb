"""Bounded waits of the attention kernels that run out, on the GPU, without a
fault: the test export shortens the waits to half a millisecond and has the first
CTA stop copying.  What waits for the next copy gives up, the kernel ends, the
workspace reports the timeout once, what other CTAs computed is right, and the
next call with the same workspace is exact."""
import time

import pytest

import few_row_packed_gb300 as lbv
from test_gpu_attend_long import Case

torch = pytest.importorskip("torch")
pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def built():
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    lbv.build()


def run_out(c, copies, safe):
    """`safe`: the rows and heads that the first CTA has no part in."""
    want, lse = c.attend()
    out = torch.full_like(want, 7.0)
    torch.cuda.synchronize()
    t0 = time.perf_counter()
    lbv.attend_test_wait(c.cache, c.batch, c.q, out, c.scale, c.workspace, copies)
    torch.cuda.synchronize()
    assert time.perf_counter() - t0 < 5.0
    with pytest.raises(lbv.LbvError) as e:
        lbv.attend_status(c.workspace)
    assert e.value.status == lbv.ERR_TIMEOUT
    lbv.attend_status(c.workspace)                      # reported once, then cleared
    assert torch.equal(safe(out), safe(want))
    again, lse2 = c.attend()
    assert torch.equal(again, want) and torch.equal(lse2, lse)


# q_len, kv_len, heads, kv_heads, dim, dtype, page
ROWS = {
    # the parts of an item joined by its last CTA, and by a launch of their own
    "many requests": (([1] * 200, [900] * 200, 12, 2, 128, "bf16", 16), lambda t: t[1:]),
    "one request": (([2], [100001], 48, 8, 64, "f16", 32), lambda t: t[:, 6:]),
}


@pytest.mark.parametrize("copies", [0, 1, 5])
@pytest.mark.parametrize("name", list(ROWS))
def test_few_row_kernel(name, copies):
    args, safe = ROWS[name]
    run_out(Case(*args), copies, safe)


TILES = {
    # items of one and of two row tiles in turn, several in each CTA
    "many items": (([40, 150, 3, 129, 64] * 24, [400, 420, 90, 500, 64] * 24, 16, 8, 128, "bf16", 16),
                   lambda t: t[772:]),
    "small heads": (([150, 40] * 60, [1500, 1300] * 60, 8, 4, 64, "f16", 32), lambda t: t[570:]),
    # one row tile over every CTA, and two
    "one request": (([16], [30011], 48, 8, 128, "f16", 16), lambda t: t[:, 6:]),
    "a chunk": (([200], [30000], 16, 8, 128, "bf16", 64), lambda t: t[:, 2:]),
}


@pytest.mark.parametrize("copies", [0, 1, 2, 3, 6, 9])
@pytest.mark.parametrize("name", list(TILES))
def test_tile_kernel(name, copies):
    args, safe = TILES[name]
    run_out(Case(*args), copies, safe)
