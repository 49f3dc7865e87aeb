"""GPU tests of attention over 4 bits where a key's or a value's group could not be held (it has
a NaN or a magnitude beyond the cache's bounds): what sees it is NaN, never a number."""
import pytest

import few_row_packed_gb300 as lbv
from kv4_setup import Setup4
from oracle import kv4
from test_gpu_step import run_attend

torch = pytest.importorskip("torch")
pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def built():
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    lbv.build()


@pytest.mark.parametrize("heads, dim, dtype, q_len, kv_len", [
    (1, 128, "f16", [3], [3]), (6, 64, "bf16", [4, 1], [4, 90]),            # few rows
    (1, 128, "f16", [26], [26]), (6, 64, "bf16", [9, 1], [9, 300]),         # a tile
    (6, 128, "bf16", [40], [40]), (4, 64, "f16", [70, 1], [70, 3000]),      # two
])
@pytest.mark.parametrize("which", [0, 1])
def test_what_sees_a_lost_group_is_nan(heads, dim, dtype, q_len, kv_len, which):
    """The first key is lost, which every row sees, the first row alone."""
    s = Setup4(q_len, kv_len, kv_heads=1, dim=dim, dtype=dtype, page=16)
    for r in range(len(q_len)):
        _, at = kv4.offsets(16, 1, dim, 0, 0, which, 0)
        s.data[int(s.table[r, 0]), at:at + 2] = torch.tensor([0xFF, 0x7F], dtype=torch.uint8).cuda()
    out, lse, _ = run_attend(s, s.rows(heads, scale=2.0))
    if which == 0:
        assert torch.isnan(out).all() and torch.isnan(lse).all()
    else:
        assert torch.isnan(out[..., :64]).all() and not torch.isnan(lse).any()
