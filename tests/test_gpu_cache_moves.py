"""GPU tests of what a program does to a paged cache between steps: keeping some
of the new tokens, and copying pages."""
import numpy as np
import pytest

import few_row_packed_gb300 as lbv
from kv4_setup import Setup4
from oracle import kv4
from test_gpu_step import Setup

torch = pytest.importorskip("torch")
pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def built():
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    lbv.build()


def words(kept):
    return torch.tensor(np.array(kept, np.uint64).view(np.int64)).cuda()


class Slots:
    """The bits of every slot of a cache, [pages, page, bytes], as they are held now."""

    def __init__(self, s, bits):
        self.s, self.bits = s, bits

    def __call__(self):
        s = self.s
        if self.bits == 16:
            both = torch.stack((s.k, s.v), 2).contiguous().view(torch.uint8)
            return both.flatten(2).cpu().numpy()
        data, rows = s.data.cpu().numpy(), []
        for slot in range(s.page):
            at = [kv4.offsets(s.page, s.heads, s.dim, h, slot, w, p)
                  for h in range(s.heads) for w in range(2) for p in range(s.dim // 64)]
            rows.append(np.concatenate([data[:, a:b] for c, d in at for a, b in ((c, c + 32), (d, d + 4))], 1))
        return np.stack(rows, 1)


def make(bits, q_len, kv_len, dim, page, order="token", dtype="f16"):
    if bits == 16:
        s = Setup(q_len, kv_len, kv_heads=3, dim=dim, dtype=dtype, page=page, order=order)
        s.k.copy_(torch.randn(s.k.shape, generator=s.g))        # the unused slots too
        s.v.copy_(torch.randn(s.v.shape, generator=s.g))
    else:
        s = Setup4(q_len, kv_len, kv_heads=3, dim=dim, dtype=dtype, page=page)
    return s, Slots(s, bits)


def expect(slots, s, kept, page, pages):
    """The slots after a keep, the lengths, and the slots whose contents do not matter."""
    want, open_, left = slots.copy(), np.zeros(slots.shape[:2], bool), []
    for r, w in enumerate(kept):
        n = int(s.start[r + 1] - s.start[r])
        first = int(s.kv_len[r]) - n
        stay = [b for b in range(min(n, 64)) if w >> b & 1]

        def place(pos):
            if pos < 0 or pos // page >= s.table.shape[1]:
                return None
            p = int(s.table[r, pos // page])
            return (p, pos % page) if 0 <= p < pages else None

        for j, b in enumerate(stay):
            src, dst = place(first + b), place(first + j)
            if src and dst:
                want[dst] = slots[src]
        left.append(first + len(stay))
        for pos in range(max(left[-1], 0), int(s.kv_len[r])):
            if place(pos):
                open_[place(pos)] = True
    return want, open_, left


@pytest.mark.parametrize("bits, dim, page, order, dtype", [
    (16, 128, 16, "token", "f16"), (16, 64, 8, "head", "bf16"), (16, 128, 64, "gap", "f16"),
    (4, 128, 8, "", "f16"), (4, 64, 64, "", "bf16"), (4, 128, 256, "", "f16"),
])
@pytest.mark.parametrize("q_len, kv_len, kept", [
    ([1], [1], [0]), ([1], [5], [1]),
    ([8, 0, 5, 3], [70, 9, 5, 40], [0b10110101, 2 ** 64 - 1, 0b11111, 0b100]),
    ([64, 63], [64, 100], [0x8000000000000000, 0x5555555555555555]),
    ([64, 80], [300, 80], [2 ** 64 - 1, 0xAAAAAAAAAAAAAAAA]),       # past the 64th: dropped
    ([6, 2], [3, 0], [0b111010, 0b11]),                             # negative positions do not exist
    ([4, 4], [20, 33], [0b11111110, 0b11110111]),                   # bits past the tokens do not count
])
def test_keep(bits, dim, page, order, dtype, q_len, kv_len, kept):
    s, slots = make(bits, q_len, kv_len, dim, page, order, dtype)
    before = slots()
    want, open_, left = expect(before, s, kept, page, before.shape[0])
    got = torch.full((len(kept) + 1,), 77, dtype=torch.int32, device="cuda")
    lbv.kv_keep(s.batch, s.cache, words(kept), got)
    assert got.tolist() == left + [77]
    after = slots()
    assert np.array_equal(after[~open_], want[~open_])
    lbv.kv_keep(s.batch, s.cache, words([2 ** 64 - 1] * len(kept)))      # all stay: nothing moves
    assert np.array_equal(after, slots())


@pytest.mark.parametrize("bits", [16, 4])
def test_keep_leaves_missing_slots(bits):
    s, slots = make(bits, [8], [24], 128, 8)
    s.table[0, 2] = 10 ** 6                             # new tokens 0..7 are slots 16..23: all outside
    s.batch.block_table.copy_(torch.from_numpy(s.table))
    before = slots()
    lbv.kv_keep(s.batch, s.cache, words([0b10101010]))
    assert np.array_equal(before, slots())


@pytest.mark.parametrize("bits", [16, 4])
def test_keep_of_many_requests(bits):
    g = np.random.default_rng(2)
    q_len = [int(n) for n in g.integers(0, 65, 50)]
    kv_len = [n + int(g.integers(0, 90)) for n in q_len]
    kept = [int(g.integers(0, 2 ** 63)) * 2 + int(g.integers(0, 2)) for _ in q_len]
    s, slots = make(bits, q_len, kv_len, 64, 16)
    before = slots()
    want, open_, left = expect(before, s, kept, 16, before.shape[0])
    got = torch.empty(50, dtype=torch.int32, device="cuda")
    lbv.kv_keep(s.batch, s.cache, words(kept), got)
    assert got.tolist() == left
    assert np.array_equal(slots()[~open_], want[~open_])


@pytest.mark.parametrize("bits, dim, page, order, dtype", [
    (16, 128, 16, "token", "f16"), (16, 64, 8, "head", "bf16"), (16, 128, 1024, "gap", "f16"), (16, 64, 64, "token", "f16"),
    (4, 128, 8, "", "f16"), (4, 64, 64, "", "bf16"), (4, 128, 512, "", "f16"),
])
def test_copy_pages(bits, dim, page, order, dtype):
    s, slots = make(bits, [1], [6 * page], dim, page, order, dtype)
    before = slots()
    src, dst = [0, 3, 3, -1, 2, 1000, 5, 7], [1, 2, 6, 4, 8, 5, 5, -3]     # page 8 does not exist
    lbv.kv_copy_pages(s.cache, *(torch.tensor(x, dtype=torch.int32, device="cuda") for x in (src, dst)))
    want = before.copy()
    want[1], want[2], want[6] = before[0], before[3], before[3]
    assert np.array_equal(slots(), want)
    none = torch.empty(0, dtype=torch.int32, device="cuda")
    lbv.kv_copy_pages(s.cache, none, none)


def test_copy_leaves_what_lies_between():
    """Gaps between heads and between pages keep their bits."""
    room = torch.randn((5, 20, 2, 72), device="cuda").half()
    k, v = room[:, 1:17, :, :64], torch.randn((5, 20, 2, 72), device="cuda").half()[:, 1:17, :, :64]
    cache = lbv.KVCache(k, v)
    before, held = room.clone(), k.clone()
    pair = torch.tensor([[0, 4], [2, 3]], dtype=torch.int32, device="cuda")
    lbv.kv_copy_pages(cache, pair[0].contiguous(), pair[1].contiguous())
    held[2], held[3] = held[0], held[4]
    assert torch.equal(k, held)
    before[:, 1:17, :, :64] = held
    assert torch.equal(room, before)
