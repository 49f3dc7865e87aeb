"""GPU tests of a step whose batch mixes prompts with drafts: one batch for the append, the
attention and the tokens that stay."""
import numpy as np
import pytest

import few_row_packed_gb300 as lbv
from test_gpu_cache_moves import expect, make, words

torch = pytest.importorskip("torch")
pytestmark = pytest.mark.gpu

ALL = 2 ** 64 - 1


@pytest.fixture(scope="module", autouse=True)
def built():
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    lbv.build()


@pytest.mark.parametrize("bits, dim, page, order, dtype", [
    (16, 128, 16, "token", "f16"), (16, 64, 64, "head", "bf16"), (4, 128, 64, "", "bf16"), (4, 64, 8, "", "f16"),
])
@pytest.mark.parametrize("q_len, kv_len, kept", [
    ([65], [65], [ALL]), ([64], [200], [ALL]),
    ([300, 8, 1, 100, 0, 65], [300, 40, 77, 450, 9, 65], [ALL, 0b10100110, 1, ALL, ALL, 0]),
    ([300, 70], [301, 70], [ALL - 1, ALL >> 1]),        # of a prompt with any bit clear, the first 64 at most
])
def test_all_ones_keep_a_whole_prompt(bits, dim, page, order, dtype, q_len, kv_len, kept):
    s, slots = make(bits, q_len, kv_len, dim, page, order, dtype)
    before = slots()
    want, open_, left = expect(before, s, kept, page, before.shape[0])
    for r, w in enumerate(kept):
        if w == ALL:                                    # nothing moves, and all of it counts
            left[r] = kv_len[r]
            for pos in range(max(0, kv_len[r] - q_len[r]), kv_len[r]):
                open_[int(s.table[r, pos // page]), pos % page] = False
    got = torch.full((len(kept),), -1, dtype=torch.int32, device="cuda")
    lbv.kv_keep(s.batch, s.cache, words(kept), got)
    assert got.tolist() == left
    after = slots()
    assert np.array_equal(after[~open_], want[~open_])


@pytest.mark.parametrize("bits", [16, 4])
def test_a_step_of_prompts_and_drafts(bits):
    """Append, attention and keep by one batch; what stays is the context of the next step: the same
    rows as after an append of the tokens that stayed alone."""
    dim, page, kv_heads, heads = 64, 16, 2, 6
    q_len, context, kept = [200, 5, 1], [0, 30, 64], [ALL, 0b10011, 1]
    kv_len = [a + b for a, b in zip(q_len, context)]
    width = max(-(-k // page) for k in kv_len)
    i32 = lambda *x: torch.tensor(x, dtype=torch.int32, device="cuda")  # noqa: E731
    g = torch.Generator(device="cuda").manual_seed(7)
    table = torch.randperm(3 * width, generator=g, device="cuda").int().view(3, width)

    def cache():
        if bits == 4:
            data = torch.zeros((3 * width, lbv.kv_cache4_page_bytes(page, kv_heads, dim)), dtype=torch.uint8, device="cuda")
            return lbv.KVCache4(data, page, kv_heads, dim, torch.float16)
        return lbv.KVCache(*(torch.zeros((3 * width, page, kv_heads, dim), dtype=torch.float16, device="cuda") for _ in "kv"))

    def starts(n):
        return i32(*np.concatenate([[0], np.cumsum(n)]).tolist())

    def step(c, batch, places, rows):
        q = torch.empty((batch.tokens, heads, dim), dtype=torch.float16, device="cuda")
        lbv.rope_append(rope, batch, c, *rows, q, positions=places)
        out = torch.empty_like(q)
        ws = torch.zeros(lbv.attend_workspace_bytes(c, batch, heads), dtype=torch.uint8, device="cuda")
        lbv.attend(c, batch, q, out, dim ** -0.5, workspace=ws)
        lbv.attend_status(ws)
        return out

    rope = lbv.Rope(lbv.rope_frequencies(dim))
    one, other = cache(), cache()
    old = [torch.randn((sum(context), h, dim), generator=g, device="cuda") for h in (heads, kv_heads, kv_heads)]
    for c in (one, other):
        step(c, lbv.Batch(starts(context), i32(*context), table, sum(context)), None, old)
    new = [torch.randn((sum(q_len), h, dim), generator=g, device="cuda") for h in (heads, kv_heads, kv_heads)]
    places = i32(*[context[r] + i for r in range(3) for i in range(q_len[r])])
    batch = lbv.Batch(starts(q_len), i32(*kv_len), table, sum(q_len))
    step(one, batch, places, new)
    left = torch.zeros(3, dtype=torch.int32, device="cuda")
    lbv.kv_keep(batch, one, words(kept), left)
    stay = [sum(q_len[:r]) + i for r in range(3) for i in range(q_len[r]) if q_len[r] > 64 or kept[r] >> i & 1]
    count = [200, 3, 1]
    assert left.tolist() == [c + n for c, n in zip(context, count)]
    step(other, lbv.Batch(starts(count), left, table, sum(count)), places[stay].contiguous(),
         [t[stay].contiguous() for t in new])
    # the next step reads both caches alike
    following = [torch.randn((3, h, dim), generator=g, device="cuda") for h in (heads, kv_heads, kv_heads)]
    after = lbv.Batch(starts([1, 1, 1]), left + 1, torch.cat([table, torch.full((3, 1), -1, device="cuda").int()], 1), 3)
    assert torch.equal(step(one, after, None, following), step(other, after, None, following))
