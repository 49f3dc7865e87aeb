"""GPU tests of the attention over long contexts, above all by the tensor-memory
kernel: items whose copies wrap the ring many times, that go on in the next CTA,
and whose parts are few, more than eight and more than 32, against a 64-bit
computation."""
import numpy as np
import pytest

import few_row_packed_gb300 as lbv
from test_gpu_step import DT, TINY, UNIT

torch = pytest.importorskip("torch")
pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def built():
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    lbv.build()


class Case:
    """Requests over a cache whose pages are in no order; unused slots hold NaN."""

    def __init__(self, q_len, kv_len, heads, kv_heads, dim, dtype, page, scale=2.0, seed=0):
        g = torch.Generator(device="cuda").manual_seed(seed)
        self.q_len, self.kv_len, self.dtype, self.page = q_len, kv_len, dtype, page
        self.heads, self.kv_heads, self.dim = heads, kv_heads, dim
        need = [-(-k // page) for k in kv_len]
        pages = sum(need) + 3
        order = torch.randperm(pages, generator=g, device="cuda").to(torch.int32)
        self.table = torch.full((len(q_len), max(need)), -1, dtype=torch.int32, device="cuda")
        self.k, self.v = (torch.randn((pages, page, kv_heads, dim), generator=g, device="cuda").to(DT[dtype])
                          for _ in range(2))
        at, used = 0, torch.zeros((pages, page), dtype=torch.bool, device="cuda")
        for r, n in enumerate(need):
            self.table[r, :n] = order[at:at + n]
            used[order[at:at + n].long()] = True
            if kv_len[r] % page:
                used[int(order[at + n - 1]), kv_len[r] % page:] = False
            at += n
        self.k[~used] = float("nan")
        self.v[~used] = float("nan")
        start = np.concatenate([[0], np.cumsum(q_len)])
        self.tokens = int(start[-1])
        self.cache = lbv.KVCache(self.k, self.v)
        self.batch = lbv.Batch(torch.tensor(start, dtype=torch.int32, device="cuda"),
                               torch.tensor(kv_len, dtype=torch.int32, device="cuda"), self.table, self.tokens)
        self.q = (scale * torch.randn((self.tokens, heads, dim), generator=g, device="cuda")).to(DT[dtype])
        self.scale = dim ** -0.5
        self.workspace = torch.zeros(lbv.attend_workspace_bytes(self.cache, self.batch, heads),
                                     dtype=torch.uint8, device="cuda")

    def attend(self, window=0, tree=None):
        out = torch.full_like(self.q, 7.0)
        lse = torch.full((self.tokens, self.heads), 7.0, device="cuda")
        lbv.attend(self.cache, self.batch, self.q, out, self.scale, window=window, tree=tree, lse=lse,
                   workspace=self.workspace)
        lbv.attend_status(self.workspace)
        return out, lse

    def check(self, out, lse, window=0, tree=None):
        group, at = self.heads // self.kv_heads, 0
        for r, (n, kv) in enumerate(zip(self.q_len, self.kv_len)):
            pages = self.table[r, :-(-kv // self.page)].long()
            key = torch.arange(kv, device="cuda")[None, :]
            mine = torch.arange(kv - n, kv, device="cuda")[:, None]
            if tree is None:
                sees = key <= mine
            else:
                j = key - (kv - n)
                sees = (j < 0) | ((j < 64) & (((tree[at:at + n, None] >> j.clamp(0, 63)) & 1) == 1))
            if window:
                sees = sees & (key > mine - window)
            for h in range(self.kv_heads):
                k, v = (t[pages, :, h].reshape(-1, self.dim)[:kv].double() for t in (self.k, self.v))
                for i in range(group):
                    self._check_head(out, lse, at, n, h * group + i, k, v, sees)
            at += n

    def _check_head(self, out, lse, at, n, head, k, v, sees):
        q = self.q[at:at + n, head].double()
        t = (q @ k.T * self.scale).masked_fill(~sees, -np.inf)
        top = t.amax(-1, keepdim=True)
        p = (t - top).exp()
        total = p.sum(-1, keepdim=True)
        want, ref = p @ v / total, (top + total.log())[:, 0]
        A, V = p @ v.abs() / total, sees.double() @ v.abs() / total
        S = (self.scale * (q.abs() @ k.abs().T)).masked_fill(~sees, 0).amax(-1)
        u = UNIT[self.dtype]
        # scores: an fp32 dot product, its scaling and the exponential; sums: an fp32
        # addition for each 16 keys in the product with V, and for each block of the rest
        e = (self.dim + 8) * 2.0 ** -24 * S + 2.0 ** -20
        add = (k.shape[0] / 16 + 64) * 2.0 ** -23
        tol = u * want.abs() + (u + 2 * e[:, None] + add) * A + TINY[self.dtype] * (1 + V)
        err = (out[at:at + n, head].double() - want).abs()
        assert torch.all(err <= tol), (head, float(err.max()))
        more = (k.shape[0] / 64 + 128) * 2.0 ** -24
        assert torch.all((lse[at:at + n, head].double() - ref).abs() <= e + more + 2.0 ** -22 * ref.abs())


CASES = {
    # one row tile over every CTA: some 140 parts
    "one tile": ([8], [70001], 6, 1, 128, "bf16", 64),
    # 8 items of one row tile, some 19 parts each
    "eight items": ([16], [30011], 48, 8, 128, "f16", 16),
    # two items of two row tiles and one of one: some 50 parts each
    "two and one": ([100], [20000], 6, 1, 128, "bf16", 128),
    # long items of two row tiles that begin and end anywhere in a CTA's share
    "ragged": ([300, 31, 700, 44], [5003, 9000, 4001, 12345], 16, 4, 128, "bf16", 32),
    "small heads": ([260, 90, 1], [7001, 16000, 20], 12, 2, 64, "f16", 8),
    # many short items beside long ones
    "long and short": ([17] * 40 + [400], [130 + 7 * i for i in range(40)] + [9001], 16, 2, 64, "bf16", 16),
    # the few-row kernel
    "few rows": ([1, 2, 1], [40001, 12, 9999], 8, 2, 128, "bf16", 32),
}


@pytest.mark.parametrize("name", list(CASES))
def test_long_contexts(name):
    c = Case(*CASES[name])
    out, lse = c.attend()
    c.check(out, lse)
    again, lse2 = c.attend()
    assert torch.equal(out, again) and torch.equal(lse, lse2)


@pytest.mark.parametrize("name, window", [("ragged", 2000), ("two and one", 5000), ("eight items", 9999)])
def test_long_contexts_with_a_window(name, window):
    c = Case(*CASES[name])
    c.check(*c.attend(window=window), window=window)


def test_long_context_with_a_tree():
    c = Case([60, 33], [20003, 800], 12, 2, 128, "bf16", 16)
    g = torch.Generator(device="cuda").manual_seed(1)
    tree = torch.randint(-2 ** 62, 2 ** 62, (93,), generator=g, device="cuda")
    c.check(*c.attend(tree=tree), tree=tree)
    c.check(*c.attend(tree=tree, window=900), window=900, tree=tree)


def test_a_few_keys_dominate_a_long_row():
    """Scores of tens here and there over a flat rest: the reference moves late, and
    parts of very different weight are joined."""
    c = Case([20], [30001], 16, 2, 64, "f16", 64, scale=0.25)
    g = torch.Generator().manual_seed(2)
    flat = c.k.view(-1, 2, 64)
    for j in torch.randint(0, 30001, (12,), generator=g).tolist():
        slot = int(c.table[0, j // 64]) * 64 + j % 64
        flat[slot] = 40 * c.q[j % 20, ::8].float().half()
    c.check(*c.attend())
