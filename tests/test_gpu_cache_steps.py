"""GPU tests of the cache's operators together, as an engine runs them: append,
attention with a window and sinks, keeping the accepted tokens, copying a forked
request's page; in CUDA graphs, over caches past 4 GB, and on a stream of their own."""
import numpy as np
import pytest

import few_row_packed_gb300 as lbv
from kv4_setup import DT
from oracle import kv4

torch = pytest.importorskip("torch")
pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def built():
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    lbv.build()


def empty_cache(bits, pages, page, heads, dim, dtype):
    if bits == 4:
        data = torch.zeros((pages, kv4.page_bytes(page, heads, dim)), dtype=torch.uint8, device="cuda")
        return lbv.KVCache4(data, page, heads, dim, DT[dtype])
    k, v = (torch.zeros((pages, page, heads, dim), dtype=DT[dtype], device="cuda") for _ in range(2))
    return lbv.KVCache(k, v)


def bits_of(cache):
    return [cache.data.clone()] if isinstance(cache, lbv.KVCache4) else [cache.k.clone(), cache.v.clone()]


class Steps:
    """Requests whose drafted rows enter the cache, attend, and are kept in part; the
    first request's last page is then copied for a fork."""

    def __init__(self, bits, q_len, kv_len, heads=8, kv_heads=2, dim=64, page=16, dtype="f16", window=40, sinks=3):
        self.args = window, sinks
        need = [-(-k // page) for k in kv_len]
        pages = sum(need) + 2
        self.cache = empty_cache(bits, pages, page, kv_heads, dim, dtype)
        g = torch.Generator(device="cuda").manual_seed(1)
        for t in ((self.cache.data,) if bits == 4 else (self.cache.k, self.cache.v)):
            if bits == 4:
                t.copy_(torch.randint(0, 256, t.shape, generator=g, device="cuda", dtype=torch.uint8))
                size, parts = min(page, 64), dim // 64
                sc = t.view(DT[dtype]).view(pages, kv_heads, page // size, -1)[..., 32 * parts * size:]
                sc.copy_(0.2 * torch.randn(sc.shape, generator=g, device="cuda"))
            else:
                t.copy_(torch.randn(t.shape, generator=g, device="cuda"))
        table = torch.zeros((len(q_len), max(need)), dtype=torch.int32)
        order = torch.randperm(pages, generator=torch.Generator().manual_seed(2)).to(torch.int32)
        at = 0
        for r, n in enumerate(need):
            table[r, :n] = order[at:at + n]
            at += n
        n = sum(q_len)
        self.batch = lbv.Batch(torch.tensor(np.concatenate([[0], np.cumsum(q_len)]), dtype=torch.int32, device="cuda"),
                               torch.tensor(kv_len, dtype=torch.int32, device="cuda"), table.cuda(), n)
        self.rope = lbv.Rope(lbv.rope_frequencies(dim))
        self.work = torch.zeros(lbv.attend_workspace_bytes(self.cache, self.batch, heads), dtype=torch.uint8, device="cuda")
        self.rows = [torch.zeros((n, h, dim), device="cuda") for h in (heads, kv_heads, kv_heads)]
        self.q, self.out = (torch.zeros((n, heads, dim), dtype=DT[dtype], device="cuda") for _ in range(2))
        self.back = [torch.zeros((n, kv_heads, dim), dtype=DT[dtype], device="cuda") for _ in range(2)]
        self.kept = torch.zeros(len(q_len), dtype=torch.int64, device="cuda")
        self.left = torch.zeros(len(q_len), dtype=torch.int32, device="cuda")
        self.src = table[0, need[0] - 1:need[0]].cuda()
        self.dst = order[at:at + 1].cuda()
        self.scale = dim ** -0.5

    def feed(self, seed):
        g = torch.Generator(device="cuda").manual_seed(seed)
        for t in self.rows:
            t.copy_(torch.randn(t.shape, generator=g, device="cuda"))
        self.kept.copy_(torch.randint(0, 2 ** 62, self.kept.shape, generator=g, device="cuda"))

    def run(self, pause=lambda: None):
        lbv.rope_append(self.rope, self.batch, self.cache, *self.rows, self.q)
        pause()
        lbv.attend(self.cache, self.batch, self.q, self.out, self.scale, window=self.args[0], sinks=self.args[1],
                   workspace=self.work)
        pause()
        lbv.kv_read(self.batch, self.cache, *self.back)
        pause()
        lbv.kv_keep(self.batch, self.cache, self.kept, self.left)
        pause()
        lbv.kv_copy_pages(self.cache, self.src, self.dst)
        pause()

    def results(self):
        return [t.clone() for t in (self.q, self.out, *self.back, self.left)] + bits_of(self.cache)


@pytest.mark.parametrize("bits", [16, 4])
@pytest.mark.parametrize("q_len, kv_len", [([1], [2000]), ([3, 1, 8], [60, 700, 33]), ([60, 2, 1], [900, 64, 70])])
def test_steps_in_one_graph(bits, q_len, kv_len):
    """Replays over new inputs give what the calls give one at a time, with the device idle
    between them; two graphs that share the workspace, too."""
    s = Steps(bits, q_len, kv_len)
    want = []
    for i in range(4):
        s.feed(i)
        s.run(torch.cuda.synchronize)
        want.append(s.results())
    first = Steps(bits, q_len, kv_len)
    stream = torch.cuda.Stream()
    stream.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(stream):
        graphs = []
        for _ in range(2):
            graphs.append(torch.cuda.CUDAGraph())
            with torch.cuda.graph(graphs[-1], stream=stream):
                first.run()
        for i in range(4):
            first.feed(i)
            graphs[i % 2].replay()
            got = first.results()
            assert all(torch.equal(a, b) for a, b in zip(got, want[i])), i
    lbv.attend_status(first.work)


@pytest.mark.parametrize("bits", [16, 4])
def test_kept_tokens_continue_the_context(bits):
    """The tokens that a step keeps are the context of the next, as if only they had been appended."""
    dim, page, heads = 64, 8, 2
    table = torch.randperm(20, generator=torch.Generator().manual_seed(0)).to(torch.int32)[None].cuda()
    i32 = lambda *x: torch.tensor(x, dtype=torch.int32, device="cuda")  # noqa: E731
    rope = lbv.Rope(lbv.rope_frequencies(dim))
    g = torch.Generator(device="cuda").manual_seed(5)
    rows = [torch.randn((13, heads, dim), generator=g, device="cuda") for _ in range(2)]
    stay = [0, 1, 2, 3, 4, 5, 8, 11]            # the prompt of 5, and drafts 0, 3 and 6 of 8
    places = i32(*range(5), 5, 6, 6, 6, 7, 7, 7, 8)     # a tree: siblings at one position
    one, other = (empty_cache(bits, 20, page, heads, dim, "f16") for _ in range(2))
    for at, n in ((0, 5), (5, 8)):
        batch = lbv.Batch(i32(0, n), i32(at + n), table, n)
        lbv.rope_append(rope, batch, one, None, *(t[at:at + n] for t in rows), None, positions=places[at:at + n])
    left = torch.zeros(1, dtype=torch.int32, device="cuda")
    lbv.kv_keep(batch, one, torch.tensor([0b01001001], device="cuda"), left)
    assert left.item() == 8
    short = lbv.Batch(i32(0, 8), i32(8), table, 8)
    lbv.rope_append(rope, short, other, None, *(t[stay].contiguous() for t in rows), None,
                    positions=places[torch.tensor(stay, device="cuda")].contiguous())
    a, b = ([torch.empty((8, heads, dim), dtype=torch.float16, device="cuda") for _ in "kv"] for _ in "ab")
    lbv.kv_read(short, one, *a)
    lbv.kv_read(short, other, *b)
    assert torch.equal(a[0], b[0]) and torch.equal(a[1], b[1])


@pytest.mark.parametrize("bits, heads", [(4, 4), (4, 48), (16, 4)])
def test_offsets_past_32_bits(bits, heads):
    """The same request at the start of a cache of 6 GB and at its end."""
    dim, page, kv_heads, n = 128, 64, 4, 500
    bytes_of = kv4.page_bytes(page, kv_heads, dim) if bits == 4 else 2 * page * kv_heads * dim
    pages = (6 << 30) // bytes_of
    cache = empty_cache(bits, pages, page, kv_heads, dim, "f16")
    g = torch.Generator(device="cuda").manual_seed(3)
    rows = [torch.randn((n, h, dim), generator=g, device="cuda") for h in (heads, kv_heads, kv_heads)]
    rope = lbv.Rope(lbv.rope_frequencies(dim))
    need = -(-n // page)
    tables = [torch.arange(need, dtype=torch.int32, device="cuda")[None], torch.arange(pages - need, pages, dtype=torch.int32,
                                                                                    device="cuda")[None].contiguous()]
    got = []
    for table in tables:
        batch = lbv.Batch(torch.tensor([0, n], dtype=torch.int32, device="cuda"),
                          torch.tensor([n], dtype=torch.int32, device="cuda"), table, n)
        q = torch.empty((n, heads, dim), dtype=torch.float16, device="cuda")
        lbv.rope_append(rope, batch, cache, *rows, q)
        few = lbv.Batch(torch.tensor([0, 2], dtype=torch.int32, device="cuda"), batch.kv_len, table, 2)
        out = []
        for b in (batch, few):
            o = torch.empty((b.tokens, heads, dim), dtype=torch.float16, device="cuda")
            ws = torch.zeros(lbv.attend_workspace_bytes(cache, b, heads), dtype=torch.uint8, device="cuda")
            lbv.attend(cache, b, q[:b.tokens], o, 0.1, workspace=ws)
            lbv.attend_status(ws)
            out.append(o)
        k, v = (torch.empty((n, kv_heads, dim), dtype=torch.float16, device="cuda") for _ in "kv")
        lbv.kv_read(batch, cache, k, v)
        kept = torch.tensor([2 ** 62 + 2 ** 40 + 2], device="cuda")
        many = lbv.Batch(torch.tensor([0, 64], dtype=torch.int32, device="cuda"), batch.kv_len, table, 64)
        lbv.kv_keep(many, cache, kept)
        k2, v2 = torch.empty_like(k), torch.empty_like(v)
        lbv.kv_read(batch, cache, k2, v2)
        assert torch.equal(k2[n - 64:n - 61], k[[n - 63, n - 24, n - 2]])
        got.append([q, *out, k, v, k2, v2])
    assert all(torch.equal(a, b) for a, b in zip(*got))
    lbv.kv_copy_pages(cache, tables[1][0], tables[0][0] + need)
    copied = lbv.Batch(torch.tensor([0, n], dtype=torch.int32, device="cuda"), batch.kv_len, tables[0] + need, n)
    k3, v3 = torch.empty_like(k), torch.empty_like(v)
    lbv.kv_read(copied, cache, k3, v3)
    assert torch.equal(k3, k2) and torch.equal(v3, v2)


def test_largest_page_and_single_head():
    """One head, pages of 1024 slots, a context that ends inside a chunk."""
    for dim in (64, 128):
        cache = empty_cache(4, 3, 1024, 1, dim, "bf16")
        g = torch.Generator(device="cuda").manual_seed(3)
        n = 1500
        rows = [torch.randn((n, h, dim), generator=g, device="cuda") for h in (1, 1, 1)]
        table = torch.tensor([[2, 0]], dtype=torch.int32, device="cuda")
        batch = lbv.Batch(torch.tensor([0, n], dtype=torch.int32, device="cuda"),
                          torch.tensor([n], dtype=torch.int32, device="cuda"), table, n)
        q = torch.empty((n, 1, dim), dtype=torch.bfloat16, device="cuda")
        lbv.rope_append(lbv.Rope(lbv.rope_frequencies(dim)), batch, cache, *rows, q)
        k, v = (torch.empty((n, 1, dim), dtype=torch.bfloat16, device="cuda") for _ in "kv")
        lbv.kv_read(batch, cache, k, v)
        out = torch.empty_like(q)
        ws = torch.zeros(lbv.attend_workspace_bytes(cache, batch, 1), dtype=torch.uint8, device="cuda")
        for few in (False, True):
            b = lbv.Batch(torch.tensor([0, 5], dtype=torch.int32, device="cuda"), batch.kv_len, table, 5) if few else batch
            m = b.tokens
            lbv.attend(cache, b, q[:m], out[:m], dim ** -0.5, workspace=ws)
            lbv.attend_status(ws)
            s = (q[:m, 0].double() @ k[:, 0].double().T) * dim ** -0.5
            at = torch.arange(n - m, n, device="cuda")[:, None]
            s = s.masked_fill(torch.arange(n, device="cuda")[None] > at, -torch.inf)
            p = torch.softmax(s, -1)
            want, size = p @ v[:, 0].double(), p @ v[:, 0].double().abs()
            # the probabilities and the output are rounded once each; scores are fp32 sums of dim terms
            e = (dim + 8) * 2.0 ** -24 * (q[:m, 0].double().abs() @ k[:, 0].double().abs().T).amax(-1) * dim ** -0.5 + 2.0 ** -20
            assert torch.all((out[:m, 0].double() - want).abs() <= 2.0 ** -8 * want.abs() + (2.0 ** -8 + 2 * e[:, None]) * size)


@pytest.mark.parametrize("dim, page, dtype", [(128, 8, "f16"), (128, 64, "bf16"), (64, 16, "f16")])
def test_two_calls_at_once(dim, page, dtype):
    """Few rows and many rows over one cache of 4 bits, on two streams with a workspace each,
    again and again: the results are those of a call alone, to the bit."""
    g = torch.Generator(device="cuda").manual_seed(page)
    requests, longest, heads, kv_heads = 24, 2100, 12, 2
    width = -(-longest // page)
    cache = empty_cache(4, requests * width, page, kv_heads, dim, dtype)
    table = torch.randperm(requests * width, generator=g, device="cuda").int().view(requests, width)
    kv_len = torch.randint(300, longest + 1, (requests,), generator=g, device="cuda").int()
    whole = lbv.Batch(torch.cat([kv_len.new_zeros(1), kv_len.cumsum(0).int()]), kv_len, table, int(kv_len.sum()))
    rows = [torch.randn((whole.tokens, kv_heads, dim), generator=g, device="cuda") for _ in "kv"]
    lbv.rope_append(lbv.Rope(lbv.rope_frequencies(dim)), whole, cache, None, *rows, None)
    calls = []
    for n in (1, 3, 9, 50):                             # 6, 18, 54 and 300 rows a request and key/value head
        start = torch.arange(0, requests * n + 1, n, dtype=torch.int32, device="cuda")
        batch = lbv.Batch(start, kv_len, table, requests * n)
        q = torch.randn((requests * n, heads, dim), generator=g, device="cuda").to(DT[dtype])
        ws = torch.zeros(lbv.attend_workspace_bytes(cache, batch, heads), dtype=torch.uint8, device="cuda")
        want = torch.empty_like(q)
        lbv.attend(cache, batch, q, want, dim ** -0.5, workspace=ws)
        lbv.attend_status(ws)
        calls.append((batch, q, ws, want))
    torch.cuda.synchronize()
    streams = [torch.cuda.Stream() for _ in calls]
    outs = [[torch.empty_like(c[1]) for _ in range(6)] for c in calls]
    torch.cuda.synchronize()
    for i in range(6):
        for (batch, q, ws, _), st, out in zip(calls, streams, outs):
            lbv.attend(cache, batch, q, out[i], dim ** -0.5, workspace=ws, stream=st)
    torch.cuda.synchronize()
    for (_, _, ws, want), out in zip(calls, outs):
        lbv.attend_status(ws)
        assert all(torch.equal(want, o) for o in out)
