"""GPU tests of the verify step's calls in one CUDA graph, between matmuls that
launch while the kernel before them drains: replays over new inputs give what
the same calls give one at a time, with the device idle between them."""
import numpy as np
import pytest

import few_row_packed_gb300 as lbv
import synth

torch = pytest.importorskip("torch")
pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def built():
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    lbv.build()


class Step:
    """q/k/v projections of the rows of a step as one grouped call, positions and
    append, attention, output projection, head, sampling: fixed buffers."""

    def __init__(self, q_len, kv_len, flags, heads=8, kv_heads=2, dim=64, hidden=512, vocab=2000):
        q, kv, page, f16 = heads * dim, kv_heads * dim, 16, torch.float16
        self.n = n = sum(q_len)
        self.qkv = lbv.Group(lbv.FMT_Q4_0, 32, lbv.F16, [(hidden, q), (hidden, kv), (hidden, kv)], flags)
        self.out = lbv.Plan(lbv.FMT_Q4_0, q, hidden, 32, lbv.F16, flags)
        self.head = lbv.Plan(lbv.FMT_AFFINE2, hidden, vocab, 64, lbv.F16, flags)
        self.w = []
        for i, (fmt, name, k, m, group) in enumerate((
                (lbv.FMT_Q4_0, synth.Q4_0, hidden, q, 32), (lbv.FMT_Q4_0, synth.Q4_0, hidden, kv, 32),
                (lbv.FMT_Q4_0, synth.Q4_0, hidden, kv, 32), (lbv.FMT_Q4_0, synth.Q4_0, q, hidden, 32),
                (lbv.FMT_AFFINE2, synth.AFFINE2, hidden, vocab, 64))):
            parts, _ = synth.gen_matrix(synth.Matrix(f"w{i}", name, k, m, group, "f16", sigma_scale=0.01),
                                        [7, i], rows=1)
            self.w.append(torch.from_numpy(lbv.pack(fmt, parts, k, m, group)).cuda())
        pages = sum(-(-k // page) for k in kv_len)
        g = torch.Generator(device="cuda").manual_seed(3)
        self.k, self.v = (torch.randn((pages, page, kv_heads, dim), generator=g, device="cuda").half()
                          for _ in range(2))
        self.cache = lbv.KVCache(self.k, self.v)
        table = torch.zeros((len(q_len), max(-(-k // page) for k in kv_len)), dtype=torch.int32, device="cuda")
        at, order = 0, torch.randperm(pages, generator=g, device="cuda").to(torch.int32)
        for r, k in enumerate(kv_len):
            table[r, :-(-k // page)] = order[at:at - (-k // page)]
            at += -(-k // page)
        start = torch.tensor(np.concatenate([[0], np.cumsum(q_len)]), dtype=torch.int32, device="cuda")
        self.batch = lbv.Batch(start, torch.tensor(kv_len, dtype=torch.int32, device="cuda"), table, n)
        self.rope = lbv.Rope(lbv.rope_frequencies(dim))
        self.workspace = torch.zeros(lbv.attend_workspace_bytes(self.cache, self.batch, heads),
                                     dtype=torch.uint8, device="cuda")
        self.x = torch.zeros((n, hidden), dtype=f16, device="cuda")
        self.rows = [torch.zeros((n, h, dim), device="cuda") for h in (heads, kv_heads, kv_heads)]
        self.q, self.attended = (torch.zeros((n, heads, dim), dtype=f16, device="cuda") for _ in range(2))
        self.y = torch.zeros((n, hidden), device="cuda")
        self.z = torch.zeros((n, vocab), device="cuda")
        self.u, self.prob = torch.zeros(n, device="cuda"), torch.zeros(n, device="cuda")
        self.token = torch.zeros(n, dtype=torch.int32, device="cuda")
        self.temperature = torch.full((n,), 0.8, device="cuda")
        self.top_k = torch.full((n,), 50, dtype=torch.int32, device="cuda")

    def feed(self, seed):
        g = torch.Generator(device="cuda").manual_seed(seed)
        self.x.copy_(torch.randn(self.x.shape, generator=g, device="cuda"))
        self.u.copy_(torch.rand(self.n, generator=g, device="cuda"))

    def run(self, pause=lambda: None):
        for a in range(0, self.n, 8):                   # matmuls take up to 8 rows
            b = min(a + 8, self.n)
            lbv.verify_grouped(self.qkv, [(self.x[a:b], b - a, w, y[a:b]) for w, y in zip(self.w, self.rows)])
            pause()
        lbv.rope_append(self.rope, self.batch, self.cache, *self.rows, self.q)
        pause()
        lbv.attend(self.cache, self.batch, self.q, self.attended, 0.125, workspace=self.workspace)
        pause()
        for a in range(0, self.n, 8):
            b = min(a + 8, self.n)
            lbv.verify_gemm(self.out, self.attended[a:b], b - a, self.w[3], self.y[a:b])
            pause()
            lbv.verify_gemm(self.head, self.attended[a:b].reshape(b - a, -1), b - a, self.w[4], self.z[a:b])
            pause()
        lbv.sample(self.z, self.u, self.token, prob=self.prob, temperature=self.temperature, top_k=self.top_k)
        pause()

    def results(self):
        return [t.clone() for t in (*self.rows, self.q, self.k, self.v, self.attended, self.y, self.z,
                                    self.token, self.prob)]


@pytest.mark.parametrize("flags", [0, lbv.PLAN_PDL])
@pytest.mark.parametrize("q_len, kv_len", [
    ([1], [2000]),              # parts joined by a launch of their own
    ([3, 1, 4], [60, 700, 33]),
    ([40, 1, 9], [900, 64, 70]),        # the tensor-memory kernel
])
def test_a_step_in_one_graph(q_len, kv_len, flags):
    s = Step(q_len, kv_len, flags)
    seeds = range(6)
    want = []
    for i in seeds:
        s.feed(i)
        s.run(torch.cuda.synchronize)
        want.append(s.results())
    stream = torch.cuda.Stream()
    stream.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(stream):
        s.run()
        graph = torch.cuda.CUDAGraph()
        with torch.cuda.graph(graph, stream=stream):
            s.run()
            s.run()             # the second pass follows the first without a pause
        for i in [*seeds, *seeds]:
            s.feed(i)
            graph.replay()
            got = s.results()
            assert all(torch.equal(a, b) for a, b in zip(got, want[i]))
        for i in seeds:         # and without a graph
            s.feed(i)
            for _ in range(3):
                s.run()
            assert all(torch.equal(a, b) for a, b in zip(s.results(), want[i]))
    lbv.attend_status(s.workspace)
    assert len({tuple(w[-2].tolist()) for w in want}) > 1
