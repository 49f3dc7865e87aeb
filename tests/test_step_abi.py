"""CPU tests of the operators around the verify matmul: refused arguments,
frequencies, and the oracles against hand-worked values."""
import ctypes
import math

import numpy as np
import pytest

import few_row_packed_gb300 as lbv
from oracle import step

INF, P = lbv.ERR_INVALID_ARG, ctypes.c_void_p


@pytest.fixture(scope="module")
def L():
    lbv.build()
    return lbv.lib()


def batch(**kw):
    a = dict(q_start=4096, kv_len=4096, block_table=4096, requests=1, tokens=1, table_stride=4,
             table_pages=4)
    a.update(kw)
    return lbv._BatchArg(*[a[f] for f, _ in lbv._BatchArg._fields_])


def rows(**kw):
    a = dict(data=4096, heads=2, dtype=lbv.F16, token_stride=256, head_stride=128)
    a.update(kw)
    return lbv._RowsArg(*[a[f] for f, _ in lbv._RowsArg._fields_])


def cache(L, pages=4, page_size=16, heads=2, dim=128, strides=None, dtype=lbv.F16, k=4096, v=8192):
    h = P()
    st = strides or (page_size * heads * dim, heads * dim, dim)
    return L.lbv_kv_cache_create(k, v, pages, page_size, heads, dim, *st, dtype, ctypes.byref(h)), h


@pytest.mark.parametrize("kw, want", [
    (dict(k=None), lbv.ERR_INVALID_ARG), (dict(v=8), lbv.ERR_INVALID_ARG),
    (dict(pages=0), lbv.ERR_INVALID_ARG), (dict(heads=0), lbv.ERR_INVALID_ARG),
    (dict(dtype=lbv.F32), lbv.ERR_INVALID_ARG), (dict(dtype=9), lbv.ERR_INVALID_ARG),
    (dict(page_size=24), lbv.ERR_UNSUPPORTED), (dict(page_size=4), lbv.ERR_UNSUPPORTED),
    (dict(page_size=2048), lbv.ERR_UNSUPPORTED), (dict(dim=96), lbv.ERR_UNSUPPORTED),
    (dict(strides=(4096, 256, 64)), lbv.ERR_INVALID_ARG),      # a head shorter than its dim
    (dict(strides=(4096, 260, 128)), lbv.ERR_INVALID_ARG),     # not a multiple of 8
    (dict(strides=(2048, 256, 128)), lbv.ERR_INVALID_ARG),     # pages overlap
    (dict(strides=(4096, 128, 128)), lbv.ERR_INVALID_ARG),     # heads overlap tokens
])
def test_cache_refusals(L, kw, want):
    st, h = cache(L, **kw)
    assert st == want and not h.value
    assert "lbv_kv_cache_create" in lbv.last_error()


def test_cache_null_out(L):
    assert L.lbv_kv_cache_create(4096, 8192, 1, 16, 1, 64, 1024, 64, 64, 0, None) == INF
    assert L.lbv_kv_cache_destroy(None) == lbv.OK


def test_rope_refusals(L):
    f = np.ones(64)
    h = P()

    def create(freqs=f, rot=128, layout=0, factor=1.0, out=ctypes.byref(h)):
        return L.lbv_rope_create(None if freqs is None else freqs.ctypes.data, rot, layout, factor, out)

    for kw in (dict(freqs=None), dict(rot=6), dict(rot=136), dict(rot=12), dict(layout=2),
               dict(factor=math.inf), dict(out=None), dict(freqs=np.full(64, math.nan))):
        assert create(**kw) == INF, kw
    r = lbv.Rope(f)
    b, k = batch(), rows()
    R = ctypes.byref
    none = P()
    assert L.lbv_rope_append(None, R(b), none, None, R(k), R(k), None, None, None) == INF
    assert L.lbv_rope_append(r.handle, None, none, None, R(k), R(k), None, None, None) == INF
    for bad in (dict(requests=0), dict(requests=5000), dict(tokens=-1), dict(q_start=None),
                dict(kv_len=4098), dict(block_table=None), dict(table_pages=0), dict(table_stride=3)):
        x = batch(**bad)
        assert L.lbv_rope_append(r.handle, R(x), none, None, R(k), R(k), None, None, None) == INF, bad
    for bad in (dict(data=None), dict(data=4097), dict(heads=0), dict(dtype=5)):
        x = rows(**bad)
        assert L.lbv_rope_append(r.handle, R(b), none, None, R(x), R(k), None, None, None) == INF, bad
        assert L.lbv_rope_append(r.handle, R(b), none, None, R(k), R(x), None, None, None) == INF, bad
        assert L.lbv_rope_append(r.handle, R(b), none, R(k), R(k), R(k), R(x), None, None) == INF, bad
    # queries without a place for them
    assert L.lbv_rope_append(r.handle, R(b), none, R(k), R(k), R(k), None, None, None) == INF
    assert L.lbv_rope_append(r.handle, R(b), none, None, R(k), R(k), None, None, None) == INF
    assert "cache is NULL" in lbv.last_error()


def test_attend_refusals(L):
    b, q = batch(), rows()
    R = ctypes.byref
    none = P()
    assert L.lbv_attend_workspace_bytes(None, R(b), 8) == 0
    call = lambda bb, qq, oo: L.lbv_attend(none, bb, qq, oo, 1.0, 0, None, None, None, 0, None)  # noqa: E731
    assert call(None, R(q), R(q)) == INF
    assert call(R(b), None, R(q)) == INF
    assert call(R(b), R(q), None) == INF
    assert call(R(b), R(rows(dtype=7)), R(q)) == INF
    assert call(R(b), R(q), R(q)) == INF and "cache is NULL" in lbv.last_error()
    assert L.lbv_attend_status(None) == INF


def test_sample_refusals(L):
    rules = lbv._RulesArg()
    R = ctypes.byref

    def call(logits=4096, m=1, n=100, ld=100, dt=lbv.F32, r=rules, u=4096, token=4096, prob=None):
        return L.lbv_sample(logits, m, n, ld, dt, None if r is None else R(r), u, token, prob, None)

    for kw in (dict(dt=3), dict(m=-1), dict(n=0), dict(m=2, ld=99), dict(r=None), dict(u=4098),
               dict(token=4097), dict(prob=4098), dict(logits=None), dict(logits=4098),
               dict(u=None), dict(token=None), dict(r=lbv._RulesArg(temperature_last=2)),
               dict(r=lbv._RulesArg(top_k=4097)),
               dict(m=2, r=lbv._RulesArg(mask=4096, mask_ld=3))):
        assert call(**kw) == INF, kw
    assert call(n=1 << 24, ld=1 << 24) == lbv.ERR_UNSUPPORTED
    assert call(m=0, logits=None, u=None, token=None) == lbv.OK


def test_frequencies(L):
    f = lbv.rope_frequencies(64, 10000.0)
    want = 10000.0 ** (-2.0 * np.arange(32) / 64)
    assert np.allclose(f, want, rtol=1e-14)
    assert np.allclose(lbv.rope_frequencies(64, 10000.0, lbv.ROPE_LINEAR, 4.0), want / 4, rtol=1e-14)
    parts = lbv.rope_frequencies(64, 10000.0, lbv.ROPE_BY_PARTS, 8.0, 4096, 1.0, 32.0)
    turns = 4096 * want / (2 * np.pi)
    assert np.allclose(parts[turns >= 32], want[turns >= 32], rtol=1e-14)       # fast pairs stay
    assert np.allclose(parts[turns <= 1], want[turns <= 1] / 8, rtol=1e-14)     # slow ones stretch
    mid = (turns > 1) & (turns < 32)
    assert mid.any() and np.all((parts[mid] < want[mid]) & (parts[mid] > want[mid] / 8))
    for bad in ((7, 1e4, 0, 1., 0., 1., 32.), (8, -1., 0, 1., 0., 1., 32.), (8, 1e4, 3, 1., 0., 1., 32.),
                (8, 1e4, 1, 0., 0., 1., 32.), (8, 1e4, 2, 8., 0., 1., 32.), (8, 1e4, 2, 8., 9., 5., 5.)):
        with pytest.raises(lbv.LbvError):
            lbv.rope_frequencies(*bad)


def test_oracle_rotation_by_hand():
    x = np.array([[[1.0, 2.0, 3.0, 4.0]]])
    quarter = np.array([np.pi / 2])
    y, _ = step.rotate(x, np.array([1]), quarter, False, 1.0)       # pair (0, 1), the rest stays
    assert np.allclose(y[0, 0], [-2, 1, 3, 4])
    y, _ = step.rotate(x, np.array([1]), np.array([np.pi / 2, np.pi]), False, 2.0)
    assert np.allclose(y[0, 0], [2 * -3, 2 * -2, 2 * 1, 2 * -4])
    y, _ = step.rotate(x, np.array([1]), np.array([np.pi / 2, np.pi]), True, 1.0)
    assert np.allclose(y[0, 0], [-2, 1, -3, -4])


def test_oracle_attention_by_hand():
    k = np.zeros((2, 2, 1, 2))
    v = np.zeros((2, 2, 1, 2))
    v[1, 0, 0] = [1, 0]         # position 0 (pages in the order 1, 0)
    v[1, 1, 0] = [0, 1]         # position 1
    v[0, 0, 0] = [9, 9]         # position 2: past the context
    q = np.ones((2, 1, 2))
    out, lse, *_ = step.attend(q, k, v, [0, 2], [2], np.array([[1, 0]]), 1.0)
    assert np.allclose(out[:, 0], [[1, 0], [.5, .5]])               # equal scores, causal
    assert np.allclose(lse[:, 0], [0, np.log(2)])
    out, lse, *_ = step.attend(q, k, v, [0, 2], [2], np.array([[1, 0]]), 1.0, tree=[0, 2])
    assert np.allclose(out[:, 0], [[0, 0], [0, 1]]) and lse[0, 0] == -np.inf


def test_oracle_sampling_by_hand():
    x = np.log(np.array([1.0, 4.0, 2.0, 1.0]))
    kept, w = step.sample_sets(x, top_k=3)
    assert list(kept) == [1, 2, 0] and np.allclose(w, [1, .5, .25])
    assert list(step.sample_sets(x, top_p=0.5)[0]) == [1]
    assert list(step.sample_sets(x, top_p=0.51)[0]) == [1, 2]
    assert list(step.sample_sets(x, min_p=0.3)[0]) == [1, 2]
    assert list(step.sample_sets(x, temperature=0.0)[0]) == [1]
    assert np.allclose(step.sample_sets(x, temperature=0.5, top_k=2, last=True)[1], [1, .25])
