"""CPU tests of the 4-bit cache, the sinks and the moves of a cache's contents: refused
arguments of the C ABI and of the binding, and the oracles against hand-worked values."""
import ctypes

import numpy as np
import pytest

import few_row_packed_gb300 as lbv
from oracle import kv4, step
from test_step_abi import batch as batch_arg
from test_step_abi import rows
from test_step_binding import Fake, batch, refused

torch = pytest.importorskip("torch")
INV, P, R = lbv.ERR_INVALID_ARG, ctypes.c_void_p, ctypes.byref


@pytest.fixture(scope="module")
def L():
    lbv.build()
    return lbv.lib()


def create(L, data=4096, pages=4, page_size=16, heads=2, dim=128, dtype=lbv.F16):
    h = P()
    return L.lbv_kv_cache4_create(data, pages, page_size, heads, dim, dtype, R(h)), h


@pytest.mark.parametrize("kw, want", [
    (dict(data=None), INV), (dict(data=4112), INV), (dict(pages=0), INV), (dict(heads=0), INV),
    (dict(heads=70000), INV), (dict(dtype=lbv.F32), INV), (dict(dtype=7), INV),
    (dict(page_size=24), lbv.ERR_UNSUPPORTED), (dict(page_size=4), lbv.ERR_UNSUPPORTED),
    (dict(page_size=2048), lbv.ERR_UNSUPPORTED), (dict(dim=96), lbv.ERR_UNSUPPORTED), (dict(dim=256), lbv.ERR_UNSUPPORTED),
])
def test_cache4_refusals(L, kw, want):
    st, h = create(L, **kw)
    assert st == want and not h.value
    assert "lbv_kv_cache4_create" in lbv.last_error()


def test_cache4_page_bytes(L):
    assert L.lbv_kv_cache4_create(4096, 1, 16, 1, 64, 0, None) == INV
    assert lbv.kv_cache4_page_bytes(64, 8, 128) == 64 * 8 * 144
    assert lbv.kv_cache4_page_bytes(1024, 65535, 128) == 1024 * 65535 * 144
    for bad in ((12, 8, 128), (64, 0, 128), (64, 8, 80), (2048, 1, 64), (64, 65536, 64)):
        assert L.lbv_kv_cache4_page_bytes(*bad) == 0
        with pytest.raises(lbv.LbvError):
            lbv.kv_cache4_page_bytes(*bad)


def test_moves_refusals(L):
    none = P()
    b, k = batch_arg(), rows()
    read, keep, copy = L.lbv_kv_read, L.lbv_kv_keep, L.lbv_kv_copy_pages
    assert read(None, none, R(k), R(k), None) == INV
    assert read(R(b), none, None, None, None) == INV and "NULL" in lbv.last_error()
    for bad in (dict(data=None), dict(data=4097), dict(heads=0), dict(dtype=5)):
        assert read(R(b), none, R(rows(**bad)), None, None) == INV, bad
        assert read(R(b), none, None, R(rows(**bad)), None) == INV, bad
    assert read(R(b), none, R(k), R(k), None) == INV and "cache is NULL" in lbv.last_error()
    assert keep(None, none, 4096, None, None) == INV
    for kept, left in ((None, None), (4100, None), (4096, 4098)):
        assert keep(R(b), none, kept, left, None) == INV and "kept" in lbv.last_error()
    assert keep(R(b), none, 4096, 8192, None) == INV and "cache is NULL" in lbv.last_error()
    for src, dst, n in ((None, 4096, 1), (4096, None, 1), (4098, 4096, 1), (4096, 4097, 1), (4096, 4096, -1)):
        assert copy(none, src, dst, n, None) == INV and "count" in lbv.last_error()
    assert copy(none, 4096, 4096, 1, None) == INV and "cache is NULL" in lbv.last_error()
    q = rows()
    call = L.lbv_attend_sinks
    assert call(none, R(b), R(q), R(q), 1.0, 5, 2, None, None, None, 0, None) == INV
    assert "lbv_attend_sinks" in lbv.last_error()


@pytest.fixture()
def setup(monkeypatch):
    lbv.build()
    monkeypatch.setattr(lbv, "_device", lambda: 0)
    n = lbv.kv_cache4_page_bytes(16, 2, 64)
    return lbv.KVCache4(Fake([4, n], dtype=torch.uint8), 16, 2, 64, torch.float16), batch(1, 4, (4, 1)), n


def test_binding_refuses_other_bytes(setup, monkeypatch):
    n, u8, half = setup[2], torch.uint8, torch.float16
    for data in (Fake([4, n + 1], dtype=u8), Fake([4, n], dtype=torch.int32), Fake([4 * n], dtype=u8),
                 Fake([4, n], (2 * n, 1), u8), Fake([4, n], dtype=u8, device=-1), Fake([4, n], dtype=u8, device=1)):
        refused(lambda: lbv.KVCache4(data, 16, 2, 64, half))
    refused(lambda: lbv.KVCache4(Fake([4, n], dtype=u8), 16, 2, 80, half), lbv.ERR_UNSUPPORTED)
    with pytest.raises(lbv.LbvError):
        lbv.KVCache4(Fake([4, n], dtype=u8), 16, 2, 64, torch.float32)


@pytest.mark.parametrize("device", [1, -1])
def test_binding_refuses_other_devices(setup, device):
    cache, b, _ = setup
    half, i32, i64 = torch.float16, torch.int32, torch.int64
    row, away = Fake([1, 2, 64], dtype=half), Fake([1, 2, 64], dtype=half, device=device)
    refused(lambda: lbv.kv_read(b, cache, away, row))
    refused(lambda: lbv.kv_read(b, cache, row, away))
    refused(lambda: lbv.kv_keep(b, cache, Fake([1], dtype=i64, device=device)))
    refused(lambda: lbv.kv_keep(b, cache, Fake([1], dtype=i64), Fake([1], dtype=i32, device=device)))
    pages = Fake([3], dtype=i32)
    refused(lambda: lbv.kv_copy_pages(cache, Fake([3], dtype=i32, device=device), pages))
    refused(lambda: lbv.kv_copy_pages(cache, pages, Fake([3], dtype=i32, device=device)))
    if device > 0:
        other = lbv.Batch(*(Fake(s, device=device) for s in ([2], [1], [1, 4])), 1)
        refused(lambda: lbv.kv_read(other, cache, row, row))
        refused(lambda: lbv.kv_keep(other, cache, Fake([1], dtype=i64)))
        refused(lambda: lbv.attend(cache, other, row, row, 1.0, window=4, sinks=2))


def test_binding_refuses_sizes_and_types(setup):
    cache, b, _ = setup
    half, i32, i64 = torch.float16, torch.int32, torch.int64
    refused(lambda: lbv.kv_read(b, cache, Fake([0, 2, 64], dtype=half), None))
    refused(lambda: lbv.kv_read(b, cache, Fake([1, 2, 32], dtype=half), None))
    refused(lambda: lbv.kv_keep(b, cache, None))
    refused(lambda: lbv.kv_keep(b, cache, Fake([1], dtype=i32)))
    refused(lambda: lbv.kv_keep(b, cache, Fake([0], dtype=i64)))
    refused(lambda: lbv.kv_keep(b, cache, Fake([1], dtype=i64), Fake([1], dtype=i64)))
    refused(lambda: lbv.kv_copy_pages(cache, Fake([3]), Fake([2])))
    refused(lambda: lbv.kv_copy_pages(cache, Fake([3]), None))
    refused(lambda: lbv.kv_copy_pages(cache, Fake([3], dtype=i64), Fake([3], dtype=i64)))
    refused(lambda: lbv.kv_copy_pages(cache, Fake([3], (2,)), Fake([3])))


def test_oracle_layout_by_hand():
    raw = kv4.pack(np.arange(64) % 16)
    # 8 codes 0..7 in a word: 0, 2, 4, 6 from the lowest bits on, 1, 3, 5, 7 in the upper half
    assert raw[:4].tolist() == [0x20, 0x64, 0x31, 0x75]
    assert np.array_equal(kv4.unpack(raw), np.arange(64) % 16)
    # page of 128 slots, 2 heads of 128: chunks of 64 slots are 64 * 144 bytes
    assert kv4.page_bytes(128, 2, 128) == 128 * 2 * 144
    assert kv4.offsets(128, 2, 128, 0, 0, 0, 0) == (0, 8192)
    assert kv4.offsets(128, 2, 128, 1, 65, 1, 1) == (9216 * 3 + (3 * 64 + 1) * 32, 9216 * 3 + 8192 + (3 * 64 + 1) * 4)


def test_oracle_quantisation_by_hand():
    x = np.concatenate([[-1.0, 2.0, 0.09, 0.11], np.zeros(60)]).astype(np.float32)
    code, scale, bias = kv4.quantise(x, lambda v: v)
    assert (scale, bias) == (np.float32(3) * (np.float32(1) / np.float32(15)), np.float32(-1))
    assert code[:5].tolist() == [0, 15, 5, 6, 5]            # 5.45, 5.55 and 5 steps of 0.2 above -1
    assert kv4.quantise(np.full(64, 3.0), lambda v: v)[1] == 0


def test_oracle_sinks_by_hand():
    k, v = np.zeros((1, 8, 1, 2)), np.zeros((1, 8, 1, 2))
    v[0, :, 0, 0] = 2.0 ** np.arange(8)
    q = np.ones((1, 1, 2))
    seen = lambda **kw: step.attend(q, k, v, [0, 1], [8], np.array([[0]]), 1.0, **kw)[0][0, 0, 0]  # noqa: E731
    assert seen(window=2) == (64 + 128) / 2                     # positions 6 and 7
    assert np.isclose(seen(window=2, sinks=1), (1 + 64 + 128) / 3)
    assert np.isclose(seen(window=2, sinks=7), 255 / 8)
    assert np.isclose(seen(window=0, sinks=3), 255 / 8)
