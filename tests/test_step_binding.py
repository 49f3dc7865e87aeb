"""CPU tests of what the Python binding refuses before anything reaches the
device: tensors are stood in for by objects with a tensor's attributes."""
import ctypes

import pytest

import few_row_packed_gb300 as lbv

torch = pytest.importorskip("torch")


class Fake:
    """A device tensor as the binding looks at it (device -1: host memory)."""

    def __init__(self, shape, stride=None, dtype=torch.int32, device=0):
        self.shape, self.dtype = tuple(shape), dtype
        if stride is None:
            stride, n = [], 1
            for s in reversed(self.shape):
                stride.insert(0, n)
                n *= s
        self._stride = tuple(stride)
        self.index, self.device, self.is_cuda = device, f"device {device}", device >= 0

    def get_device(self):
        return self.index

    def element_size(self):
        return {torch.float16: 2, torch.uint8: 1, torch.int64: 8}.get(self.dtype, 4)

    def dim(self):
        return len(self.shape)

    def stride(self, i=None):
        return self._stride if i is None else self._stride[i]

    def numel(self):
        n = 1
        for s in self.shape:
            n *= s
        return n

    def is_contiguous(self):
        return self._stride == Fake(self.shape)._stride

    def data_ptr(self):
        return 4096


def batch(requests, pages, stride):
    return lbv.Batch(Fake([requests + 1]), Fake([requests]), Fake([requests, pages], stride), requests)


@pytest.mark.parametrize("requests, pages, stride", [
    (2, 5, (0, 1)),             # one row for all requests
    (4096, 64, (0, 1)),
    (3, 8, (4, 1)),             # rows that overlap
    (2, 8, (7, 1)),
    (2, 1, (0, 1)),
])
def test_batch_refuses_tables_whose_rows_overlap(requests, pages, stride):
    """The kernels address row r at r * stride: a stride below the row's length
    would have to be replaced by one that leaves the tensor."""
    with pytest.raises(lbv.LbvError) as e:
        batch(requests, pages, stride)
    assert e.value.status == lbv.ERR_INVALID_ARG


@pytest.mark.parametrize("requests, pages, stride, want", [
    (2, 5, (5, 1), 5), (2, 5, (9, 1), 9), (1, 5, (5, 1), 5),
    (1, 5, (0, 1), 5),          # one row: its stride is not used
    (1, 5, (1, 1), 5),
])
def test_batch_keeps_the_tables_stride(requests, pages, stride, want):
    b = batch(requests, pages, stride)
    assert (b.arg.table_stride, b.arg.table_pages, b.arg.requests) == (want, pages, requests)


def test_attend_test_wait_refusals():
    lbv.build()
    call = lbv.lib().lbv_attend_test_wait
    assert call(None, None, None, None, 1.0, 0, None, None, None, 0, -1, None) == lbv.ERR_INVALID_ARG
    assert "copies" in lbv.last_error()
    assert call(None, None, None, None, 1.0, 0, None, None, None, 0, 0, None) == lbv.ERR_INVALID_ARG
    assert "batch is NULL" in lbv.last_error()


@pytest.fixture()
def setup(monkeypatch):
    lbv.build()
    monkeypatch.setattr(lbv, "_device", lambda: 0)
    shape, half = [4, 16, 2, 64], torch.float16
    cache = lbv.KVCache(Fake(shape, dtype=half), Fake(shape, dtype=half))
    return cache, batch(1, 4, (4, 1))


def refused(call, status=lbv.ERR_INVALID_ARG):
    """A refusal of the binding's own: the library, which has no device here, was not reached."""
    with pytest.raises(lbv.LbvError) as e:
        call()
    assert e.value.status == status
    assert "lbv_" not in str(e.value)


def test_cache_on_another_than_the_current_device_is_refused(monkeypatch):
    """Its handle, with the size and maps of the current device, would otherwise launch there."""
    lbv.build()
    shape, half = [4, 16, 2, 64], torch.float16
    k, v = (Fake(shape, dtype=half, device=1) for _ in range(2))
    monkeypatch.setattr(lbv, "_device", lambda: 0)
    refused(lambda: lbv.KVCache(k, v))
    monkeypatch.setattr(lbv, "_device", lambda: 1)
    assert lbv.KVCache(k, v).device == 1


@pytest.mark.parametrize("device", [1, -1])
def test_tensors_on_another_device_are_refused(setup, device):
    cache, b = setup
    half, f32, i32 = torch.float16, torch.float32, torch.int32
    shape = [4, 16, 2, 64]
    refused(lambda: lbv.KVCache(Fake(shape, dtype=half, device=device), Fake(shape, dtype=half)))
    refused(lambda: lbv.KVCache(Fake(shape, dtype=half), Fake(shape, dtype=half, device=device)))
    for which in range(3):
        at = [device if i == which else 0 for i in range(3)]
        refused(lambda: lbv.Batch(Fake([2], device=at[0]), Fake([1], device=at[1]), Fake([1, 4], device=at[2]), 1))
    rope = lbv.Rope(lbv.rope_frequencies(64))
    if device > 0:
        other = lbv.Batch(*(Fake(s, device=device) for s in ([2], [1], [1, 4])), 1)
        row = Fake([1, 2, 64], dtype=half)
        refused(lambda: lbv.rope_append(rope, other, cache, None, row, row, None))
        refused(lambda: lbv.attend(cache, other, row, row, 1.0))
    for which in range(5):
        at = [device if i == which else 0 for i in range(5)]
        q, k, v, out = (Fake([1, 2, 64], dtype=half, device=i) for i in at[:4])
        refused(lambda: lbv.rope_append(rope, b, cache, q, k, v, out, positions=Fake([1], device=at[4])))
    for which in range(5):
        at = [device if i == which else 0 for i in range(5)]
        q, out = (Fake([1, 2, 64], dtype=half, device=i) for i in at[:2])
        refused(lambda: lbv.attend(cache, b, q, out, 1.0, tree=Fake([1], dtype=torch.int64, device=at[2]),
                                   lse=Fake([1, 2], dtype=f32, device=at[3]),
                                   workspace=Fake([1 << 26], dtype=torch.uint8, device=at[4])),
                lbv.ERR_WORKSPACE if which == 4 else lbv.ERR_INVALID_ARG)
    for which in range(9):
        at = [device if i == which else 0 for i in range(9)]
        f = [Fake([3], dtype=f32, device=i) for i in at[:5]]
        w = [Fake([3], dtype=i32, device=i) for i in at[5:7]]
        refused(lambda: lbv.sample(Fake([3, 50], dtype=f32, device=at[7]), f[0], w[0], prob=f[1], temperature=f[2],
                                   top_k=w[1], top_p=f[3], min_p=f[4], mask=Fake([3, 2], device=at[8])))


def test_workspace_that_repeats_its_bytes_is_refused(setup):
    cache, b = setup
    q = Fake([1, 2, 64], dtype=torch.float16)
    refused(lambda: lbv.attend(cache, b, q, q, 1.0, workspace=Fake([1 << 26], (0,), torch.uint8)),
            lbv.ERR_WORKSPACE)


@pytest.mark.parametrize("pages, strides", [
    # 2^31 pages of 2^34 elements: their extent wraps 64 bits, and tokens and pages overlap
    (2 ** 31 - 1, (2 ** 34, 2 ** 37, 128)),
    (2 ** 31 - 1, (2 ** 37, 256, 128)),
])
def test_cache_whose_extent_passes_64_bits_is_refused(pages, strides):
    lbv.build()
    h = ctypes.c_void_p()
    st = lbv.lib().lbv_kv_cache_create(4096, 8192, pages, 16, 2, 128, *strides, lbv.F16, ctypes.byref(h))
    assert st == lbv.ERR_INVALID_ARG and not h.value
