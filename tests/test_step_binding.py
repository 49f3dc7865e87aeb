"""CPU tests of what the Python binding refuses before anything reaches the
device: tensors are stood in for by objects with a tensor's attributes."""
import pytest

import few_row_packed_gb300 as lbv

torch = pytest.importorskip("torch")


class Fake:
    """A device tensor as the binding looks at it."""
    is_cuda = True

    def __init__(self, shape, stride=None, dtype=torch.int32):
        self.shape, self.dtype = tuple(shape), dtype
        if stride is None:
            stride, n = [], 1
            for s in reversed(self.shape):
                stride.insert(0, n)
                n *= s
        self._stride = tuple(stride)
        self.device = "cuda:0"

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
