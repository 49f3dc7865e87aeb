"""A batch over a cache held in 4 bits whose pages are in no order, for the GPU
tests: bytes made on the host, and the values they stand for."""
import numpy as np
import torch

import few_row_packed_gb300 as lbv
from oracle import kv4

DT = {"f16": torch.float16, "bf16": torch.bfloat16, "f32": torch.float32}
UNIT = {"f16": 2.0 ** -11, "bf16": 2.0 ** -8}       # half an ulp, relative
TINY = {"f16": 2.0 ** -25, "bf16": 2.0 ** -134}     # half a subnormal step


def f64(t):
    return t.double().cpu().numpy()


def round16(x, dtype):
    """x rounded to the 16-bit type, as fp64."""
    return torch.as_tensor(np.asarray(x, np.float32)).to(DT[dtype]).double().numpy()


def words16(x, dtype):
    """The 16-bit patterns of values of the type."""
    return torch.as_tensor(np.asarray(x, np.float32)).to(DT[dtype]).view(torch.int16).numpy().view(np.uint16)


def values(data, page, heads, dim, dtype):
    """Bytes [pages, page_bytes] -> keys and values [pages, page, heads, dim] in fp64."""
    data = np.ascontiguousarray(data)
    out = np.zeros((2, data.shape[0], page, heads, dim))
    for slot in range(page):
        for h in range(heads):
            for which in range(2):
                for part in range(dim // 64):
                    c, s = kv4.offsets(page, heads, dim, h, slot, which, part)
                    raw = np.ascontiguousarray(data[:, c:c + 32]).view("<u4")
                    code = ((raw[..., None] >> kv4.BITS) & 15).reshape(-1, 64).astype(np.float64)
                    pair = torch.from_numpy(np.ascontiguousarray(data[:, s:s + 4])).view(DT[dtype]).double().numpy()
                    with np.errstate(invalid="ignore"):
                        v = code * pair[:, :1] + pair[:, 1:]
                    out[which, :, slot, h, part * 64:(part + 1) * 64] = round16(v, dtype)
    return out


class Setup4:
    """As the setup of the 16-bit tests; unused slots hold NaN scales."""

    def __init__(self, q_len, kv_len, kv_heads=2, dim=128, dtype="f16", page=16, seed=0, pad=0, spare=2):
        g = np.random.default_rng(seed)
        self.g = torch.Generator().manual_seed(seed)
        self.dtype, self.dim, self.page, self.heads = dtype, dim, page, kv_heads
        need = [max(0, -(-k // page)) for k in kv_len]
        self.pages = pages = sum(need) + spare
        order = g.permutation(pages).astype(np.int32)
        width = max(max(need), 1) + 1
        self.table = np.full((len(q_len), width), -1, np.int32)
        at = 0
        used = np.zeros((pages, page), bool)
        for r, n in enumerate(need):
            self.table[r, :n] = order[at:at + n]
            at += n
            for j in range(max(kv_len[r], 0)):
                used[self.table[r, j // page], j % page] = True
        self.used = used
        self.start = np.concatenate([[0], np.cumsum(q_len)]).astype(np.int32)
        self.kv_len = np.array(kv_len, np.int32)
        self.tokens = int(self.start[-1]) + pad
        data = g.integers(0, 256, (pages, kv4.page_bytes(page, kv_heads, dim)), dtype=np.uint8)
        for slot in range(page):
            for h in range(kv_heads):
                for which in range(2):
                    for part in range(dim // 64):
                        _, s = kv4.offsets(page, kv_heads, dim, h, slot, which, part)
                        scale, bias = 0.1 + 0.3 * g.random(pages), -1.5 + g.standard_normal(pages)
                        scale[~used[:, slot]] = np.nan
                        pair = np.stack((words16(scale, dtype), words16(bias, dtype)), -1)
                        data[:, s:s + 4] = pair.astype("<u2").view(np.uint8)
        self.data = torch.from_numpy(data).cuda()
        self.cache = lbv.KVCache4(self.data, page, kv_heads, dim, DT[dtype])
        self.batch = lbv.Batch(torch.from_numpy(self.start).cuda(), torch.from_numpy(self.kv_len).cuda(),
                               torch.from_numpy(self.table).cuda(), self.tokens)

    def values(self):
        """Keys and values as they are held now."""
        return values(self.data.cpu().numpy(), self.page, self.heads, self.dim, self.dtype)

    def rows(self, heads, dtype=None, scale=1.0):
        x = scale * torch.randn((self.tokens, heads, self.dim), generator=self.g)
        return x.to(DT[dtype or self.dtype]).cuda()
