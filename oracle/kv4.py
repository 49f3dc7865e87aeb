"""fp64 oracle of the paged cache held in 4 bits (test infrastructure only):
its layout and its values, from the definitions in include/lbv.h."""
from __future__ import annotations

import numpy as np

GROUP = 64
BITS = np.array([4 * (i // 2) + 16 * (i % 2) for i in range(8)], np.uint32)


def page_bytes(page, heads, dim):
    return page * heads * (dim // GROUP) * 72


def offsets(page, heads, dim, head, slot, which, part):
    """Bytes of a page where 64 elements have their codes, and their (scale, bias)."""
    size, parts = min(page, 64), dim // GROUP
    chunk = (head * (page // size) + slot // size) * size * parts * 72
    plane, at = which * parts + part, slot % size
    return chunk + (plane * size + at) * 32, chunk + 2 * parts * size * 32 + (plane * size + at) * 4


def pack(codes):
    """64 codes -> 32 bytes."""
    words = (np.asarray(codes, np.uint32).reshape(8, 8) << BITS).sum(1, dtype=np.uint32)
    return words.astype("<u4").view(np.uint8)


def unpack(raw):
    """32 bytes -> 64 codes."""
    return ((np.ascontiguousarray(raw).view("<u4")[:, None] >> BITS) & 15).reshape(64).astype(np.int64)


def quantise(x, round16):
    """Codes, scale and bias of 64 fp32 values, as the append defines them: fp32
    arithmetic; round16 rounds an fp32 number to the cache's dtype."""
    x = np.asarray(x, np.float32)
    f = np.float32
    bias, scale = f(round16(x.min())), f(round16(f(x.max() - x.min()) * (f(1) / f(15))))
    if scale < f(2.0 ** -126):
        return np.zeros(64, np.int64), f(0), bias
    code = np.rint((x - bias) * (f(1) / scale))
    return np.clip(code, 0, 15).astype(np.int64), scale, bias
