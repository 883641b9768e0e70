"""Microscaled numbers in 64-bit numpy (test infrastructure): the format as include/fh_ops.h
states it, written from the definition, element tables and all."""
from __future__ import annotations

import numpy as np

TOP = {"mxfp8": 448.0, "mxfp4": 6.0}


def element_table(fmt: str) -> np.ndarray:
    """Value of every code."""
    if fmt == "mxfp4":
        pos = [0.0, 0.5, 1.0, 1.5, 2.0, 3.0, 4.0, 6.0]
        return np.array(pos + [-v for v in pos])
    v = np.empty(256)
    for code in range(256):
        s, e, f = code >> 7, (code >> 3) & 15, code & 7
        m = np.nan if (code & 127) == 127 else (f / 8 * 2.0 ** -6 if e == 0 else (1 + f / 8) * 2.0 ** (e - 7))
        v[code] = -m if s else m
    return v


def round_element(r: np.ndarray, fmt: str) -> np.ndarray:
    """Nearest element value to each r, ties to the even code."""
    tab = element_table(fmt)
    pos = tab[:127] if fmt == "mxfp8" else tab[:8]
    a = np.abs(r)
    hi = np.minimum(np.searchsorted(pos, a, side="left"), len(pos) - 1)
    lo = np.maximum(hi - 1, 0)
    dl, dh = a - pos[lo], pos[hi] - a
    code = np.where(dl < dh, lo, np.where(dh < dl, hi, np.where(lo % 2 == 0, lo, hi)))
    return np.where(np.signbit(r), -pos[code], pos[code])


def scale_exponent(amax: np.ndarray, fmt: str) -> np.ndarray:
    """Smallest e >= -127 with amax <= top * 2^e."""
    e = np.full(amax.shape, -127)
    ok = amax > 0
    f, x = np.frexp(np.where(ok, amax, 1.0) / TOP[fmt])   # f in [0.5, 1): amax / top = f * 2^x
    e = np.where(ok, np.where(f == 0.5, x - 1, x), e)
    return np.maximum(e, -127)


def quantize(x: np.ndarray, fmt: str):
    """(element values [M, K], scale bytes [M, K / 32]) of a float64 matrix."""
    M, K = x.shape
    b = x.astype(np.float64).reshape(M, K // 32, 32)
    bad = ~np.isfinite(b).all(-1)
    b = np.where(bad[..., None], 0.0, b)
    e = scale_exponent(np.abs(b).max(-1), fmt)
    v = round_element(b * 2.0 ** -e[..., None].astype(np.float64), fmt)
    return v.reshape(M, K), np.where(bad, 255, e + 127).astype(np.uint8)


def scale_values(byte: np.ndarray) -> np.ndarray:
    return np.where(byte == 255, np.nan, 2.0 ** (byte.astype(np.float64) - 127))


def values(elements: np.ndarray, byte: np.ndarray) -> np.ndarray:
    M, K = elements.shape
    return (elements.reshape(M, K // 32, 32) * scale_values(byte)[..., None]).reshape(M, K)


def offsets(M: int, K: int) -> np.ndarray:
    """Where each [row, block] scale byte lies."""
    r, k = np.arange(M)[:, None], np.arange(K // 32)[None, :]
    return (r // 128 * -(-K // 128) + k // 4) * 512 + r % 32 * 16 + r % 128 // 32 * 4 + k % 4


def scale_count(M: int, K: int) -> int:
    return -(-M // 128) * -(-K // 128) * 512


def tile(byte: np.ndarray, K: int) -> np.ndarray:
    flat = np.zeros(scale_count(byte.shape[0], K), dtype=np.uint8)
    flat[offsets(byte.shape[0], K)] = byte
    return flat


def unpack(data: np.ndarray, fmt: str) -> np.ndarray:
    """Element values of the code bytes."""
    if fmt == "mxfp8":
        return element_table(fmt)[data]
    codes = np.empty((data.shape[0], data.shape[1] * 2), dtype=np.uint8)
    codes[:, 0::2], codes[:, 1::2] = data & 15, data >> 4
    return element_table(fmt)[codes]


def read(q):
    """(element values, scale bytes, all scale bytes as they lie) of a library MXTensor."""
    data, flat = q.data.cpu().numpy(), q.scales.cpu().numpy()
    M, K = q.shape
    return unpack(data, q.fmt), flat[offsets(M, K)], flat


def padding(flat: np.ndarray, M: int, K: int) -> np.ndarray:
    """The scale bytes past the tensor."""
    used = np.zeros(flat.shape, dtype=bool)
    used[offsets(M, K)] = True
    return flat[~used]


def check_result(q, y: np.ndarray, tol: np.ndarray):
    """A microscaled result against float64 values y that the kernel knows to within tol: scales
    are those of some amax within tol, elements are off by the rounding (half a step of e4m3,
    2^-4 relative or half its smallest step 2^-9; of e2m1, 2^-2 relative or 1/4) and tol."""
    M, K = y.shape
    el, byte, flat = read(q)
    assert not padding(flat, M, K).any()
    blk = lambda t: t.reshape(M, K // 32, 32)  # noqa: E731
    amax, slack = np.abs(blk(y)).max(-1), blk(tol).max(-1)
    lo = scale_exponent(np.maximum(amax - slack, 0.0), q.fmt) + 127
    hi = scale_exponent(amax + slack, q.fmt) + 127
    assert ((byte >= lo) & (byte <= hi)).all()
    got = values(el, byte)
    unit = np.repeat(scale_values(byte), 32, axis=1)
    rel, step = (2.0 ** -4, 2.0 ** -10) if q.fmt == "mxfp8" else (2.0 ** -2, 0.25)
    allowed = np.maximum(rel * np.abs(y), step * unit) + 2 * tol
    assert (np.abs(got - y) <= allowed).all(), float((np.abs(got - y) - allowed).max())
