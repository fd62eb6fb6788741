"""CPU fp64 oracle of the 8-bit operators.  TEST INFRASTRUCTURE ONLY (as
dora_oracle, and sharing no code with the HIP path).

The format: e4m3 values (sign, 4 exponent bits with bias 7, 3 fraction bits;
0x7f and 0xff are NaN, there is no infinity, the largest value is 448) in
blocks of 128, each with a power of two 2^e, e the smallest whole number >= -126
for which the block's largest finite magnitude is at most 448 * 2^e.  A stored
value is the e4m3 value nearest to v * 2^-e, the one with an even fraction where
two are equally near; a value that is not finite is NaN.

``held_rows`` and ``held_weight`` are the fp64 values that a matrix is held as;
the operators are the plain products of those values.
"""
from __future__ import annotations

import numpy as np

BLOCK = 128


def _table():
    """Every e4m3 byte's value, from the format's definition."""
    v = np.empty(256)
    for b in range(256):
        s, ex, fr = b >> 7, (b >> 3) & 15, b & 7
        if ex == 15 and fr == 7:
            v[b] = np.nan
        else:
            v[b] = (-1.0) ** s * ((fr / 8.0) * 2.0**-6 if ex == 0 else (1 + fr / 8.0) * 2.0 ** (ex - 7))
    return v


E4M3 = _table()
_POS = E4M3[:127]  # 0 .. 448 in order; the byte's lowest bit is the fraction's


def block_exponent(amax: float) -> int:
    e = -126
    while amax > 448.0 * 2.0**e:
        e += 1
    return e


def _exponents(amax: np.ndarray) -> np.ndarray:
    """block_exponent of every entry (a search over the exponents)."""
    lim = 448.0 * np.exp2(np.arange(-126, 128, dtype=np.float64))
    return np.searchsorted(lim, amax, side="left") - 126


def nearest_byte(v: np.ndarray) -> np.ndarray:
    """The e4m3 byte nearest to each v (|v| <= 448), ties to the even byte; NaN is 0x7f."""
    a = np.abs(np.where(np.isfinite(v), v, 0.0))
    hi = np.clip(np.searchsorted(_POS, a, side="left"), 0, 126)
    lo = np.maximum(hi - 1, 0)
    dl, dh = a - _POS[lo], _POS[hi] - a
    pick = np.where((dl < dh) | ((dl == dh) & (lo % 2 == 0)), lo, hi)
    out = (pick | np.where(np.signbit(v), 128, 0)).astype(np.uint8)
    return np.where(np.isfinite(v), out, np.uint8(0x7F))


def _padded(x: np.ndarray, rows: int, cols: int) -> np.ndarray:
    p = np.zeros((rows, cols))
    p[: x.shape[0], : x.shape[1]] = x
    return p


def _up(n, k):
    return -(-n // k) * k


def _amax(b, axis):
    return np.max(np.where(np.isfinite(b), np.abs(b), 0.0), axis=axis, initial=0.0)


def pack_rows(x: np.ndarray):
    """(bytes [T x P], exponent bytes [T x E]) of fp64 rows."""
    T, K = x.shape
    P = _up(K, BLOCK)
    b = _padded(x, T, P).reshape(T, P // BLOCK, BLOCK)
    e = _exponents(_amax(b, 2))
    q = nearest_byte(b * np.exp2(-e.astype(np.float64))[:, :, None]).reshape(T, P)
    eb = np.full((T, _up(P // BLOCK, 4)), 127, np.uint8)
    eb[:, : P // BLOCK] = e + 127
    return q, eb


def pack_weight(W: np.ndarray):
    o, i = W.shape
    O_, I_ = _up(o, BLOCK), _up(i, BLOCK)
    b = _padded(W, O_, I_).reshape(O_ // BLOCK, BLOCK, I_ // BLOCK, BLOCK)
    e = _exponents(_amax(b, (1, 3)))
    q = nearest_byte(b * np.exp2(-e.astype(np.float64))[:, None, :, None]).reshape(O_, I_)
    eb = np.full((O_ // BLOCK, _up(I_ // BLOCK, 4)), 127, np.uint8)
    eb[:, : I_ // BLOCK] = e + 127
    return q, eb


def held_rows(q: np.ndarray, eb: np.ndarray, cols: int) -> np.ndarray:
    s = np.exp2(eb[:, : q.shape[1] // BLOCK].astype(np.float64) - 127)
    return (E4M3[q] * np.repeat(s, BLOCK, axis=1))[:, :cols]


def held_weight(q: np.ndarray, eb: np.ndarray, rows: int, cols: int) -> np.ndarray:
    s = np.exp2(eb[:, : q.shape[1] // BLOCK].astype(np.float64) - 127)
    return (E4M3[q] * np.repeat(np.repeat(s, BLOCK, axis=0), BLOCK, axis=1))[:rows, :cols]


def linear(x, W):
    """y = x W^T of held values."""
    return x @ W.T


def linear_bwd(g, W):
    """dx = g W of held values."""
    return g @ W


def grad_a(dh, x):
    """d_A = d_h^T x, x the held values."""
    return dh.T @ x
