"""CPU fp64 oracle of the 4-bit weight and of the operators on sorted tokens.  TEST
INFRASTRUCTURE ONLY (as dora_oracle, and sharing no code with the HIP path).

The format: e2m1 codes (sign, 2 exponent bits with bias 1, 1 fraction bit: 0, 0.5, 1,
1.5, 2, 3, 4, 6 and their negatives) in blocks of 32 columns of a row, each with a
power of two 2^e, e the smallest whole number in [-23, 13] for which the block's
largest magnitude is at most 7 * 2^e (13 where none is).  A stored value is the e2m1
value nearest to v * 2^-e, the one of even code where two are equally near; a block
with a value that is not finite is NaN as a whole.

Sorting: slots with an adapter in order of (adapter, slot), then the others by slot.
"""
from __future__ import annotations

import numpy as np



def _value(c: int) -> float:
    """The value of a code, from the format's definition."""
    sign, ex, half = -1.0 if c & 8 else 1.0, (c >> 1) & 3, 0.5 * (c & 1)
    return sign * (half if ex == 0 else (1 + half) * 2.0 ** (ex - 1))


E2M1 = np.array([_value(c) for c in range(16)])
NAN_BYTE = 255


def block_exponent(amax: float) -> int:
    e = -23
    while e < 13 and amax > 7.0 * 2.0**e:
        e += 1
    return e


def nearest_code(v: np.ndarray) -> np.ndarray:
    """The e2m1 code nearest to each finite v, ties to the even code, 6 at most."""
    a = np.minimum(np.abs(v), 6.0)
    d = np.abs(a[..., None] - E2M1[:8])
    best = d.min(axis=-1, keepdims=True)
    near = d == best  # one or two of them
    even = near & (np.arange(8) % 2 == 0)
    pick = np.where(even.any(axis=-1), even.argmax(axis=-1), near.argmax(axis=-1))
    return (pick | np.where(np.signbit(v), 8, 0)).astype(np.uint8)


def blocks(W: np.ndarray):
    """(codes [out x P], exponent bytes [out x P / 32]) of W, P = in rounded up to 64."""
    out, in_ = W.shape
    P = -(-in_ // 64) * 64
    v = np.zeros((out, P))
    v[:, :in_] = W
    v = v.reshape(out, P // 32, 32)
    bad = ~np.isfinite(v).all(axis=2)
    amax = np.where(bad, 0.0, np.abs(np.where(np.isfinite(v), v, 0.0)).max(axis=2))
    e = np.vectorize(block_exponent, otypes=[np.int64])(amax) if amax.size else np.zeros(amax.shape, np.int64)
    c = nearest_code(np.where(bad[:, :, None], 0.0, v) * 2.0 ** -e[:, :, None].astype(np.float64))
    return c.reshape(out, P), np.where(bad, NAN_BYTE, e + 127).astype(np.uint8)


def held(W: np.ndarray) -> np.ndarray:
    """The fp64 values that W is held as."""
    c, e = blocks(W)
    s = np.where(e == NAN_BYTE, np.nan, 2.0 ** (e.astype(np.float64) - 127))
    return (E2M1[c] * np.repeat(s, 32, axis=1))[:, : W.shape[1]]


def pack(W: np.ndarray):
    """(q, e) in the layout of tiles of 32 x 64, byte by byte."""
    out, in_ = W.shape
    rt, ct = -(-out // 32), -(-in_ // 64)
    full = np.zeros((rt * 32, ct * 64))
    full[:out, :in_] = W
    c, ex = blocks(full)
    q, e = np.zeros((rt, ct, 1024), np.uint8), np.zeros((rt, ct, 64), np.uint8)
    for row in range(32):
        g, i = divmod(row, 8)
        for b in range(2):
            codes = c[row::32].reshape(rt, ct, 2, 16, 2)[:, :, b]
            at = 128 * i + 32 * g + 16 * (b ^ (i // 2 % 2))
            q[:, :, at : at + 16] = codes[..., 0] | codes[..., 1] << 4
            e[:, :, 32 * b + 8 * g + 2 * (i % 4) + i // 4] = ex[row::32].reshape(rt, ct, 2)[:, :, b]
    return q, e


# ------------------------------------------------------------------ sorted tokens


def sort(ids: np.ndarray, n: int):
    """(order, place, bounds) of ids [T x k]."""
    T, k = ids.shape
    flat = [int(v) if 0 <= v < n else n for v in ids.reshape(-1)]
    slots = sorted(range(T * k), key=lambda s: (flat[s], s))
    order, place = np.zeros(T * k, np.int64), np.zeros(T * k, np.int64)
    for p, s in enumerate(slots):
        has = flat[s] < n
        order[p], place[s] = (s, p) if has else (~s, ~p)
    bounds = np.array([sum(1 for f in flat if f < a) for a in range(n + 1)], np.int64)
    return order, place.reshape(T, k), bounds


def gather(x: np.ndarray, place: np.ndarray) -> np.ndarray:
    rows = np.zeros((place.size, x.shape[1]))
    for t in range(place.shape[0]):
        for p in place[t]:
            if p >= 0:
                rows[p] = x[t]
    return rows


def combine(rows, weights, place, base):
    y = np.zeros((place.shape[0], rows.shape[1])) if base is None else base.copy()
    for t in range(place.shape[0]):
        for j, p in enumerate(place[t]):
            if p >= 0:
                y[t] += (1.0 if weights is None else weights[t, j]) * rows[p]
    return y


def combine_bwd(dy, rows, weights, place):
    d_rows, d_w = np.zeros(rows.shape), np.zeros(place.shape)
    for t in range(place.shape[0]):
        for j, p in enumerate(place[t]):
            if p >= 0:
                d_rows[p] = (1.0 if weights is None else weights[t, j]) * dy[t]
                d_w[t, j] = dy[t] @ rows[p]
    return d_rows, d_w
