"""Plain 64-bit reference of the quantised key/value cache (numpy only).

Written from the definitions: a block of 32 values shares one power of two,
its codes are the nearest representable values (ties to the even code), and
attention is softmax(scale * q k^T) v over the values that the codes stand
for.  Shares no code with the GPU path.
"""
from __future__ import annotations

import math

import numpy as np

E4M3, E5M2, E2M1 = 0, 1, 2
FLOOR, CEIL, NEAREST = 0, 1, 2
BLOCK = 32
#: exponent bits, mantissa bits, bias, largest finite value
_FORMAT = {E4M3: (4, 3, 7, 448.0), E5M2: (5, 2, 15, 57344.0), E2M1: (2, 1, 1, 6.0)}


def grid(fmt: int) -> np.ndarray:
    """The finite magnitudes in code order."""
    ebits, mbits, bias, top = _FORMAT[fmt]
    got = []
    for code in range(1 << (ebits + mbits)):
        f, m = code >> mbits, code & ((1 << mbits) - 1)
        v = math.ldexp(m, 1 - bias - mbits) if f == 0 else math.ldexp((1 << mbits) + m, f - bias - mbits)
        if v <= top:
            got.append(v)
    return np.array(got)


def _exponent(amax: float, fmt: int, rule: int, headroom: int = 0) -> int:
    if amax == 0:
        return -127
    top = _FORMAT[fmt][3]
    mu, k = math.frexp(amax)
    mu, k = 2 * mu, k - 1                          # amax = mu * 2^k, mu in [1, 2)
    tmu, tk = math.frexp(top)
    tmu, tk = 2 * tmu, tk - 1
    e = k - tk
    if rule == CEIL and mu > tmu:
        e += 1
    if rule == NEAREST and 2 * mu * mu < tmu * tmu:    # log2(amax / top) below the middle
        e -= 1
    return min(127, max(-127, e + headroom))


def encode(x: np.ndarray, fmt: int, rule: int = FLOOR, headroom: int = 0):
    """x [..., D] -> (codes uint8 [..., D], one per element, E8M0 uint8 [..., D / 32])."""
    x = np.asarray(x, dtype=np.float64)
    g = grid(fmt)
    mids = (g[1:] + g[:-1]) / 2
    sign_bit = 8 if fmt == E2M1 else 128
    b = x.reshape(*x.shape[:-1], -1, BLOCK)
    finite = np.isfinite(b).all(-1)
    amax = np.where(finite, np.abs(np.where(np.isfinite(b), b, 0)).max(-1), 0)
    e = np.vectorize(lambda a: _exponent(a, fmt, rule, headroom), otypes=[np.int64])(amax)
    m = np.abs(np.where(finite[..., None], b, 0)) * np.exp2(-e.astype(np.float64))[..., None]
    low = np.searchsorted(mids, m)                 # on a middle: the lower neighbour
    at = np.minimum(low, len(mids) - 1)
    tie = (low < len(mids)) & (m == mids[at])
    code = low + (tie & (low % 2 == 1))
    code = np.where(finite[..., None], code, sign_bit - 1) | np.where(np.signbit(b), sign_bit, 0)
    return code.reshape(x.shape).astype(np.uint8), np.where(finite, e + 127, 255).astype(np.uint8)


def pack(codes: np.ndarray, fmt: int) -> np.ndarray:
    return codes if fmt != E2M1 else codes[..., 0::2] | (codes[..., 1::2] << 4)


def unpack(packed: np.ndarray, fmt: int) -> np.ndarray:
    if fmt != E2M1:
        return packed
    out = np.empty((*packed.shape[:-1], 2 * packed.shape[-1]), dtype=np.uint8)
    out[..., 0::2], out[..., 1::2] = packed & 15, packed >> 4
    return out


def decode(packed: np.ndarray, e8m0: np.ndarray, fmt: int) -> np.ndarray:
    """Packed codes and E8M0 bytes -> float64 values (E8M0 0xFF: NaN)."""
    ebits, mbits = _FORMAT[fmt][:2]
    g = np.full(1 << (ebits + mbits), np.nan)
    v = grid(fmt)
    g[:len(v)] = v
    if fmt == E5M2:
        g[len(v)] = np.inf
    table = np.concatenate([g, -g])
    scale = np.exp2(e8m0.astype(np.float64) - 127)
    scale[e8m0 == 255] = np.nan
    return table[unpack(packed, fmt)] * np.repeat(scale, BLOCK, axis=-1)


def attention(q: np.ndarray, k: np.ndarray, v: np.ndarray, scale: float, window: int = 0, hidden=None):
    """One sequence, one key/value head: q [n, G, D], k and v [len, D] ->
    (out [n, G, D], log of the softmax sum [n, G]).  hidden: bool [len], keys
    that no query sees."""
    n, length = q.shape[0], k.shape[0]
    out = np.zeros(q.shape)
    lse = np.full(q.shape[:2], -np.inf)
    for i in range(n):
        pos = length - n + i
        j = np.arange(length)
        seen = j <= pos
        if window:
            seen &= j > pos - window
        if hidden is not None:
            seen &= ~hidden
        if not seen.any():
            continue
        s = scale * (q[i].astype(np.float64) @ k[seen].T)
        top = s.max(-1, keepdims=True)
        top = np.where(np.isfinite(top), top, 0)
        p = np.exp(s - top)
        total = p.sum(-1, keepdims=True)
        out[i] = p @ v[seen] / total
        lse[i] = (top + np.log(total))[:, 0]
    return out, lse
