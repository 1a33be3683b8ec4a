"""fp64 CPU oracle of the 4-bit paged key/value cache -- TEST INFRASTRUCTURE ONLY.

The format and the operators as the header states them, in numpy and 64 bits, one value or
one row at a time where that is the plainest way to say it:

    m    = the value of largest magnitude of a group of 32 (the positive one of an equal pair)
    s    = -m / 8, rounded to 5 significant bits, ties to even
    code = clamp(rint(x / s), -8, 7) + 8, ties to even; it stands for (code - 8) * s

A group that holds a value that is not finite or above 2^120 stands for NaN, one whose values
are all below 2^-107 for zeros.  A scale of 2^118 or more in magnitude, which no group has, stands
for NaN too.
"""
from __future__ import annotations

import numpy as np

GROUP = 32


def scale_of(group: np.ndarray) -> float:
    """Scale of one group of 32 values (float64)."""
    if not np.all(np.isfinite(group)) or np.abs(group).max() > 2.0 ** 120:
        return float("nan")
    top = float(np.abs(group).max())
    if top < 2.0 ** -107:
        return 0.0
    m = top if top in group else -top
    mantissa, exponent = np.frexp(m)                 # 0.5 <= |mantissa| < 1
    return float(-np.ldexp(np.rint(mantissa * 32.0), exponent - 5 - 3))


def quantise(x: np.ndarray):
    """float64 [..., d] -> (codes uint8 [..., d] in 0..15, scales float64 [..., d/32])."""
    x = np.asarray(x, np.float64)
    g = x.reshape(-1, GROUP)
    scales = np.array([scale_of(row) for row in g])
    codes = np.full(g.shape, 8, np.uint8)
    for i, s in enumerate(scales):
        if np.isfinite(s) and s != 0.0:
            codes[i] = np.clip(np.rint(g[i] / s), -8, 7) + 8
    return codes.reshape(x.shape), scales.reshape(*x.shape[:-1], x.shape[-1] // GROUP)


def values(codes: np.ndarray, scales: np.ndarray) -> np.ndarray:
    """What codes [..., d] with scales [..., d/32] stand for (float64)."""
    s = np.asarray(scales, np.float64)
    s = np.where(np.abs(s) < 2.0 ** 118, s, np.nan)
    return (codes.astype(np.float64) - 8.0) * np.repeat(s, GROUP, axis=-1)


def pack(codes: np.ndarray) -> np.ndarray:
    """Codes [..., d] -> bytes [..., d/2], the even channel in the low half."""
    return (codes[..., 0::2] | (codes[..., 1::2] << 4)).astype(np.uint8)


def unpack(packed: np.ndarray) -> np.ndarray:
    codes = np.empty((*packed.shape[:-1], packed.shape[-1] * 2), np.uint8)
    codes[..., 0::2] = packed & 15
    codes[..., 1::2] = packed >> 4
    return codes


def place(pos: int, b: int, table, page_size: int, max_pages: int, num_pages: int):
    """(page, token in it) of a position of sequence b, or None where the cache has no place for it."""
    if pos < 0 or pos >= max_pages * page_size:
        return None
    page = b * max_pages + pos // page_size if table is None else int(table[b][pos // page_size])
    return (page, pos % page_size) if 0 <= page < num_pages else None


def attend(q, k, v, visible, scale):
    """One head: q [N, d], k and v [L, d], visible [N, L] (all float64) -> (O [N, d], LSE [N]).

    Keys that a query does not see take no part, whatever they hold."""
    o = np.zeros(q.shape)
    lse = np.full(q.shape[0], -np.inf)
    for i in range(q.shape[0]):
        seen = np.nonzero(visible[i])[0]
        if seen.size == 0:
            continue
        s = scale * (k[seen] @ q[i])
        m = s.max()
        p = np.exp(s - m)
        o[i] = (p @ v[seen]) / p.sum()
        lse[i] = m + np.log(p.sum())
    return o, lse


def visible_keys(n_q, q_len, key_len, positions, causal, window):
    """[n_q, positions]: query i of q_len stands at key_len - q_len + i."""
    i = np.arange(n_q)[:, None]
    j = np.arange(positions)[None, :]
    at = key_len - q_len + i
    seen = (j < key_len) & (i < q_len)
    if causal:
        seen &= j <= at
    if window >= 0:
        seen &= j >= at - window
    return seen
