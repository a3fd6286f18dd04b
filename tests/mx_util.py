"""The microscaled (MX) formats and operators in 64 bits, for the tests: a
plain restatement of the formulas on numpy arrays, written apart from the
CUDA code."""
from __future__ import annotations

import numpy as np
import torch

E4M3, E2M1 = 0, 1
MOST = {E4M3: 448.0, E2M1: 6.0}
TORCH = {0: torch.bfloat16, 1: torch.float16, 2: torch.float32}


def grid(fmt):
    """Values of the codes without their sign, in code order."""
    if fmt == E2M1:
        return np.array([0, 0.5, 1, 1.5, 2, 3, 4, 6])
    v = [m / 8 * 2.0 ** -6 for m in range(8)]
    v += [(1 + m / 8) * 2.0 ** (e - 7) for e in range(1, 16) for m in range(8)]
    return np.array(v[:127])  # the last code is NaN


def scale_code(amax, fmt):
    """Smallest c in [0, 254] with amax <= MOST 2^(c - 127); 255 for a value that is not finite."""
    tops = MOST[fmt] * 2.0 ** (np.arange(255) - 127.0)
    amax = np.asarray(amax, np.float64)
    c = np.searchsorted(tops, np.where(np.isfinite(amax), amax, 0.0))
    return np.where(np.isfinite(amax), c, 255).astype(np.int64)


def scale_value(code):
    return np.where(code == 255, np.nan, 2.0 ** (np.asarray(code, np.float64) - 127))


def quantize(x, fmt):
    """(codes [rows, cols] with the sign in the top bit, scale codes [rows, cols / 32])."""
    g = grid(fmt)
    sign = 128 if fmt == E4M3 else 8
    x = np.asarray(x, np.float64)
    b = x.reshape(x.shape[0], -1, 32)
    with np.errstate(invalid="ignore"):
        sc = scale_code(np.abs(b).max(axis=2), fmt)  # max passes NaN on
        t = np.abs(b) / scale_value(np.minimum(sc, 254))[..., None]
    t = np.where(sc[..., None] == 255, 0.0, t)
    mid = (g[1:] + g[:-1]) / 2
    at = np.searchsorted(mid, t)
    tie = (at < len(mid)) & (t == mid[np.minimum(at, len(mid) - 1)]) & (at % 2 == 1)
    c = at + tie + np.where(np.signbit(b), sign, 0)
    return np.where(sc[..., None] == 255, 0, c).reshape(x.shape), sc


def values(codes, sc, fmt):
    """fp64 values of codes and scale codes."""
    g = np.concatenate([grid(fmt), [np.nan]]) if fmt == E4M3 else grid(fmt)
    n = 128 if fmt == E4M3 else 8
    v = np.where(codes >= n, -1.0, 1.0) * g[codes % n]
    return (v.reshape(*sc.shape, 32) * scale_value(sc)[..., None]).reshape(codes.shape)


def pack(codes, fmt):
    """Codes as the library stores them."""
    if fmt == E4M3:
        return codes.astype(np.uint8)
    return (codes[..., 0::2] | codes[..., 1::2] << 4).astype(np.uint8)


def unpack(q, fmt):
    q = np.asarray(q).astype(np.int64)
    if fmt == E4M3:
        return q
    out = np.empty((*q.shape[:-1], q.shape[-1] * 2), np.int64)
    out[..., 0::2], out[..., 1::2] = q & 15, q >> 4
    return out


def pitch(cols):
    return -(-(cols // 32) // 16) * 16


def scale_rows(sc, fill=0):
    """Scale codes as rows of pitch bytes."""
    out = np.full((*sc.shape[:-1], pitch(sc.shape[-1] * 32)), fill, np.uint8)
    out[..., :sc.shape[-1]] = sc
    return out


class Matrix:
    """A random matrix [.., rows, cols] in microscaled form: `q`, `s` (uint8
    CUDA tensors as the library takes them) and `v`, its fp64 values."""

    def __init__(self, rng, shape, fmt, sigma=1.0):
        x = rng.standard_normal((int(np.prod(shape[:-1])), shape[-1])) * sigma
        c, sc = quantize(x, fmt)
        self.v = values(c, sc, fmt).reshape(shape)
        self.q = torch.from_numpy(pack(c, fmt)).view(*shape[:-1], -1).cuda()
        self.s = torch.from_numpy(scale_rows(sc)).view(*shape[:-1], -1).cuda()


def code_error(q, sc, n, slack):
    """Whether e4m3 codes and scale codes are right for values known to be
    n (1 + d), |d| <= slack: the scale is the one of a magnitude within the
    slack, the value within half a step (2^-4 relative, 2^-10 below the
    smallest normal) of n / scale.  Returns the worst excess (<= 0 is right)."""
    b = n.reshape(n.shape[0], -1, 32)
    amax = np.abs(b).max(axis=2)
    lo, hi = scale_code(amax * (1 - slack), E4M3), scale_code(amax * (1 + slack), E4M3)
    assert ((sc >= lo) & (sc <= hi)).all()
    t = b / scale_value(sc)[..., None]
    v = values(q, np.full_like(sc, 127), E4M3).reshape(b.shape)
    # half a step: 2^(floor(log2 |t|) - 4), at least 2^-10
    e = np.floor(np.log2(np.maximum(np.abs(t) * (1 + slack), 2.0 ** -6)))
    return float((np.abs(v - t) - 2.0 ** (e - 4) - slack * np.abs(t)).max())
