"""Rotary positions, the quantized key/value cache and attention over it, in
plain numpy.  TEST INFRASTRUCTURE ONLY (see the package docstring).

The pages name 4-bit inference and batched generation as the deployment mode
of the quantized model (project page, inference features); what stands between
the q/k/v linears and the output linear there is the usual decoder attention:

  rotation  pair i of a head, (a, b), at position p becomes
            (a c - b s, b c + a s) with (c, s) = (cos, sin)(p f_i) * amplitude,
            f_i = base^(-2 i / rot); the pairs are (i, i + rot/2) or (2i, 2i+1).
  cache     a row x of one token and head, all in fp32 with top = max |x| and
            u = 1 / top:  int8: code = rint(x * (127 u)), scale = top * (1/127);
            4 bit: the level #{m : x u > m} over the fp32 midpoints m of the
            type's levels, scale = top.  top < 1e-30: zeros with scale 0; a row
            with an infinity or a NaN: scale NaN.
  attention query i of n new tokens stands at p = length - n + i and sees
            stored token j if j < length, j <= p (causal), j > p - window
            (window > 0); softmax over the seen ones of scale q.k, times v;
            nothing seen: zeros and a log-sum of -inf.

The cache's rule is stated in fp32, so its oracle works in fp32 (each operation
rounded); rotation and attention are fp64.
"""

from __future__ import annotations

import math

import numpy as np

from . import baselines

KV_TYPES = ("bf16", "int8", "nf4", "int4", "fp4")
TINY = np.float32(1e-30)


def frequencies(rot: int, base: float = 10000.0, scaling: str = "none", factor: float = 1.0, original: float = 0.0,
                low: float = 1.0, high: float = 32.0) -> np.ndarray:
    i = np.arange(rot // 2, dtype=np.float64)
    if scaling == "base":
        base = base * factor ** (rot / (rot - 2))
    f = base ** (-2.0 * i / rot)
    if scaling == "linear":
        f = f / factor
    if scaling == "bands":
        turns = original * f / (2.0 * math.pi)
        keep = np.clip((turns - low) / (high - low), 0.0, 1.0)
        f = keep * f + (1.0 - keep) * f / factor
    return f


def rope_table(positions: int, rot: int, amplitude: float = 1.0, **kw) -> np.ndarray:
    """fp64 [positions, rot/2, 2]."""
    angle = np.arange(positions, dtype=np.float64)[:, None] * frequencies(rot, **kw)
    return np.stack((np.cos(angle), np.sin(angle)), -1) * amplitude


def rotate(x, table, positions, layout: str = "half", inverse: bool = False) -> np.ndarray:
    """[tokens, heads, dim] in the arithmetic of x's and the table's type."""
    x = np.array(x)
    half = table.shape[1]
    c, s = (table[positions][:, None, :, k] for k in (0, 1))
    s = -s if inverse else s
    first, second = ((slice(0, half), slice(half, 2 * half)) if layout == "half"
                     else (slice(0, 2 * half, 2), slice(1, 2 * half, 2)))
    a, b = x[..., first].copy(), x[..., second].copy()
    x[..., first] = a * c - b * s
    x[..., second] = b * c + a * s
    return x


def _levels(kind):
    """(fp32 levels ascending, their codes); codes that are never produced left out."""
    table = baselines.type_table(kind)
    codes = [c for c in range(16) if kind == "nf4" or c != 8]
    codes.sort(key=lambda c: float(table[c]))
    return table[codes], np.array(codes, dtype=np.uint8)


def quantize_rows(x, kind: str):
    """Rows (last axis) of fp32 x -> (codes one per element, scale per row)."""
    x = np.asarray(x, dtype=np.float32)
    top = np.max(np.abs(x), axis=-1)
    odd = ~np.isfinite(x).all(axis=-1)
    fine = (top >= TINY) & ~odd
    unit = np.divide(np.float32(1), top, out=np.zeros_like(top), where=fine)
    if kind == "int8":
        y = np.rint(np.where(odd[..., None], np.float32(0), x) * (unit * np.float32(127))[..., None])
        codes = np.clip(y, -127, 127).astype(np.int8)
        scale = np.where(fine, top * np.float32(1 / 127), np.float32(0))
    else:
        lv, order = _levels(kind)
        mids = ((lv[1:].astype(np.float64) + lv[:-1].astype(np.float64)) / 2).astype(np.float32)
        y = np.where(odd[..., None], np.float32(0), x) * unit[..., None]
        codes = order[np.searchsorted(mids, y, side="left")]
        scale = np.where(fine, top, np.float32(0))
    return codes, np.where(odd, np.float32("nan"), scale).astype(np.float32)


def stored_values(codes, scale, kind: str) -> np.ndarray:
    """fp32 values that codes (one per element) and scales stand for."""
    if kind == "int8":
        return codes.astype(np.float32) * scale[..., None]
    return baselines.type_table(kind)[codes] * scale[..., None]


def seen(n: int, length: int, causal: bool = True, window: int = 0) -> np.ndarray:
    """[n, length] truth values."""
    p = np.arange(length - n, length)[:, None]
    j = np.arange(length)[None]
    ok = np.ones((n, length), dtype=bool)
    if causal:
        ok &= j <= p
    if window > 0:
        ok &= j > p - window
    return ok


def attend(q, k, v, scale: float, causal: bool = True, window: int = 0):
    """One sequence: q [n, Hq, D], k and v [length, H, D] -> (out [n, Hq, D],
    lse [n, Hq], mass [n, Hq, D]), fp64; mass = sum_j w_j |v_j|, the scale of
    the output's rounding errors."""
    q, k, v = (np.asarray(t, dtype=np.float64) for t in (q, k, v))
    n, hq, d = q.shape
    length, h = k.shape[:2]
    out, mass = np.zeros((n, hq, d)), np.zeros((n, hq, d))
    lse = np.full((n, hq), -np.inf)
    ok = seen(n, length, causal, window)
    for x in range(hq):
        s = scale * (q[:, x] @ k[:, x // (hq // h)].T) if length else np.zeros((n, 0))
        for i in range(n):
            js = np.nonzero(ok[i])[0]
            if js.size == 0:
                continue
            t = s[i, js]
            top = t.max()
            w = np.exp(t - top)
            total = w.sum()
            lse[i, x] = top + math.log(total)
            out[i, x] = (w / total) @ v[js, x // (hq // h)]
            mass[i, x] = (w / total) @ np.abs(v[js, x // (hq // h)])
    return out, lse, mass
