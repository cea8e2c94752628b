"""The operators around a training step beside the linears, in fp64: the gated
feed-forward block, the softmax cross entropy over a vocabulary, and the global
gradient norm with clipping.  TEST INFRASTRUCTURE ONLY (see the package
docstring).

Readings:
  R29  Gated block: H = act(G) * U with G and U the adapted linears of R7 over
       one input; act one of SiLU, GELU (erf) and GELU (tanh).  Gradients
       follow from H being a product: dG = dH act'(G) U, dU = dH act(G), then
       R8 for both linears, their dX summed.
  R30  Cross entropy: loss = lse - z_target per token, lse = log sum exp(z) over
       the head's rows; tokens with a negative target are not learned (loss,
       lse and gradient 0); the mean is over the learned tokens (0 if none).
       The head is frozen: only the input gets a gradient.
"""

from __future__ import annotations

import math

import numpy as np

from .lora import linear_bwd, linear_fwd

_erf = np.vectorize(math.erf, otypes=[np.float64])


def activation(g, act):
    """(act(g), act'(g)) in fp64."""
    g = np.asarray(g, dtype=np.float64)
    if act == "silu":
        s = 1.0 / (1.0 + np.exp(-g))
        return g * s, s * (1.0 + g * (1.0 - s))
    if act == "gelu":
        phi = 0.5 * (1.0 + _erf(g / math.sqrt(2.0)))
        return g * phi, phi + g * np.exp(-0.5 * g * g) / math.sqrt(2.0 * math.pi)
    if act == "gelu_tanh":
        c = math.sqrt(2.0 / math.pi)
        t = np.tanh(c * (g + 0.044715 * g ** 3))
        return 0.5 * g * (1.0 + t), 0.5 * (1.0 + t) + 0.5 * g * (1.0 - t * t) * c * (1.0 + 3 * 0.044715 * g * g)
    raise ValueError(act)


def gated_fwd(X, gate, up, alpha, r, act):
    """gate, up: (W' [N,K], A, B).  Returns (H, P1, P2, G, U, [XAg, XAu])."""
    G, XAg = linear_fwd(X, *gate, alpha, r)
    U, XAu = linear_fwd(X, *up, alpha, r)
    a, slope = activation(G, act)
    return a * U, slope * U, a, G, U, [XAg, XAu]


def gated_bwd(dH, X, gate, up, alpha, r, act):
    """Returns (dX, dAg, dBg, dAu, dBu)."""
    _, p1, p2, _, _, _ = gated_fwd(X, gate, up, alpha, r, act)
    dH = np.asarray(dH, dtype=np.float64)
    g = linear_bwd(dH * p1, X, *gate, alpha, r)
    u = linear_bwd(dH * p2, X, *up, alpha, r)
    return g[0] + u[0], g[1], g[2], u[1], u[2]


def head_loss(X, W, targets, dloss=None):
    """Returns (loss [T], lse [T], mean, dX [T,K], p [T,V])."""
    X, W = np.asarray(X, dtype=np.float64), np.asarray(W, dtype=np.float64)
    t = np.asarray(targets)
    z = X @ W.T
    top = z.max(1)
    e = np.exp(z - top[:, None])
    lse = top + np.log(e.sum(1))
    on = t >= 0
    rows = np.arange(len(t))
    at = np.where(on, t, 0)
    # The others' share, without the target: exact where the target is all but certain.
    rest = e.copy()
    rest[rows, at] = 0.0
    a = e[rows, at]
    loss = np.where(on, np.log1p(rest.sum(1) / a) if len(t) else 0.0, 0.0)
    p = e / e.sum(1, keepdims=True)
    n = max(int(on.sum()), 1)
    g = np.where(on, np.full(len(t), 1.0 / n) if dloss is None else np.asarray(dloss, dtype=np.float64), 0.0)
    q = rest / e.sum(1, keepdims=True)
    q[rows, at] = -q.sum(1)
    dX = g[:, None] * (q @ W)
    return loss, np.where(on, lse, 0.0), loss.sum() / n, dX, p


def clip(grads, max_norm):
    """(norm, clipped gradients) in fp64, the rule of R21."""
    grads = [np.asarray(g, dtype=np.float64) for g in grads]
    norm = math.sqrt(sum(float(np.sum(g * g)) for g in grads))
    c = min(1.0, max_norm / (norm + 1e-6)) if max_norm > 0 else 1.0
    return norm, [c * g for g in grads]


def multiplier(x):
    """A kept multiplier: 10 significant bits from 2^-30 to 2^33, multiples of
    2^-39 below, infinite from there on (ties away from zero)."""
    x = np.asarray(x, dtype=np.float64)
    _, e = np.frexp(np.abs(x))                     # |x| in [2^(e-1), 2^e)
    unit = np.ldexp(1.0, np.maximum(e - 10, -39))
    y = np.copysign(np.floor(np.abs(x) / unit + 0.5) * unit, x)
    return np.where(np.abs(y) >= 2.0 ** 33 - 2.0 ** 23, np.copysign(np.inf, x), y)
