"""Pins of oracle/train.py against what does not depend on it: differences,
torch in fp64 on the CPU, and closed forms."""

import math

import numpy as np
import pytest
import torch

from oracle import train

RNG = np.random.Generator(np.random.PCG64(5))


@pytest.mark.parametrize("act", ["silu", "gelu", "gelu_tanh"])
def test_activations(act):
    g = np.concatenate((np.linspace(-12, 12, 241), [0.0, -30.0, 30.0]))
    a, slope = train.activation(g, act)
    t = torch.from_numpy(g).requires_grad_()
    ref = {"silu": torch.nn.functional.silu, "gelu": torch.nn.functional.gelu,
           "gelu_tanh": lambda x: torch.nn.functional.gelu(x, approximate="tanh")}[act](t)
    (d,) = torch.autograd.grad(ref.sum(), t)
    np.testing.assert_allclose(a, ref.detach().numpy(), atol=1e-14)
    np.testing.assert_allclose(slope, d.numpy(), atol=1e-13)
    h = 1e-6
    np.testing.assert_allclose(slope, (train.activation(g + h, act)[0] - train.activation(g - h, act)[0]) / (2 * h),
                               atol=1e-8)


@pytest.mark.parametrize("act", ["silu", "gelu", "gelu_tanh"])
def test_gated_gradients_are_the_differences(act):
    T, K, N, r, alpha = 3, 6, 4, 2, 3.0
    X = RNG.normal(size=(T, K))
    gate, up = ([RNG.normal(size=s) for s in ((N, K), (K, r), (r, N))] for _ in range(2))
    dH = RNG.normal(size=(T, N))
    got = train.gated_bwd(dH, X, gate, up, alpha, r, act)

    def value():
        return float(np.sum(dH * train.gated_fwd(X, gate, up, alpha, r, act)[0]))
    for x, d in zip((X, gate[1], gate[2], up[1], up[2]), got):
        for i in np.ndindex(x.shape):
            keep = x[i]
            h = 1e-6
            x[i] = keep + h
            hi = value()
            x[i] = keep - h
            lo = value()
            x[i] = keep
            assert abs((hi - lo) / (2 * h) - d[i]) < 1e-6 * (1 + abs(d[i]))


def test_gated_by_loops():
    T, K, N, r = 2, 3, 2, 1
    X = RNG.normal(size=(T, K))
    gate, up = ([RNG.normal(size=s) for s in ((N, K), (K, r), (r, N))] for _ in range(2))
    H = train.gated_fwd(X, gate, up, 2.0, r, "silu")[0]
    for t in range(T):
        for n in range(N):
            side = [sum(X[t, k] * (w[n, k] + 2.0 * a[k, 0] * b[0, n]) for k in range(K)) for w, a, b in (gate, up)]
            assert abs(H[t, n] - side[0] / (1 + math.exp(-side[0])) * side[1]) < 1e-12


def test_loss_against_torch_and_differences():
    T, K, V = 5, 4, 7
    X, W = RNG.normal(size=(T, K)), RNG.normal(size=(V, K))
    t = np.array([0, 6, -1, 3, -100])
    loss, lse, mean, dX, p = train.head_loss(X, W, t)
    x = torch.from_numpy(X).requires_grad_()
    ref = torch.nn.functional.cross_entropy(x @ torch.from_numpy(W).t(), torch.from_numpy(np.where(t < 0, -100, t)))
    (d,) = torch.autograd.grad(ref, x)
    assert abs(mean - ref.item()) < 1e-12
    np.testing.assert_allclose(dX, d.numpy(), atol=1e-13)
    np.testing.assert_allclose(p.sum(1), 1.0)
    assert loss[2] == loss[4] == lse[2] == lse[4] == 0 and not dX[2].any()
    g = RNG.normal(size=T)
    dX = train.head_loss(X, W, t, g)[3]
    for i in np.ndindex(X.shape):
        keep, h = X[i], 1e-6
        X[i] = keep + h
        hi = np.sum(g * train.head_loss(X, W, t)[0])
        X[i] = keep - h
        lo = np.sum(g * train.head_loss(X, W, t)[0])
        X[i] = keep
        assert abs((hi - lo) / (2 * h) - dX[i]) < 1e-7


def test_loss_of_a_certain_token_keeps_its_digits():
    # z = (40, 0): loss = log1p(e^-40), dX = -(1 - p) (w_t - w_o).
    X, W = np.array([[1.0]]), np.array([[40.0], [0.0]])
    loss, _, _, dX, _ = train.head_loss(X, W, np.array([0]))
    assert abs(loss[0] / math.exp(-40) - 1) < 1e-12 and abs(dX[0, 0] / (-40 * math.exp(-40)) - 1) < 1e-12


def test_loss_of_nothing():
    loss, lse, mean, dX, _ = train.head_loss(np.ones((2, 3)), np.ones((4, 3)), np.array([-1, -2]))
    assert mean == 0 and not loss.any() and not lse.any() and not dX.any()


def test_clip():
    g = [np.array([3.0]), np.array([0.0, 4.0])]
    norm, out = train.clip(g, 1.0)
    assert norm == 5.0
    np.testing.assert_allclose(np.concatenate(out), np.array([3, 0, 4]) / (5 + 1e-6))
    assert train.clip(g, 10.0)[1][1][1] == 4.0 and train.clip(g, 0.0)[1][0][0] == 3.0
    p = [torch.nn.Parameter(torch.zeros(x.shape, dtype=torch.float64)) for x in g]
    for q, x in zip(p, g):
        q.grad = torch.from_numpy(x.copy())
    assert abs(torch.nn.utils.clip_grad_norm_(p, 1.0).item() - norm) < 1e-12
    for q, x in zip(p, out):
        np.testing.assert_allclose(q.grad.numpy(), x, rtol=1e-12)


def test_multiplier():
    m = train.multiplier
    assert m(1.0) == 1.0 and m(-1.5) == -1.5 and m(0.0) == 0.0
    assert m(1 + 2.0 ** -9) == 1 + 2.0 ** -9 and m(1 + 2.0 ** -10) == 1 + 2.0 ** -9    # a tie, away from zero
    assert m(1 + 1.9 * 2.0 ** -11) == 1.0 and m(-1 - 2.0 ** -10) == -1 - 2.0 ** -9
    assert m(1 + 3 * 2.0 ** -10) == 1 + 2.0 ** -8                               # the next one
    assert m(2.0 ** -39) == 2.0 ** -39 and m(2.0 ** -40) == 2.0 ** -39 and m(2.0 ** -41) == 0.0
    assert m(2.0 ** 33) == np.inf and m(-2.0 ** 40) == -np.inf and m(2.0 ** 32) == 2.0 ** 32
    assert m(2.0 ** 33 - 2.0 ** 24) == 2.0 ** 33 - 2.0 ** 24 and m(2.0 ** 33 - 2.0 ** 23) == np.inf
    x = RNG.normal(size=1000) * 10.0 ** RNG.uniform(-8, 9, 1000)
    assert np.all(np.abs(m(x) - x) <= 2.0 ** -10 * np.abs(x) + 2.0 ** -40)
