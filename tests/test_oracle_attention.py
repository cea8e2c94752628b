"""Pins of the attention-side oracle, each against something else: complex
products, closed forms, brute force with fractions, torch's softmax."""

import math
from fractions import Fraction

import numpy as np
import pytest

from oracle import attention as at
from oracle import baselines, nf4


def _rng(seed):
    return np.random.Generator(np.random.PCG64(seed))


@pytest.mark.parametrize("layout", ["half", "interleaved"])
def test_rotation_is_a_complex_product(layout):
    rng = _rng(1)
    x = rng.normal(size=(5, 3, 32))
    t = at.rope_table(100, 16)
    p = rng.integers(0, 100, 5)
    y = at.rotate(x, t, p, layout)
    i, j = (np.arange(8), np.arange(8) + 8) if layout == "half" else (2 * np.arange(8), 2 * np.arange(8) + 1)
    z = (x[..., i] + 1j * x[..., j]) * np.exp(1j * p[:, None] * 10000.0 ** (-np.arange(8) / 8))[:, None]
    np.testing.assert_allclose(y[..., i] + 1j * y[..., j], z, atol=1e-14)
    assert np.array_equal(y[..., 16:], x[..., 16:])
    np.testing.assert_allclose(at.rotate(y, t, p, layout, inverse=True), x, atol=1e-14)


def test_rotated_products_depend_on_the_distance_alone():
    rng = _rng(2)
    q, k = rng.normal(size=(1, 1, 64)), rng.normal(size=(1, 1, 64))
    t = at.rope_table(5000, 64)
    one = np.sum(at.rotate(q, t, [40]) * at.rotate(k, t, [7]))
    assert abs(one - np.sum(at.rotate(q, t, [4040]) * at.rotate(k, t, [4007]))) < 1e-10


def test_inverse_rotation_is_the_gradient():
    rng = _rng(3)
    x, dy = rng.normal(size=(4, 2, 32)), rng.normal(size=(4, 2, 32))
    t, p = at.rope_table(64, 32, amplitude=1.3), rng.integers(0, 64, 4)
    grad = at.rotate(dy, t, p, inverse=True)
    for _ in range(20):
        e = np.zeros_like(x)
        idx = tuple(rng.integers(0, s) for s in x.shape)
        e[idx] = 1e-3
        diff = np.sum(dy * (at.rotate(x + e, t, p) - at.rotate(x - e, t, p))) / 2e-3
        assert abs(diff - grad[idx]) < 1e-9


def test_scalings():
    f = at.frequencies(64)
    np.testing.assert_allclose(at.frequencies(64, scaling="linear", factor=4.0), f / 4)
    b = at.frequencies(64, scaling="base", factor=4.0)
    assert b[0] == 1.0 and abs(b[-1] - f[-1] / 4) < 1e-15
    z = at.frequencies(64, scaling="bands", factor=8.0, original=4096, low=1, high=32)
    turns = 4096 * f / (2 * math.pi)
    assert np.array_equal(z[turns >= 32], f[turns >= 32])
    np.testing.assert_allclose(z[turns <= 1], f[turns <= 1] / 8)
    assert np.all((z <= f) & (z >= f / 8))


@pytest.mark.parametrize("kind", ["nf4", "int4", "fp4"])
def test_four_bit_rows_take_the_nearest_level(kind):
    """Against exact fractions: the nearest level to x / top wherever the fp32
    rule does not sit within rounding (2^-22) of a boundary."""
    rng = _rng(4)
    x = nf4.bf16_round(rng.normal(size=(20, 32)).astype(np.float32))
    codes, scale = at.quantize_rows(x, kind)
    table = [Fraction(float(v)) for v in baselines.type_table(kind)]
    for row, c, s in zip(x, codes, scale):
        top = max(abs(Fraction(float(v))) for v in row)
        assert Fraction(float(s)) == top
        for v, code in zip(row, c):
            u = Fraction(float(v)) / top
            gaps = [abs(u - t) for t in table]
            assert gaps[code] <= min(gaps) + Fraction(1, 1 << 22)
    assert kind == "nf4" or not np.any(codes == 8)


def test_int8_rows():
    rng = _rng(5)
    x = nf4.bf16_round(rng.normal(size=(50, 64)).astype(np.float32))
    codes, scale = at.quantize_rows(x, "int8")
    assert np.all(np.abs(codes).max(-1) == 127)
    assert np.max(np.abs(at.stored_values(codes, scale, "int8") - x) / scale[:, None]) <= 0.5 + 1e-4


@pytest.mark.parametrize("kind", ["int8", "nf4", "int4", "fp4"])
def test_rows_of_nothing_and_of_no_numbers(kind):
    x = np.zeros((4, 16), np.float32)
    x[1, 3] = 1e-31
    x[2, 5] = np.inf
    x[3, 0] = np.nan
    codes, scale = at.quantize_rows(x, kind)
    v = at.stored_values(codes, scale, kind)
    assert np.all(v[:2] == 0) and np.all(np.isnan(v[2:]))


@pytest.mark.parametrize("causal,window", [(True, 0), (False, 0), (True, 3), (False, 4)])
def test_attention_against_torch(causal, window):
    torch = pytest.importorskip("torch")
    rng = _rng(6)
    n, length = 7, 11
    q, k, v = rng.normal(size=(n, 4, 16)), rng.normal(size=(length, 2, 16)), rng.normal(size=(length, 2, 16))
    out, lse, mass = at.attend(q, k, v, 0.25, causal, window)
    qt, kt, vt = torch.tensor(q), torch.tensor(k).repeat_interleave(2, 1), torch.tensor(v).repeat_interleave(2, 1)
    s = 0.25 * torch.einsum("ihd,jhd->hij", qt, kt)
    p, j = torch.arange(length - n, length)[:, None], torch.arange(length)[None]
    hide = torch.zeros(n, length, dtype=torch.bool)
    if causal:
        hide |= j > p
    if window:
        hide |= j <= p - window
    s = s.masked_fill(hide, -math.inf)
    np.testing.assert_allclose(out, torch.einsum("hij,jhd->ihd", s.softmax(-1), vt).numpy(), atol=1e-13)
    np.testing.assert_allclose(lse, s.logsumexp(-1).T.numpy(), atol=1e-13)
    assert np.all(mass >= np.abs(out) - 1e-15)


def test_attention_of_empty_rows():
    rng = _rng(7)
    q, k = rng.normal(size=(5, 2, 16)), rng.normal(size=(3, 2, 16))
    out, lse, _ = at.attend(q, k, k, 1.0)        # five new tokens, three stored: two stand before the first
    assert np.all(out[:2] == 0) and np.all(lse[:2] == -np.inf) and np.all(np.isfinite(lse[2:]))
    np.testing.assert_allclose(out[2], k[0])
    out, lse, _ = at.attend(q, k[:0], k[:0], 1.0)
    assert np.all(out == 0) and np.all(lse == -np.inf)
