"""The kernel for few rows keeps the bits that it claims: weights and NF4 levels as two bf16 values.  The inputs and bounds
are such that one value in the place of two would not pass (tests/attention_bounds.py, and test_attention_bounds.py,
where that is planted)."""

import numpy as np
import pytest

import attention_bounds as bounds
from oracle import attention as at
from oracle.compare import ulp_bf16
from test_gpu_generate import Batch, _host, _lib

pytestmark = pytest.mark.gpu

torch = pytest.importorskip("torch")


def _check(b, terms, scale):
    """Outputs and log-sums of a batch whose q has `terms` dims that are not 0."""
    out, lse = b.run(scale=scale)
    out, lse = _host(out), lse.cpu().numpy().astype(np.float64)
    assert max(b.n) * (b.hq // b.h) <= 32                # the kernel for few rows
    for i, (n, m) in enumerate(b.seqs):
        rows = slice(b.starts[i], b.starts[i + 1])
        q = b.q[rows].astype(np.float64)
        ref, rl, mass = at.attend(q, b.k[i], b.v[i], scale)
        for x in range(b.hq):
            key = np.abs(b.k[i][:, x // (b.hq // b.h)].astype(np.float64))
            d = abs(scale) * (np.abs(q[:, x]) @ key.T).max(1)
            off = np.abs(out[rows][:, x] - ref[:, x])
            factor = bounds.mass_factor(b.kv, m, terms, d)[:, None]
            assert np.all(off <= 0.5 * ulp_bf16(np.maximum(np.abs(ref[:, x]), np.abs(out[rows][:, x]))) + mass[:, x] * factor), (i, x)
            assert np.all(np.abs(lse[rows][:, x] - rl[:, x]) <= bounds.lse_bound(b.kv, terms, d, rl[:, x])), (i, x)
    _lib().device_status()


@pytest.mark.parametrize("kv", at.KV_TYPES)
@pytest.mark.parametrize("hq,h,D", [(4, 4, 128), (8, 1, 64), (32, 2, 80), (6, 2, 256)])
def test_weights(hq, h, D, kv):
    """q of one dim: the scores are exact to a few fp32 roundings, the weights are not."""
    b = Batch([(1, 17), (1, 64), (1, 200), (2, 130), (1, 700)], hq, h, D, kv, 16, seed=50)
    keep = np.zeros_like(b.q)
    for x in range(hq):
        keep[:, x, (7 * x) % D] = b.q[:, x, (7 * x) % D]
    b.q = keep
    _check(b, 1, 1.0)


@pytest.mark.parametrize("kv", ["nf4", "int4", "fp4"])
@pytest.mark.parametrize("hq,h,D", [(4, 4, 128), (8, 1, 64), (20, 1, 128), (6, 2, 256)])
def test_levels_of_the_values(hq, h, D, kv):
    """q = 0: every stored token has the same weight."""
    b = Batch([(1, 1), (1, 64), (1, 700), (1, 4000)], hq, h, D, kv, 64, seed=51)
    b.q = np.zeros_like(b.q)
    _check(b, 0, 1.0)


@pytest.mark.parametrize("hq,h,D", [(4, 4, 128), (8, 1, 64), (7, 7, 16), (24, 1, 96), (6, 2, 256)])
def test_levels_of_the_keys(hq, h, D):
    """One stored token: its score is the log-sum."""
    b = Batch([(1, 1)] * 40, hq, h, D, "nf4", 16, seed=52)
    _check(b, D, D ** -0.5)


def test_a_long_context_by_its_norm():
    """10^5 keys: an error that every row has alike does not average out."""
    b = Batch([(1, 100000)], 4, 2, 64, "nf4", 64, seed=53)
    out, _ = b.run()
    ref, _, mass = at.attend(b.q, b.k[0], b.v[0], 0.125)
    out = _host(out)
    for x in range(4):
        ratio = np.linalg.norm(mass[0, x]) / np.linalg.norm(ref[0, x])
        # 32 splits of 8 waves: 13 steps to a wave, four matrix instructions to a step, each up to 8 additions.
        off = np.linalg.norm(out[0, x] - ref[0, x]) / np.linalg.norm(ref[0, x])
        assert off <= bounds.norm_factor("nf4", ratio, 512), (x, off)
