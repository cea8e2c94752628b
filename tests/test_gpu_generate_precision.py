"""The kernel for few rows keeps the bits that it claims: weights and NF4 levels as two bf16 values.  The inputs and bounds
are such that one value in the place of two would not pass (tests/attention_bounds.py, and test_attention_bounds.py,
where that is planted)."""

import numpy as np
import pytest

import attention_bounds as bounds
from oracle import attention as at
from oracle import nf4
from oracle.compare import ulp_bf16
from test_gpu_generate import Batch, _dev, _host, _lib

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


def _many(kv, n, m, hq, h, D, seed):
    b = Batch([(n, m)], hq, h, D, kv, 16, seed=seed)
    assert n * hq // h > 32                              # the kernel for many rows
    return b


@pytest.mark.parametrize("kv", at.KV_TYPES)
@pytest.mark.parametrize("n,m,hq,h,D", [(100, 300, 2, 1, 64), (200, 1100, 4, 4, 128), (70, 700, 8, 2, 80), (150, 900, 2, 2, 256)])
def test_many_rows_by_their_norm(n, m, hq, h, D, kv):
    """The roundings of weights, keys and values are as good as independent of each other and of the outputs' own, so the
    squares of their norms add up.  Rounding a number of b significant bits leaves on average 2^-b / sqrt(3) times 0.7 of it
    (mantissas are spread over [1, 2)): the outputs' own is known; a weight in bf16 adds as much again (so sqrt(2), 1.5 with
    its spread), while fp16 weights, keys and values (NF4) add 3 times an 8th of it, squared: 1.02, 1.2 with all else."""
    b = _many(kv, n, m, hq, h, D, 60)
    out, lse = b.run()
    b.check(out, lse)
    ref, _, _ = at.attend(b.q, b.k[0], b.v[0], D ** -0.5)
    own = np.linalg.norm(nf4.bf16_round(ref.astype(np.float32)) - ref)
    off = np.linalg.norm(_host(out) - ref)
    assert off <= (1.2 if kv == "nf4" else 1.5) * own, off / own


@pytest.mark.parametrize("kv", ["nf4", "int8", "bf16", "fp4"])
@pytest.mark.parametrize("n,m", [(2, 300), (100, 300), (140, 1100)])
@pytest.mark.parametrize("what", ["values", "keys", "queries", "all", "zeros", "huge values", "tiny values", "large scores"])
def test_rows_of_every_size(what, n, m, kv):
    """Scales from 2^-90 to 2^100, side by side: no operand may leave its range, and what a row sees most of decides how
    exact it is, not what is largest."""
    lib = _lib()
    b = _many(kv, n, m, 4, 1, 64, 61) if n > 8 else Batch([(n, m)], 4, 1, 64, kv, 16, seed=61)
    rng = np.random.Generator(np.random.PCG64(62))

    def sizes(rows, lo, hi):
        return np.exp2(rng.integers(lo, hi + 1, rows)).astype(np.float32)[:, None, None]
    k, v = (nf4.bf16_round(rng.normal(size=(m, 1, 64)).astype(np.float32)) for _ in range(2))
    if what in ("values", "all"):
        v = v * sizes(m, -60, 40)
    if what in ("keys", "all"):
        k = k * sizes(m, -80, 2)
    if what in ("queries", "all"):
        b.q = nf4.bf16_round(b.q * sizes(n, -70, 3))
    if what == "zeros":
        k[rng.random(m) < 0.3] = 0
        v[rng.random(m) < 0.3] = 0
    if what == "huge values":
        v = v * sizes(m, 80, 96)
    if what == "tiny values":
        v = v * sizes(m, -92, -80)
    if what == "large scores":
        k, b.q = k * np.float32(2.0 ** 14), nf4.bf16_round(b.q * np.float32(2.0 ** 12))
    k, v = nf4.bf16_round(k.astype(np.float32)), nf4.bf16_round(v.astype(np.float32))
    j = np.arange(m)
    lib.kv_write(b.cache, _dev(k), _dev(v), torch.tensor(b.table[0, j // 16] * 16 + j % 16).cuda())
    b.k, b.v = ([x] if kv == "bf16" else [at.stored_values(*at.quantize_rows(x, kv), kv)] for x in (k, v))
    for kw in (dict(), dict(window=90), dict(causal=False)):
        out, lse = b.run(**kw)
        assert bool(torch.isfinite(out).all())
        if what != "large scores":
            b.check(out, lse, **kw)
        else:                                            # a score's own rounding exceeds 1: one key takes all
            hit = np.zeros(out.shape[0], bool)
            o = _host(out)
            for x in range(4):
                near = np.abs(o[:, x, None] - b.v[0][None, :, 0]).max(-1) <= 2.0 ** -7 * np.abs(b.v[0][None, :, 0]).max(-1)
                hit |= near.any(1)
            assert hit.mean() > 0.9
