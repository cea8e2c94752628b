"""The bounds that the few-row attention tests use notice what they are for: one
bf16 value in the place of two, planted in numpy."""

import numpy as np
import pytest

import attention_bounds as bounds
from oracle import attention as at
from oracle import baselines, nf4
from oracle.compare import ulp_bf16


def _problem(kv, keys, dim, seed):
    rng = np.random.Generator(np.random.PCG64(seed))
    q = nf4.bf16_round(rng.normal(size=dim).astype(np.float32))
    x = [nf4.bf16_round(rng.normal(size=(keys, dim)).astype(np.float32)) for _ in range(2)]
    if kv == "bf16":
        return q, [(t, np.ones(keys)) for t in x], None, x
    pairs = [at.quantize_rows(t, kv) for t in x]
    table = None if kv == "int8" else baselines.type_table(kv).astype(np.float64)
    return q, [(c, s.astype(np.float64)) for c, s in pairs], table, [at.stored_values(c, s, kv) for c, s in pairs]


def _run(kv, keys, dim, seed, terms, scale, **words):
    """(share of the outputs outside of their bound, whether the log-sum is)."""
    q, stored, table, (k, v) = _problem(kv, keys, dim, seed)
    q[terms:] = 0
    if kv in ("int4", "fp4"):
        words["level_words"] = 3          # the kernel has their levels as integers and halves, exactly
    out, lse = bounds.attend_few(q, *stored, table, scale, **words)
    ref, rl, mass = at.attend(q[None, None], k[:, None], v[:, None], scale)
    d = scale * (np.abs(k.astype(np.float64)) @ np.abs(q.astype(np.float64))).max()
    bound = 0.5 * ulp_bf16(np.maximum(np.abs(ref[0, 0]), np.abs(out))) + mass[0, 0] * bounds.mass_factor(kv, keys, terms, d)
    return np.mean(np.abs(out - ref[0, 0]) > bound), abs(lse - rl[0, 0]) > bounds.lse_bound(kv, terms, d, rl[0, 0])


@pytest.mark.parametrize("kv", at.KV_TYPES)
@pytest.mark.parametrize("keys", [17, 64, 200])
def test_one_bf16_value_to_a_weight_is_noticed(kv, keys):
    for seed in range(4):
        assert _run(kv, keys, 128, seed, 1, 1.0) == (0, False)
        assert _run(kv, keys, 128, seed, 1, 1.0, weight_words=1)[0] > 0.1


@pytest.mark.parametrize("keys", [1, 64, 700, 4000])
def test_one_bf16_value_to_a_level_of_the_values_is_noticed(keys):
    for seed in range(4):
        assert _run("nf4", keys, 128, seed, 0, 1.0) == (0, False)
        assert _run("nf4", keys, 128, seed, 0, 1.0, level_words=1)[0] > 0.1


@pytest.mark.parametrize("dim", [16, 64, 128, 256])
def test_one_bf16_value_to_a_level_of_the_keys_is_noticed(dim):
    assert not any(_run("nf4", 1, dim, seed, dim, dim ** -0.5)[1] for seed in range(50))
    assert np.mean([_run("nf4", 1, dim, seed, dim, dim ** -0.5, level_words=1)[1] for seed in range(50)]) > 0.5


def test_norm_bound_of_a_long_context():
    for seed in range(2):
        q, stored, table, (k, v) = _problem("nf4", 100000, 64, seed)
        ref, _, mass = (x[0, 0] for x in at.attend(q[None, None], k[:, None], v[:, None], 0.125))
        ratio = np.linalg.norm(mass) / np.linalg.norm(ref)
        tolerance = bounds.norm_factor("nf4", ratio, 512)
        off = [np.linalg.norm(bounds.attend_few(q, *stored, table, 0.125, level_words=n)[0] - ref) / np.linalg.norm(ref)
               for n in (2, 1)]
        assert off[0] <= tolerance < off[1], (off, tolerance)
