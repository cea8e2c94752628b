"""How far attention over the cache may be from the oracle where its rows are
few (at most 32 rows of a key/value head), and what it computes there, in numpy,
for planting mistakes.

There the weights, and the levels of an NF4 cache, enter the products as two
bf16 values each.  bf16 has 8 significant bits: rounding leaves at most 2^-8 of a
value, and rounding the rest leaves at most 2^-16.  So an output is off by half
a bf16 unit of itself, and by mass = sum_j w_j |v_j| times
    2^-16            the weights,
  + 2^-16            the values' levels (NF4),
  + 2 e              the scores, off by e = d ((terms + 8) 2^-24 + 2^-21 + 2^-16
                     (NF4)) with d = |scale| max_j sum |q k_j| over `terms` dims
                     where q is not 0: the fp32 sum, its scaling to base 2 and
                     the exponential, the keys' levels,
  + a 2^-24          the fp32 sums of weights and outputs: a additions,
  + 2^-20            scales and the join of a few splits.
A wave adds up every fourth (or eighth) step of 32 keys of its split, four
matrix instructions to a step, each of which may round at every fourth of its 32
products: a = 32 keys / 128 + 64.  With q of many terms e hides what a single
bf16 value in the place of two would change, so the inputs have q of one term
(the weights), of none (the values' levels), or one stored key (the keys'
levels: its score is the log-sum)."""

import numpy as np

from oracle import nf4


def score_error(kv, terms, d):
    return d * ((terms + 8) * 2.0 ** -24 + 2.0 ** -21 + (2.0 ** -16 if kv == "nf4" else 0.0))


def mass_factor(kv, keys, terms, d):
    """Of the mass (without the output's own rounding)."""
    two = 2.0 ** -16 if kv == "nf4" else 0.0
    return (2.0 ** -16 + two + 2 * score_error(kv, terms, d) + (keys / 4 + 64) * 2.0 ** -24 + 2.0 ** -20) * 1.05


def lse_bound(kv, terms, d, lse):
    return score_error(kv, terms, d) + 2.0 ** -22 * (4 + np.abs(lse))


def norm_factor(kv, ratio, adds):
    """||error|| / ||output|| with ratio = ||mass|| / ||output|| and keys that are independent of the values (errors of
    the scores then do not add up): the output's rounding, weights, levels, and `adds` fp32 additions."""
    two = 2.0 ** -16 if kv == "nf4" else 0.0
    return 2.0 ** -8 + ratio * (2.0 ** -16 + two + adds * 2.0 ** -24)


def _parts(x, words):
    """x as the sum of `words` bf16 values."""
    x = np.asarray(x, dtype=np.float64)
    out = np.zeros_like(x)
    for _ in range(words):
        out += nf4.bf16_round((x - out).astype(np.float32)).astype(np.float64)
    return out


def attend_few(q, k, v, table, scale, weight_words=2, level_words=2):
    """One new token over stored rows that all are seen, one head: (outputs, log-sum) as the kernel rounds them.  k and v:
    (codes [keys, dim], scales [keys]); codes index `table`, or are the values themselves where it is None."""
    (ck, sk), (cv, sv) = k, v
    k, v = ((_parts(table, level_words)[c] if table is not None else c.astype(np.float64)) for c in (ck, cv))
    s = scale * (k @ q.astype(np.float64)) * sk
    w = np.exp(s - s.max())
    p = _parts(w * sv, weight_words)
    return nf4.bf16_round(((p @ v) / w.sum()).astype(np.float32)).astype(np.float64), s.max() + np.log(w.sum())
