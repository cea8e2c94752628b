"""GPU parity of the attention side: rotary positions and their table, rows
quantized as they are written and read back (bit for bit), and attention over
the paged cache, against the oracle, at the sizes and masks where each can go
wrong.

Tolerances.  Rotation: two fp32 products and a sum (3 roundings, 2^-24 each of
|a c| + |b s|) and half a bf16 unit.  Attention, elementwise: half a bf16 unit
of the result plus mass * (u + 2 d + ...), where mass = sum_j w_j |v_j|,
u = 2^-8 is the rounding of the weights to bf16 (8 significant bits: half a unit
in the last place of 1 is 2^-8), and d bounds the error of a score:
(dim + 8) 2^-24 sum |scale q k| for the fp32 sum, 2^-22 |s| for its scaling to
base 2 and the exponential.  An NF4 row may enter the products rounded to bf16
(u of every |q k| in d, and u of mass).  A weight below fp32's normal range,
relative to the largest, counts as nothing: 2^-100 per output.  lse: d and 2^-22 of its size."""

import numpy as np
import pytest

from oracle import attention as at
from oracle import baselines, nf4
from oracle.compare import ulp_bf16

pytestmark = pytest.mark.gpu

torch = pytest.importorskip("torch")


def _lib():
    import bit_nf4_quantized_21_amd as lib
    return lib


def _rng(seed):
    return np.random.Generator(np.random.PCG64(seed))


def _bf16(rng, *shape, scale=1.0):
    return nf4.bf16_round((rng.normal(size=shape) * scale).astype(np.float32))


def _dev(x):
    return torch.from_numpy(np.ascontiguousarray(nf4.f32_to_bf16_bits(x)).view(np.int16).reshape(x.shape)).cuda().view(torch.bfloat16)


def _host(t):
    return t.float().cpu().numpy().astype(np.float64)


def _i32(x):
    return torch.tensor(np.asarray(x), dtype=torch.int32, device="cuda")


def _status_ok():
    _lib().device_status()


# ------------------------------------------------------------------ rotation

@pytest.mark.parametrize("kw", [dict(), dict(scaling="linear", factor=4.0), dict(scaling="base", factor=8.0, base=5e5),
                                dict(scaling="bands", factor=8.0, original=4096.0, low=1.0, high=4.0, amplitude=1.2)])
@pytest.mark.parametrize("positions,rot", [(1, 16), (4097, 128), (300, 80)])
def test_rope_table(positions, rot, kw):
    t = _lib().rope_table(positions, rot, **kw)
    ref = at.rope_table(positions, rot, **kw)
    # Angles in fp64 (relative 2^-48 with the power's rounding), one rounding to fp32.
    err = np.abs(t.cpu().numpy().astype(np.float64) - ref)
    amp = kw.get("amplitude", 1.0)
    assert t.shape == ref.shape and np.all(err <= amp * (2.0 ** -24 + positions * 2.0 ** -48))


def test_rope_table_of_a_long_context():
    t = _lib().rope_table(1 << 20, 64).cpu().numpy().astype(np.float64)
    p = np.array([0, 1, 131071, (1 << 20) - 1])
    angle = p[:, None] * at.frequencies(64)
    ref = np.stack((np.cos(angle), np.sin(angle)), -1)
    assert np.all(np.abs(t[p] - ref) <= 2.0 ** -24 + (1 << 20) * 2.0 ** -48)


def _check_rope(got, x, table, pos, layout, inverse):
    ref = at.rotate(x.astype(np.float64), table.astype(np.float64), pos, layout, inverse)
    half = table.shape[1]
    a, b = ((slice(0, half), slice(half, 2 * half)) if layout == "half" else (slice(0, 2 * half, 2), slice(1, 2 * half, 2)))
    c, s = np.abs(table[pos][:, None, :, 0]).astype(np.float64), np.abs(table[pos][:, None, :, 1]).astype(np.float64)
    size = np.zeros_like(ref)
    ax = np.abs(x.astype(np.float64))
    size[..., a] = ax[..., a] * c + ax[..., b] * s
    size[..., b] = ax[..., b] * c + ax[..., a] * s
    assert np.all(np.abs(got - ref) <= 0.5 * ulp_bf16(np.maximum(np.abs(ref), np.abs(got))) + 2.0 ** -22 * size)
    assert np.array_equal(got[..., 2 * half:], ref[..., 2 * half:])


@pytest.mark.parametrize("inverse", [False, True])
@pytest.mark.parametrize("layout", ["half", "interleaved"])
@pytest.mark.parametrize("T,hq,hk,D,rot", [(1, 1, 1, 16, 16), (3, 4, 2, 128, 128), (257, 7, 7, 80, 32), (33, 5, 1, 256, 96),
                                           (130, 64, 8, 64, 64)])
def test_rope(T, hq, hk, D, rot, layout, inverse):
    lib = _lib()
    rng = _rng(T + D)
    q, k = _bf16(rng, T, hq, D), _bf16(rng, T, hk, D)
    table = at.rope_table(1000, rot, amplitude=1.1).astype(np.float32)
    pos = rng.integers(0, 1000, T)
    tq, tk = lib.rope(_dev(q), _dev(k), torch.from_numpy(table).cuda(), _i32(pos), layout=layout, inverse=inverse)
    _check_rope(_host(tq), q, table, pos, layout, inverse)
    _check_rope(_host(tk), k, table, pos, layout, inverse)
    one, none = lib.rope(_dev(q), None, torch.from_numpy(table).cuda(), _i32(pos), layout=layout, inverse=inverse)
    assert none is None and torch.equal(one.view(torch.int16), tq.view(torch.int16))
    _status_ok()


@pytest.mark.parametrize("layout", ["half", "interleaved"])
def test_rope_strides_in_place_and_gradient(layout):
    """Views of a fused buffer (token stride of all heads), head-major memory,
    in place; forward and inverse undo each other; dq.y' = (inverse dq).x."""
    lib = _lib()
    rng = _rng(8)
    T, hq, hk, D, rot = 37, 6, 2, 64, 48
    x = _bf16(rng, T, hq + 2 * hk, D)
    table = at.rope_table(64, rot).astype(np.float32)
    pos = rng.integers(0, 64, T)
    tt, tp = torch.from_numpy(table).cuda(), _i32(pos)
    fused = _dev(x)
    q, k = fused[:, :hq], fused[:, hq:hq + hk]
    a, b = lib.rope(q, k, tt, tp, layout=layout)
    _check_rope(_host(a), x[:, :hq], table, pos, layout, False)
    _check_rope(_host(b), x[:, hq:hq + hk], table, pos, layout, False)
    major = q.transpose(0, 1).contiguous().transpose(0, 1)       # [T, heads, D] over [heads, T, D] memory
    c, _ = lib.rope(major, None, tt, tp, layout=layout)
    assert torch.equal(a.view(torch.int16), c.view(torch.int16))
    rest = fused[:, hq + hk:].clone()
    lib.rope(q, k, tt, tp, layout=layout, q_out=q, k_out=k)
    assert torch.equal(q.contiguous().view(torch.int16), a.view(torch.int16))
    assert torch.equal(k.contiguous().view(torch.int16), b.view(torch.int16))
    assert torch.equal(fused[:, hq + hk:].contiguous().view(torch.int16), rest.view(torch.int16))
    dy = _bf16(rng, T, hq, D)
    dx, _ = lib.rope(_dev(dy), None, tt, tp, layout=layout, inverse=True)
    left, right = np.sum(dy.astype(np.float64) * _host(a)), np.sum(_host(dx) * x[:, :hq].astype(np.float64))
    assert abs(left - right) <= 2.0 ** -8 * np.sqrt(np.sum(dy ** 2.0) * np.sum(x[:, :hq] ** 2.0)) / np.sqrt(T * hq * D) * 8
    with pytest.raises(lib.QLoRAError):
        lib.rope(fused.view(-1)[4:4 + 2 * D].view(1, 2, D), None, tt, tp)   # not on 16 bytes


def test_rope_positions_out_of_range_are_reported():
    lib = _lib()
    q = torch.zeros(3, 2, 32, dtype=torch.bfloat16, device="cuda")
    t = lib.rope_table(8, 32)
    lib.rope(q, None, t, _i32([0, 7, 3]))
    _status_ok()
    for bad in (8, -1, 2 ** 31 - 1):
        lib.rope(q, None, t, _i32([0, bad, 3]))
        with pytest.raises(lib.QLoRAError, match="QLORA_ERR_INDEX"):
            lib.device_status()
    _status_ok()


# --------------------------------------------------------------------- cache

def _rows(rng, T, h, D):
    """Rows of every kind: normal, tiny, huge, zero, one element, ties."""
    x = rng.normal(size=(T, h, D)).astype(np.float32)
    flat = x.reshape(-1, D)
    flat[0] = 0
    if len(flat) > 8:
        flat[1] *= 1e-33
        flat[2] *= 1e30
        flat[3] *= 1e-29
        flat[4] = 0
        flat[4, D // 2] = -3.0
        flat[5] = np.arange(D) % 15 - 7            # int4's levels
        flat[6] = (np.arange(D) % 29 - 14) / 2     # halfway between them
        flat[7] = np.array([0, .25, .5, .75, 1, 1.25, 1.5, 1.75, 2, 2.5, 3, 3.5, 4, 5, 6, -6])[np.arange(D) % 16]
    return nf4.bf16_round(x)


def _unpack(codes):
    return np.stack((codes & 15, codes >> 4), -1).reshape(*codes.shape[:-1], -1)


@pytest.mark.parametrize("turn", [None, "half", "interleaved"])
@pytest.mark.parametrize("kv", at.KV_TYPES)
@pytest.mark.parametrize("T,h,D,page", [(1, 1, 16, 16), (45, 3, 80, 16), (70, 2, 128, 64), (19, 5, 256, 32), (33, 8, 64, 1024)])
def test_write_and_read(T, h, D, page, kv, turn):
    """Codes, scales and the values read back equal the oracle's, bit for bit;
    skipped tokens and untouched rows stay as they were."""
    lib = _lib()
    rng = _rng(T * D + len(kv))
    pages = -(-T // page) + 2
    cache = lib.KVCache.empty(pages, h, page, D, kv_type=kv)
    buffers = [t for t in (cache.k, cache.v, cache.k_scale, cache.v_scale) if t is not None]
    for t in buffers:
        t.view(torch.uint8).fill_(0x55)
    before = [t.clone() for t in buffers]
    k, v = _rows(rng, T, h, D), _rows(rng, T, h, D)
    slots = rng.permutation(pages * page)[:T]
    slots[rng.random(T) < 0.2] = -1
    kw, kf = {}, k.astype(np.float32)
    if turn:
        rot = max(16, D // 32 * 16)
        table, pos = at.rope_table(500, rot).astype(np.float32), rng.integers(0, 500, T)
        kw = dict(table=torch.from_numpy(table).cuda(), positions=_i32(pos), layout=turn)
        kf = at.rotate(kf, table, pos, turn)
    lib.kv_write(cache, _dev(k), _dev(v), torch.tensor(slots).cuda(), **kw)
    got = [t.cpu().numpy() if t.dtype != torch.bfloat16 else t.view(torch.int16).cpu().numpy().view(np.uint16) for t in buffers]
    old = [t.cpu().numpy() if t.dtype != torch.bfloat16 else t.view(torch.int16).cpu().numpy().view(np.uint16) for t in before]
    kept = slots >= 0
    where = (slots[kept] // page, slice(None), slots[kept] % page)
    values = {}
    for n, (side, x) in enumerate((("k", kf), ("v", v))):
        if kv == "bf16":
            old[n][where] = nf4.f32_to_bf16_bits(x[kept])
            values[side] = nf4.bf16_round(x)
        else:
            codes, scale = at.quantize_rows(x, kv)
            values[side] = nf4.bf16_round(at.stored_values(codes, scale, kv))
            if kv != "int8":
                codes = codes[..., 0::2] | (codes[..., 1::2] << 4)
            old[n][where] = codes[kept]
            old[2 + n].view(np.uint32)[where] = scale[kept].view(np.uint32)
    for a, b in zip(got, old):
        assert np.array_equal(a.view(np.uint8), b.view(np.uint8))
    back = rng.integers(0, T, 2 * T + 3)
    ks, vs = lib.kv_read(cache, torch.tensor(slots[back]).cuda())
    for t, side in ((ks, "k"), (vs, "v")):
        ref = np.where((slots[back] >= 0)[:, None, None], values[side][back], np.float32(0))
        assert np.array_equal(_host(t), ref.astype(np.float64))
    _status_ok()


@pytest.mark.parametrize("kv", ["int8", "nf4", "fp4"])
def test_rows_that_are_no_numbers_read_back_as_nan(kv):
    lib = _lib()
    x = np.ones((4, 1, 64), np.float32)
    x[1, 0, 7] = np.inf
    x[2, 0, 63] = -np.inf
    x[3, 0, 0] = np.nan
    t = torch.from_numpy(x).cuda().to(torch.bfloat16)
    cache = lib.KVCache.empty(1, 1, 16, 64, kv_type=kv)
    slots = torch.arange(4, device="cuda")
    lib.kv_write(cache, t, t, slots)
    for r in lib.kv_read(cache, slots):
        r = _host(r)
        assert np.all(r[0] == 1) and np.all(np.isnan(r[1:]))


def test_strided_views_and_empty_calls():
    lib = _lib()
    rng = _rng(10)
    x = _dev(_bf16(rng, 9, 8, 64))
    a, b = (lib.KVCache.empty(1, 2, 16, 64) for _ in range(2))
    slots = torch.arange(9, device="cuda")
    lib.kv_write(a, x[:, 4:6], x[:, 6:8], slots)
    lib.kv_write(b, x[:, 4:6].contiguous(), x[:, 6:8].contiguous(), slots)
    for p, q in zip(lib.kv_read(a, slots), lib.kv_read(b, slots)):
        assert torch.equal(p.view(torch.int16), q.view(torch.int16))
    none = torch.zeros(0, dtype=torch.int64, device="cuda")
    lib.kv_write(a, x[:0, 4:6], x[:0, 6:8], none)
    k, v = lib.kv_read(a, none)
    assert k.shape == (0, 2, 64) and v.shape == (0, 2, 64)
    q, _ = lib.rope(x[:0], None, lib.rope_table(4, 64), _i32([]))
    assert q.shape == (0, 8, 64)


def test_slots_out_of_range_are_reported():
    lib = _lib()
    x = torch.ones(2, 1, 16, dtype=torch.bfloat16, device="cuda")
    cache = lib.KVCache.empty(2, 1, 16, 16)
    lib.kv_write(cache, x, x, torch.tensor([5, 32], device="cuda"))
    with pytest.raises(lib.QLoRAError, match="QLORA_ERR_INDEX"):
        lib.device_status()
    k, _ = lib.kv_read(cache, torch.tensor([1 << 40, 5], device="cuda"))
    with pytest.raises(lib.QLoRAError, match="QLORA_ERR_INDEX"):
        lib.device_status()
    assert torch.all(k[0] == 0) and torch.all(k[1] == 1)


# ----------------------------------------------------------------- attention

class Batch:
    """Sequences of (new, stored) tokens over a cache of scattered pages whose
    unused rows hold what must not matter."""

    def __init__(self, seqs, hq, h, D, kv, page, seed=0, garbage=True, pad=0):
        lib, rng = _lib(), _rng(seed + 77)
        self.seqs, self.hq, self.h, self.D, self.kv = seqs, hq, h, D, kv
        need = [-(-m // page) for _, m in seqs]
        pages = sum(need) + 3
        self.cache = c = lib.KVCache.empty(pages, h, page, D, kv_type=kv)
        if garbage:
            for t in (c.k, c.v):
                t.view(torch.uint8).fill_(0xFF)          # bf16: NaN everywhere
            if kv != "bf16":
                c.k_scale.fill_(float("nan"))
                c.v_scale.fill_(float("inf"))
        ids = rng.permutation(pages)
        self.table = np.full((len(seqs), max(max(need), 1) + pad), 0)
        first, slots, ks, vs = 0, [], [], []
        self.k, self.v = [], []
        for b, ((n, m), w) in enumerate(zip(seqs, need)):
            self.table[b, :w] = ids[first:first + w]
            first += w
            j = np.arange(m)
            slots.append(self.table[b, j // page] * page + j % page)
            ks.append(_bf16(rng, m, h, D))
            vs.append(_bf16(rng, m, h, D))
            if kv == "bf16":
                self.k.append(ks[-1]), self.v.append(vs[-1])
            else:
                self.k.append(at.stored_values(*at.quantize_rows(ks[-1], kv), kv) if m else ks[-1])
                self.v.append(at.stored_values(*at.quantize_rows(vs[-1], kv), kv) if m else vs[-1])
        slots = np.concatenate(slots)
        if slots.size:
            lib.kv_write(c, _dev(np.concatenate(ks)), _dev(np.concatenate(vs)), torch.tensor(slots).cuda())
        self.n = [n for n, _ in seqs]
        self.starts = np.concatenate(([0], np.cumsum(self.n)))
        self.q = _bf16(rng, int(self.starts[-1]), hq, D)
        self.pages, self.dstarts, self.lengths = _i32(self.table), _i32(self.starts), _i32([m for _, m in seqs])
        self.bounds = dict(max_new=max(self.n), max_len=max(m for _, m in seqs))

    def run(self, q=None, lse=True, **kw):
        return _lib().attend_paged(_dev(self.q) if q is None else q, self.cache, self.pages, self.dstarts, self.lengths,
                                   lse=lse, **{**self.bounds, **kw})

    def check(self, out, lse, scale=None, causal=True, window=0, skip=()):
        scale = self.D ** -0.5 if scale is None else scale
        out, lse = _host(out), lse.cpu().numpy().astype(np.float64)
        for b, (n, m) in enumerate(self.seqs):
            if b in skip or n == 0:
                continue
            rows = slice(self.starts[b], self.starts[b + 1])
            q = self.q[rows].astype(np.float64)
            ref, rl, mass = at.attend(q, self.k[b], self.v[b], scale, causal, window)
            aq = np.abs(q)
            d = np.zeros((n, self.hq))
            for x in range(self.hq):
                if m:
                    d[:, x] = abs(scale) * (aq[:, x] @ np.abs(self.k[b][:, x // (self.hq // self.h)].astype(np.float64)).T).max(1)
            four = 2.0 ** -8 if self.kv == "nf4" else 0.0
            err = d * ((self.D + 8) * 2.0 ** -24 + 2.0 ** -21 + four)
            bound = (0.5 * ulp_bf16(np.maximum(np.abs(ref), np.abs(out[rows])))
                     + mass * (2.0 ** -8 + four + 2 * err[..., None] + 2.0 ** -20) * 1.05
                     + 2.0 ** -100)
            worst = np.abs(out[rows] - ref) - bound
            assert np.all(worst <= 0), (b, n, m, float(worst.max()))
            none = rl == -np.inf
            assert np.array_equal(lse[rows] == -np.inf, none)
            fine = ~none
            assert np.all(np.abs(lse[rows][fine] - rl[fine]) <= (err + 2.0 ** -22 * (4 + np.abs(rl)))[fine])
        _status_ok()


SMALL = [(1, 1), (1, 17), (1, 64), (1, 33), (1, 200)]
MIXED = [(5, 5), (0, 9), (3, 70), (1, 1), (9, 4), (2, 0), (0, 0), (6, 130), (1, 65)]
LARGE = [(40, 40), (0, 5), (131, 200), (1, 300), (70, 20), (3, 0), (64, 64), (129, 641)]


@pytest.mark.parametrize("kv", at.KV_TYPES)
@pytest.mark.parametrize("hq,h,D,page", [(4, 4, 128, 16), (8, 1, 64, 64), (10, 2, 80, 16), (6, 2, 256, 32), (7, 7, 16, 16),
                                         (24, 1, 96, 128)])
def test_single_tokens(hq, h, D, page, kv):
    b = Batch(SMALL, hq, h, D, kv, page)
    b.check(*b.run())


@pytest.mark.parametrize("kv", at.KV_TYPES)
@pytest.mark.parametrize("seqs", [MIXED, LARGE], ids=["mixed", "large"])
@pytest.mark.parametrize("hq,h,D,page", [(2, 2, 128, 16), (8, 2, 64, 32), (5, 1, 80, 16), (2, 1, 256, 64)])
def test_chunks(hq, h, D, page, seqs, kv):
    b = Batch(seqs, hq, h, D, kv, page)
    b.check(*b.run())


@pytest.mark.parametrize("kv", ["bf16", "int8", "nf4"])
@pytest.mark.parametrize("causal,window", [(False, 0), (True, 1), (True, 40), (False, 33), (True, 10 ** 6)])
@pytest.mark.parametrize("seqs", [SMALL, MIXED, LARGE], ids=["small", "mixed", "large"])
def test_masks(seqs, causal, window, kv):
    b = Batch(seqs, 4, 2, 64, kv, 16, seed=3)
    b.check(*b.run(causal=causal, window=window), causal=causal, window=window)


@pytest.mark.parametrize("kv", ["bf16", "int8", "nf4", "int4"])
@pytest.mark.parametrize("seqs,hq,h", [([(1, 4000), (1, 1), (1, 2047)], 8, 2), ([(20, 3000), (2, 4001)], 2, 1),
                                       ([(150, 3001), (0, 0), (150, 150)], 2, 1)])
def test_split_keys(seqs, hq, h, kv):
    """Long contexts of few rows: the keys are cut over workgroups and joined."""
    b = Batch(seqs, hq, h, 128, kv, 64, seed=5, pad=3)
    b.check(*b.run())
    b.check(*b.run(window=1500), window=1500)
    one, two = b.run(), b.run()
    for x, y in zip(one, two):
        assert torch.equal(x.view(torch.uint8), y.view(torch.uint8))


@pytest.mark.parametrize("kv", ["bf16", "int8", "nf4"])
@pytest.mark.parametrize("hq,h,n", [(2, 2, 1), (2, 1, 10), (4, 1, 30), (2, 1, 150)])
def test_split_and_whole_sequences_together(hq, h, n, kv):
    """Sequences whose keys are cut over workgroups beside such that fit one, in any order of lengths."""
    b = Batch([(min(n, 3), 40), (n, 2600), (n, 640), (1, 641), (n, 5200), (0, 5200), (n, max(n, 639)), (2, 0), (n, 2600)],
              hq, h, 128, kv, 32, seed=8)
    b.check(*b.run())
    b.check(*b.run(causal=False), causal=False)


@pytest.mark.parametrize("kv", ["bf16", "nf4"])
def test_a_long_context_beside_short_ones(kv):
    """Many splits of one sequence (a workgroup joins each row), one of the others'."""
    b = Batch([(1, 20000), (1, 5), (1, 512), (2, 700), (0, 30), (2, 1)], 4, 2, 64, kv, 128, seed=10)
    b.check(*b.run())
    b.check(*b.run(window=9000), window=9000)


@pytest.mark.parametrize("n,batch", [(1, 70), (40, 64), (40, 65)])
def test_many_sequences(n, batch):
    seqs = [(n, n + (37 * i) % 90) for i in range(batch)]
    b = Batch(seqs, 2, 1, 64, "int8", 16, seed=9)
    b.check(*b.run())


@pytest.mark.parametrize("n", [1, 20, 90])
def test_nothing_stored(n):
    for kv in ("bf16", "int8"):
        b = Batch([(n, 0), (0, 0), (n, 0)], 4, 2, 64, kv, 16, seed=18)
        assert b.bounds["max_len"] == 0
        out, lse = b.run()
        assert torch.all(out == 0) and torch.all(lse == float("-inf"))
        b.check(out, lse)


@pytest.mark.parametrize("scale", [-0.2, 0.0, 1.0])
@pytest.mark.parametrize("seqs", [SMALL, LARGE], ids=["small", "large"])
def test_scales(seqs, scale):
    for kv in ("bf16", "int8"):
        b = Batch(seqs, 2, 1, 64, kv, 32, seed=6)
        b.check(*b.run(scale=scale), scale=scale)


@pytest.mark.parametrize("seqs", [SMALL, MIXED, LARGE], ids=["small", "mixed", "large"])
def test_large_scores(seqs):
    """Scores of some hundreds: one key takes nearly all of the weight."""
    for kv in ("bf16", "int8", "fp4"):
        b = Batch(seqs, 2, 2, 64, kv, 16, seed=7)
        b.q = nf4.bf16_round(b.q * np.float32(64))
        b.check(*b.run())


@pytest.mark.parametrize("kv", ["bf16", "int8", "nf4"])
@pytest.mark.parametrize("n", [4, 100])
@pytest.mark.parametrize("bad", [float("nan"), float("inf")])
def test_a_later_tokens_bad_row_reaches_only_those_that_see_it(n, kv, bad):
    """The 3rd last stored token's key and value are no numbers: the tokens
    before it must not notice, those that see it must."""
    lib = _lib()
    b = Batch([(n, 150), (n, 90)], 2, 1, 64, kv, 16, seed=9)
    m = 150
    slot = int(b.table[0, (m - 3) // 16] * 16 + (m - 3) % 16)
    x = torch.full((1, 1, 64), 1.0, dtype=torch.bfloat16, device="cuda")
    x[0, 0, 5] = bad
    lib.kv_write(b.cache, x, x, torch.tensor([slot], device="cuda"))
    out, lse = b.run()
    o = _host(out)
    ok = n - 3
    ref, _, mass = at.attend(b.q[:n], b.k[0], b.v[0], 64 ** -0.5)
    assert np.all(np.isfinite(o[:ok])) and np.all(np.abs(o[:ok] - ref[:ok]) <= 2.0 ** -6 * mass[:ok])
    assert np.all(np.isnan(o[ok:n, :, 5]))
    b.check(out, lse, skip=(0,))


@pytest.mark.parametrize("kv", at.KV_TYPES)
@pytest.mark.parametrize("D", [64, 80, 128, 256])
def test_the_same_bits_every_time(D, kv):
    for seqs in (SMALL, MIXED, LARGE):
        b = Batch(seqs, 2, 1, D, kv, 16, seed=17)
        q = _dev(b.q)
        first = [t.clone() for t in b.run(q=q)]
        for _ in range(10):
            for x, y in zip(b.run(q=q), first):
                assert torch.equal(x.view(torch.uint8), y.view(torch.uint8))


def test_strided_queries_and_given_outputs():
    lib = _lib()
    for seqs in (SMALL, LARGE):
        b = Batch(seqs, 4, 2, 64, "int8", 16, seed=11)
        T = b.q.shape[0]
        fused = torch.zeros(T, 8, 64, dtype=torch.bfloat16, device="cuda")
        fused[:, :4] = _dev(b.q)
        out = torch.empty(T, 4, 64, dtype=torch.bfloat16, device="cuda")
        lse = torch.empty(T, 4, dtype=torch.float32, device="cuda")
        o, s = b.run(q=fused[:, :4], out=out, lse=lse)
        assert o.data_ptr() == out.data_ptr() and s.data_ptr() == lse.data_ptr()
        b.check(out, lse)
        o, s = b.run(lse=False)
        assert s is None and torch.equal(o.view(torch.int16), out.view(torch.int16))
        need = lib.attend_paged_workspace_bytes(b.cache, T, 4, len(seqs), **b.bounds)
        if need:
            with pytest.raises(ValueError):
                b.run(workspace=torch.empty(need - 1, dtype=torch.uint8, device="cuda"))


def test_a_cache_past_32_bits():
    """Rows whose byte offsets pass 2^32 and whose numbers pass 2^31 elements."""
    lib = _lib()
    h, D, page = 8, 128, 1024
    pages = (1 << 32) // (h * page * D * 2) * 2 + 3                      # 8 GiB of keys, and of values
    cache = lib.KVCache.empty(pages, h, page, D, kv_type="bf16")
    rng = _rng(12)
    m = 1030
    table = np.array([[pages - 1, pages - 2]])
    j = np.arange(m)
    slots = table[0, j // page] * page + j % page
    k, v = _bf16(rng, m, h, D), _bf16(rng, m, h, D)
    lib.kv_write(cache, _dev(k), _dev(v), torch.tensor(slots).cuda())
    kr, vr = lib.kv_read(cache, torch.tensor(slots).cuda())
    assert np.array_equal(_host(kr), k) and np.array_equal(_host(vr), v)
    for n in (1, 70):
        q = _bf16(rng, n, h, D)
        out, _ = lib.attend_paged(_dev(q), cache, _i32(table), _i32([0, n]), _i32([m]), max_new=n, max_len=m)
        ref, _, mass = at.attend(q, k, v, D ** -0.5)
        assert np.all(np.abs(_host(out) - ref) <= 2.0 ** -8 * mass + 2.0 ** -8 * np.abs(ref))
    _status_ok()


def test_indices_out_of_range_are_reported():
    lib = _lib()
    for seqs in (SMALL, LARGE):
        good = Batch(seqs, 2, 1, 64, "int8", 16, seed=13)
        for what in ("page", "negative page", "length", "negative length", "starts", "end", "new"):
            b = Batch(seqs, 2, 1, 64, "int8", 16, seed=13)
            table, starts, lengths = b.table.copy(), b.starts.copy(), np.array([m for _, m in seqs])
            if what == "page":
                table[2, 0] = b.cache.pages
            elif what == "negative page":
                table[2, 0] = -1
            elif what == "length":
                lengths[2] = 10 ** 6
            elif what == "negative length":
                lengths[2] = -4
            elif what == "starts":
                starts[2] = -5
            elif what == "end":
                starts[-1] += 1000
            else:
                b.bounds["max_new"] = max(b.n) - 1
                if b.bounds["max_new"] == 0:
                    continue
            b.pages, b.dstarts, b.lengths = _i32(table), _i32(starts), _i32(lengths)
            b.run()
            with pytest.raises(lib.QLoRAError, match="QLORA_ERR_INDEX"):
                lib.device_status()
        good.check(*good.run())


def test_another_stream_and_a_captured_graph():
    """Work on a stream of its own, and a captured decode step replayed with
    new contents, equal the eager result every time."""
    lib = _lib()
    b = Batch([(1, 700), (1, 40), (1, 1)], 8, 2, 128, "int8", 16, seed=14)
    want = [t.clone() for t in b.run()]
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    q = _dev(b.q)
    ws = torch.empty(max(16, lib.attend_paged_workspace_bytes(b.cache, 3, 8, 3, **b.bounds)), dtype=torch.uint8, device="cuda")
    table = lib.rope_table(1024, 128)
    pos = _i32([699, 39, 0])
    new_k, new_v = _dev(_bf16(_rng(15), 3, 2, 128)), _dev(_bf16(_rng(16), 3, 2, 128))
    slots = torch.tensor([int(b.table[i, (m - 1) // 16] * 16 + (m - 1) % 16) for i, (_, m) in enumerate(b.seqs)], device="cuda")
    turned, out = torch.empty_like(q), torch.empty_like(q)
    with torch.cuda.stream(side):
        got = b.run(q=q, workspace=ws)
    side.synchronize()
    for x, y in zip(got, want):
        assert torch.equal(x.view(torch.uint8), y.view(torch.uint8))

    def step():
        lib.rope(q, None, table, pos, q_out=turned)
        lib.kv_write(b.cache, new_k, new_v, slots, table=table, positions=pos)
        lib.attend_paged(turned, b.cache, b.pages, b.dstarts, b.lengths, out=out, workspace=ws, **b.bounds)

    step()
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        step()
    for i in range(4):
        rng = _rng(20 + i)
        q.copy_(_dev(_bf16(rng, 3, 8, 128)))
        new_k.copy_(_dev(_bf16(rng, 3, 2, 128)))
        new_v.copy_(_dev(_bf16(rng, 3, 2, 128)))
        out.zero_()
        graph.replay()
        torch.cuda.synchronize()
        first = out.clone()
        out.zero_()
        step()
        torch.cuda.synchronize()
        assert torch.equal(first.view(torch.int16), out.view(torch.int16)) and bool(out.abs().sum() > 0)


@pytest.mark.parametrize("seed", range(10))
def test_random_problems(seed):
    rng = _rng(1000 + seed)
    h = int(rng.integers(1, 5))
    hq, D = h * int(rng.integers(1, 9)), 16 * int(rng.integers(1, 17))
    page, kv = int(rng.choice([16, 32, 64, 256])), at.KV_TYPES[seed % 5]
    top = int(rng.choice([1, 4, 200]))
    seqs = [(int(rng.integers(0, top + 1)), int(rng.integers(0, 500))) for _ in range(int(rng.integers(1, 6)))]
    seqs[0] = (top, 500)
    causal, window = bool(rng.random() < 0.8), int(rng.choice([0, 0, 30, 250]))
    print(seed, h, hq, D, page, kv, seqs, causal, window, flush=True)
    b = Batch(seqs, hq, h, D, kv, page, seed=seed)
    b.check(*b.run(causal=causal, window=window), causal=causal, window=window)
