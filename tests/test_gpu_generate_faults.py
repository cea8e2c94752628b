"""Calls of the attention side that once went wrong: one test per fault, on the
mended code."""

import ctypes

import numpy as np
import pytest

from oracle import attention as at
from test_gpu_generate import Batch, _dev, _host, _i32, _lib

pytestmark = pytest.mark.gpu

torch = pytest.importorskip("torch")


@pytest.mark.parametrize("kv", ["bf16", "int8", "nf4", "fp4"])
@pytest.mark.parametrize("n", [1, 20, 90])
def test_nothing_stored_needs_no_table_of_pages(n, kv):
    """max_len = 0 with a null table, though a sequence may have pages (the
    single-token kernel read its entries before it knew the lengths)."""
    from bit_nf4_quantized_21_amd import qlora
    lib = _lib()
    cache = lib.KVCache.empty(3, 2, 16, 64, kv_type=kv)
    q = torch.ones(2 * n, 4, 64, dtype=torch.bfloat16, device="cuda")
    out = torch.full((2 * n, 4, 64), 7.0, dtype=torch.bfloat16, device="cuda")
    lse = torch.zeros(2 * n, 4, dtype=torch.float32, device="cuda")
    starts, lengths = _i32([0, n, 2 * n]), _i32([0, 0])
    heads = qlora.Heads(q.data_ptr(), 256, 64, 4)
    for window in (0, 9):
        rc = qlora.lib().qlora_attend_paged(ctypes.byref(cache._desc), 2 * n, ctypes.byref(heads), 2, None, 4, starts.data_ptr(),
                                            lengths.data_ptr(), n, 0, 0.125, 1, window, out.data_ptr(), lse.data_ptr(), None,
                                            0, None)
        assert rc == 0
        torch.cuda.synchronize()
        assert torch.all(out == 0) and torch.all(lse == float("-inf"))
        out.fill_(7.0)
        lse.zero_()
    lib.device_status()


def _busy(cycles=200_000_000):
    """Keep the current stream at work for a while."""
    torch.cuda._sleep(cycles)


def test_workspace_and_outputs_of_a_call_on_another_stream():
    """A block that work queued on the current stream still has to read is not
    taken by a call on another stream, and an output dropped on the current
    stream is not given to the other stream's next call before that work ran."""
    lib = _lib()
    b = Batch([(1, 4000), (1, 1), (1, 2047)], 8, 2, 128, "int8", 64, seed=5, pad=3)
    want, want_lse = (t.clone() for t in b.run())
    q = _dev(b.q)
    nbytes = lib.attend_paged_workspace_bytes(b.cache, 3, 8, 3, **b.bounds)
    assert nbytes > 0
    side = torch.cuda.Stream()
    sizes = (nbytes, want.numel() * 2, want_lse.numel() * 4)
    torch.cuda.synchronize()
    torch.cuda.empty_cache()
    held = [torch.full((n,), 3, dtype=torch.uint8, device="cuda") for n in sizes]
    side.wait_stream(torch.cuda.current_stream())
    _busy()
    copies = [t.clone() for t in held]
    del held
    out, lse = b.run(q=q, stream=side)
    torch.cuda.current_stream().wait_stream(side)
    torch.cuda.synchronize()
    assert all(bool((c == 3).all()) for c in copies)
    assert torch.equal(out.view(torch.int16), want.view(torch.int16)) and torch.equal(lse, want_lse)

    torch.cuda.current_stream().wait_stream(side)
    _busy()
    copy = out.clone()
    del out, lse
    other, _ = b.run(q=-q, stream=side)
    torch.cuda.synchronize()
    assert torch.equal(copy.view(torch.int16), want.view(torch.int16))
    assert not torch.equal(other.view(torch.int16), want.view(torch.int16))


def test_other_calls_on_another_stream():
    """Rotation, cache and linear calls with stream=: what they allocate is not
    what the current stream still reads."""
    lib = _lib()
    side = torch.cuda.Stream()
    T, K, N, r = 64, 512, 512, 16
    g = torch.Generator(device="cuda").manual_seed(1)
    w = torch.randn(N, K, generator=g, device="cuda") * 0.02
    x = torch.randn(T, K, generator=g, device="cuda").bfloat16()
    a, bb = (torch.randn(*s, generator=g, device="cuda").bfloat16() for s in ((K, r), (r, N)))
    heads = x.view(T, 4, 128)
    table, pos = lib.rope_table(64, 128), _i32(range(T))
    cache = lib.KVCache.empty(5, 4, 16, 128)
    slots = torch.arange(T, device="cuda")
    lib.kv_write(cache, heads, heads, slots)
    codes, q8, s2 = lib.quantize_dq(w)

    def calls(**kw):
        codes1, q81, s21 = lib.quantize_dq(w, **kw)
        y, xa = lib.linear_fwd(x, codes, q8, s2, a, bb, 16.0, N, **kw)
        grads = lib.linear_bwd(y, x, xa, codes, q8, s2, a, bb, 16.0, **kw)
        turned, _ = lib.rope(heads, None, table, pos, **kw)
        return (codes1, q81, s21, y, xa, *grads, turned, *lib.kv_read(cache, slots, **kw), lib.rope_table(64, 128, **kw),
                lib.dequantize_nf4(codes, q8, s2, N * K, **kw))

    want = calls()
    sizes = [t.numel() * t.element_size() for t in want]
    sizes += [lib.linear_fwd_workspace_bytes(T, K, N, r), lib.linear_bwd_workspace_bytes(T, K, N, r)]
    torch.cuda.synchronize()
    torch.cuda.empty_cache()
    held = [torch.full((max(1, n),), 3, dtype=torch.uint8, device="cuda") for n in sizes]
    side.wait_stream(torch.cuda.current_stream())
    _busy()
    copies = [t.clone() for t in held]
    del held
    got = calls(stream=side)
    torch.cuda.synchronize()
    assert all(bool((c == 3).all()) for c in copies)
    for t, u in zip(got, want):
        assert torch.equal(t.view(torch.uint8), u.view(torch.uint8))


@pytest.mark.parametrize("kv", ["bf16", "int8", "nf4", "fp4"])
@pytest.mark.parametrize("n,hq,h,D", [(4, 2, 1, 64), (100, 2, 1, 64), (130, 4, 2, 128), (100, 2, 2, 80)])
@pytest.mark.parametrize("bad", [float("nan"), float("inf"), float("-inf")])
def test_a_value_that_is_no_number_leaves_the_log_sum_alone(n, hq, h, D, kv, bad):
    """lse is a function of the scores, so a value (or its scale) that is no
    number must not change a bit of it, whether the key lies at the edge of what
    the rows see or where all of them see it.  Rows that do not see the key keep
    every bit of their outputs; those that see it are no numbers in its dim."""
    b = Batch([(n, 900), (n, 0), (n, 701)], hq, h, D, kv, 16, seed=21)
    first = b.run()
    b.check(*first)
    for kw in (dict(), dict(window=200), dict(causal=False)):
        out, lse = b.run(**kw)
        for key in (899, 898 - n // 2, 900 - n, 890 - n, 300):
            page, off = int(b.table[0, key // 16]), key % 16
            where = (page, h - 1, off, 5) if kv == "bf16" else (page, h - 1, off)
            buffer = b.cache.v if kv == "bf16" else b.cache.v_scale
            kept = buffer[where].clone()
            buffer[where] = bad
            got, got_lse = b.run(**kw)
            buffer[where] = kept
            assert torch.equal(got_lse.view(torch.int32), lse.view(torch.int32)), (key, kw)
            at = torch.arange(900 - n, 900, device="cuda")
            sees = (at >= key) if kw.get("causal", True) else torch.ones_like(at, dtype=torch.bool)
            if "window" in kw:
                sees &= key > at - kw["window"]
            mine = torch.zeros(got.shape[0], hq, dtype=torch.bool, device="cuda")
            mine[:n, hq - hq // h:] = sees[:, None]
            assert torch.equal(got[~mine].view(torch.int16), out[~mine].view(torch.int16)), (key, kw)
            assert not bool(torch.isfinite(got[mine][:, 5]).any()), (key, kw)


@pytest.mark.parametrize("n", [1, 20, 90])
def test_rows_outside_of_all_sequences_are_reported(n):
    """starts that begin after the first token or end before the last one leave
    rows unwritten; a padding sequence of length 0 gives zeros instead."""
    lib = _lib()
    b = Batch([(n, n + 40), (n, n + 3), (4, 0)], 4, 2, 64, "int8", 16, seed=31)
    out, lse = b.run()
    b.check(out, lse)
    assert torch.all(out[2 * n:] == 0) and torch.all(lse[2 * n:] == float("-inf"))
    full = b.dstarts.clone()
    for starts in ([1, n, 2 * n, 2 * n + 4], [0, n, 2 * n, 2 * n + 3], [0, n, 2 * n, 2 * n]):
        b.dstarts = _i32(starts)
        got, _ = b.run()
        with pytest.raises(lib.QLoRAError, match="QLORA_ERR_INDEX"):
            lib.device_status()
        rows = slice(n, 2 * n)                     # a sequence that is whole keeps its results
        assert torch.equal(got[rows].view(torch.int16), out[rows].view(torch.int16))
    b.dstarts = full
    b.check(*b.run())


def test_tokens_of_no_sequence_are_refused():
    lib = _lib()
    b = Batch([(2, 9)], 4, 2, 64, "int8", 16, seed=32)
    q = _dev(b.q)
    with pytest.raises(ValueError, match="tokens of no sequence"):
        lib.attend_paged(q, b.cache, b.pages, b.dstarts, b.lengths, max_new=0, max_len=9)
    with pytest.raises(ValueError, match="tokens of no sequence"):
        lib.attend_paged(q, b.cache, b.pages[:0], b.dstarts[:1], b.lengths[:0], max_new=2, max_len=9)
    out, _ = lib.attend_paged(q[:0], b.cache, b.pages[:0], b.dstarts[:1], b.lengths[:0], max_new=0, max_len=0)
    assert out.shape == (0, 4, 64)


@pytest.mark.parametrize("kv,n,D", [("bf16", 40, 64), ("bf16", 40, 80), ("int8", 40, 64), ("int8", 130, 64), ("nf4", 130, 128),
                                    ("fp4", 33, 48)])
def test_keys_past_a_list_of_pages(kv, n, D):
    """Row tiles that fill the chip walk all keys of a sequence, past what their
    list of pages holds at a time (8192 keys), once and more than once, and to
    lengths around its end; nothing is split, so there is no workspace."""
    lib = _lib()
    long = [8176, 8177, 8192, 8193, 8257, 17000]
    h, batch = (8 if n <= 128 else 4), 128
    seqs = [(n, m) for m in long] + [(n, n + 7 * i) for i in range(batch - len(long))]
    b = Batch(seqs, h, h, D, kv, 16, seed=40)
    assert lib.attend_paged_workspace_bytes(b.cache, n * batch, h, batch, **b.bounds) == 0
    few = range(len(long), batch - 3)               # the oracle takes its time: the long ones and three short ones
    b.check(*b.run(), skip=few)
    b.check(*b.run(window=8400), window=8400, skip=few)


def test_a_long_prompt_needs_no_workspace():
    """One prompt of 9000 tokens and 52 heads: rows at its ends and in between against the oracle's."""
    lib = _lib()
    n, h, D, page = 9000, 52, 64, 16
    g = torch.Generator(device="cuda").manual_seed(3)
    q, k, v = (torch.randn(n, h, D, generator=g, device="cuda").bfloat16() for _ in range(3))
    pages = -(-n // page)
    cache = lib.KVCache.empty(pages, h, page, D, kv_type="bf16")
    lib.kv_write(cache, k, v, torch.arange(n, device="cuda"))
    table = torch.arange(pages, dtype=torch.int32, device="cuda")[None].contiguous()
    assert lib.attend_paged_workspace_bytes(cache, n, h, 1, n, n) == 0
    out, lse = lib.attend_paged(q, cache, table, _i32([0, n]), _i32([n]), max_new=n, max_len=n, lse=True)
    for i in (0, 63, 127, 128, 4500, 8191, 8192, 8300, 8999):
        ref, rl, mass = at.attend(_host(q[i:i + 1]), _host(k[:i + 1]), _host(v[:i + 1]), D ** -0.5)
        # The weights' rounding to bf16 and the output's; scores in fp32 (sum |q k| below 100 of the scale here).
        assert np.all(np.abs(_host(out[i:i + 1]) - ref) <= mass * (2.0 ** -8 + 2.0 ** -13) + 2.0 ** -8 * np.abs(ref))
        assert np.all(np.abs(lse[i:i + 1].cpu().numpy() - rl) <= 2.0 ** -14)
    lib.device_status()


def test_given_outputs_of_another_shape_are_refused():
    """A buffer with the output's axes in another order would be filled as if
    they were its own; longer and flat ones hold the rows in order."""
    lib = _lib()
    b = Batch([(3, 20), (2, 9)], 4, 2, 64, "int8", 16, seed=33)
    want, want_lse = b.run()
    bf16, f32 = dict(dtype=torch.bfloat16, device="cuda"), dict(dtype=torch.float32, device="cuda")
    for shape in ((4, 5, 64), (5, 64, 4), (10, 2, 64)):
        with pytest.raises(ValueError, match="out must be"):
            b.run(out=torch.empty(shape, **bf16))
    with pytest.raises(ValueError, match="lse must be"):
        b.run(lse=torch.empty((4, 5), **f32))
    with pytest.raises(ValueError, match="elements"):
        b.run(out=torch.empty((4, 4, 64), **bf16))
    for shape in ((5, 4, 64), (7, 4, 64), (5, 256), (2000,)):
        out, lse = torch.empty(shape, **bf16), torch.empty(shape[:1] + (4,), **f32)
        b.run(out=out, lse=lse)
        assert torch.equal(out.view(-1)[:1280].view(torch.int16), want.view(-1).view(torch.int16))
        assert torch.equal(lse.view(-1)[:20], want_lse.view(-1))
    slots = torch.arange(6, device="cuda")
    k, v = lib.kv_read(b.cache, slots)
    with pytest.raises(ValueError, match="k_out must be"):
        lib.kv_read(b.cache, slots, k_out=torch.empty((2, 6, 64), **bf16))
    with pytest.raises(ValueError, match="v_out must be"):
        lib.kv_read(b.cache, slots, v_out=torch.empty((64, 6, 2), **bf16))
    longer = torch.empty((9, 2, 64), **bf16)
    lib.kv_read(b.cache, slots, k_out=longer, v_out=torch.empty(6 * 128, **bf16))
    assert torch.equal(longer[:6].view(torch.int16), k.view(torch.int16))
