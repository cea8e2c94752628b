"""Weights of more elements than one launch counts threads for: what lies around
the cut between two launches, and at the end, equals what the same weights give
on their own."""

import pytest

pytestmark = pytest.mark.gpu

torch = pytest.importorskip("torch")

CUT, SPAN = 1 << 33, 1 << 15          # elements of a launch; elements looked at on each side (groups of 2^14)


def _room(gigabytes):
    torch.cuda.empty_cache()
    if torch.cuda.mem_get_info()[0] < gigabytes * 1e9:
        pytest.skip("not enough free memory")


@pytest.fixture(autouse=True)
def _give_back():
    yield
    torch.cuda.empty_cache()


def _random(n, seed):
    g = torch.Generator(device="cuda").manual_seed(seed)
    return torch.randn(n, generator=g, device="cuda").bfloat16()


def test_quantizers_past_one_launch():
    import bit_nf4_quantized_21_amd as lib
    _room(40)
    n = CUT + SPAN
    w = torch.zeros(n, dtype=torch.bfloat16, device="cuda")
    w[CUT - SPAN:] = _random(2 * SPAN, 1)
    last = w[CUT - SPAN:].clone()
    codes, absmax = lib.quantize_nf4(w)
    want, want_max = lib.quantize_nf4(last)
    assert torch.equal(codes[(CUT - SPAN) // 2:], want) and torch.equal(absmax[(CUT - SPAN) // 64:], want_max)
    del codes, absmax
    for t, u in zip(lib.quantize_dq(w), lib.quantize_dq(last)):
        assert torch.equal(t[t.numel() - u.numel():], u)


def test_double_quant_past_one_launch():
    import bit_nf4_quantized_21_amd as lib
    _room(60)
    absmax = torch.zeros(CUT + 1024, dtype=torch.float32, device="cuda")
    absmax[CUT - 1024:] = _random(2048, 2).float().abs()
    last = absmax[CUT - 1024:].clone()
    for t, u in zip(lib.double_quant(absmax), lib.double_quant(last)):
        assert torch.equal(t[t.numel() - u.numel():], u)


def test_dequantize_past_32_bits_of_threads():
    """2^35 weights take 2^32 threads: the last ones were not written."""
    import bit_nf4_quantized_21_amd as lib
    _room(100)
    n = (1 << 35) + SPAN
    codes8, q88, s28 = lib.quantize_dq(_random(2 * SPAN, 3))
    codes = torch.zeros(n // 2, dtype=torch.uint8, device="cuda")
    q8 = torch.full((n // 64,), 128, dtype=torch.uint8, device="cuda")
    s2 = torch.ones(n // 16384, dtype=torch.float32, device="cuda")
    for big, small in ((codes, codes8), (q8, q88), (s2, s28)):
        big[big.numel() - small.numel():] = small
        half = small.numel() // 2
        at = CUT * small.numel() // (2 * SPAN)
        big[at - half:at + half] = small
    out = lib.dequantize_nf4(codes, q8, s2, n)
    want = lib.dequantize_nf4(codes8, q88, s28, 2 * SPAN)
    assert torch.equal(out[n - 2 * SPAN:].view(torch.int16), want.view(torch.int16))
    assert torch.equal(out[CUT - SPAN:CUT + SPAN].view(torch.int16), want.view(torch.int16))
