"""Refusals of the attention side's entry points: argument errors come back as
the documented status before anything is enqueued (no GPU is touched), and the
binding's own checks."""

import ctypes

import pytest

from bit_nf4_quantized_21_amd import generate, qlora

OK, ENULL, ESHAPE, EALIGN, EUNSUP, EHIP, EWS = 0, -1, -2, -3, -4, -5, -6
A = 0x10000                       # aligned, never dereferenced: validation fails first
P, MIS = ctypes.c_void_p(A), ctypes.c_void_p(A + 4)


@pytest.fixture(scope="module")
def L():
    return qlora.lib()


def H(data=A, token=256, head=64, heads=4):
    return ctypes.byref(qlora.Heads(data, token, head, heads))


def C(k=A, v=A, ks=A, vs=A, pages=10, type=1, heads=4, dim=64, page=16):
    return ctypes.byref(qlora.KVCacheDesc(k, v, ks, vs, pages, type, heads, dim, page))


def test_index_status_string(L):
    assert L.qlora_status_string(-10).startswith(b"QLORA_ERR_INDEX")


def test_rope_table(L):
    f = L.qlora_rope_table
    assert f(8, 24, 1e4, 0, 1.0, 0.0, 1.0, 32.0, 1.0, P, None) == EUNSUP
    assert f(8, 272, 1e4, 0, 1.0, 0.0, 1.0, 32.0, 1.0, P, None) == EUNSUP
    assert f(8, 64, 0.0, 0, 1.0, 0.0, 1.0, 32.0, 1.0, P, None) == EUNSUP
    assert f(8, 64, float("nan"), 0, 1.0, 0.0, 1.0, 32.0, 1.0, P, None) == EUNSUP
    assert f(8, 64, 1e4, 4, 1.0, 0.0, 1.0, 32.0, 1.0, P, None) == EUNSUP
    assert f(8, 64, 1e4, 1, 0.5, 0.0, 1.0, 32.0, 1.0, P, None) == EUNSUP
    assert f(8, 64, 1e4, 3, 2.0, 0.0, 1.0, 32.0, 1.0, P, None) == EUNSUP      # no original context
    assert f(8, 64, 1e4, 3, 2.0, 4096.0, 32.0, 32.0, 1.0, P, None) == EUNSUP  # low = high
    assert f(8, 64, 1e4, 0, 1.0, 0.0, 1.0, 32.0, 0.0, P, None) == EUNSUP      # amplitude
    assert f(-1, 64, 1e4, 0, 1.0, 0.0, 1.0, 32.0, 1.0, P, None) == ESHAPE
    assert f(8, 64, 1e4, 0, 1.0, 0.0, 1.0, 32.0, 1.0, None, None) == ENULL
    assert f(8, 64, 1e4, 0, 1.0, 0.0, 1.0, 32.0, 1.0, MIS, None) == EALIGN
    assert f(0, 64, 1e4, 0, 1.0, 0.0, 1.0, 32.0, 1.0, None, None) == OK


def test_rope(L):
    def f(T=3, dim=64, rot=64, inter=0, inv=0, table=P, n=16, pos=P, q=H(), qo=H(), k=H(), ko=H()):
        return L.qlora_rope(T, dim, rot, inter, inv, table, n, pos, q, qo, k, ko, None)
    assert f(dim=72) == EUNSUP and f(dim=0) == EUNSUP and f(dim=272) == EUNSUP
    assert f(rot=80) == EUNSUP and f(rot=24) == EUNSUP and f(rot=0) == EUNSUP
    assert f(inter=2) == EUNSUP and f(inv=-1) == EUNSUP
    assert f(T=-1) == ESHAPE and f(n=0) == ESHAPE
    assert f(table=None) == ENULL and f(pos=None) == ENULL and f(q=None) == ENULL and f(qo=None) == ENULL
    assert f(k=None) == ENULL and f(ko=None) == ENULL                  # one without the other
    assert f(table=MIS) == EALIGN and f(pos=ctypes.c_void_p(A + 2)) == EALIGN
    assert f(q=H(data=A + 8)) == EALIGN and f(q=H(token=255)) == EALIGN and f(qo=H(head=60)) == EALIGN
    assert f(q=H(heads=0)) == ESHAPE and f(qo=H(heads=5)) == ESHAPE and f(ko=H(heads=2)) == ESHAPE
    assert f(q=H(data=None)) == ENULL
    assert f(T=0, table=None, q=None, qo=None, k=None, ko=None) == OK


def test_cache_write_and_read(L):
    def w(c=C(), T=3, k=H(), v=H(), slots=P, table=None, n=0, pos=None, rot=0, inter=0):
        return L.qlora_kv_write(c, T, k, v, slots, table, n, pos, rot, inter, None)

    def r(c=C(), T=3, slots=P, k=P, v=P):
        return L.qlora_kv_read(c, T, slots, k, v, None)
    for f in (w, r):
        assert f(c=None) == ENULL
        assert f(c=C(type=5)) == EUNSUP and f(c=C(type=-1)) == EUNSUP
        assert f(c=C(dim=40)) == EUNSUP and f(c=C(dim=512)) == EUNSUP
        assert f(c=C(page=24)) == EUNSUP and f(c=C(page=8)) == EUNSUP and f(c=C(page=2048)) == EUNSUP
        assert f(c=C(heads=0)) == ESHAPE and f(c=C(pages=0)) == ESHAPE
        assert f(c=C(k=None)) == ENULL and f(c=C(v=A + 8)) == EALIGN
        assert f(c=C(ks=None)) == ENULL and f(c=C(vs=A + 4)) == EALIGN
        assert f(T=-1) == ESHAPE and f(slots=None) == ENULL and f(slots=MIS) == EALIGN
        assert f(T=0, slots=None, k=None, v=None) == OK
    assert w(k=None) == ENULL and w(v=H(heads=3)) == ESHAPE and w(k=H(data=A + 2)) == EALIGN
    assert w(table=P, n=8, pos=P, rot=24) == EUNSUP and w(table=P, n=8, pos=P, rot=80) == EUNSUP
    assert w(table=P, n=0, pos=P, rot=64) == ESHAPE and w(table=P, n=8, pos=None, rot=64) == ENULL
    assert r(k=None) == ENULL and r(v=MIS) == EALIGN


def test_attend(L):
    def f(c=C(), tokens=8, q=H(), batch=2, pages=P, width=4, starts=P, lengths=P, new=4, length=64, scale=0.1, causal=1,
          window=0, out=P, lse=None, ws=P, wsb=1 << 30):
        return L.qlora_attend_paged(c, tokens, q, batch, pages, width, starts, lengths, new, length, scale, causal,
                                    window, out, lse, ws, wsb, None)
    assert f(c=None) == ENULL and f(q=None) == ENULL and f(c=C(dim=24)) == EUNSUP
    assert f(tokens=-1) == ESHAPE and f(batch=-1) == ESHAPE and f(new=-1) == ESHAPE and f(length=-1) == ESHAPE
    assert f(batch=1 << 17) == ESHAPE and f(window=-1) == ESHAPE
    assert f(length=65) == ESHAPE                                      # more than the pages hold
    assert f(q=H(heads=6)) == ESHAPE and f(q=H(heads=0)) == ESHAPE     # not a multiple of the cache's heads
    assert f(causal=2) == EUNSUP and f(scale=float("inf")) == EUNSUP
    assert f(pages=None) == ENULL and f(starts=None) == ENULL and f(lengths=None) == ENULL and f(out=None) == ENULL
    assert f(out=ctypes.c_void_p(A + 8)) == EALIGN and f(lse=ctypes.c_void_p(A + 2)) == EALIGN
    assert f(q=H(token=4)) == EALIGN
    need = L.qlora_attend_paged_workspace_bytes(C(), 1, 4, 1, 1, 4096, 1, 0)
    assert need > 0
    one = dict(tokens=1, batch=1, new=1, length=4096, width=256)
    assert f(wsb=need - 1, **one) == EWS and f(ws=None, **one) == EWS and f(ws=MIS, wsb=need, **one) == EALIGN
    assert f(tokens=0, starts=None, lengths=None, out=None) == OK
    assert f(batch=0) == OK and f(new=0) == OK
    assert L.qlora_attend_paged_workspace_bytes(C(dim=24), 1, 4, 1, 1, 4096, 1, 0) == 0
    assert L.qlora_attend_paged_workspace_bytes(None, 1, 4, 1, 1, 4096, 1, 0) == 0


def test_binding_refusals():
    torch = pytest.importorskip("torch")
    with pytest.raises(ValueError):
        generate.rope_table(8, 64, scaling="sideways", device="cpu")
    with pytest.raises(ValueError):
        generate.KVCache.empty(4, 2, 16, 64, kv_type="int3", device="cpu")
    with pytest.raises(ValueError):
        generate.KVCache.empty(4, 2, 16, 64, device="cpu")            # not on the GPU
    with pytest.raises(ValueError):
        generate._heads(torch.zeros(2, 3, 16, dtype=torch.bfloat16), "q")
    with pytest.raises(TypeError):
        generate._heads([1], "q")
