"""Refusals of the training step's entry points: argument errors come back as
the documented status before anything is enqueued (no GPU is touched), and the
binding's own checks."""

import ctypes

import pytest

from bit_nf4_quantized_21_amd import qlora, train

OK, ENULL, ESHAPE, EALIGN, EUNSUP, EHIP, EWS = 0, -1, -2, -3, -4, -5, -6
A = 0x10000                       # aligned, never dereferenced: validation fails first
P, MIS = ctypes.c_void_p(A), ctypes.c_void_p(A + 4)


@pytest.fixture(scope="module")
def L():
    return qlora.lib()


def W(codes=A, q8=A, s2=A, a=A, b=A):
    return ctypes.byref(qlora.AdaptedWeight(codes, q8, s2, a, b))


def test_gated_fwd(L):
    def f(qtype=0, act=0, X=P, T=32, K=128, N=64, gate=W(), up=W(), r=8, H=P, saved=P, XA=P, ws=P, wsb=1 << 30):
        return L.qlora_gated_fwd(qtype, act, X, T, K, N, gate, up, r, 16.0, H, saved, XA, ws, wsb, None)
    assert f(qtype=3) == EUNSUP and f(act=3) == EUNSUP and f(act=-1) == EUNSUP
    assert f(r=7) == EUNSUP and f(r=136) == EUNSUP and f(r=0) == EUNSUP
    assert f(K=96) == ESHAPE and f(K=0) == ESHAPE and f(N=12) == ESHAPE and f(N=0) == ESHAPE and f(T=-1) == ESHAPE
    assert f(T=1 << 30) == ESHAPE                                    # T*K*2 past a 32-bit view
    for side in ("gate", "up"):
        assert f(**{side: None}) == ENULL
        for name in ("codes", "q8", "s2", "a", "b"):
            assert f(**{side: W(**{name: None})}) == ENULL and f(**{side: W(**{name: A + 8})}) == EALIGN
    assert f(X=None) == ENULL and f(H=None) == ENULL and f(XA=None) == ENULL
    assert f(X=MIS) == EALIGN and f(H=MIS) == EALIGN and f(XA=MIS) == EALIGN and f(saved=MIS) == EALIGN
    for T in (1, 16, 17, 32):
        need = L.qlora_gated_fwd_workspace_bytes(T, 128, 64, 8)
        assert need > 0 and f(T=T, wsb=need - 1) == EWS and f(T=T, ws=None) == EWS
    assert f(ws=MIS) == EALIGN
    assert f(T=0, X=None, gate=None, up=None, H=None, XA=None, ws=None) == OK


def test_gated_bwd(L):
    def f(qtype=0, dH=P, X=P, saved=P, XA=P, T=32, K=128, N=64, gate=W(), up=W(), r=8, dX=P, dAg=P, dBg=P, dAu=P, dBu=P,
          ws=P, wsb=1 << 30):
        return L.qlora_gated_bwd(qtype, dH, X, saved, XA, T, K, N, gate, up, r, 16.0, dX, dAg, dBg, dAu, dBu, ws, wsb,
                                 None)
    assert f(qtype=-1) == EUNSUP and f(r=12) == EUNSUP and f(K=65) == ESHAPE and f(N=4) == ESHAPE and f(T=-5) == ESHAPE
    for name in ("dH", "X", "saved", "dX", "dAg", "dBg", "dAu", "dBu"):
        assert f(**{name: None}) == ENULL, name
        assert f(**{name: MIS}) == EALIGN, name
    assert f(XA=MIS) == EALIGN
    assert f(gate=None) == ENULL and f(up=W(s2=None)) == ENULL and f(up=W(b=A + 2)) == EALIGN
    for T in (1, 32):
        need = L.qlora_gated_bwd_workspace_bytes(T, 128, 64, 8)
        assert need > 0 and f(T=T, wsb=need - 1) == EWS and f(T=T, ws=None) == EWS
    assert f(T=0, dAg=None) == ENULL and f(T=0, dBu=MIS) == EALIGN


def test_gated_workspace(L):
    assert L.qlora_gated_fwd_workspace_bytes(0, 128, 64, 8) == 0 and L.qlora_gated_bwd_workspace_bytes(0, 128, 64, 8) == 0
    for bad in ((32, 100, 64, 8), (32, 128, 63, 8), (32, 128, 64, 9), (-1, 128, 64, 8)):
        assert L.qlora_gated_fwd_workspace_bytes(*bad) == 0 and L.qlora_gated_bwd_workspace_bytes(*bad) == 0
    # dG and dU (2 T N 2 bytes) at the least, and not many times that.
    for T, K, N in ((512, 8192, 22016), (2048, 4096, 11008), (4096, 6656, 17920)):
        assert 4 * T * N <= L.qlora_gated_bwd_workspace_bytes(T, K, N, 64) < 8 * T * N + (1 << 30)


def test_head_loss(L):
    def f(X=P, T=5, K=128, w=P, V=1000, targets=P, dloss=None, loss=P, lse=P, mean=P, dX=P, ws=P, wsb=1 << 33):
        return L.qlora_head_loss(X, T, K, w, V, targets, dloss, loss, lse, mean, dX, ws, wsb, None)
    assert f(T=-1) == ESHAPE and f(K=32) == ESHAPE and f(K=100) == ESHAPE and f(K=(1 << 20) + 64) == ESHAPE
    assert f(V=0) == ESHAPE and f(V=(1 << 30) + 1) == ESHAPE and f(T=(1 << 23) + 1, K=64, V=10) == ESHAPE
    assert f(T=1 << 23) == ESHAPE                              # T*K*2 = 2^31
    assert f(T=1 << 20, K=64, V=1 << 20) == ESHAPE             # too many sums
    for name in ("X", "w", "targets", "loss", "lse", "mean"):
        assert f(**{name: None}) == ENULL, name
        assert f(**{name: MIS}) == EALIGN, name
    assert f(dX=MIS) == EALIGN and f(dloss=MIS) == EALIGN
    for T, dX in ((5, P), (5, None), (300, P), (5000, P)):
        need = L.qlora_head_loss_workspace_bytes(T, 128, 1000, 0 if dX is None else 1)
        assert need > 0 and f(T=T, dX=dX, wsb=need - 1) == EWS and f(T=T, dX=dX, ws=None) == EWS
    assert f(ws=MIS) == EALIGN
    assert f(T=0, mean=None) == ENULL


def test_head_loss_workspace(L):
    f = L.qlora_head_loss_workspace_bytes
    assert f(0, 128, 1000, 1) == 0 and f(5, 100, 1000, 1) == 0 and f(5, 128, 0, 1) == 0
    # Without a gradient: sums and lists; with one, no more than is said, however many tokens.
    assert f(4096, 4096, 128000, 0) < 8 * 4096 * 1000 + (1 << 20)
    for T, K, V in ((4096, 4096, 128000), (16384, 4096, 128000), (512, 8192, 32000), (65, 64, 1 << 20)):
        assert f(T, K, V, 1) < (130 << 20) + max(4 * 4096 * K, 64 << 20) + 8 * min(T, 4096) * (V // 128 + 1) + 16 * T + (1 << 20)


def G(*entries):
    arr = (qlora.Grad * max(1, len(entries)))()
    for i, e in enumerate(entries):
        arr[i] = qlora.Grad(*e)
    return arr


def test_clip_grads(L):
    def f(*entries, count=None, max_norm=1.0, norm=P, ws=P, wsb=1 << 30):
        return L.qlora_clip_grads(len(entries) if count is None else count, G(*entries) if entries else None, max_norm, norm,
                                  ws, wsb, None)
    one = (A, A + 4096, 100, 0, 0)
    assert f(count=-1) == ESHAPE and f(count=65537) == ESHAPE and f(count=1) == ENULL
    assert f((A, A, -1, 0, 0)) == ESHAPE and f((A, A, (1 << 40) + 1, 0, 0)) == ESHAPE
    assert f((A, A, 4, 2, 0)) == EUNSUP and f((A, A, 4, 0, -1)) == EUNSUP and f(one, max_norm=float("nan")) == EUNSUP
    assert f((None, A, 4, 0, 0)) == ENULL
    assert f((A + 1, A, 4, 0, 0)) == EALIGN and f((A + 2, A, 4, 1, 1)) == EALIGN and f((A, A + 2, 4, 1, 1)) == EALIGN
    assert f((A, A, 4, 0, 1)) == ESHAPE                              # in place, but of another type
    assert f(one, one) == ESHAPE                                     # the same output twice
    assert f((A, A, 100, 0, 0), (A + 198, A + 198, 10, 0, 0)) == ESHAPE    # one value shared
    assert f((A, A + 8192, 100, 0, 0), (A + 4096, A + 8192 + 198, 100, 0, 0)) == ESHAPE
    assert f((A, A + 100, 100, 0, 0)) == ESHAPE                      # an output inside its gradient
    assert f((A, A + 8192, 100, 0, 0), (A + 4096, A + 100, 10, 0, 0)) == ESHAPE    # ... inside another's
    assert f(one, norm=MIS) == EALIGN
    need = L.qlora_clip_grads_workspace_bytes(1)
    assert f(one, wsb=need - 1) == EWS and f(one, ws=None) == EWS and f(one, ws=MIS) == EALIGN
    # What is accepted comes as far as the workspace: neighbours, in place, no output, the norm alone.
    short = dict(wsb=8)
    assert f((A, A, 100, 0, 0), (A + 200, A + 200, 10, 0, 0), **short) == EWS
    assert f((A, None, 100, 0, 0), (A, None, 100, 0, 0), **short) == EWS
    assert f(one, one, max_norm=0.0, **short) == EWS
    assert f((None, None, 0, 0, 0), **short) == EWS
    assert f((A + 2, A + 8194, 7, 0, 0), **short) == EWS             # aligned to the elements


def test_clip_grads_workspace(L):
    f = L.qlora_clip_grads_workspace_bytes
    assert f(-1) == 0 and f(65537) == 0 and 0 < f(0) <= f(1) <= f(448) < 1 << 20


def test_binding_refuses_what_is_no_gpu_tensor():
    import torch
    x = torch.zeros(4, 64, dtype=torch.bfloat16)
    with pytest.raises(ValueError):
        train.gated_fwd(x, {}, {}, 16.0)
    with pytest.raises(ValueError):
        train.head_loss(x, x, torch.zeros(4, dtype=torch.int64))
    with pytest.raises(ValueError):
        train.clip_grads([x], 1.0)
    with pytest.raises(TypeError):
        train.clip_grads([1.0], 1.0)
    with pytest.raises(TypeError):
        train.clip_grads([x.half()], 1.0)
    with pytest.raises(ValueError):
        train.GradSet([x], [])
