"""ctypes binding of the operators of libqlora (include/qlora.h) around a
training step beside the linears: the gated feed-forward block with its
backward, the cross entropy over a vocabulary with its gradient, and the global
norm and clipping of many gradients.  Argument marshalling only, as in qlora.py.
"""

from __future__ import annotations

import ctypes

from .generate import _choice, _given
from .qlora import (AdaptedWeight, Grad, _check, _dev, _empty, _need, _p, _qtype, _stream, _torch, _weight, _workspace,
                    lib)

ACTS = {"silu": 0, "gelu": 1, "gelu_tanh": 2}


def _together(device, **tensors):
    """All of a call's tensors are on one GPU, and that is the current one (whose
    status word and stream the call uses)."""
    if device.index != _torch()._C._cuda_getDevice():
        raise ValueError(f"the tensors are on {device}, which is not the current device")
    for name, t in tensors.items():
        if t is not None and t.device != device:
            raise ValueError(f"{name} is on {t.device}, not on {device}")


def _adapted(w, K, name):
    """qlora_adapted_weight of a dict of codes, q8, s2, A [K,r] and B [r,N], and its N and r."""
    torch = _torch()
    A, B = _dev(w["A"], torch.bfloat16, f"A of {name}"), _dev(w["B"], torch.bfloat16, f"B of {name}")
    if A.dim() != 2 or B.dim() != 2 or A.shape[0] != K or B.shape[0] != A.shape[1]:
        raise ValueError(f"A of {name} must be [K,r] and its B [r,N]")
    codes, q8, s2 = (_dev(w[k], t, f"{k} of {name}")
                     for k, t in (("codes", torch.uint8), ("q8", torch.uint8), ("s2", torch.float32)))
    N, r = B.shape[1], A.shape[1]
    _weight(codes, q8, s2, N, K)
    _together(A.device, B=B, codes=codes, q8=q8, s2=s2)
    return AdaptedWeight(codes.data_ptr(), q8.data_ptr(), s2.data_ptr(), A.data_ptr(), B.data_ptr()), N, r


def _pair(gate, up, X):
    K = X.shape[1]
    g, N, r = _adapted(gate, K, "gate")
    u, N2, r2 = _adapted(up, K, "up")
    _together(X.device, gate=gate["A"], up=up["A"])
    if (N, r) != (N2, r2):
        raise ValueError("gate and up must have the same features and rank")
    return g, u, N, r


def _matrix(t, name):
    torch = _torch()
    _dev(t, torch.bfloat16, name)
    if t.dim() != 2:
        raise ValueError(f"{name} must have two axes")
    return t


def _exactly(t, shape, dtype, name):
    """An input: of these axes and no others (a longer one would be read as if it
    ended sooner, and every axis after the first from the wrong place)."""
    if tuple(_dev(t, dtype, name).shape) != shape:
        raise ValueError(f"{name} must be {list(shape)}, got {list(t.shape)}")
    return t


def _written(t, shape, dtype, name):
    """A given output, and as a tensor of `shape` the part of it that is written
    (the tensor itself where that is all of it)."""
    if tuple(_given(t, shape, dtype, name).shape) == shape:
        return t
    n = 1
    for x in shape:
        n *= x
    return t.view(-1)[:n].view(shape)


def gated_fwd_workspace_bytes(T, K, N, r):
    return int(lib().qlora_gated_fwd_workspace_bytes(T, K, N, r))


def gated_bwd_workspace_bytes(T, K, N, r):
    return int(lib().qlora_gated_bwd_workspace_bytes(T, K, N, r))


def gated_fwd(X, gate, up, alpha, act="silu", save=False, H=None, saved=None, XA=None, workspace=None, stream=None,
              qtype="nf4"):
    """H = act(G) * U of the adapted 4-bit linears gate and up (see
    qlora_gated_fwd): dicts of codes, q8, s2, A [K,r] and B [r,N].

    act: "silu", "gelu" (erf) or "gelu_tanh".  save=True (or a given `saved`)
    keeps what gated_bwd needs.  Returns (H bf16 [T,N], saved int16 [2,T,N] or
    None, XA f32 [2,T,r]); of a given longer `saved` or XA the part that was
    written, which is what gated_bwd takes."""
    torch = _torch()
    T, K = _matrix(X, "X").shape
    g, u, N, r = _pair(gate, up, X)
    code = _choice(ACTS, act, "act")
    H = _empty((T, N), torch.bfloat16, X.device, stream) if H is None else _given(H, (T, N), torch.bfloat16, "H")
    if saved is not None:
        saved = _written(saved, (2, T, N), torch.int16, "saved")
    elif save:
        saved = _empty((2, T, N), torch.int16, X.device, stream)
    if XA is None:
        XA = _empty((2, T, r), torch.float32, X.device, stream)
    else:
        XA = _written(XA, (2, T, r), torch.float32, "XA")
    _together(X.device, H=H, saved=saved, XA=XA, workspace=workspace)
    nbytes = gated_fwd_workspace_bytes(T, K, N, r)
    workspace = _workspace(nbytes, X.device, workspace, stream)
    _check(lib().qlora_gated_fwd(_qtype(qtype), code, _p(X), T, K, N, ctypes.byref(g), ctypes.byref(u), r, float(alpha),
                                 _p(H), _p(saved), _p(XA), _p(workspace), nbytes, _stream(stream)))
    return H, saved, XA


def gated_bwd(dH, X, saved, XA, gate, up, alpha, dX=None, dA_gate=None, dB_gate=None, dA_up=None, dB_up=None,
              workspace=None, stream=None, qtype="nf4"):
    """Gradients of gated_fwd from its saved and XA (XA may be None: recomputed).
    Returns (dX bf16 [T,K], dA_gate, dB_gate, dA_up, dB_up)."""
    torch = _torch()
    T, K = _matrix(X, "X").shape
    g, u, N, r = _pair(gate, up, X)
    if tuple(_matrix(dH, "dH").shape) != (T, N):
        raise ValueError("dH must be [T,N]")
    _exactly(saved, (2, T, N), torch.int16, "saved")
    if XA is not None:
        _exactly(XA, (2, T, r), torch.float32, "XA")
    outs = []
    for t, shape, name in ((dX, (T, K), "dX"), (dA_gate, (K, r), "dA_gate"), (dB_gate, (r, N), "dB_gate"),
                           (dA_up, (K, r), "dA_up"), (dB_up, (r, N), "dB_up")):
        outs.append(_empty(shape, torch.bfloat16, X.device, stream) if t is None
                    else _given(t, shape, torch.bfloat16, name))
    _together(X.device, dH=dH, saved=saved, XA=XA, dX=dX, dA_gate=dA_gate, dB_gate=dB_gate, dA_up=dA_up, dB_up=dB_up,
              workspace=workspace)
    nbytes = gated_bwd_workspace_bytes(T, K, N, r)
    workspace = _workspace(nbytes, X.device, workspace, stream)
    _check(lib().qlora_gated_bwd(_qtype(qtype), _p(dH), _p(X), _p(saved), _p(XA), T, K, N, ctypes.byref(g),
                                 ctypes.byref(u), r, float(alpha), *(_p(t) for t in outs), _p(workspace), nbytes,
                                 _stream(stream)))
    return tuple(outs)


def head_loss_workspace_bytes(T, K, V, grad=True):
    return int(lib().qlora_head_loss_workspace_bytes(T, K, V, 1 if grad else 0))


def head_loss(X, W, targets, dloss=None, grad=True, loss=None, lse=None, mean=None, dX=None, workspace=None,
              stream=None):
    """Cross entropy of the tokens X [T,K] over the rows of the head W [V,K] (see
    qlora_head_loss); targets int64 [T], a negative one is not learned.

    targets and dloss may be views that start anywhere (labels[1:], weights[1:]).
    dloss: fp32 [T], the gradient of each token's loss; None: that of the mean.
    grad=False leaves dX out.  Returns (loss f32 [T], lse f32 [T], mean f32 [1],
    dX bf16 [T,K] or None)."""
    torch = _torch()
    T, K = _matrix(X, "X").shape
    V, K2 = _matrix(W, "W").shape
    if K2 != K:
        raise ValueError("X must be [T,K] and W [V,K]")
    _exactly(targets, (T,), torch.int64, "targets")
    if dloss is not None:
        _exactly(dloss, (T,), torch.float32, "dloss")
    given = []
    for t, n, name in ((loss, T, "loss"), (lse, T, "lse"), (mean, 1, "mean")):
        given.append(_empty((n,), torch.float32, X.device, stream) if t is None
                     else _given(t, (n,), torch.float32, name))
    loss, lse, mean = given
    if dX is not None:
        if not grad:
            raise ValueError("dX is given, but grad is False")
        _given(dX, (T, K), torch.bfloat16, "dX")
    elif grad:
        dX = _empty((T, K), torch.bfloat16, X.device, stream)
    _together(X.device, W=W, targets=targets, dloss=dloss, loss=loss, lse=lse, mean=mean, dX=dX, workspace=workspace)
    if dloss is not None and dloss.data_ptr() % 16:   # the library takes it on 16 bytes
        if stream is None:
            dloss = dloss.clone()
        else:
            with torch.cuda.stream(stream):           # from and in the order of the call's stream
                dloss = dloss.clone()
    nbytes = head_loss_workspace_bytes(T, K, V, grad)
    workspace = _workspace(nbytes, X.device, workspace, stream)
    _check(lib().qlora_head_loss(_p(X), T, K, _p(W), V, _p(targets), _p(dloss), _p(loss), _p(lse), _p(mean), _p(dX),
                                 _p(workspace), nbytes, _stream(stream)))
    return loss, lse, mean, dX


def _grad_type(t, name):
    torch = _torch()
    if not isinstance(t, torch.Tensor):
        raise TypeError(f"{name} must be a torch.Tensor")
    if t.dtype not in (torch.bfloat16, torch.float32):
        raise TypeError(f"{name} must be bfloat16 or float32, got {t.dtype}")
    _dev(t, t.dtype, name)
    return 1 if t.dtype == torch.float32 else 0


class GradSet:
    """Gradients that keep their places from step to step, with the places of
    their clipped values: the list that clip_grads takes, looked over once (2 us a
    tensor, which a plain list costs on every call).  It keeps addresses: a tensor
    that is given other memory (set_, .data, resize_) needs a new set.

    grads: contiguous bf16 or fp32 tensors of any lengths.  out: None (in place)
    or a tensor for each, of the same length, bf16 or fp32; no output may
    overlap another output or gradient."""

    def __init__(self, grads, out=None):
        self.grads = list(grads)
        self.out = self.grads if out is None else list(out)
        if len(self.out) != len(self.grads):
            raise ValueError("out must hold a tensor for each gradient")
        self.descs = (Grad * max(1, len(self.grads)))()
        device = None
        for i, (g, o) in enumerate(zip(self.grads, self.out)):
            kinds = _grad_type(g, "a gradient"), _grad_type(o, "an output")
            if o.numel() != g.numel():
                raise ValueError(f"output {i} holds {o.numel()} values, its gradient {g.numel()}")
            if device is None:
                device = g.device
            if (g.device, o.device) != (device, device):
                raise ValueError("all gradients and outputs must be on one GPU")
            self.descs[i] = Grad(g.data_ptr(), o.data_ptr(), g.numel(), *kinds)
        self.device = device
        self.workspace_bytes = clip_grads_workspace_bytes(len(self.grads))

    def __len__(self):
        return len(self.grads)


def clip_grads_workspace_bytes(count):
    return int(lib().qlora_clip_grads_workspace_bytes(count))


def clip_grads(grads, max_norm, out=None, norm=None, workspace=None, stream=None):
    """Global norm of the gradients, and their values clipped to it (see
    qlora_clip_grads).  grads: a GradSet, or a list of tensors (then `out` as
    GradSet takes it).  max_norm 0: only the norm.  Returns the norm, fp32 [1]."""
    torch = _torch()
    if isinstance(grads, GradSet):
        if out is not None:
            raise ValueError("a GradSet has its outputs already")
    else:
        grads = GradSet(grads, out)
    device = grads.device if len(grads) else "cuda"
    if len(grads):
        _together(device, norm=norm, workspace=workspace)
    norm = _empty((1,), torch.float32, device, stream) if norm is None else _given(norm, (1,), torch.float32, "norm")
    nbytes = grads.workspace_bytes
    workspace = _workspace(nbytes, device, workspace, stream)
    _check(lib().qlora_clip_grads(len(grads), grads.descs, float(max_norm), _p(norm), _p(workspace), nbytes,
                                  _stream(stream)))
    return norm
