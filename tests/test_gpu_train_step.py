"""The training step's operators together, as they are used: the example's
gradients against fp64 autograd on the same values and against differences, the
step captured into a graph and replayed, calls on another stream, two calls that
share nothing but the card, and repeated calls bit for bit."""

import os
import sys

import numpy as np
import pytest

pytestmark = pytest.mark.gpu

torch = pytest.importorskip("torch")
sys.path.insert(0, os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))), "examples"))

U = 2.0 ** -8


def _block(**kw):
    import training_step
    return training_step.LastBlock(**{**dict(width=256, features=576, vocabulary=777, rank=8), **kw})


def _inputs(block, tokens, vocabulary=777, seed=1):
    g = torch.Generator(device="cuda").manual_seed(seed)
    x = torch.randn(tokens, block.width, generator=g, device="cuda").bfloat16()
    t = torch.randint(0, vocabulary, (tokens,), generator=g, device="cuda")
    t[::5] = -100
    return x, t


def _reference(block, x, t):
    """(mean loss, gradients by name, dx) in fp64."""
    import bit_nf4_quantized_21_amd as lib
    scale = block.alpha / block.rank
    leaf = {n: block.linears[n[0]][n[1]].double().requires_grad_() for n in block.NAMES}
    x = x.double().requires_grad_()

    def linear(v, name, n, k):
        w = block.linears[name]
        dense = lib.dequantize_nf4(w["codes"], w["q8"], w["s2"], n * k).double().view(n, k)
        return v @ dense.t() + scale * (v @ leaf[name, "A"]) @ leaf[name, "B"]
    h = torch.nn.functional.silu(linear(x, "gate", block.features, block.width)) * linear(x, "up", block.features, block.width)
    y = x + linear(h, "down", block.width, block.features)
    loss = torch.nn.functional.cross_entropy(y @ block.head.double().t(), t)
    grads = torch.autograd.grad(loss, [leaf[n] for n in block.NAMES] + [x])
    return loss.item(), dict(zip(block.NAMES, grads)), grads[-1]


def _rel(a, b):
    return float((a.double() - b).norm() / b.norm())


@pytest.mark.parametrize("tokens", [10, 300])
def test_step_gradients(tokens):
    """Roundings on the way to a gradient, each at most u / sqrt 3 of the norm: of
    h, of y twice (linear, sum), of dy, of dh, of dG and dU, and its own; between
    them the head's and the linears' condition (at most 2 here, since y's parts
    and the logits' are of one size)."""
    block = _block()
    x, t = _inputs(block, tokens)
    mean, dx = block.forward_backward(x, t)
    loss, grads, gx = _reference(block, x, t)
    assert abs(float(mean) - loss) < 2 * U * abs(loss)
    bound = 2 * np.sqrt(8) * U / np.sqrt(3)
    for n in block.NAMES:
        assert _rel(block.grads[n], grads[n]) < bound, n
    assert _rel(dx, gx) < bound


def test_step_runs_and_clips():
    import bit_nf4_quantized_21_amd as lib
    block = _block()
    x, t = _inputs(block, 100)
    before = block.param.clone()
    for i in range(3):
        mean, norm = block.step(x, t, max_norm=1e-3)
        assert np.isfinite(float(mean)) and float(norm) > 1e-3
        got = float(block.grad.double().norm())
        assert abs(got - 1e-3) < 1e-3 * U              # clipped to the bound, each value rounded
    assert not torch.equal(before, block.param) and torch.equal(block.param, block.master.bfloat16())
    lib.device_status()


def test_step_in_a_graph():
    """Captured once, replayed with other inputs in the same places, with eager
    work between the replays: every replay equals the eager result bit for bit."""
    block, again = _block(), _block()
    x, t = _inputs(block, 150)
    eager = [_inputs(block, 150, seed=s) for s in (2, 3, 4)]
    block.forward_backward(x, t)        # what is looked up once per process
    import bit_nf4_quantized_21_amd as lib
    lib.clip_grads(block.set, 0.5)
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        mean, dx = block.forward_backward(x, t)
        norm = lib.clip_grads(block.set, 0.5)
    for nx, nt in eager:
        want_mean, want_dx = again.forward_backward(nx, nt)
        want_norm = lib.clip_grads(again.set, 0.5)
        x.copy_(nx)
        t.copy_(nt)
        graph.replay()
        torch.cuda.synchronize()
        assert torch.equal(mean, want_mean) and torch.equal(dx, want_dx) and torch.equal(norm, want_norm)
        assert torch.equal(block.grad, again.grad)
    lib.device_status()


def test_two_graphs_of_their_own():
    """Two captured calls, replayed in turn: each has its own workspace."""
    import bit_nf4_quantized_21_amd as lib
    a, b = _block(seed=1), _block(seed=2)
    xa, ta = _inputs(a, 90, seed=5)
    xb, tb = _inputs(b, 130, seed=6)
    want = [[v.clone() for v in blk.forward_backward(x, t)] for blk, x, t in ((a, xa, ta), (b, xb, tb))]
    torch.cuda.synchronize()
    graphs, got = [], []
    for blk, x, t in ((a, xa, ta), (b, xb, tb)):
        graphs.append(torch.cuda.CUDAGraph())
        with torch.cuda.graph(graphs[-1]):
            got.append(blk.forward_backward(x, t))
    for i in (0, 1, 0, 0, 1, 1, 0):
        graphs[i].replay()
        torch.cuda.synchronize()
        assert all(torch.equal(g, w) for g, w in zip(got[i], want[i]))
    lib.device_status()


def test_other_stream():
    """Every call on another stream than the current one, behind work of that
    stream; what the calls allocate may be dropped and reused at once."""
    import bit_nf4_quantized_21_amd as lib
    block = _block()
    x, t = _inputs(block, 200)
    gate, up = block.linears["gate"], block.linears["up"]
    h, saved, xa = lib.gated_fwd(x, gate, up, block.alpha, save=True)
    back = lib.gated_bwd(h, x, saved, xa, gate, up, block.alpha)
    loss = lib.head_loss(x, block.head, t)
    norm = lib.clip_grads(list(back), 0.1, out=[torch.empty_like(g) for g in back])
    torch.cuda.synchronize()
    side = torch.cuda.Stream()
    for _ in range(3):
        side.wait_stream(torch.cuda.current_stream())
        h2, saved2, xa2 = lib.gated_fwd(x, gate, up, block.alpha, save=True, stream=side)
        back2 = lib.gated_bwd(h2, x, saved2, xa2, gate, up, block.alpha, stream=side)
        loss2 = lib.head_loss(x, block.head, t, stream=side)
        out2 = [torch.empty_like(g) for g in back2]
        side.wait_stream(torch.cuda.current_stream())
        norm2 = lib.clip_grads(list(back2), 0.1, out=out2, stream=side)
        torch.cuda.current_stream().wait_stream(side)
        junk = [torch.randn(1 << 20, device="cuda") for _ in range(4)]
        assert torch.equal(h, h2) and torch.equal(xa, xa2) and torch.equal(norm, norm2)
        assert all(torch.equal(a, b) for a, b in zip(back, back2)) and all(torch.equal(a, b) for a, b in zip(loss, loss2))
        del junk
    lib.device_status(side)


def test_calls_at_once():
    """Two streams run different calls at the same time; each gets what it gets alone."""
    import bit_nf4_quantized_21_amd as lib
    block = _block()
    x, t = _inputs(block, 300)
    want = lib.head_loss(x, block.head, t)
    h = lib.gated_fwd(x, block.linears["gate"], block.linears["up"], block.alpha, save=True)
    torch.cuda.synchronize()
    s1, s2 = torch.cuda.Stream(), torch.cuda.Stream()
    got1 = [lib.head_loss(x, block.head, t, stream=s1) for _ in range(5)]
    got2 = [lib.gated_fwd(x, block.linears["gate"], block.linears["up"], block.alpha, save=True, stream=s2) for _ in range(5)]
    torch.cuda.synchronize()
    assert all(torch.equal(a, b) for g in got1 for a, b in zip(g, want))
    assert all(torch.equal(a, b) for g in got2 for a, b in zip(g, h))


@pytest.mark.parametrize("tokens", [1, 16, 400])
def test_repeated_calls_are_the_same(tokens):
    block = _block()
    x, t = _inputs(block, tokens)
    t[0] = 3
    first = block.forward_backward(x, t)
    grads = {n: g.clone() for n, g in block.grads.items()}
    for _ in range(3):
        again = block.forward_backward(x, t)
        assert all(torch.equal(a, b) for a, b in zip(first, again))
        assert all(torch.equal(grads[n], block.grads[n]) for n in block.NAMES)
