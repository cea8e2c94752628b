"""What calls around a training step must not do: tests that failed on earlier
kernels, one for each fault."""

import numpy as np
import pytest

pytestmark = pytest.mark.gpu

torch = pytest.importorskip("torch")


def _lib():
    import bit_nf4_quantized_21_amd as lib
    return lib


def _normal(g, *shape, scale=1.0):
    return (torch.randn(*shape, generator=g, device="cuda") * scale).bfloat16()


def _adapted(g, N, K, r):
    codes, q8, s2 = _lib().quantize_dq(torch.randn(N, K, generator=g, device="cuda") * 0.05)
    return dict(codes=codes, q8=q8, s2=s2, A=_normal(g, K, r, scale=K ** -0.5), B=_normal(g, r, N, scale=0.05))


@pytest.mark.parametrize("T,N", [(5, 776), (20, 776), (300, 776), (300, 8), (257, 1000), (40, 640)])
@pytest.mark.parametrize("value", [float("inf"), float("nan")])
def test_input_gradient_of_a_token_is_its_own(T, N, value):
    """An infinity or NaN in one token's output gradient reaches the input
    gradient of that token and of no other, whatever features are left over in
    the last step of 64: bit for bit."""
    print(f"own row T={T} N={N} {value}", flush=True)
    lib = _lib()
    g = torch.Generator(device="cuda").manual_seed(T + N)
    K, r, alpha = 320, 8, 16.0
    gate, up = _adapted(g, N, K, r), _adapted(g, N, K, r)
    X, dH = _normal(g, T, K), _normal(g, T, N)
    _, saved, XA = lib.gated_fwd(X, gate, up, alpha, save=True)
    w = (gate["codes"], gate["q8"], gate["s2"], gate["A"], gate["B"], alpha)
    clean = lib.gated_bwd(dH, X, saved, XA, gate, up, alpha)[0], lib.linear_bwd(dH, X, None, *w)[0]
    for token in {1, T // 2, T - 1}:
        for feature in {0, 7, min(N - 1, 50)}:
            bad = dH.clone()
            bad[token, feature] = value
            got = lib.gated_bwd(bad, X, saved, XA, gate, up, alpha)[0], lib.linear_bwd(bad, X, None, *w)[0]
            others = torch.arange(T, device="cuda") != token
            for a, b in zip(got, clean):
                assert torch.equal(a[others], b[others]), (token, feature)
                assert not bool(torch.isfinite(a[token]).any())
    lib.device_status()


@pytest.mark.parametrize("T", [3, 40])
@pytest.mark.parametrize("act", ["silu", "gelu", "gelu_tanh"])
@pytest.mark.parametrize("side", ["gate", "up"])
def test_what_is_no_number_reaches_the_gradients(T, act, side):
    """Where G or U is no number the kept multipliers are infinite (both where G is,
    act'(G) U alone where U is), so no gradient they enter comes out finite."""
    print(f"no number T={T} {act} {side}", flush=True)
    lib = _lib()
    g = torch.Generator(device="cuda").manual_seed(T)
    K, N, r, n = 128, 72, 8, 11
    gate, up = _adapted(g, N, K, r), _adapted(g, N, K, r)
    (gate if side == "gate" else up)["B"][:, n] = float("nan")
    X, dH = _normal(g, T, K), _normal(g, T, N)
    H, saved, XA = lib.gated_fwd(X, gate, up, 16.0, act=act, save=True)
    assert bool(torch.isnan(H[:, n]).all()) and bool(torch.isfinite(H[:, :n]).all())
    infinite = (saved & 0x7FFF) == 0x7FFF
    assert bool(infinite[0, :, n].all()) and bool(infinite[1, :, n].all()) == (side == "gate")
    dX, _, dB_gate, _, dB_up = lib.gated_bwd(dH, X, saved, XA, gate, up, 16.0)
    assert not bool(torch.isfinite(dX).any()) and not bool(torch.isfinite(dB_gate[:, n]).any())
    assert bool(torch.isfinite(dB_up[:, n]).any()) == (side == "up")
    assert bool(torch.isfinite(dB_gate[:, :n]).all()) and bool(torch.isfinite(dB_up[:, :n]).all())
    lib.device_status()


@pytest.mark.parametrize("T", [2, 65, 301])
@pytest.mark.parametrize("other_stream", [False, True])
def test_loss_of_shifted_labels(T, other_stream):
    """labels[1:] and weights[1:], contiguous but off 16 bytes, give what their copies give."""
    print(f"shifted T={T}", flush=True)
    lib = _lib()
    g = torch.Generator(device="cuda").manual_seed(T)
    X, W = _normal(g, T, 192), _normal(g, 500, 192, scale=0.1)
    labels = torch.randint(0, 500, (T,), generator=g, device="cuda")
    labels[T // 2] = -100
    weights = torch.rand(T, generator=g, device="cuda")
    want = lib.head_loss(X[:-1], W, labels[1:].clone(), dloss=weights[1:].clone())
    torch.cuda.synchronize()
    stream = torch.cuda.Stream() if other_stream else None
    for _ in range(3):
        got = lib.head_loss(X[:-1], W, labels[1:], dloss=weights[1:], stream=stream)
        junk = [torch.full((T - 1,), 9.0, device="cuda") for _ in range(8)]     # what was freed may be given away
        torch.cuda.synchronize()
        assert all(torch.equal(a, b) for a, b in zip(got, want))
        del junk
    assert all(torch.equal(a, b) for a, b in zip(lib.head_loss(X[:-1], W, labels[1:])[:3], want[:3]))
    lib.device_status()


def test_loss_of_shifted_labels_in_a_graph():
    lib = _lib()
    g = torch.Generator(device="cuda").manual_seed(1)
    T = 130
    X, W = _normal(g, T, 128), _normal(g, 700, 128, scale=0.1)
    labels = torch.randint(0, 700, (T,), generator=g, device="cuda")
    weights = torch.rand(T, generator=g, device="cuda")
    lib.head_loss(X[:-1], W, labels[1:], dloss=weights[1:])      # what is looked up once per process
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        got = lib.head_loss(X[:-1], W, labels[1:], dloss=weights[1:])
    for _ in range(4):
        labels.copy_(torch.randint(0, 700, (T,), generator=g, device="cuda"))
        weights.copy_(torch.rand(T, generator=g, device="cuda"))
        want = lib.head_loss(X[:-1], W, labels[1:].clone(), dloss=weights[1:].clone())
        graph.replay()
        torch.cuda.synchronize()
        assert all(torch.equal(a, b) for a, b in zip(got, want))
    lib.device_status()


def test_inputs_of_another_length_are_refused():
    """An input that is too long is no input: T states with T + 1 unshifted labels
    would pair every token with the wrong word, what was kept for more tokens
    would be read from the wrong place."""
    lib = _lib()
    g = torch.Generator(device="cuda").manual_seed(3)
    T, K, N, r = 20, 128, 72, 8
    gate, up = _adapted(g, N, K, r), _adapted(g, N, K, r)
    X, dH, W = _normal(g, T, K), _normal(g, T, N), _normal(g, 50, K)
    labels = torch.randint(0, 50, (T + 1,), generator=g, device="cuda")
    weights = torch.rand(T + 1, generator=g, device="cuda")

    def refused(f, *a, **k):
        with pytest.raises(ValueError, match="must be"):
            f(*a, **k)
    refused(lib.head_loss, X, W, labels)
    refused(lib.head_loss, X, W, labels[:T - 1])
    refused(lib.head_loss, X, W, labels[:T].view(1, T))
    refused(lib.head_loss, X, W, labels[1:], dloss=weights)
    want = lib.head_loss(X, W, labels[1:].clone(), dloss=weights[:T].clone())
    assert all(torch.equal(a, b) for a, b in zip(lib.head_loss(X, W, labels[1:], dloss=weights[:T]), want))

    H, saved, XA = lib.gated_fwd(X, gate, up, 16.0, save=True)
    want = lib.gated_bwd(dH, X, saved, XA, gate, up, 16.0)
    long_saved = torch.zeros(2 * (T + 5) * N, dtype=torch.int16, device="cuda")
    long_XA = torch.zeros(2 * (T + 5) * r, device="cuda")
    for shape in ((2, T + 5, N), (-1,), (T + 5, 2 * N)):
        refused(lib.gated_bwd, dH, X, long_saved.view(shape), XA, gate, up, 16.0)
    for shape in ((2, T + 5, r), (-1,)):
        refused(lib.gated_bwd, dH, X, saved, long_XA.view(shape), gate, up, 16.0)
    # A buffer kept for more tokens is written at its start, and that part comes back.
    H2, part, partXA = lib.gated_fwd(X, gate, up, 16.0, saved=long_saved, XA=long_XA)
    assert part.shape == (2, T, N) and partXA.shape == (2, T, r)
    assert part.data_ptr() == long_saved.data_ptr() and partXA.data_ptr() == long_XA.data_ptr()
    assert torch.equal(part, saved) and torch.equal(partXA, XA) and torch.equal(H2, H)
    assert not bool(long_saved[2 * T * N:].any()) and not bool(long_XA[2 * T * r:].any())
    assert all(torch.equal(a, b) for a, b in zip(lib.gated_bwd(dH, X, part, partXA, gate, up, 16.0), want))
    same = lib.gated_fwd(X, gate, up, 16.0, saved=saved, XA=XA)
    assert same[1] is saved and same[2] is XA
    lib.device_status()


@pytest.mark.parametrize("T", [20, 300])
def test_exponentials_of_lifted_rows_are_rounded_once(T):
    """Every stretch of words lies far above the target, each by another amount, so
    all of them take references of their own and are then brought to one.  Each
    word has a column of its own, so that an element of dX is one exponential times
    a power of two: it is off by that exponential's rounding to bf16 and its own,
    u = 2^-8 each, and 2^-15 for what happens in fp32 (arguments up to 58 powers of
    two, an exponential and a division to an ulp, a sum of 640 terms)."""
    print(f"lifted T={T}", flush=True)
    lib = _lib()
    V = K = 640
    g = torch.Generator(device="cuda").manual_seed(T)
    W = (2 * torch.eye(V, device="cuda")).bfloat16()
    X = (10 + 6 * torch.rand(T, K, generator=g, device="cuda")).bfloat16()        # logits of 20 to 32
    t = torch.randint(0, V, (T,), generator=g, device="cuda")
    rows = torch.arange(T, device="cuda")
    X[rows, t] = -15.0
    loss, lse, mean, dX = lib.head_loss(X, W, t)
    z = 2 * X.double()
    p = torch.softmax(z, 1)
    rest = p.clone()
    rest[rows, t] = 0
    want = 2 * rest / T
    want[rows, t] = -2 * rest.sum(1) / T
    u = 2.0 ** -8
    off = (dX.double() - want).abs() / want.abs()
    print(float(off.max()) / u)
    assert float(off.max()) <= (1 + u) ** 2 - 1 + 2.0 ** -15
    ref = torch.logsumexp(z, 1)
    # Logits are exact; 2^-17 for exponentials and sum, and 4 roundings of the result.
    assert bool(((loss.double() - (ref + 30)).abs() <= 2.0 ** -17 + 2.0 ** -22 * (ref + 30)).all())
    alone = lib.head_loss(X, W, t, grad=False)
    assert torch.equal(alone[0], loss) and torch.equal(alone[1], lse) and torch.equal(alone[2], mean)
    lib.device_status()


@pytest.mark.parametrize("T,far", [(20, 1e4), (300, 1e4), (70, 1e6), (7, 1e8)])
def test_log_sum_beside_a_target_far_below(T, far):
    """The log-sum is that of the other words, whose logits lie between 20 and 32: off
    by 2^-17 for exponentials and sum and by 2^-22 of itself, however large the loss."""
    print(f"far target T={T} {far}", flush=True)
    lib = _lib()
    V = K = 640
    g = torch.Generator(device="cuda").manual_seed(T)
    W = (2 * torch.eye(V, device="cuda")).bfloat16()
    X = (10 + 6 * torch.rand(T, K, generator=g, device="cuda")).bfloat16()
    t = torch.randint(0, V, (T,), generator=g, device="cuda")
    X[torch.arange(T, device="cuda"), t] = -far / 2
    z = 2 * X.double()
    ref = torch.logsumexp(z, 1)
    want = ref - z.gather(1, t[:, None])[:, 0]
    for grad in (True, False):
        loss, lse, _, _ = lib.head_loss(X, W, t, grad=grad)
        assert bool(((lse.double() - ref).abs() <= 2.0 ** -17 + 2.0 ** -22 * ref).all())
        assert bool(((loss.double() - want).abs() <= 2.0 ** -17 + 2.0 ** -22 * want).all())
    lib.device_status()


@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16])
def test_norm_of_equal_values_is_rounded_once(dtype):
    """Roundings that all go the same way add up: of many equal values the norm is
    off by its own rounding, 2^-24, and what fp64 leaves (50000 terms of 2^-53)."""
    lib = _lib()
    n = 50000
    for i in range(40):
        v = torch.full((n,), 1.0 + i / 41, device="cuda").to(dtype)
        ref = float(n ** 0.5 * v[0].double())
        assert abs(float(lib.clip_grads([v], 0.0)) - ref) <= 2.0 ** -24 * (1 + 2.0 ** -12) * ref, i


@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16])
def test_clip_of_gradients_that_are_all_zero(dtype):
    """As every dA is while B = 0: the norm is that of the others, and all stay as they are said."""
    lib = _lib()
    zeros = [torch.zeros(n, dtype=dtype, device="cuda") for n in (70000, 3, 16384)]
    others = [torch.full((n,), 2.0, dtype=dtype, device="cuda") for n in (4, 60000)]
    assert float(lib.clip_grads(zeros, 1.0)) == 0 and not any(bool(z.any()) for z in zeros)
    norm = lib.clip_grads(zeros + others, 1.0)
    ref = 2 * 60004 ** 0.5
    assert abs(float(norm) - ref) <= 2.0 ** -24 * 1.01 * ref
    assert not any(bool(z.any()) for z in zeros)
    want = 2 / ref
    half = 2.0 ** -24 if dtype == torch.float32 else 2.0 ** -8
    for o in others:   # the coefficient in fp32 (2^-24), the product in fp32, its rounding; 1e-6 beside the norm
        assert bool(((o.double() - want).abs() <= (half + 2 * 2.0 ** -24 + 1e-6 / ref) * want).all())


def test_clip_of_hundreds_of_tensors_in_a_graph():
    """More tensors than the kernels' arguments hold: their table is written to the
    workspace by launches of its own, in a captured call on every replay."""
    lib = _lib()
    g = torch.Generator(device="cuda").manual_seed(2)
    lengths = [1 + (i * 7919) % 5000 for i in range(300)]
    kinds = [torch.float32 if i % 3 else torch.bfloat16 for i in range(300)]
    grads = [torch.randn(n, generator=g, device="cuda").to(k) for n, k in zip(lengths, kinds)]
    flat = torch.zeros(sum(lengths), dtype=torch.bfloat16, device="cuda")
    out = list(flat.split(lengths))
    other = [torch.zeros_like(x) for x in grads]
    lib.clip_grads(grads, 0.5, out=out)      # what is looked up once per process
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        norm = lib.clip_grads(grads, 0.5, out=out)
        norm2 = lib.clip_grads(other, 0.5)
    for i in range(4):
        for x, y in zip(grads, other):
            x.copy_(torch.randn(x.shape, generator=g, device="cuda") * 10.0 ** -i)
            y.copy_(x)
        torch.cuda.synchronize()
        graph.replay()
        torch.cuda.synchronize()
        got = flat.clone()
        want = torch.zeros_like(flat)
        assert torch.equal(lib.clip_grads(grads, 0.5, out=list(want.split(lengths))), norm)
        assert torch.equal(got, want) and torch.equal(norm, norm2)
        lib.clip_grads(grads, 0.5)
        assert all(torch.equal(x, y) for x, y in zip(grads, other))
