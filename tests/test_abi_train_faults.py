"""What the training step's entry points must not refuse or accept: tests that
failed on earlier versions, one for each fault (no GPU is touched)."""

import ctypes

import pytest

from bit_nf4_quantized_21_amd import qlora, train

ESHAPE, EALIGN, EWS = -2, -3, -6
A = 0x10000                       # aligned, never dereferenced: validation fails first
P = ctypes.c_void_p(A)


def test_head_loss_takes_shifted_labels():
    """targets is read one element at a time: a view on 8 bytes comes as far as the workspace."""
    L = qlora.lib()

    def f(targets):
        return L.qlora_head_loss(P, 5, 128, P, 1000, ctypes.c_void_p(targets), None, P, P, P, P, P, 8, None)
    assert f(A + 8) == EWS and f(A + 24) == EWS and f(A) == EWS
    for off in (1, 2, 4, 12):
        assert f(A + off) == EALIGN


@pytest.mark.parametrize("shape", [(6,), (4,), (1, 5), (5, 1), ()])
def test_inputs_have_exactly_their_axes(monkeypatch, shape):
    import torch
    monkeypatch.setattr(train, "_dev", lambda t, dtype, name: t)      # (host tensors)
    with pytest.raises(ValueError, match="must be"):
        train._exactly(torch.zeros(shape), (5,), torch.float32, "targets")
    t = torch.zeros(5)
    assert train._exactly(t, (5,), torch.float32, "targets") is t


class _OnGPU:
    """What GradSet looks at in a tensor on one of several GPUs."""

    def __init__(self, index, n=4):
        import torch
        self.device, self._n = torch.device("cuda", index), n

    def numel(self):
        return self._n

    def data_ptr(self):
        return A


@pytest.mark.parametrize("grads,outs", [((0,), (1,)), ((1,), (0,)), ((0, 0), (1, 0)), ((0, 1), (0, 1)), ((0, 0), (0, 1))])
def test_gradients_and_outputs_on_two_gpus_are_refused(monkeypatch, grads, outs):
    """The first gradient's output, too."""
    monkeypatch.setattr(train, "_grad_type", lambda t, name: 0)
    with pytest.raises(ValueError, match="one GPU"):
        train.GradSet([_OnGPU(i) for i in grads], [_OnGPU(i) for i in outs])
    train.GradSet([_OnGPU(1), _OnGPU(1)], [_OnGPU(1), _OnGPU(1)])


@pytest.mark.parametrize("T", [1, 17, 64, 65, 100, 512, 2048, 4095, 4096, 4097, 10000])
def test_head_loss_workspace_is_what_the_header_says(T):
    f = qlora.lib().qlora_head_loss_workspace_bytes
    for K in (64, 4096, 8192, 65536):
        for V in (1, 31, 1000, 16384, 32000, 50021, 128000, 1 << 20, 1 << 25):
            if T * K * 2 >= 1 << 31 or T * -(-V // 32) >= 1 << 31:
                continue
            B = min(T, 4096)
            plain = 16 * T + 8 * B * -(-V // (32 if T <= 64 else 128)) + 9 * 256
            # (A call without a gradient takes the vocabulary in one piece.)
            assert 0 < f(T, K, V, 0) <= plain + 4 * -(-T // 4096), (T, K, V)
            pieces = 4 * (V * B // (1 << 25) + 1) * -(-T // 4096)
            assert 0 < f(T, K, V, 1) <= plain + (129 << 20) + pieces + max(4 * B * K, 64 << 20), (T, K, V)
