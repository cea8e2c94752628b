"""Calls of the attention side that once went wrong: one test per fault, on the
mended code."""

import ctypes

import pytest

from test_gpu_generate import _i32, _lib

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
