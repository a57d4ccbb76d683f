"""The Python binding and the C calls behind it, on the host."""
import ctypes
import importlib.util

import pytest
import torch

from quantized_moe_expert_quantize_amd import ftq


def test_imports_without_the_gpu_names_of_torch(monkeypatch):
    """A torch without GPU support lacks the raw-handle queries; the import and the host calls work, GPU calls refuse."""
    for name in [n for n in dir(torch._C) if n.startswith("_cuda_")]:
        monkeypatch.delattr(torch._C, name)
    spec = importlib.util.spec_from_file_location("ftq_without_gpu", ftq.__file__)
    m = importlib.util.module_from_spec(spec)
    spec.loader.exec_module(m)
    assert m.select_path(8, 64, 256, 4, 2) in (m.PATH_GEMV, m.PATH_GROUPED)
    assert m.fp8_select_path(8, 64, 256, 4, 2) in (m.PATH_GEMV, m.PATH_GROUPED)
    x = torch.zeros(4, 128)
    for f in (lambda: m.quantize_q8_1(x), lambda: m.moe_topk(x, 2), lambda: m.quantize_fp8(x), lambda: m.quantize_fp8_weight(x[None])):
        with pytest.raises(ValueError):
            f()


def test_exact_products_are_a_flag_of_the_out_type():
    f, P, A = ftq.lib().ftq_moe_fp8, ctypes.c_void_p, 0x100000

    def call(out_dtype, T=4, out=A):
        return f(P(A), P(A), P(A), P(A), P(A), P(out), out_dtype, 8, 64, 256, T, 2, 0, 0, None, 0, ftq.PATH_GROUPED, None)
    for dt in (ftq.F32, ftq.F16, ftq.BF16):
        assert call(dt | ftq.EXACT) == ftq.ERR_WORKSPACE      # past the checks of the arguments
        assert call(dt | ftq.EXACT, T=0) == ftq.OK
        assert call(dt | 0x200) == ftq.ERR_INVALID_ARG and "type" in ftq.last_error()
    assert call(ftq.EXACT | 3) == ftq.ERR_INVALID_ARG
    assert call(ftq.EXACT | ftq.BF16, out=A + 1) == ftq.ERR_INVALID_ARG
    assert call(ftq.EXACT | ftq.F32, out=A + 2) == ftq.ERR_INVALID_ARG
