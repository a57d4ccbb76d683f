"""The Python binding without a GPU build of torch."""
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
