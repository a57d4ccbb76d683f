"""Balance loss, router, combine and adapter gradients on the host: refusals and
workspace sizes (no call here touches a device)."""
import ctypes

import pytest
import torch

from quantized_moe_expert_quantize_amd import ftq

P = ctypes.c_void_p
A = 0x100000   # an address that passes the alignment checks; never read
BIG = 1 << 40


def _call(name, args, kw):
    d = {**args, **kw}
    assert set(d) == set(args), set(d) - set(args)
    return getattr(ftq.lib(), name)(*d.values())


BALANCE = dict(logits=A, dtype=0, ld=64, ids=A, valid=None, offsets=A, counts=A, tokens=A, loss=A, T=100, E=64, k=4, S=3, score=0, ws=A,
               ws_n=BIG, stream=None)


@pytest.mark.parametrize("kw", [
    dict(dtype=3), dict(score=2), dict(T=-1), dict(E=0), dict(k=0), dict(S=0), dict(ld=63), dict(offsets=None), dict(logits=None),
    dict(ids=None), dict(counts=None), dict(tokens=None), dict(loss=None), dict(logits=A + 2), dict(logits=A + 1, dtype=2), dict(ids=A + 2),
    dict(offsets=A + 1), dict(counts=A + 2), dict(tokens=A + 2), dict(loss=A + 2), dict(ws=A + 128),
])
def test_balance_refuses(kw):
    assert _call("ftq_moe_balance", BALANCE, kw) == ftq.ERR_INVALID_ARG and ftq.last_error()


def test_balance_limits_and_workspace():
    for kw in (dict(E=1025, ld=1025), dict(k=65), dict(T=2 ** 30, k=2), dict(S=2 ** 31), dict(T=2 ** 30, k=1, ld=2 ** 40)):
        assert _call("ftq_moe_balance", BALANCE, kw) == ftq.ERR_UNSUPPORTED, kw
    need = ftq.balance_workspace_bytes(100, 64, 4, 3)
    assert need > 0 and need % 256 == 0
    for kw in (dict(ws_n=need - 1), dict(ws=None)):
        assert _call("ftq_moe_balance", BALANCE, kw) == ftq.ERR_WORKSPACE
    for args in ((-1, 64, 4, 1), (100, 0, 4, 1), (100, 2000, 4, 1), (100, 64, 4, 0)):
        with pytest.raises(ftq.FtqError):
            ftq.balance_workspace_bytes(*args)


TOPK = dict(logits=A, dtype=0, ld=64, ids=A, d_gates=A, counts=A, tokens=A, d_loss=A, valid=None, offsets=A, out=A, ld_d=64, T=100, E=64, k=4,
            S=3, score=0, renorm=1, scale=ctypes.c_float(1.0), stream=None)


@pytest.mark.parametrize("kw", [
    dict(dtype=-1), dict(score=5), dict(T=-1), dict(E=0), dict(k=0), dict(S=0), dict(ld=63), dict(ld_d=63), dict(d_gates=None, d_loss=None),
    dict(offsets=None), dict(logits=None), dict(out=None), dict(ids=None), dict(counts=None), dict(tokens=None), dict(logits=A + 2),
    dict(out=A + 2), dict(ids=A + 1), dict(d_gates=A + 2), dict(counts=A + 2), dict(tokens=A + 2), dict(d_loss=A + 2), dict(offsets=A + 2),
])
def test_topk_backward_refuses(kw):
    assert _call("ftq_moe_topk_backward", TOPK, kw) == ftq.ERR_INVALID_ARG and ftq.last_error()


def test_topk_backward_limits():
    for kw in (dict(E=1025, ld=1025, ld_d=1025), dict(k=65), dict(T=2 ** 30, k=2), dict(T=2 ** 30, k=1, ld_d=2 ** 40)):
        assert _call("ftq_moe_topk_backward", TOPK, kw) == ftq.ERR_UNSUPPORTED, kw
    assert _call("ftq_moe_topk_backward", TOPK, dict(T=0, logits=None, out=None, d_gates=None, d_loss=None)) == ftq.OK


COMBINE = dict(d_out=A, y=A, gates=A, d_y=A, dtype=0, d_gates=A, T=10, k=2, N=64, stream=None)


def test_combine_backward_refuses():
    for kw in (dict(T=-1), dict(k=0), dict(N=0), dict(dtype=4), dict(d_y=None, d_gates=None), dict(d_out=None), dict(gates=None), dict(y=None),
               dict(d_out=A + 2), dict(y=A + 2), dict(gates=A + 1), dict(d_y=A + 2), dict(d_y=A + 1, dtype=1), dict(d_gates=A + 2)):
        assert _call("ftq_moe_combine_topk_backward", COMBINE, kw) == ftq.ERR_INVALID_ARG, kw
    assert _call("ftq_moe_combine_topk_backward", COMBINE, dict(T=2 ** 40, k=2 ** 10, N=2 ** 20)) == ftq.ERR_UNSUPPORTED
    assert _call("ftq_moe_combine_topk_backward", COMBINE, dict(T=0, d_out=None, y=None, gates=None, d_y=None, d_gates=None)) == ftq.OK


LORA = dict(x=A, ldx=256, a=A, b=A, scale=A, ids=A, base=A, ld_base=128, out=2 * A, ld_out=128, h=A, dtype=2, out_dtype=2, L=4, R=16, K=256, N=128,
            T=10, k=1, per_pair=0, ws=A, ws_n=BIG, path=0, stream=None)


@pytest.mark.parametrize("kw", [
    dict(dtype=3), dict(out_dtype=7), dict(L=0), dict(R=0), dict(R=12), dict(K=0), dict(K=252), dict(N=0), dict(N=100), dict(T=-1), dict(k=0),
    dict(ldx=248), dict(ldx=260), dict(ld_base=120), dict(ld_out=132), dict(path=3), dict(path=-1), dict(x=None), dict(a=None), dict(b=None),
    dict(ids=None), dict(out=None), dict(x=A + 8), dict(a=A + 8), dict(b=A + 8), dict(base=A + 8), dict(out=A + 8), dict(h=A + 8), dict(scale=A + 2),
    dict(ids=A + 2), dict(out=A, ld_out=256),
])
def test_lora_refuses(kw):
    assert _call("ftq_lora", LORA, kw) == ftq.ERR_INVALID_ARG and ftq.last_error()


def test_lora_limits_paths_and_workspace():
    for kw in (dict(R=136), dict(T=2 ** 30, k=2), dict(L=2 ** 31), dict(K=2 ** 32, ldx=2 ** 32), dict(L=5000, path=ftq.PATH_GROUPED)):
        assert _call("ftq_lora", LORA, kw) == ftq.ERR_UNSUPPORTED, kw
    assert _call("ftq_lora", LORA, dict(T=0, x=None, a=None, b=None, ids=None, out=None, base=None, ws=None)) == ftq.OK
    assert _call("ftq_lora", LORA, dict(T=1, base=None, ld_base=0, ws=None, ws_n=0)) == ftq.ERR_WORKSPACE
    need = ftq.lora_workspace_bytes(4, 16, 256, 128, 10, 1, torch.bfloat16, ftq.PATH_GROUPED)
    assert need > 0
    assert _call("ftq_lora", LORA, dict(ws_n=need - 1, path=ftq.PATH_GROUPED)) == ftq.ERR_WORKSPACE
    assert _call("ftq_lora", LORA, dict(ws=A + 64, path=ftq.PATH_GROUPED)) == ftq.ERR_INVALID_ARG
    assert ftq.lora_select_path(4, 10 ** 6, 1) == ftq.PATH_GEMV     # a request's rows lie together
    assert ftq.lora_select_path(5000, 10 ** 6, 8) == ftq.PATH_GEMV  # more adapters than a sort takes
    for args in ((0, 10, 1), (4, -1, 1), (4, 10, 0)):
        with pytest.raises(ftq.FtqError):
            ftq.lora_select_path(*args)
    with pytest.raises(ftq.FtqError):
        ftq.lora_workspace_bytes(5000, 16, 256, 128, 10, 1, torch.bfloat16, ftq.PATH_GROUPED)


BACK = dict(d_out=A, ld_d=128, x=A, ldx=256, a=A, b=A, scale=A, ids=A, h=A, base=None, d_x=A, d_a=A, d_b=A, dtype=2, L=4, R=16, K=256, N=128, T=10,
            k=1, per_pair=0, ws=A, ws_n=BIG, stream=None)


@pytest.mark.parametrize("kw", [
    dict(dtype=3), dict(L=0), dict(R=12), dict(K=252), dict(N=100), dict(T=-1), dict(k=0), dict(ld_d=120), dict(ldx=252), dict(d_out=None),
    dict(x=None), dict(a=None), dict(b=None), dict(ids=None), dict(h=None), dict(d_x=None, d_a=None, d_b=None), dict(d_out=A + 8), dict(x=A + 8),
    dict(a=A + 8), dict(b=A + 8), dict(h=A + 4), dict(base=A + 8), dict(d_x=A + 8), dict(d_a=A + 4), dict(d_b=A + 8), dict(scale=A + 1), dict(ids=A + 1),
    dict(ws=A + 8),
])
def test_lora_backward_refuses(kw):
    assert _call("ftq_lora_backward", BACK, kw) == ftq.ERR_INVALID_ARG and ftq.last_error()


def test_lora_backward_limits_and_workspace():
    for kw in (dict(R=136), dict(T=2 ** 30, k=2), dict(L=4096), dict(k=65)):
        assert _call("ftq_lora_backward", BACK, kw) == ftq.ERR_UNSUPPORTED, kw
    need = ftq.lora_backward_workspace_bytes(4, 16, 256, 128, 10, 1, torch.bfloat16)
    assert need > 0
    for kw in (dict(ws_n=need - 1), dict(ws=None)):
        assert _call("ftq_lora_backward", BACK, kw) == ftq.ERR_WORKSPACE
    assert _call("ftq_lora_backward", BACK, dict(T=0, d_out=None, x=None, a=None, b=None, ids=None, h=None, d_a=None, d_b=None, ws=None)) == ftq.OK
    with pytest.raises(ftq.FtqError):
        ftq.lora_backward_workspace_bytes(4096, 16, 256, 128, 10, 1, torch.bfloat16)


def test_binding_refuses_host_tensors():
    x, a, b = torch.zeros(4, 16), torch.zeros(2, 8, 16), torch.zeros(2, 8, 8)
    ids = torch.zeros(4, 1, dtype=torch.int32)
    for call in (lambda: ftq.lora(x, a, b, ids), lambda: ftq.lora_backward(torch.zeros(4, 8), x, a, b, ids, torch.zeros(4, 8)),
                 lambda: ftq.moe_balance(x, ids), lambda: ftq.moe_topk_backward(x, ids, torch.zeros(4, 1)),
                 lambda: ftq.combine_topk_backward(x, x, torch.zeros(4, 1))):
        with pytest.raises(ValueError, match="GPU tensor"):
            call()


def test_lora_takes_rows_of_any_length_below_2_31():
    """Strides past 2^26 elements; refused only where offsets overflow.  (Without a workspace, which is asked for last.)"""
    for wide in (2 ** 26 + 8, 2 ** 31 - 8):
        for kw in (dict(K=wide, ldx=wide), dict(ldx=wide), dict(N=wide, ld_out=wide, ld_base=wide), dict(ld_out=2 ** 40, ld_base=2 ** 40)):
            assert _call("ftq_lora", LORA, dict(kw, ws_n=0)) == ftq.ERR_WORKSPACE, kw
        for kw in (dict(K=wide, ldx=wide), dict(ldx=wide), dict(N=wide, ld_d=wide), dict(ld_d=2 ** 40)):
            assert _call("ftq_lora_backward", BACK, dict(kw, ws_n=0)) == ftq.ERR_WORKSPACE, kw
    for kw in (dict(ldx=2 ** 60), dict(ld_out=2 ** 60), dict(ld_base=2 ** 60), dict(T=2 ** 30, ldx=2 ** 30)):
        assert _call("ftq_lora", LORA, kw) == ftq.ERR_UNSUPPORTED, kw
    for kw in (dict(ldx=2 ** 60), dict(ld_d=2 ** 60), dict(T=2 ** 30, ldx=2 ** 30)):
        assert _call("ftq_lora_backward", BACK, kw) == ftq.ERR_UNSUPPORTED, kw


def test_lora_backward_workspace_of_few_pairs():
    """Room for the tiles that there can be: pieces of at most ten tiles of 32 pairs (both sets, 6 bytes a value of 128 ranks, 24 KiB each), g and its
    parts (10 KiB), parts of the sums of at most three runs (6 x 64 KiB), and the tables of 4096 buckets (counts, offsets, first
    tiles, descriptors of 16 bytes)."""
    need = ftq.lora_backward_workspace_bytes(4095, 128, 64, 64, 10, 1, torch.bfloat16)
    assert need <= 2 * 10 * 128 * 32 * 6 + 2 * 10 * 128 * 4 + 2 * 6 * 128 * 64 * 4 + 4096 * (3 * 4 + 16) + 12 * 256
