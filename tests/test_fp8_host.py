"""Router and 8-bit floating-point calls on the host: refusals, path choice and
workspace sizes (no call here touches a device), and the test definitions of
the format against torch's own conversions."""
import ctypes

import numpy as np
import pytest
import torch

from quantized_moe_expert_quantize_amd import ftq
from tests import _fp8

P = ctypes.c_void_p
A = 0x100000   # an address that passes the alignment checks; never read


def _topk(logits=A, dtype=0, ld=256, bias=None, ids=A, gates=A, T=4, E=256, k=8, score=0, ng=1, tg=1, gt=1):
    return ftq.lib().ftq_moe_topk(P(logits), dtype, ld, P(bias), P(ids), P(gates), T, E, k, score, ng, tg, gt, 1, 1.0, None)


@pytest.mark.parametrize("kw", [
    dict(dtype=3), dict(dtype=-1), dict(score=2), dict(T=-1), dict(E=0, ld=0), dict(k=0), dict(ld=255), dict(ng=0),
    dict(ng=7), dict(ng=8, tg=0), dict(ng=8, tg=9), dict(gt=0), dict(gt=3), dict(ng=256, tg=256, gt=2), dict(k=257, E=256),
    dict(ng=8, tg=1, k=33), dict(logits=None), dict(ids=None), dict(gates=None), dict(logits=A + 2), dict(logits=A + 1, dtype=1),
    dict(ids=A + 2), dict(gates=A + 2), dict(bias=A + 1),
])
def test_topk_refuses(kw):
    assert _topk(**kw) == ftq.ERR_INVALID_ARG
    assert ftq.last_error()


@pytest.mark.parametrize("kw", [dict(E=1025, ld=1025), dict(k=65), dict(E=130, ld=130, ng=65, tg=65), dict(T=2 ** 52, ld=2 ** 20)])
def test_topk_unsupported(kw):
    assert _topk(**kw) == ftq.ERR_UNSUPPORTED
    assert ftq.last_error()


def test_topk_zero_rows():
    assert _topk(T=0, logits=None, ids=None, gates=None) == ftq.OK


def test_quantize_refuses():
    q = ftq.lib().ftq_quantize_fp8
    ok = dict(x=A, dtype=2, ld=256, T=4, K=256, y=A, s=A)

    def call(**kw):
        d = {**ok, **kw}
        return q(P(d["x"]), d["dtype"], d["ld"], d["T"], d["K"], P(d["y"]), P(d["s"]), None)
    for kw in (dict(dtype=5), dict(K=0), dict(K=-16), dict(K=24), dict(ld=240), dict(ld=260), dict(T=-1), dict(x=None), dict(y=None),
               dict(s=None), dict(x=A + 8), dict(y=A + 8), dict(s=A + 2)):
        assert call(**kw) == ftq.ERR_INVALID_ARG, kw
        assert ftq.last_error()
    assert call(T=2 ** 60) == ftq.ERR_UNSUPPORTED
    assert call(T=0, x=None) == ftq.OK


def test_quantize_weight_refuses():
    q = ftq.lib().ftq_quantize_fp8_weight
    ok = dict(w=A, dtype=2, E=2, N=40, K=256, y=A, s=A)

    def call(**kw):
        d = {**ok, **kw}
        return q(P(d["w"]), d["dtype"], d["E"], d["N"], d["K"], P(d["y"]), P(d["s"]), None)
    for kw in (dict(dtype=5), dict(K=0), dict(K=24), dict(E=-1), dict(N=-1), dict(E=-1, N=-1), dict(E=2 ** 62, N=4), dict(w=None),
               dict(y=None), dict(s=None), dict(w=A + 8), dict(y=A + 8), dict(s=A + 2)):
        assert call(**kw) == ftq.ERR_INVALID_ARG, kw
    assert call(E=2 ** 30, N=2 ** 30) == ftq.ERR_UNSUPPORTED
    assert call(E=0, w=None) == ftq.OK and call(N=0, w=None) == ftq.OK


def _moe(w=A, ws=A, a=A, as_=A, ids=A, out=A, od=0, E=8, N=64, K=256, T=4, k=2, pp=0, act=0, wk=None, wkb=0, path=1, routed=False):
    f = ftq.lib().ftq_moe_fp8_routed if routed else ftq.lib().ftq_moe_fp8
    return f(P(w), P(ws), P(a), P(as_), P(ids), P(out), od, E, N, K, T, k, pp, act, P(wk), wkb, path, None)


@pytest.mark.parametrize("kw", [
    dict(K=0), dict(K=-16), dict(K=40), dict(E=0), dict(N=0), dict(k=0), dict(T=-1), dict(k=9), dict(path=7), dict(od=3), dict(act=9),
    dict(act=1, N=65), dict(w=None), dict(ws=None), dict(a=None), dict(as_=None), dict(ids=None), dict(out=None), dict(w=A + 8),
    dict(ws=A + 2), dict(a=A + 8), dict(as_=A + 2), dict(ids=A + 2), dict(out=A + 2), dict(out=A + 1, od=2),
])
@pytest.mark.parametrize("routed", [False, True])
def test_moe_refuses(kw, routed):
    assert _moe(**kw, routed=routed) == ftq.ERR_INVALID_ARG
    assert ftq.last_error()


@pytest.mark.parametrize("kw", [dict(act=1, N=48), dict(E=4096, k=1), dict(T=2 ** 31, E=2, k=1, path=2), dict(T=2049, path=1),
                                dict(K=2 ** 58), dict(N=2 ** 60), dict(T=2 ** 29, K=2 ** 32, path=2)])
def test_moe_unsupported(kw):
    assert _moe(**kw) == ftq.ERR_UNSUPPORTED
    assert ftq.last_error()


def test_moe_workspace():
    need = ftq.fp8_workspace_bytes(8, 64, 256, 4, 2, ftq.PATH_GROUPED)
    assert need > 0 and need % 256 == 0
    assert ftq.fp8_workspace_bytes(8, 64, 256, 4, 2, ftq.PATH_GEMV) == 0
    assert ftq.fp8_workspace_bytes(8, 64, 256, 0, 2, ftq.PATH_GROUPED) == 0
    assert _moe(path=2) == ftq.ERR_WORKSPACE
    assert _moe(path=2, wk=A, wkb=need - 1) == ftq.ERR_WORKSPACE
    assert _moe(path=2, wk=A + 16, wkb=need) == ftq.ERR_INVALID_ARG
    route = ftq.lib().ftq_moe_fp8_route
    assert route(P(A), 8, 4, 2, P(A), need - 1, 2, None) == ftq.ERR_WORKSPACE
    assert route(None, 8, 4, 2, P(A), need, 2, None) == ftq.ERR_INVALID_ARG
    assert route(P(A), 8, 4, 2, None, 0, ftq.PATH_GEMV, None) == ftq.OK   # nothing to route
    assert _moe(T=0, w=None, ids=None, out=None, path=0) == ftq.OK
    with pytest.raises(ftq.FtqError):
        ftq.fp8_workspace_bytes(8, 64, 250, 4, 2)
    with pytest.raises(ftq.FtqError):
        ftq.fp8_select_path(8, 64, 250, 4, 2)


def test_path_choice():
    # one token, a decode batch, a prefill chunk
    assert ftq.fp8_select_path(128, 1408, 2816, 1, 8) == ftq.PATH_GEMV
    assert ftq.fp8_select_path(8, 14336, 4096, 8, 2) == ftq.PATH_GEMV
    assert ftq.fp8_select_path(128, 1408, 2816, 8191, 8) == ftq.PATH_GROUPED
    # the GEMV path is never chosen where it would be refused
    for E, k in ((8, 2), (128, 8), (1024, 8), (4095, 64)):
        for T in (1, 64, 512, 513, 2048, 100000):
            if T * k > 4096:
                assert ftq.fp8_select_path(E, 64, 256, T, k) == ftq.PATH_GROUPED
    # at most 2 pairs an expert, or little work in all
    assert ftq.fp8_select_path(128, 1408, 2816, 32, 8) == ftq.PATH_GEMV
    assert ftq.fp8_select_path(128, 1408, 2816, 33, 8) == ftq.PATH_GROUPED
    assert ftq.fp8_select_path(8, 704, 1024, 128, 2) == ftq.PATH_GEMV
    assert ftq.fp8_select_path(8, 704, 1024, 1024, 2) == ftq.PATH_GROUPED


def test_routed_calls_name_their_path():
    route = ftq.lib().ftq_moe_fp8_route
    assert route(P(A), 8, 4, 2, P(A), 1 << 20, ftq.PATH_AUTO, None) == ftq.ERR_INVALID_ARG
    assert _moe(path=0, wk=A, wkb=1 << 20, routed=True) == ftq.ERR_INVALID_ARG
    assert "path" in ftq.last_error()


def test_binding_refuses_host_tensors():
    x = torch.zeros(4, 128)
    for f in (lambda: ftq.moe_topk(x, 2), lambda: ftq.quantize_fp8(x), lambda: ftq.quantize_fp8_weight(x[None])):
        with pytest.raises(ValueError):
            f()


def test_definitions_agree_with_torch():
    """The tests' e4m3 tables against torch's conversions, over every code and many quotients."""
    codes = torch.arange(256, dtype=torch.uint8)
    assert np.array_equal(codes.view(torch.float8_e4m3fn).double().numpy(), _fp8.TABLE, equal_nan=True)
    rng = np.random.default_rng(0)
    q = np.concatenate([rng.uniform(-460, 460, 20000), rng.normal(0, 1, 20000), rng.normal(0, 0.01, 20000),
                        (_fp8.TABLE[:126] + _fp8.TABLE[1:127]) / 2, _fp8.TABLE[:127], [0.0, 2.0 ** -10, 2.0 ** -11]]).astype(np.float32)
    t = torch.from_numpy(np.clip(q, -448, 448)).to(torch.float8_e4m3fn).view(torch.uint8).numpy()
    assert np.array_equal(_fp8.e4m3_codes(q), t)
