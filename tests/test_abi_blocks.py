"""Refusals of the norm, e4m3 and grouped entry points, on the host before any device work."""
import ctypes

import pytest
import torch

from quantized_lora_fine_b200 import _lib, api, build

NULL, SHAPE, ALIGN, DTYPE, UNSUPPORTED, WORKSPACE = 1, 2, 3, 4, 5, 7
P, Q = 0x10000, 0x10008      # an aligned address and one that is not


@pytest.fixture(scope="module")
def lib():
    build.build()
    return _lib.load()


def _weight(**kw):
    w = _lib.ExpertWeight()
    w.experts, w.out, w.in_, w.is_bf16, w.codes, w.scale, w.w_bf16 = 1, 256, 128, 0, P, P, P
    for k, v in kw.items():
        setattr(w, k, v)
    return ctypes.byref(w)


def _norm(lib, **kw):
    a = dict(x=P, r=P, w=P, dt=0, M=4, H=64, eps=1e-6, h=P, y=P, y8=None, ys=None, rstd=P)
    a.update(kw)
    return lib.qlora_rms_norm_fwd(a["x"], a["r"], a["w"], a["dt"], a["M"], a["H"], a["eps"], a["h"], a["y"], a["y8"],
                                  a["ys"], a["rstd"], None)


def test_norm_forward(lib):
    assert _norm(lib, dt=2) == DTYPE
    for kw in (dict(M=0), dict(M=-1), dict(M=(1 << 30) + 1), dict(H=0), dict(H=12), dict(H=32776)):
        assert _norm(lib, **kw) == SHAPE, kw
    assert _norm(lib, eps=-1.0) == UNSUPPORTED
    assert _norm(lib, eps=float("nan")) == UNSUPPORTED
    for kw in (dict(x=None), dict(w=None), dict(rstd=None), dict(h=None), dict(y=None), dict(y8=P)):
        assert _norm(lib, **kw) == NULL, kw
    for kw in (dict(x=Q), dict(r=Q), dict(w=Q), dict(h=Q), dict(y=Q), dict(y8=Q, ys=P), dict(y8=P, ys=P + 2),
               dict(rstd=P + 1)):
        assert _norm(lib, **kw) == ALIGN, kw


def _norm_bwd(lib, **kw):
    a = dict(dy=P, dh=P, h=P, rstd=P, w=P, dt=0, M=4, H=64, dx=P, dw=P, ws=P, n=1 << 20)
    a.update(kw)
    return lib.qlora_rms_norm_bwd(a["dy"], a["dh"], a["h"], a["rstd"], a["w"], a["dt"], a["M"], a["H"], a["dx"],
                                  a["dw"], a["ws"], a["n"], None)


def test_norm_backward(lib):
    assert _norm_bwd(lib, dt=7) == DTYPE
    for kw in (dict(M=0), dict(H=4), dict(H=1 << 20)):
        assert _norm_bwd(lib, **kw) == SHAPE, kw
    for kw in (dict(dy=None), dict(h=None), dict(rstd=None), dict(w=None), dict(dx=None)):
        assert _norm_bwd(lib, **kw) == NULL, kw
    for kw in (dict(dy=Q), dict(dh=Q), dict(h=Q), dict(w=Q), dict(dx=Q), dict(dw=Q)):
        assert _norm_bwd(lib, **kw) == ALIGN, kw
    need = lib.qlora_rms_norm_bwd_workspace_size(4, 64)
    assert need >= 4 * 64 * 4
    for kw in (dict(ws=None), dict(ws=Q), dict(n=need - 1)):
        assert _norm_bwd(lib, **kw) == WORKSPACE, kw
    for m, h in ((0, 64), (4, 0), (4, 12), (-1, 64), (4, 32776)):
        assert lib.qlora_rms_norm_bwd_workspace_size(m, h) == 0


def test_quantizers(lib):
    for M, n in ((0, 128), (4, 0), (4, 120), (1 << 31, 128), (4, (1 << 24) + 16)):
        assert lib.fp8_quantize_rows(P, M, n, P, P, None) == SHAPE
    assert lib.fp8_quantize_rows(None, 4, 128, P, P, None) == NULL
    assert lib.fp8_quantize_rows(Q, 4, 128, P, P, None) == ALIGN
    assert lib.fp8_quantize_rows(P, 4, 128, P, P + 2, None) == ALIGN
    ok = (P, 256)
    assert lib.fp8_quantize_weight(P, 3, 1, 128, 128, P, P, *ok, None) == DTYPE
    for E, o, i in ((0, 128, 128), (1025, 128, 128), (1, 0, 128), (1, 128, 100), (1, 130, 128)):
        assert lib.fp8_quantize_weight(P, 0, E, o, i, P, P, *ok, None) == SHAPE
    assert lib.fp8_quantize_weight(P, 0, 1, 128, 128, None, P, *ok, None) == NULL
    assert lib.fp8_quantize_weight(P, 0, 1, 128, 128, P + 4, P, *ok, None) == ALIGN
    assert lib.fp8_quantize_weight(P, 0, 1, 128, 128, P, P, None, 256, None) == WORKSPACE
    assert lib.fp8_quantize_weight(P, 0, 1, 128, 128, P, P, P, 255, None) == WORKSPACE


@pytest.mark.parametrize("fn", ["fp8_linear_fwd", "fp8_linear_bwd"])
def test_fp8_linear(lib, fn):
    f = getattr(lib, fn)
    assert f(None, P, P, 4, P, P, 256, None) == NULL
    for kw in (dict(out=0), dict(in_=8), dict(out=100), dict(in_=(1 << 24) + 16), dict(experts=2), dict(experts=0)):
        assert f(_weight(**kw), P, P, 4, P, P, 256, None) == SHAPE, kw
    assert f(_weight(is_bf16=1), P, P, 4, P, P, 256, None) == UNSUPPORTED
    assert f(_weight(is_bf16=2), P, P, 4, P, P, 256, None) == DTYPE
    for kw in (dict(codes=None), dict(scale=None)):
        assert f(_weight(**kw), P, P, 4, P, P, 256, None) == NULL
    assert f(_weight(codes=Q), P, P, 4, P, P, 256, None) == ALIGN
    for M in (0, -5, (1 << 30) + 1):
        assert f(_weight(), P, P, M, P, P, 256, None) == SHAPE
    assert f(_weight(), None, P, 4, P, P, 256, None) == NULL
    assert f(_weight(), P, None, 3, P, P, 256, None) == NULL      # bf16 rows: up to 2, forward only
    if fn == "fp8_linear_bwd":
        assert f(_weight(), P, None, 4, P, P, 256, None) == NULL
    assert f(_weight(), P, P, 4, None, P, 256, None) == NULL
    assert f(_weight(), Q, P, 4, P, P, 256, None) == ALIGN
    assert f(_weight(), P, P, 4, Q, P, 256, None) == ALIGN
    assert f(_weight(), P, P, 4, P, None, 256, None) == WORKSPACE
    assert f(_weight(), P, P, 4, P, P, 16, None) == WORKSPACE
    assert lib.qlora_expert_workspace_size() == 256
    assert lib.fp8_linear_bf16_rows() == 2


def test_grouped_linear(lib):
    f, b = lib.qlora_grouped_linear_fwd, lib.qlora_grouped_linear_bwd
    bf = dict(is_bf16=1, experts=8)
    assert f(_weight(experts=1025), P, P, 4, P, P, P, 256, None) == SHAPE
    assert f(_weight(**bf), P, None, 0, P, P, P, 256, None) == SHAPE
    assert f(_weight(**bf, w_bf16=None), P, None, 4, P, P, P, 256, None) == NULL
    assert f(_weight(**bf), None, None, 4, P, P, P, 256, None) == NULL
    assert f(_weight(**bf), P, None, 4, None, P, P, 256, None) == NULL
    assert f(_weight(experts=8), P, None, 4, P, P, P, 256, None) == NULL        # 8-bit rows without scales
    assert f(_weight(**bf), P, None, 4, P + 2, P, P, 256, None) == ALIGN
    assert f(_weight(**bf), P, None, 4, P, Q, P, 256, None) == ALIGN
    assert f(_weight(**bf), P, None, 4, P, P, None, 0, None) == WORKSPACE
    assert b(_weight(experts=8), P, P, P, 4, P, P, P, P, 256, None) == UNSUPPORTED   # dW of a frozen weight
    assert b(_weight(**bf), None, P, None, 4, P, P, P, P, 256, None) == NULL         # dW without X
    assert b(_weight(**bf), P, P, None, 4, P, None, None, P, 256, None) == NULL      # nothing to compute
    assert b(_weight(**bf), P, P, None, 4, P, P, P + 4, P, 256, None) == ALIGN
    assert b(_weight(**bf), Q, P, None, 4, P, P, P, P, 256, None) == ALIGN


def test_binding_refuses_cpu_tensors():
    x, w = torch.zeros(4, 64, dtype=torch.bfloat16), torch.ones(64, dtype=torch.bfloat16)
    off = torch.zeros(2, dtype=torch.int32)
    for call in (lambda: api.rms_norm_fwd(x, w), lambda: api.rms_norm_bwd(x, x, w.float(), w),
                 lambda: api.fp8_quantize_rows(x), lambda: api.fp8_quantize_weight(x),
                 lambda: api.FP8Rows(x.to(torch.float8_e4m3fn), torch.zeros(4, 1)),
                 lambda: api.grouped_linear_fwd(x.view(1, 4, 64), x, off)):
        with pytest.raises(ValueError, match="CUDA tensor"):
            call()


@pytest.mark.parametrize("shape", [(), (16,), (1, 2, 16, 16)])
def test_binding_refuses_weights_of_other_ranks(shape):
    W, X = torch.zeros(shape, dtype=torch.bfloat16), torch.zeros(4, 16, dtype=torch.bfloat16)
    off = torch.zeros(2, dtype=torch.int32)
    with pytest.raises(ValueError, match="experts, out, in"):
        api.grouped_linear_fwd(W, X, off)
    with pytest.raises(ValueError, match="experts, out, in"):
        api.grouped_linear_bwd(W, X, X, off)


def test_status_word_is_not_set_up_while_capturing(monkeypatch):
    """The first call on a device allocates the status word; under capture that is refused in words."""
    monkeypatch.setattr(api.Workspace, "_bufs", {})
    monkeypatch.setattr(torch.cuda, "is_current_stream_capturing", lambda: True)
    with pytest.raises(RuntimeError, match="before capturing"):
        api.Workspace.status_word(0)
