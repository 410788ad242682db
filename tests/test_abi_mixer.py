"""Refusals of the mixer block's entry points: errors come back before any launch,
and the Python layer names what is wrong with a tensor."""
import ctypes as C
import re

import pytest


@pytest.fixture(scope="module")
def L():
    from byte_level_lm_amd import _lib
    return _lib.lib()


P = C.c_void_p(4096)
ODD = C.c_void_p(4100)


def test_norm_refusals(L):
    norm = lambda x=P, r=None, w=P, dt=1, rows=4, d=64, eps=1e-6, ro=None, y=P: L.bllm_rmsnorm(  # noqa: E731
        x, r, w, dt, rows, d, eps, ro, y, None)
    assert norm(x=None) == norm(w=None) == norm(y=None) == norm(rows=-1) == norm(d=0) == norm(eps=-1.0) == -1
    assert norm(eps=float("nan")) == norm(ro=P) == -1
    assert norm(dt=2) == norm(d=60) == norm(dt=0, d=6) == norm(x=ODD) == norm(w=ODD) == norm(y=ODD) == norm(r=ODD) == -2
    assert norm(d=1 << 24) == norm(rows=1 << 31) == -2
    assert norm(rows=0, x=None, y=None) == 0
    q8 = lambda x=P, q=P, s=P, d=64, rows=4: L.bllm_rmsnorm_q8(x, None, P, 1, rows, d, 1e-6, None, q, s, None)  # noqa: E731
    assert q8(q=None) == q8(s=None) == q8(x=None) == -1
    assert q8(q=ODD) == q8(s=C.c_void_p(4098)) == q8(d=4) == -2
    assert L.bllm_quant_rows_q8(None, 1, 4, 64, P, P, None) == L.bllm_quant_rows_q8(P, 1, 4, 64, None, P, None) == -1
    assert L.bllm_quant_rows_q8(P, 1, 4, 63, P, P, None) == -2 and L.bllm_quant_rows_q8(None, 1, 0, 64, None, None, None) == 0


def test_linear_refusals(L):
    lin = lambda x=P, sx=P, w=P, sw=P, dt=1, m=4, n=4, k=64, y=P: L.bllm_linear_i8(  # noqa: E731
        x, sx, w, sw, None, dt, m, n, k, y, None)
    assert lin(x=None) == lin(sx=None) == lin(w=None) == lin(sw=None) == lin(y=None) == lin(m=-1) == lin(n=0) == lin(k=0) == -1
    assert lin(dt=3) == lin(k=24) == lin(k=131072) == lin(x=ODD) == lin(w=ODD) == lin(y=ODD) == lin(m=1 << 31) == -2
    assert lin(n=1 << 31) == -2
    assert lin(m=0, x=None, sx=None, y=None) == 0


def test_delta_refusals(L):
    def prompt(q=P, off=P, nseq=2, total=8, hk=2, hv=4, dk=64, dv=64, qs=128, ks=128, vs=256, scale=1.0, dt=1, o=P,
               ws=P, wsb=1 << 40, g=P):
        return L.bllm_gated_delta(q, P, P, g, P, dt, off, nseq, total, hk, hv, dk, dv, qs, ks, vs, scale, 1, None, None, o,
                                  ws, wsb, None)
    assert prompt(q=None) == prompt(off=None) == prompt(g=None) == prompt(o=None) == prompt(nseq=0) == prompt(total=-1) == -1
    assert prompt(hk=0) == prompt(hv=3) == prompt(hv=1) == prompt(dk=0) == prompt(dv=0) == prompt(qs=127) == prompt(vs=248) == -1
    assert prompt(scale=float("nan")) == -1
    assert prompt(dt=0) == prompt(dk=60) == prompt(dv=60) == prompt(dk=136, qs=512, ks=512) == prompt(qs=132) == prompt(q=ODD) == -2
    assert prompt(dv=1032, vs=1 << 14) == prompt(nseq=65536) == prompt(total=1 << 31) == prompt(o=ODD) == -2
    assert prompt(ws=None) == prompt(wsb=8) == -3
    assert L.bllm_gated_delta_workspace(0, 8, 4, 64, 64) == 0 and L.bllm_gated_delta_workspace(2, 8, 4, 64, 64) > 0

    def step(si=P, so=P, slots=None, nslots=2, nseq=2, q=P, dk=64):
        return L.bllm_gated_delta_step(q, P, P, P, P, 1, nseq, 2, 4, dk, 64, 128, 128, 256, 1.0, 1, si, so, slots, nslots, P,
                                       None)
    assert step(si=None) == step(so=None) == step(nslots=0) == step(nslots=1) == step(q=None) == step(nseq=0) == -1
    assert step(si=ODD) == step(so=ODD) == step(dk=60) == step(nseq=65536, nslots=65536) == -2


def test_python_layer_names_the_argument():
    """Shapes, dtypes and places are checked before the library is called."""
    import torch
    import byte_level_lm_amd as B
    x = torch.zeros(4, 64)
    with pytest.raises(ValueError, match="GPU"):
        B.rmsnorm(x, torch.ones(64))
    with pytest.raises(ValueError, match="GPU"):
        B.linear_i8(x.to(torch.int8), torch.ones(4), x.to(torch.int8), torch.ones(4))
    with pytest.raises(ValueError, match="GPU"):
        B.gated_delta(x[:, None], x[:, None], x[:, None], x, x, torch.tensor([0, 4]))


@pytest.mark.gpu
def test_python_layer_refuses_wrong_tensors():
    import torch
    import byte_level_lm_amd as B
    dev = "cuda"
    x, w = torch.zeros(4, 64, device=dev), torch.ones(64, device=dev)
    for bad, word in [(dict(residual=x[:3]), "residual"), (dict(residual_out=x), "residual"), (dict(y_out=x.half()), "y_out")]:
        with pytest.raises(ValueError, match=word):
            B.rmsnorm(x, w, **bad)
    with pytest.raises(ValueError, match="w must"):
        B.rmsnorm(x, w[:8])
    with pytest.raises(ValueError, match="contiguous"):
        B.rmsnorm_q8(x[:, ::2], w[::2])
    with pytest.raises(TypeError):
        B.rmsnorm(x.half(), w.half())
    xq, s = x.to(torch.int8), torch.ones(4, device=dev)
    with pytest.raises(ValueError, match="x_scale"):
        B.linear_i8(xq, s[:3], xq, s)
    with pytest.raises(TypeError):
        B.linear_i8(x, s, xq, s)
    with pytest.raises(B.BllmError, match="unsupported"):
        B.linear_i8(xq[:, :24].contiguous(), s, xq[:, :24].contiguous(), s)
    q = torch.zeros(4, 2, 64, device=dev, dtype=torch.bfloat16)
    g, off = torch.zeros(4, 2, device=dev), torch.tensor([0, 4], device=dev)
    for args, word in [((q, q, q, g[:3], g, off), "g must"), ((q, q[:, :1], q, g, g, off), "k must"),
                       ((q, q, q[:2], g, g, off), "same tokens"), ((q, q, q, g, g, off.int()), "offsets"),
                       ((q.transpose(1, 2), q.transpose(1, 2), q, g, g, off), "dense")]:
        with pytest.raises(ValueError, match=re.escape(word)):
            B.gated_delta(*args)
    with pytest.raises(B.BllmError, match="unsupported"):
        B.gated_delta(q.float(), q.float(), q.float(), g, g, off)
    st = torch.zeros(4, 2, 64, 64, device=dev)
    with pytest.raises(ValueError, match="slots"):
        B.gated_delta_step(q, q, q, g, g, st, slots=torch.zeros(4, device=dev, dtype=torch.int64))
    with pytest.raises(ValueError, match="state_out"):
        B.gated_delta_step(q, q, q, g, g, st, state_out=st[:2])
