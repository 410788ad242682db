"""Refusals of the attention calls: errors come back before any launch, and the
Python layer names what is wrong with a tensor."""
import ctypes as C
import re

import pytest


@pytest.fixture(scope="module")
def L():
    from byte_level_lm_amd import _lib
    return _lib.lib()


P = C.c_void_p(4096)
ODD = C.c_void_p(4100)


def _write(L, k=P, v=P, dt=1, off=P, nseq=2, total=8, hkv=2, d=64, ks=128, vs=128, start=None, table=P, cols=4, pdt=1,
           npages=9, page=64, kp=P, vp=P, kc=None, vc=None):
    return L.bllm_kv_write(k, v, dt, off, nseq, total, hkv, d, ks, vs, start, table, cols, pdt, npages, page, kp, vp, kc,
                           vc, None)


def test_write_refusals(L):
    for bad in (dict(k=None), dict(v=None), dict(nseq=0), dict(total=-1), dict(hkv=0), dict(d=0), dict(ks=127), dict(vs=64),
                dict(table=None), dict(cols=0), dict(npages=0), dict(page=0), dict(kp=None), dict(vp=None), dict(off=None),
                dict(pdt=2), dict(pdt=2, kc=P), dict(kc=P), dict(vc=P)):
        assert _write(L, **bad) == -1, bad
    for bad in (dict(dt=0), dict(dt=2), dict(d=60, ks=512, vs=512), dict(d=264, ks=1024, vs=1024), dict(page=8), dict(page=48),
                dict(page=512), dict(pdt=0), dict(pdt=2, kc=P, vc=P, d=24), dict(pdt=2, kc=C.c_void_p(4098), vc=P),
                dict(k=ODD), dict(v=ODD), dict(kp=ODD), dict(vp=ODD), dict(ks=132), dict(vs=1 << 22), dict(nseq=65536),
                dict(cols=1 << 25), dict(npages=1 << 31), dict(total=(1 << 30) + 1), dict(hkv=1025, ks=1 << 20, vs=1 << 20)):
        assert _write(L, **bad) == -2, bad
    assert _write(L, total=0, k=None, v=None) == 0


def test_read_refusals(L):
    def read(kp=P, vp=P, kc=None, vc=None, pdt=1, npages=9, page=64, hkv=2, d=64, table=P, cols=4, off=P, nseq=2, total=8,
             start=None, dt=1, ko=P, vo=P):
        return L.bllm_kv_read(kp, vp, kc, vc, pdt, npages, page, hkv, d, table, cols, off, nseq, total, start, dt, ko, vo, None)
    for bad in (dict(kp=None), dict(vp=None), dict(table=None), dict(off=None), dict(nseq=0), dict(total=-1), dict(ko=None),
                dict(vo=None), dict(pdt=2), dict(kc=P, vc=P), dict(hkv=0)):
        assert read(**bad) == -1, bad
    for bad in (dict(dt=0), dict(d=12), dict(page=20), dict(ko=ODD), dict(vo=ODD), dict(kp=ODD), dict(pdt=0),
                dict(total=(1 << 30) + 1)):
        assert read(**bad) == -2, bad
    assert read(total=0, ko=None, vo=None) == 0


def test_attention_refusals(L):
    def att(q=P, k=P, v=P, dt=1, off=P, koff=P, nseq=2, total=8, total_k=9, hq=4, hkv=2, d=64, qs=256, ks=128, vs=128,
            scale=1.0, causal=1, window=0, cap=0.0, o=P, ws=P, wsb=1 << 40):
        return L.bllm_attention(q, k, v, dt, off, koff, nseq, total, total_k, hq, hkv, d, qs, ks, vs, scale, causal, window,
                                cap, None, None, o, ws, wsb, None)
    nan = float("nan")
    for bad in (dict(q=None), dict(k=None), dict(v=None), dict(off=None), dict(koff=None), dict(o=None), dict(nseq=0),
                dict(total=-1), dict(total_k=-1), dict(hq=0), dict(hkv=0), dict(hq=3), dict(d=0), dict(qs=255), dict(ks=127),
                dict(vs=120), dict(scale=nan), dict(window=-1), dict(cap=-1.0), dict(cap=nan), dict(cap=float("inf"))):
        assert att(**bad) == -1, bad
    for bad in (dict(dt=0), dict(dt=2), dict(d=60), dict(d=264, qs=2048, ks=1024, vs=1024), dict(qs=260), dict(ks=1 << 22),
                dict(q=ODD), dict(k=ODD), dict(v=ODD), dict(o=ODD), dict(nseq=65536), dict(total=(1 << 30) + 1),
                dict(total_k=(1 << 30) + 1), dict(hq=2048, hkv=2, qs=1 << 20), dict(cap=1025.0), dict(cap=1e-4), dict(ws=ODD)):
        assert att(**bad) == -2, bad
    assert att(ws=None) == att(wsb=8) == -3
    assert att(total=0, q=None, o=None) == 0
    assert L.bllm_attention_workspace(0, 8, 8, 4, 2, 64) == 0 and L.bllm_attention_workspace(2, 8, 8, 4, 2, 64) > 0


def test_step_refusals(L):
    def step(q=P, dt=1, nseq=2, hq=4, hkv=2, d=64, qs=256, kp=P, vp=P, kc=None, vc=None, pdt=1, npages=9, page=64, table=P,
             cols=4, lengths=P, scale=1.0, window=0, cap=0.0, o=P, ws=P, wsb=1 << 40):
        return L.bllm_attention_step(q, dt, nseq, hq, hkv, d, qs, kp, vp, kc, vc, pdt, npages, page, table, cols, lengths,
                                     scale, window, cap, None, None, o, ws, wsb, None)
    for bad in (dict(q=None), dict(kp=None), dict(vp=None), dict(table=None), dict(lengths=None), dict(o=None), dict(nseq=0),
                dict(hq=3), dict(hq=0), dict(qs=128), dict(pdt=2), dict(kc=P), dict(scale=float("nan")), dict(window=-1),
                dict(cap=-2.0), dict(cols=0)):
        assert step(**bad) == -1, bad
    for bad in (dict(dt=0), dict(d=60), dict(page=17), dict(pdt=0), dict(q=ODD), dict(o=ODD), dict(kp=ODD), dict(qs=1 << 22),
                dict(nseq=65536), dict(cols=1 << 26), dict(hq=2048, qs=1 << 18), dict(cap=2000.0), dict(ws=ODD)):
        assert step(**bad) == -2, bad
    assert step(ws=None) == step(wsb=8) == -3
    assert L.bllm_attention_step_workspace(0, 4, 2, 64, 256) == 0 and L.bllm_attention_step_workspace(2, 4, 2, 64, 256) > 0


def test_python_layer_names_the_argument():
    """Shapes, dtypes and places are checked before the library is called."""
    import torch
    import byte_level_lm_amd as B
    q, pages, table = torch.zeros(4, 2, 64), torch.zeros(3, 2, 16, 64), torch.zeros(1, 3, dtype=torch.int32)
    with pytest.raises(ValueError, match="GPU"):
        B.attention(q, q, q, torch.tensor([0, 4]))
    with pytest.raises(ValueError, match="GPU"):
        B.attention_step(q[:1], pages, pages, table, torch.ones(1, dtype=torch.int32))
    with pytest.raises(ValueError, match="GPU"):
        B.kv_write(q, q, pages, pages, table, offsets=torch.tensor([0, 4]))
    with pytest.raises(ValueError, match="GPU"):
        B.kv_read(pages, pages, table, torch.tensor([0, 4]), 4)


@pytest.mark.gpu
def test_python_layer_refuses_wrong_tensors():
    import torch
    import byte_level_lm_amd as B
    dev, bf16, i32 = "cuda", torch.bfloat16, torch.int32
    q = torch.zeros(4, 2, 64, device=dev, dtype=bf16)
    off, pages = torch.tensor([0, 4], device=dev), torch.zeros(3, 2, 16, 64, device=dev, dtype=bf16)
    table, one = torch.zeros(1, 3, device=dev, dtype=i32), torch.ones(1, device=dev, dtype=i32)
    scale, codes = torch.zeros(3, 2, 16, device=dev), pages.to(torch.int8)
    cases = [
        (lambda: B.attention(q, q[:3], q[:3], off), "k_offsets"), (lambda: B.attention(q, q, q[:3], off), "v must"),
        (lambda: B.attention(q, q, q, off.int()), "offsets"), (lambda: B.attention(q, q, q, off, k_offsets=off[:1]), "k_offsets"),
        (lambda: B.attention(q.transpose(1, 2), q, q, off), "dense"), (lambda: B.attention(q, q, q, off, window=0), "window"),
        (lambda: B.attention(q, q, q, off, cap=0.0), "cap"), (lambda: B.attention(q, q, q, off, slopes=scale), "slopes"),
        (lambda: B.attention(q, q, q, off, prefix=off), "prefix"), (lambda: B.attention(q, q, q, off, o_out=q[:2]), "o_out"),
        (lambda: B.attention(q, q, q, off, ws=q[:0]), "workspace"), (lambda: B.attention(q, q, q, off.cpu()), "GPU"),
        (lambda: B.attention_step(q, pages, pages, table, one), "q must"),
        (lambda: B.attention_step(q[:1], pages, pages, table, one.long()), "lengths"),
        (lambda: B.attention_step(q[:1], pages, pages, table.long(), one), "table"),
        (lambda: B.attention_step(q[:1], pages, pages[:2], table, one), "one shape"),
        (lambda: B.attention_step(q[:1], codes, codes, table, one), "8-bit"),
        (lambda: B.attention_step(q[:1], pages, pages, table, one, k_scale=scale), "8-bit"),
        (lambda: B.kv_write(q, q, pages, pages, table), "without offsets"),
        (lambda: B.kv_write(q[:, :1], q, pages, pages, table, offsets=off), "k must"),
        (lambda: B.kv_write(q, q, pages, pages, table, offsets=off, start=off), "start"),
        (lambda: B.kv_write(q, q, codes, codes, table, offsets=off, k_scale=scale, v_scale=scale[:2]), "v_scale"),
        (lambda: B.kv_read(pages, pages, table, off, 4, k_out=q[:2]), "k_out"),
        (lambda: B.kv_read(pages.transpose(1, 2), pages.transpose(1, 2), table, off, 4), "contiguous"),
    ]
    for call, word in cases:
        with pytest.raises(ValueError, match=re.escape(word)):
            call()
    for call in (lambda: B.attention(q, q.float(), q, off), lambda: B.attention(q.half(), q.half(), q.half(), off),
                 lambda: B.kv_read(pages.float(), pages.float(), table, off, 4)):
        with pytest.raises(TypeError):
            call()
    with pytest.raises(B.BllmError, match="unsupported"):
        B.attention(q.float(), q.float(), q.float(), off)
