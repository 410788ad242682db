"""8-bit pages whose scales lie on 4 bytes, as the calls allow, and on no more."""
import numpy as np
import pytest

import oracle
from tests.helpers import to_dev, to_np
from tests.test_gpu_attention import _bf16, _cache, _check, _dev16, _offsets

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("first", [1, 2, 3])
@pytest.mark.parametrize("d", [64, 128, 256])
def test_scales_on_4_bytes(first, d):
    import torch

    import byte_level_lm_amd as B
    rng = np.random.default_rng(d + first)
    lengths = [700, 3, 0, 65]
    pages, scales, table, dev, sc = _cache(rng, lengths, 2, d, 16, True)
    moved = {}
    for name, x in sc.items():
        buf = torch.full((x.numel() + 8,), 5.0, device="cuda")
        moved[name] = buf[first:first + x.numel()].view(x.shape)
        moved[name].copy_(x)
        assert moved[name].data_ptr() % 16 == 4 * first
    q, n = _bf16(rng, (4, 4, d)), to_dev(np.array(lengths, np.int32))
    want = oracle.attention_step(q, *pages, table, lengths, k_scale=scales[0], v_scale=scales[1], sizes=True)
    o = B.attention_step(_dev16(q), *dev, to_dev(table), n, **moved)
    _check(o, want, 2.0 ** -16, d)
    assert torch.equal(o, B.attention_step(_dev16(q), *dev, to_dev(table), n, **sc))
    off = to_dev(_offsets(lengths))
    back = [B.kv_read(*dev, to_dev(table), off, sum(lengths), **s) for s in (moved, sc)]
    assert all(torch.equal(a, b) for a, b in zip(*back))
    B.kv_write(*back[0], *dev, to_dev(table), offsets=off, **moved)
    again = B.kv_read(*dev, to_dev(table), off, sum(lengths), **moved)
    for a, b in zip(again, back[0]):  # half a code of the row and the rounding to bf16
        top = np.abs(to_np(b)).max(-1, keepdims=True)
        assert np.all(np.abs(to_np(a) - to_np(b)) <= 1.01 * top * (0.5 / 127 + 2.0 ** -8))
