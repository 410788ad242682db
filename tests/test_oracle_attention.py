"""Pins for the attention half of the oracle: closed forms, invariants, PyTorch's softmax."""
import numpy as np
import pytest

import oracle


def _qkv(rng, n, m, hq=2, hkv=1, d=16):
    return rng.standard_normal((n, hq, d)), rng.standard_normal((m, hkv, d)), rng.standard_normal((m, hkv, d))


def test_equal_scores_give_the_mean_of_what_is_seen():
    rng = np.random.default_rng(0)
    _, _, v = _qkv(rng, 6, 6)
    q, k, off = np.zeros((6, 2, 16)), np.ones((6, 1, 16)), np.array([0, 4, 6])
    o = oracle.attention(q, k, v, off)
    for s in range(2):
        for i in range(off[s], off[s + 1]):
            np.testing.assert_allclose(o[i, 1], v[off[s]:i + 1, 0].mean(0))
    o = oracle.attention(q, k, v, off, window=2)
    np.testing.assert_allclose(o[3, 0], v[2:4, 0].mean(0))
    o = oracle.attention(q, k, v, off, window=2, prefix=[1, 0])
    np.testing.assert_allclose(o[3, 0], v[[0, 2, 3], 0].mean(0))
    o = oracle.attention(q, k, v, off, causal=False, window=2)
    np.testing.assert_allclose(o[2, 0], v[1:4, 0].mean(0))


def test_against_torch_softmax_in_64_bits():
    import torch
    rng = np.random.default_rng(1)
    q, k, v = _qkv(rng, 9, 9, hq=4, hkv=2)
    o = oracle.attention(q, k, v, np.array([0, 9]))
    for h in range(4):
        x = torch.from_numpy(q[:, h]) @ torch.from_numpy(k[:, h // 2]).T * 16 ** -0.5
        x = x.masked_fill(torch.ones(9, 9).triu(1).bool(), -np.inf)
        np.testing.assert_allclose(o[:, h], (torch.softmax(x, 1) @ torch.from_numpy(v[:, h // 2])).numpy())


def test_cap_slopes_and_rows_that_see_nothing():
    rng = np.random.default_rng(2)
    q, k, v = _qkv(rng, 5, 3)
    off, koff = np.array([0, 5]), np.array([0, 3])
    o = oracle.attention(q, k, v, off, k_offsets=koff)
    assert not o[:2].any() and np.allclose(o[2], v[0, 0]) and o[3].any()
    # a large cap is none; a tiny one makes every score the same
    np.testing.assert_allclose(oracle.attention(q, k, v, off, k_offsets=koff, cap=1e6), o, atol=1e-9)
    np.testing.assert_allclose(oracle.attention(q, k, v, off, k_offsets=koff, cap=1e-9)[4, 0], v[:, 0].mean(0), atol=1e-8)
    # a steep slope leaves the nearest key
    np.testing.assert_allclose(oracle.attention(q, k, v, off, k_offsets=koff, slopes=[1e3, 0.0])[4, 0], v[2, 0])


@pytest.mark.parametrize("q8", [False, True])
def test_pages_give_the_rows_back(q8):
    rng = np.random.default_rng(3)
    rows, off = rng.standard_normal((20, 2, 16)).astype(np.float32), np.array([0, 13, 13, 20])
    table = np.array([[5, -1], [0, 1], [2, 99]], np.int32)
    start = np.array([14, 0, -2])
    pages = np.zeros((6, 2, 16, 16), np.int8 if q8 else np.float32)
    scale = np.zeros((6, 2, 16), np.float32) if q8 else None
    pages, scale = oracle.kv_write(rows, off, table, pages, start=start, scale=scale)
    back = oracle.kv_read(pages, off, table, start=start, scale=scale)
    assert not back[2:13].any() and not back[13:15].any()
    step = np.abs(rows).max(2, keepdims=True) / 127 * 0.5001 if q8 else 1e-12
    for r in [0, 1, *range(15, 20)]:
        assert np.all(np.abs(back[r] - rows[r]) <= (step[r] if q8 else step))


def test_step_is_the_last_row_of_the_prompt():
    rng = np.random.default_rng(4)
    q, k, v = _qkv(rng, 37, 37)
    table = np.array([[2, 0, 1]], np.int32)
    pages = [oracle.kv_write(x, [0, 37], table, np.zeros((3, 1, 16, 16)))[0] for x in (k, v)]
    for more in [{}, {"window": 9, "prefix": [3]}, {"cap": 2.0, "slopes": [0.1, 0.2]}]:
        want = oracle.attention(q, k, v, [0, 37], **more)[-1:]
        np.testing.assert_allclose(oracle.attention_step(q[-1:], *pages, table, np.array([37]), **more), want)
