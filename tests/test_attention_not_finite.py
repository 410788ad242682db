"""Values that are not finite in attention of packed prompts: what they do to the queries that see them, that the others
have the bits they have without them, and that a call with them takes no longer than a few passes."""
import numpy as np
import pytest

import oracle
from tests.helpers import say, to_dev, to_np
from tests.test_gpu_attention import _bf16, _check, _dev16, _mask, _offsets, _strided

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def B():
    import byte_level_lm_amd as B
    B.lib()
    return B


def _time(f, n=5):
    import torch
    f()
    ms = []
    for _ in range(n):
        a, b = (torch.cuda.Event(enable_timing=True) for _ in range(2))
        a.record()
        f()
        b.record()
        torch.cuda.synchronize()
        ms.append(a.elapsed_time(b))
    return sorted(ms)[n // 2]


@pytest.mark.parametrize("hq,hkv,d", [(12, 4, 128), (8, 8, 64), (4, 2, 256)])
def test_the_time_of_a_call_with_values_that_are_not_finite(B, hq, hkv, d):
    """512 causal queries a sequence with a NaN in the first row, in the middle, or an infinite column: some passes more."""
    import torch
    gen = torch.Generator(device="cuda").manual_seed(d)
    q, k, v = (torch.randn(4 * 512, h, d, device="cuda", generator=gen).to(torch.bfloat16) for h in (hq, hkv, hkv))
    off = torch.arange(5, device="cuda") * 512
    clean = _time(lambda: B.attention(q, k, v, off))
    for rows, value in ((0, float("nan")), (256, float("nan")), (slice(None), float("inf"))):
        v2 = v.clone()
        v2.view(4, 512, hkv, d)[:, rows, :, 3] = value
        ms = _time(lambda: B.attention(q, k, v2, off))
        say("d", d, "rows", rows, value, "%.1f us, without it %.1f" % (1e3 * ms, 1e3 * clean))
        assert ms < 20 * clean


def _seen(n, m, causal=True, window=None, prefix=0):
    t, j = np.arange(n)[:, None] + m - n, np.arange(m)[None, :]
    seen = np.ones((n, m), bool)
    if causal:
        seen &= j <= t
    if window:
        seen &= abs(t - j) < window
    return seen | (j < prefix)


# lengths of queries and keys
SHAPES = [([70, 300, 90], None), ([1, 40, 0, 5], [700, 40, 8, 3000]), ([130], [6000]), ([33, 20], [5, 20])]


@pytest.mark.parametrize("lengths,keys", SHAPES)
@pytest.mark.parametrize("hq,hkv,d", [(6, 2, 64), (2, 1, 128), (4, 4, 40), (3, 1, 200)])
@pytest.mark.parametrize("more", [{}, {"window": 45}, {"window": 700, "prefix": 20}, {"causal": False}, {"cap": 6.0, "slopes": True}],
                         ids=lambda m: "-".join(m) or "plain")
def test_what_a_query_sees_of_values_that_are_not_finite(B, lengths, keys, hq, hkv, d, more):
    """Infinities of one sign stay, of both or NaN give NaN, in the columns and heads that have them; everything else is bit for bit as
    without them."""
    rng = np.random.default_rng(sum(lengths) + d)
    off, koff = _offsets(lengths), _offsets(lengths if keys is None else keys)
    q, k, v = _bf16(rng, (int(off[-1]), hq, d), 0.5), _bf16(rng, (int(koff[-1]), hkv, d), 0.5), _bf16(rng, (int(koff[-1]), hkv, d))
    host, dev = _mask(more, rng, len(lengths), hq)
    if "slopes" in host:  # no weight becomes zero
        host["slopes"] = np.full(hq, 2.0 ** -9, np.float32)
        dev["slopes"] = to_dev(host["slopes"])
    args = dict(k_offsets=to_dev(koff), **dev)
    clean = to_np(B.attention(*_strided(q), *_strided(k, v), to_dev(off), **args)).astype(np.float64)
    v2 = v.copy()
    for _ in range(12):
        v2[rng.integers(koff[-1]), rng.integers(hkv), rng.integers(d)] = rng.choice([np.nan, np.inf, -np.inf])
    at = int(koff[-1]) // 2  # and two beside each other
    v2[at, 0, 1], v2[max(at - 1, 0), 0, 1], v2[-1, 0, 0] = np.inf, -np.inf, np.nan
    got = to_np(B.attention(*_strided(q), *_strided(k, v2), to_dev(off), **args)).astype(np.float64)
    want = clean.copy()
    for s in range(len(lengths)):
        rows, ks = slice(off[s], off[s + 1]), slice(koff[s], koff[s + 1])
        prefix = 0 if host.get("prefix") is None else int(host["prefix"][s])
        seen = _seen(lengths[s], int(koff[s + 1] - koff[s]), host.get("causal", True), host.get("window"), prefix).astype(np.float64)
        for h in range(hq):
            x = v2[ks, h * hkv // hq]
            nan, up, down = (seen @ c.astype(np.float64) > 0 for c in (np.isnan(x), x == np.inf, x == -np.inf))
            part = want[rows, h]
            part[up] = np.inf
            part[down] = -np.inf
            part[nan | (up & down)] = np.nan
    assert np.array_equal(got, want, equal_nan=True)


@pytest.mark.parametrize("keys", [100, 3000])
@pytest.mark.parametrize("d", [64, 128, 256])
def test_a_weight_of_zero_times_an_infinity(B, keys, d):
    """Keys whose weight beside the others is below what fp32 holds: zero times an infinity is NaN for who sees it, wherever
    in a tile it lies, and nothing for who does not."""
    rng = np.random.default_rng(d)
    n = 40
    q, k, v = np.ones((n, 2, d), np.float32), np.ones((keys, 2, d), np.float32), _bf16(rng, (keys, 2, d))
    for at in (5, keys - 33, keys - 17, keys - 1):
        k2, v2 = k.copy(), v.copy()
        k2[at], v2[at, 1, 7] = -200.0, np.inf
        off, koff = to_dev(_offsets([n])), to_dev(_offsets([keys]))
        clean = to_np(B.attention(*map(_dev16, (q, k2, v)), off, k_offsets=koff))
        got = to_np(B.attention(*map(_dev16, (q, k2, v2)), off, k_offsets=koff))
        want = clean.copy()
        want[max(at - (keys - n), 0):, 1, 7] = np.nan
        if at == keys - 1 and keys > n:  # the last query sees other keys too
            assert np.isnan(got[-1, 1, 7])
        assert np.array_equal(got, want, equal_nan=True)


@pytest.mark.parametrize("d", [64, 128, 256])
def test_large_values_whose_mean_fp32_holds(B, d):
    """The maximum that weights are taken against may lag by 2^8: sums that pass fp32 only for that are finite."""
    rng = np.random.default_rng(d + 1)
    n, keys, h = 5, 96, 2
    q, k = np.zeros((n, h, d), np.float32), np.zeros((keys, h, d), np.float32)
    q[:, :, 0], k[40:44, :, 0] = 1.0, 5.0  # weights of e^5 beside 1
    v = _bf16(rng, (keys, h, d)) * np.float32(2.0 ** 121)
    want = oracle.attention(q, k, v, _offsets([n]), k_offsets=_offsets([keys]), scale=1.0, sizes=True)
    o = B.attention(_dev16(q), _dev16(k), _dev16(v), to_dev(_offsets([n])), k_offsets=to_dev(_offsets([keys])), scale=1.0)
    _check(o, want, 2.0 ** -8, d)
