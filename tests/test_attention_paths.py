"""Orders of work and joins that shapes of their own bring about: blocks in the order of their keys together with shares, and with
keys of their own; a join of 9 to 64 shares by one wave a query (more than 2048 queries and heads).  The cards' places that the
host's rules count with: 4, 3 and 2 workgroups on each of 256 CUs up to d 64, 128 and 256; 8, 4 and 2 in a step."""
import numpy as np
import pytest

import oracle
from tests.helpers import to_dev, to_np
from tests.test_attention_not_finite import _seen
from tests.test_gpu_attention import _bf16, _cache, _check, _dev16, _mask, _offsets, _strided

pytestmark = pytest.mark.gpu

MASKS = [{}, {"prefix": 90}, {"cap": 4.0, "slopes": True}]

# in the order of their keys (two fifths of the places or more have a unit of work): with shares, 4 of each; with keys in front of the queries too; whole, 1 of each
RANKED = [([3300], None, 4, 4, 64), ([2000, 40, 0, 1500], None, 4, 4, 64), ([1800, 1, 1700], None, 4, 4, 32),
          ([1600, 30, 1200], None, 6, 3, 128), ([1300, 5, 1000], None, 4, 2, 200),
          ([1024, 1024], [2048, 2048], 12, 4, 128), ([1000, 700], [1500, 1200], 8, 8, 64), ([900, 700], [1200, 1300], 4, 2, 256),
          ([300] * 8, [500] * 8, 8, 8, 64), (30, 200, 8, 8, 64), (40, 200, 6, 2, 128), (35, 200, 4, 2, 200)]

# 9 to 64 shares of more than 2048 queries' heads, joined by a wave each
JOINED = [([275] * 4, [8192] * 4, 8, 8, 64), ([300, 0, 61], [9000, 50, 4000], 12, 2, 128), ([150, 60], [7000, 5000], 16, 2, 256),
          ([280, 300], [6000, 9000], 8, 4, 32), ([600], [9000], 4, 1, 128), ([400, 33], [9000, 9000], 8, 1, 200)]


@pytest.fixture(scope="module")
def B():
    import byte_level_lm_amd as B
    B.lib()
    return B


def _case(lengths, keys, hq, hkv, d):
    rng = np.random.default_rng(hq * d)
    if isinstance(lengths, int):  # so many of up to 330, behind up to `keys`
        lengths = rng.integers(0, 330, lengths)
        keys = lengths + rng.integers(0, keys, len(lengths))
    off = _offsets(lengths)
    koff = off if keys is None else _offsets(keys)
    q, k, v = _bf16(rng, (int(off[-1]), hq, d)), _bf16(rng, (int(koff[-1]), hkv, d)), _bf16(rng, (int(koff[-1]), hkv, d))
    return rng, off, koff, q, k, v


def _run(B, off, koff, q, k, v, **dev):
    return B.attention(*_strided(q), *_strided(k, v), to_dev(off), k_offsets=None if koff is off else to_dev(koff), **dev)


@pytest.mark.parametrize("lengths,keys,hq,hkv,d", RANKED, ids=lambda x: str(x)[:24])
@pytest.mark.parametrize("more", MASKS, ids=lambda m: "-".join(m) or "plain")
def test_blocks_in_the_order_of_their_keys(B, lengths, keys, hq, hkv, d, more):
    rng, off, koff, q, k, v = _case(lengths, keys, hq, hkv, d)
    host, dev = _mask(more, rng, len(off) - 1, hq)
    want = oracle.attention(q, k, v, off, k_offsets=koff, sizes=True, **host)
    o = _run(B, off, koff, q, k, v, **dev)
    _check(o, want, 2.0 ** -8, d, host.get("slopes"), int(np.max(np.diff(koff))))


@pytest.mark.parametrize("lengths,keys,hq,hkv,d", JOINED, ids=lambda x: str(x)[:24])
@pytest.mark.parametrize("more", [{}, {"window": 300, "prefix": 40}, {"causal": False}, {"cap": 4.0, "slopes": True}],
                         ids=lambda m: "-".join(m) or "plain")
def test_many_queries_of_many_shares(B, lengths, keys, hq, hkv, d, more):
    """With the window most shares hold no key that a query sees."""
    import torch
    rng, off, koff, q, k, v = _case(lengths, keys, hq, hkv, d)
    host, dev = _mask(more, rng, len(off) - 1, hq)
    want = oracle.attention(q, k, v, off, k_offsets=koff, sizes=True, **host)
    size = B.attention_workspace(len(off) - 1, len(q), len(k), hq, hkv, d)
    buf = torch.full((size + 4096,), 77, device="cuda", dtype=torch.uint8)
    o = _run(B, off, koff, q, k, v, ws=buf[:size], **dev)
    assert torch.all(buf[size:] == 77)
    _check(o, want, 2.0 ** -8, d, host.get("slopes"), int(np.max(np.diff(koff))))


@pytest.mark.parametrize("lengths,keys,hq,hkv,d", [RANKED[1], RANKED[3], RANKED[4], RANKED[6], JOINED[0], JOINED[1], JOINED[2]],
                         ids=lambda x: str(x)[:24])
def test_values_that_are_not_finite_in_these_orders(B, lengths, keys, hq, hkv, d):
    rng, off, koff, q, k, v = _case(lengths, keys, hq, hkv, d)
    q *= np.float32(0.25)  # no weight is zero
    clean = to_np(_run(B, off, koff, q, k, v))
    v2 = v.copy()
    for _ in range(6):
        v2[rng.integers(koff[-1]), rng.integers(hkv), rng.integers(d)] = np.nan
    v2[-1, 0, 0] = np.nan
    want = clean.copy()
    for s in range(len(off) - 1):
        seen = _seen(int(off[s + 1] - off[s]), int(koff[s + 1] - koff[s])).astype(np.float32)
        for h in range(hq):
            bad = np.isnan(v2[koff[s]:koff[s + 1], h * hkv // hq]).astype(np.float32)
            want[off[s]:off[s + 1], h][seen @ bad > 0] = np.nan
    assert np.array_equal(to_np(_run(B, off, koff, q, k, v2)), want, equal_nan=True)


@pytest.mark.parametrize("d,q8", [(64, False), (64, True), (24, False), (16, True)])
@pytest.mark.parametrize("more", [{}, {"window": 70, "prefix": 30}, {"cap": 3.0, "slopes": True}], ids=lambda m: "-".join(m) or "plain")
def test_a_step_of_many_heads_in_many_shares(B, d, q8, more):
    """17 streams, 128 heads on 8: 16 shares of a table of 2112 positions."""
    rng = np.random.default_rng(d)
    lengths = np.array([2112, 0, 1, 700, 2000, 128, 129, 33, 1500, 2111, 16, 900, 64, 31, 1999, 5, 1024], np.int32)
    pages, scales, table, dev, sc = _cache(rng, lengths, 8, d, 16, q8)
    q = _bf16(rng, (17, 128, d))
    host, dmask = _mask(more, rng, 17, 128)
    want = oracle.attention_step(q, *pages, table, lengths, k_scale=scales[0], v_scale=scales[1], sizes=True, **host)
    o = B.attention_step(_dev16(q), *dev, to_dev(table), to_dev(lengths), **sc, **dmask)
    _check(o, want, 2.0 ** -16, d, host.get("slopes"), 2112)


def test_first_keys_that_stay_visible_behind_a_window_and_are_not_seen_ahead(B):
    """The first tokens in a call of their own without window and prefix, the others with both; then a step."""
    from oracle.attention import _attend
    rng = np.random.default_rng(1)
    n, first, window, d = 200, 30, 16, 64
    q, k, v = (_bf16(rng, (n, 2, d)) for _ in range(3))
    t = np.arange(n)
    near = t[:, None] - t[None, :]
    seen = (near >= 0) & ((near < window) | (t < first)[None, :])
    want = [np.stack(x, 1) for x in zip(*(_attend(*(a[:, h].astype(np.float64) for a in (q, k, v)), t, seen, d ** -0.5, None, 0.0, t)
                                          for h in range(2)))]
    off = [to_dev(_offsets([x])) for x in (first, n - first, n)]
    prefix = to_dev(np.array([first], np.int32))
    o = [B.attention(*(_dev16(a[:first]) for a in (q, k, v)), off[0]),
         B.attention(_dev16(q[first:]), _dev16(k), _dev16(v), off[1], k_offsets=off[2], window=window, prefix=prefix)]
    _check(to_dev(np.concatenate([to_np(x).astype(np.float64) for x in o])), want, 2.0 ** -8, d)
    table = to_dev(np.arange(-(-n // 16), dtype=np.int32)[None])
    pools = [_dev16(np.zeros((table.shape[1], 2, 16, d), np.float32)) for _ in range(2)]
    B.kv_write(_dev16(k), _dev16(v), *pools, table, offsets=off[2])
    for at in (0, 10, first, n - 1):
        one = B.attention_step(_dev16(q[at:at + 1]), *pools, table, to_dev(np.array([at + 1], np.int32)), window=window, prefix=prefix)
        _check(one, [x[at:at + 1] for x in want], 2.0 ** -8, d)
