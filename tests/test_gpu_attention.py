"""GPU parity of the paged cache and of attention against the 64-bit oracle.

Tolerances, from the roundings each result goes through:
  * rows into bf16 pages and back, and 8-bit codes, are exact; a row's scale takes one division (2^-24),
    a value read back from 8 bits one product (2^-24) and the rounding to bf16 (2^-8);
  * o = sum w v.  With A = sum w |v|: the output's rounding is 2^-8 |o|; weights rounded to bf16 and divided by the sum
    of the rounded ones move o by sum w delta (v - o) <= 2^-8 (A + |o|) (2^-16 with two terms);
    a score off by e moves every weight by a factor within e^(+-2e), o by 2 e (A + |o|).  A score is a
    sum of d products in fp32, off by (d + 16) 2^-24 sum |q k|, then scaled, capped, lowered by the distance,
    multiplied by log2 e and reduced by the maximum: 2^-21 of the sizes involved covers these steps and the
    exponential's own error.  Products and sums with v in fp32 add 2^-20 A.
"""
import numpy as np
import pytest

import oracle
from synthdata import bf16_round
from tests.helpers import to_dev, to_np, say

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def B():
    import byte_level_lm_amd as B
    B.lib()
    return B


def _bf16(rng, shape, scale=1.0):
    return bf16_round((scale * rng.standard_normal(shape)).astype(np.float32))


def _dev16(x):
    import torch
    return to_dev(x, torch.bfloat16)


def _strided(*parts):
    """Tensors [n, heads, d] as column slices of one row-major array, as a projection gives them."""
    n = parts[0].shape[0]
    row = _dev16(np.concatenate([a.reshape(n, -1) for a in parts], axis=1))
    cut = np.cumsum([0] + [a[0].size if n else a.shape[1] * a.shape[2] for a in parts])
    return [row[:, cut[i]:cut[i + 1]].unflatten(1, a.shape[1:]) for i, a in enumerate(parts)]


def _offsets(lengths):
    return np.concatenate([[0], np.cumsum(lengths)]).astype(np.int64)


def _table(rng, positions, page, spare=3, cols=None):
    """Pages anywhere in a pool for streams with so many positions: (table, npages); -1 where none is needed."""
    used = [-(-int(n) // page) for n in positions]
    cols = max(max(used), 1) if cols is None else cols
    npages = sum(used) + spare
    names, table, at = rng.permutation(npages), np.full((len(used), cols), -1, np.int32), 0
    for s, u in enumerate(used):
        table[s, :u] = names[at:at + u]
        at += u
    return table, npages


def _check(o, want, weights_rel, d, slopes=None, far=0):
    want, size, reach = want
    o = to_np(o).astype(np.float64)
    slope = np.zeros(o.shape[1]) if slopes is None else np.abs(slopes.astype(np.float64))
    e = (d + 16) * 2.0 ** -24 * reach + 2.0 ** -21 * (1 + reach + slope[None, :] * far)
    both = size + np.abs(want)
    tol = 1.02 * (2.0 ** -8 * np.abs(want) + weights_rel * both + 2 * e[..., None] * both) + 2.0 ** -20 * size + 1e-30
    assert np.isfinite(o).all()
    bad = np.abs(o - want) > tol
    assert not bad.any(), (int(bad.sum()), float(np.max(np.abs(o - want) / tol)), np.argwhere(bad)[:4].tolist())


# ---------------------------------------------------------------- rows into pages and back

KV = [([1], 1, 32, 16, [0]), ([3, 0, 70], 2, 64, 16, None), ([64, 65, 63], 4, 128, 64, [0, 1, 63]),
      ([1] * 33, 4, 128, 64, list(range(33))), ([130, 7], 3, 96, 32, [5, 300]), ([20, 300, 1], 1, 256, 128, None),
      ([500], 8, 16, 256, [9]), ([2, 5] * 50, 5, 80, 16, None), ([40], 130, 16, 16, None), ([0, 0, 9, 0], 2, 48, 16, None)]


@pytest.mark.parametrize("lengths,heads,d,page,start", KV)
@pytest.mark.parametrize("q8", [False, True])
def test_rows_into_pages_and_back(B, lengths, heads, d, page, start, q8):
    import torch
    rng = np.random.default_rng(sum(lengths) + d)
    say("kv", lengths[:5], heads, d, page, q8)
    off = _offsets(lengths)
    total = int(off[-1])
    k, v = _bf16(rng, (total + 2, heads, d), 2.0), _bf16(rng, (total + 2, heads, d))
    k[0, 0] = 0.0
    table, npages = _table(rng, [n + (0 if start is None else start[s]) for s, n in enumerate(lengths)], page)
    shape = (npages, heads, page, d)
    dt, want, pools, scales = (torch.int8 if q8 else torch.bfloat16), [], [], [None, None]
    for i, x in enumerate((k, v)):
        old = rng.integers(-127, 128, shape).astype(np.int8 if q8 else np.float32)
        old_scale = rng.random(shape[:3]).astype(np.float32) if q8 else None
        want.append(oracle.kv_write(x[:total], off, table, old, start=start, scale=old_scale))
        pools.append(to_dev(old).to(dt))
        scales[i] = to_dev(old_scale) if q8 else None
    start_d = None if start is None else to_dev(np.array(start, np.int32))
    more = {"start": start_d, "k_scale": scales[0], "v_scale": scales[1]}
    dk, dv = _strided(k, v)  # two rows more than the sequences have
    kp, vp = B.kv_write(dk, dv, *pools, to_dev(table), offsets=to_dev(off), **more)
    assert kp.data_ptr() == pools[0].data_ptr()
    for got, scale, (pages, want_scale) in zip((kp, vp), scales, want):
        assert np.array_equal(to_np(got), pages)
        if q8:
            np.testing.assert_allclose(to_np(scale), want_scale, rtol=2.0 ** -23)
    outs = [torch.full((total + 2, heads, d), 7.0, device="cuda", dtype=torch.bfloat16) for _ in range(2)]
    B.kv_read(kp, vp, to_dev(table), to_dev(off), total + 2, k_out=outs[0], v_out=outs[1], **more)
    for got, scale, (pages, _), x in zip(outs, scales, want, (k, v)):
        got = to_np(got)
        assert np.all(got[total:] == 7.0)
        if q8:
            back = oracle.kv_read(pages, off, table, start=start, scale=to_np(scale))
            assert np.all(np.abs(got[:total] - back) <= 2.0 ** -8 * 1.001 * np.abs(back))
        else:
            assert np.array_equal(got[:total], x[:total])


@pytest.mark.parametrize("q8", [False, True])
def test_one_row_of_each_stream_and_places_without_a_page(B, q8):
    """Without offsets; pages of -1 and past the pool, positions below zero and behind the table: not written, read as zero."""
    import torch
    rng = np.random.default_rng(5)
    heads, d, page, npages = 2, 64, 16, 6
    table = np.array([[0, 1], [2, -1], [3, 6], [4, 5], [1 << 30, 5], [-(1 << 31), -7]], np.int32)
    start = np.array([3, 16, 17, 32, 0, 5], np.int32)
    k, v = _bf16(rng, (6, heads, d)), _bf16(rng, (6, heads, d))
    shape = (npages, heads, page, d)
    old = np.zeros(shape, np.int8 if q8 else np.float32)
    scale = np.zeros(shape[:3], np.float32) if q8 else None
    want = [oracle.kv_write(x, np.arange(7), table, old, start=start, scale=scale) for x in (k, v)]
    pools = [to_dev(old).to(torch.int8 if q8 else torch.bfloat16) for _ in range(2)]
    sc = [to_dev(scale) if q8 else None for _ in range(2)]
    B.kv_write(*_strided(k, v), *pools, to_dev(table), start=to_dev(start), k_scale=sc[0], v_scale=sc[1])
    for got, w in zip(pools, want):
        assert np.array_equal(to_np(got), w[0])
    assert sum(int(np.any(w[0] != 0, axis=(1, 3)).sum()) for w in want) == 2  # stream 0 alone has a place
    off = _offsets([40, 30, 20, 33, 16, 3])
    start = np.array([-4, 0, 10, 0, 3, (1 << 31) - 2], np.int32)
    got = B.kv_read(*pools, to_dev(table), to_dev(off), int(off[-1]), start=to_dev(start), k_scale=sc[0], v_scale=sc[1])
    for x, w, s in zip(got, want, sc):
        back = oracle.kv_read(w[0], off, table, start=start, scale=None if s is None else to_np(s))
        assert np.all(np.abs(to_np(x) - back) <= (2.0 ** -8 * 1.001 * np.abs(back) if q8 else 0))


def test_8_bit_rows_at_their_ends(B):
    """Zeros, rows too small to divide by, NaN and infinity in one row: its scale is not finite, and only its."""
    import torch
    x = np.zeros((6, 1, 32), np.float32)
    x[1, 0, 5] = 1e-35
    x[2] = 1.0; x[2, 0, 9] = np.nan
    x[3] = 1.0; x[3, 0, 30] = -np.inf
    x[4, 0, :5] = [127.0, 0.5, 1.5, 2.5, -2.5]
    x[5, 0] = bf16_round(np.linspace(-1, 1, 32).astype(np.float32))
    pools = [torch.zeros(1, 1, 16, 32, device="cuda", dtype=torch.int8) for _ in range(2)]
    sc = [torch.ones(1, 1, 16, device="cuda") for _ in range(2)]
    dx = _dev16(x)
    B.kv_write(dx, dx, *pools, to_dev(np.zeros((1, 1), np.int32)), offsets=to_dev(_offsets([6])), k_scale=sc[0], v_scale=sc[1])
    q, s = to_np(pools[1])[0, 0], to_np(sc[1])[0, 0]
    assert not q[0].any() and s[0] == 0 and not q[1].any() and s[1] == 0
    assert np.isnan(s[2]) and np.isinf(s[3]) and list(q[4, :5]) == [127, 0, 2, 2, -2] and s[4] == 1.0
    assert np.array_equal(q[5], oracle.quant_rows_q8(x[5])[0][0]) and np.all(s[6:] == 1.0)
    assert torch.equal(pools[0], pools[1])


# ---------------------------------------------------------------- packed prompts

# lengths of queries, of keys (None: the same), query heads, key heads, d
PROMPTS = [([1], None, 1, 1, 8), ([5], None, 1, 1, 64), ([63, 64, 65], None, 2, 1, 128), ([0, 3, 0, 130, 1], None, 4, 2, 64),
           ([200], None, 6, 2, 96), ([77, 128], None, 3, 3, 40), ([300, 17], None, 2, 2, 256), ([129, 31, 33], None, 2, 1, 32),
           ([7] * 40, None, 4, 1, 64), ([520], None, 1, 1, 72), ([1000, 0, 10], None, 2, 1, 128), ([2] * 70 + [90], None, 1, 1, 128),
           ([257, 255], None, 2, 2, 16), ([33, 1, 100], [500, 1, 100], 4, 2, 128), ([1, 1, 1], [1000, 0, 65], 12, 4, 64),
           ([40, 64], [7, 64], 2, 1, 64), ([16], [2500], 2, 1, 128), ([3, 0, 5], [0, 9, 300], 8, 1, 64), ([700], [1500], 1, 1, 160),
           ([260], [1300], 2, 1, 248), ([64], [4096], 1, 1, 64)]
MASKS = [{}, {"causal": False}, {"window": 20}, {"window": 1}, {"window": 100, "prefix": 9}, {"causal": False, "window": 33},
         {"prefix": 70}, {"cap": 5.0, "slopes": True}, {"causal": False, "window": 40, "prefix": 30, "cap": 2.0, "slopes": True}]


def _mask(more, rng, nseq, hq):
    """The mask's arguments for the oracle and for the call."""
    host, dev = dict(more), dict(more)
    if "prefix" in more:
        host["prefix"] = rng.integers(0, more["prefix"] + 1, nseq).astype(np.int32)
        host["prefix"][0] = more["prefix"]
        dev["prefix"] = to_dev(host["prefix"])
    if "slopes" in more:
        host["slopes"] = (2.0 ** -rng.integers(0, 8, hq)).astype(np.float32)
        host["slopes"][0] = 0.0
        dev["slopes"] = to_dev(host["slopes"])
    return host, dev


@pytest.mark.parametrize("lengths,keys,hq,hkv,d", PROMPTS)
@pytest.mark.parametrize("more", MASKS, ids=lambda m: "-".join(m) or "plain")
def test_attention(B, lengths, keys, hq, hkv, d, more):
    rng = np.random.default_rng(sum(lengths) + 10 * d + hq)
    say("attention", lengths[:5], keys, hq, hkv, d, more)
    off, koff = _offsets(lengths), None if keys is None else _offsets(keys)
    q = _bf16(rng, (int(off[-1]), hq, d), 1.5)
    k, v = (_bf16(rng, (int((off if koff is None else koff)[-1]), hkv, d)) for _ in range(2))
    host, dev = _mask(more, rng, len(lengths), hq)
    want = oracle.attention(q, k, v, off, k_offsets=koff, sizes=True, **host)
    if koff is None:
        dq, dk, dv = _strided(q, k, v)
    else:
        dq, (dk, dv) = _dev16(q), _strided(k, v)
    o = B.attention(dq, dk, dv, to_dev(off), k_offsets=None if koff is None else to_dev(koff), **dev)
    _check(o, want, 2.0 ** -8, d, host.get("slopes"), max(keys or lengths))


def test_attention_scale_of_any_sign_and_rows_behind_the_last_sequence(B):
    import torch
    rng = np.random.default_rng(9)
    off, d = _offsets([100, 60]), 64
    q, k, v = (_bf16(rng, (170, 2, d)) for _ in range(3))
    for scale in (-0.2, 0.0, 1.0, 1e-6):
        want = oracle.attention(q[:160], k[:160], v[:160], off, scale=scale, sizes=True)
        out = torch.full((170, 2, d), 7.0, device="cuda", dtype=torch.bfloat16)
        o = B.attention(*_strided(q, k, v), to_dev(off), scale=scale, o_out=out)
        assert o.data_ptr() == out.data_ptr() and torch.all(o[160:] == 7.0)
        _check(o[:160], want, 2.0 ** -8, d)


def test_attention_no_tokens_and_no_keys(B):
    import torch
    q = torch.zeros(0, 2, 64, device="cuda", dtype=torch.bfloat16)
    off = to_dev(np.zeros(3, np.int64))
    assert B.attention(q, q, q, off).shape == (0, 2, 64)
    some = torch.ones(5, 2, 64, device="cuda", dtype=torch.bfloat16)
    o = B.attention(some, q, q, to_dev(np.array([0, 2, 5])), k_offsets=off)
    assert o.shape == (5, 2, 64) and not o.any()
    assert B.attention(q, some, some, off, k_offsets=to_dev(np.array([0, 2, 5]))).shape == (0, 2, 64)


@pytest.mark.parametrize("d", [64, 128, 256])
@pytest.mark.parametrize("value", [np.nan, np.inf, -np.inf])
@pytest.mark.parametrize("more", [{}, {"window": 50}, {"window": 30, "prefix": 4}, {"cap": 20.0}], ids=str)
def test_keys_that_a_query_does_not_see_have_no_part_in_it(B, d, value, more):
    """k and v of token 100 of sequence 1 are not finite: the other sequences and the queries that do not see it are as
    without it; of those that see v's only column 3 of the head is lost."""
    rng = np.random.default_rng(d)
    off = _offsets([70, 300, 90])
    q, k, v = (_bf16(rng, (460, 2, d)) for _ in range(3))
    host, dev = _mask(more, rng, 3, 2)
    at = 70 + 100
    want = oracle.attention(q, k, v, off, sizes=True, **host)
    seen = np.zeros(460, bool)
    seen[at:370] = True
    if "window" in more:
        seen[at + more["window"]:] = False
    for what in ("v", "k"):
        k2, v2 = k.copy(), v.copy()
        (v2 if what == "v" else k2)[at, 1, 3] = value
        o = to_np(B.attention(*_strided(q, k2, v2), to_dev(off), **dev)).astype(np.float64)
        lost = np.zeros(o.shape, bool)
        lost[seen, 1] = True
        if what == "v":
            lost[:] = False
            lost[seen, 1, 3] = True
            assert not np.isfinite(o[lost]).any()
        elif np.isnan(value):
            assert np.isnan(o[lost]).all()
        o[lost] = want[0][lost]
        _check(to_dev(o), want, 2.0 ** -8, d)


def test_keys_of_no_score_and_queries_that_are_not_finite(B):
    """A query row of NaN is lost and no other; keys of the lowest bf16 value give finite outputs."""
    rng = np.random.default_rng(12)
    off, d = _offsets([150]), 128
    q, k, v = (_bf16(rng, (150, 2, d)) for _ in range(3))
    want = oracle.attention(q, k, v, off, sizes=True)
    q2 = q.copy()
    q2[77, 0] = np.nan
    o = to_np(B.attention(*_strided(q2, k, v), to_dev(off))).astype(np.float64)
    assert np.isnan(o[77, 0]).all()
    o[77, 0] = want[0][77, 0]
    _check(to_dev(o), want, 2.0 ** -8, d)
    low = -3.3895313892515355e38
    k2, q3 = k.copy(), np.abs(q) + bf16_round(np.float32(0.5))
    k2[40:60] = low  # scores of the lowest value: keys without weight behind the others
    o = to_np(B.attention(*_strided(q3, k2, v), to_dev(off)))
    assert np.isfinite(o).all()
    keep = np.r_[0:40, 60:150]
    want = oracle.attention(q3[keep], k[keep], v[keep], np.array([0, 130]), sizes=True)
    _check(to_dev(o[keep].astype(np.float64)), want, 2.0 ** -8, d)


# ---------------------------------------------------------------- one token over its pages

# lengths, query heads, key heads, d, page
STEPS = [([1], 1, 1, 32, 16), ([5, 0, 64], 2, 1, 64, 16), ([2048], 12, 4, 128, 64), ([63, 64, 65, 127, 128, 129], 4, 4, 128, 64),
         ([300] * 20, 8, 1, 64, 32), ([31, 33, 1000], 16, 1, 128, 128), ([700, 3], 40, 2, 96, 16), ([513, 1], 6, 3, 256, 256),
         ([17, 2000, 0, 255], 3, 1, 48, 16), ([5000, 9], 2, 2, 128, 64), ([90] * 300, 2, 1, 64, 16), ([1200, 70], 4, 2, 192, 32),
         ([40000, 20], 4, 1, 64, 64), ([128, 257], 7, 7, 80, 32)]
STEP_MASKS = [{}, {"window": 1}, {"window": 100}, {"window": 40, "prefix": 50}, {"window": 500, "prefix": 3, "cap": 4.0},
              {"cap": 10.0, "slopes": True, "prefix": 5}]


def _cache(rng, lengths, heads, d, page, q8, cols=None):
    """A pool of random rows: host arrays (pages, scales) of k and v, the table, and the call's arguments."""
    import torch
    table, npages = _table(rng, lengths, page, cols=cols)
    shape = (npages, heads, page, d)
    if q8:
        pages = [rng.integers(-127, 128, shape).astype(np.int8) for _ in range(2)]
        scales = [(np.exp(0.3 * rng.standard_normal(shape[:3])) / 64).astype(np.float32) for _ in range(2)]
    else:
        pages, scales = [_bf16(rng, shape) for _ in range(2)], [None, None]
    dev = [to_dev(x).to(torch.int8 if q8 else torch.bfloat16) for x in pages]
    return pages, scales, table, dev, {"k_scale": to_dev(scales[0]) if q8 else None, "v_scale": to_dev(scales[1]) if q8 else None}


@pytest.mark.parametrize("lengths,hq,hkv,d,page", STEPS)
@pytest.mark.parametrize("q8", [False, True])
@pytest.mark.parametrize("more", STEP_MASKS, ids=lambda m: "-".join(m) or "plain")
def test_attention_step(B, lengths, hq, hkv, d, page, q8, more):
    rng = np.random.default_rng(sum(lengths) + d + hq)
    say("attention_step", lengths[:5], hq, hkv, d, page, q8, more)
    pages, scales, table, dev, sc = _cache(rng, lengths, hkv, d, page, q8)
    q = _bf16(rng, (len(lengths), hq, d), 1.5)
    host, mask = _mask(more, rng, len(lengths), hq)
    n = np.array(lengths, np.int32)
    want = oracle.attention_step(q, *pages, table, n, k_scale=scales[0], v_scale=scales[1], sizes=True, **host)
    dq = _strided(q, q)[1]
    o = B.attention_step(dq, *dev, to_dev(table), to_dev(n), **sc, **mask)
    _check(o, want, 2.0 ** -16, d, host.get("slopes"), max(lengths))


@pytest.mark.parametrize("q8", [False, True])
def test_step_without_pages_and_lengths_past_the_table(B, q8):
    """Entries outside the pool hold no key; lengths are cut at the table, below zero there are none."""
    rng = np.random.default_rng(21)
    lengths = [100, 400, 64, 130, 90]
    pages, scales, table, dev, sc = _cache(rng, lengths, 2, 64, 16, q8, cols=25)
    table[0, :7] = -1                      # no key at all
    table[1, [0, 3, 4, 24]] = [len(pages[0]), -1, 1 << 30, -(1 << 31)]
    n = np.array([100, 1 << 30, -5, 130, 0], np.int32)
    q = _bf16(rng, (5, 4, 64))
    for more in ({}, {"window": 70, "prefix": 40}):
        host, mask = _mask(more, rng, 5, 4)
        want = oracle.attention_step(q, *pages, table, n, k_scale=scales[0], v_scale=scales[1], sizes=True, **host)
        o = B.attention_step(_dev16(q), *dev, to_dev(table), to_dev(n), **sc, **mask)
        _check(o, want, 2.0 ** -16, 64)
        assert not o[[0, 2, 4]].any()


@pytest.mark.parametrize("q8", [False, True])
@pytest.mark.parametrize("d", [64, 128, 256])
def test_step_does_not_see_what_lies_behind_its_length_or_window(B, q8, d):
    import torch
    rng = np.random.default_rng(22)
    lengths = [37, 3000]
    pages, scales, table, dev, sc = _cache(rng, [64, 3008], 1, d, 32, q8)
    q, n = _bf16(rng, (2, 3, d)), np.array(lengths, np.int32)
    want = oracle.attention_step(q, *pages, table, n, k_scale=scales[0], v_scale=scales[1], window=300, sizes=True)
    hide = [(0, p) for p in range(37, 64)] + [(1, p) for p in list(range(0, 2700)) + list(range(3000, 3008))]
    for s, p in hide:
        for i in range(2):
            if q8:
                sc["kv"[i] + "_scale"][int(table[s, p // 32]), :, p % 32] = float("nan")
            else:
                dev[i][int(table[s, p // 32]), :, p % 32] = float("inf") if p % 2 else float("nan")
    o = B.attention_step(_dev16(q), *dev, to_dev(table), to_dev(n), window=300, **sc)
    _check(o, want, 2.0 ** -16, d)
    # one that it sees is lost: v's in its column, k's in the whole head
    s, p = 1, 2999
    if q8:
        sc["v_scale"][int(table[s, p // 32]), 0, p % 32] = float("nan")
    else:
        dev[1][int(table[s, p // 32]), 0, p % 32, 7] = float("nan")
    o = to_np(B.attention_step(_dev16(q), *dev, to_dev(table), to_dev(n), window=300, **sc))
    assert np.isfinite(o[0]).all() and (np.isnan(o[1]).all() if q8 else np.isnan(o[1, :, 7]).all())
    assert q8 or np.isfinite(np.delete(o[1], 7, axis=1)).all()
    torch.cuda.synchronize()


def test_a_pool_whose_offsets_pass_32_bits(B):
    """Pages behind 2^31 values of a pool: written, read back and attended to."""
    import torch
    rng = np.random.default_rng(23)
    heads, page, d = 8, 256, 128
    npages = (1 << 31) // (heads * page * d) + 40
    pools = [torch.zeros(npages, heads, page, d, device="cuda", dtype=torch.bfloat16) for _ in range(2)]
    table = np.array([[npages - 1, 2], [npages - 7, npages - 3]], np.int32)
    off = _offsets([300, 400])
    k, v = _bf16(rng, (700, heads, d)), _bf16(rng, (700, heads, d))
    B.kv_write(_dev16(k), _dev16(v), *pools, to_dev(table), offsets=to_dev(off))
    back = B.kv_read(*pools, to_dev(table), to_dev(off), 700)
    assert np.array_equal(to_np(back[0]), k) and np.array_equal(to_np(back[1]), v)
    q = _bf16(rng, (2, heads, d))
    o = B.attention_step(_dev16(q), *pools, to_dev(table), to_dev(np.array([300, 400], np.int32)))
    want = oracle.attention(q, k, v, np.arange(3), k_offsets=off, sizes=True)
    _check(o, want, 2.0 ** -16, d)


# ---------------------------------------------------------------- together

@pytest.mark.parametrize("q8", [False, True])
@pytest.mark.parametrize("more", [{}, {"window": 150, "prefix": 20}], ids=str)
def test_prompts_in_pieces_and_steps_equal_one_prompt(B, q8, more):
    """Write, read back and attend piece by piece, then token by token; every row against the whole prompt's. With 8-bit
    pages the whole prompt takes the keys and values that the codes stand for."""
    import torch
    rng = np.random.default_rng(31)
    hq, hkv, d, page = 6, 2, 64, 32
    lengths, pieces, tail = [333, 200, 64], 100, 3
    off = _offsets(lengths)
    q, k, v = (_bf16(rng, (int(off[-1]), h, d)) for h in (hq, hkv, hkv))
    table, npages = _table(rng, lengths, page)
    dt = torch.int8 if q8 else torch.bfloat16
    pools = [torch.zeros(npages, hkv, page, d, device="cuda", dtype=dt) for _ in range(2)]
    sc = {x: torch.zeros(npages, hkv, page, device="cuda") if q8 else None for x in ("k_scale", "v_scale")}
    dq, dk, dv, dtable = _dev16(q), _dev16(k), _dev16(v), to_dev(table)
    host, dev = _mask(more, rng, 3, hq)
    o = torch.zeros_like(dq)
    done = np.zeros(3, np.int64)
    while (done < np.array(lengths) - tail).any():
        n = np.minimum(np.array(lengths) - tail - done, pieces)
        rows = np.concatenate([np.arange(off[s] + done[s], off[s] + done[s] + n[s]) for s in range(3)])
        at = to_dev(rows)
        B.kv_write(dk[at], dv[at], *pools, dtable, offsets=to_dev(_offsets(n)), start=to_dev(done.astype(np.int32)), **sc)
        done = done + n
        koff = _offsets(done)
        kk, vv = B.kv_read(*pools, dtable, to_dev(koff), int(koff[-1]), **sc)
        o[at] = B.attention(dq[at], kk, vv, to_dev(_offsets(n)), k_offsets=to_dev(koff), **dev)
    lens = to_dev(done.astype(np.int32))
    for i in range(tail):
        at = to_dev(off[1:] - tail + i)
        B.kv_write(dk[at], dv[at], *pools, dtable, start=lens, **sc)
        lens += 1
        o[at] = B.attention_step(dq[at], *pools, dtable, lens, **sc, **dev)
    if q8:
        k, v = (to_np(x) for x in B.kv_read(*pools, dtable, to_dev(off), int(off[-1]), **sc))
    want = oracle.attention(q, k, v, off, sizes=True, **host)
    # 8-bit values go into the step as they are, and into a prompt rounded to bf16 (2^-8 of k in the scores, of v in the sum)
    extra = (want[0], want[1], want[2] * (1 + (2.0 ** -8 * 2 ** 24 / (d + 16) if q8 else 0)))
    _check(o, extra, 2.0 ** -8 + (2.0 ** -8 if q8 else 0), d)


def test_on_another_stream_in_a_graph_and_twice_the_same(B):
    """A step of the cache and the attention captured once, replayed with other tokens and lengths while eager calls run in
    between; every replay gives bit for bit what the eager calls give."""
    import torch
    rng = np.random.default_rng(33)
    nseq, hq, hkv, d, page, cols = 5, 8, 2, 128, 64, 40
    lengths = np.array([1, 700, 64, 2000, 2500], np.int32)
    table, npages = _table(rng, [cols * page] * nseq, page)
    base = [_dev16(_bf16(rng, (npages, hkv, page, d))) for _ in range(2)]
    dtable = to_dev(table)
    tokens = [[_dev16(_bf16(rng, (nseq, h, d))) for h in (hq, hkv, hkv)] for _ in range(4)]
    off, slots = to_dev(_offsets([3, 40, 9, 0, 200])), to_dev(lengths)
    prompt = [_dev16(_bf16(rng, (252, h, d))) for h in (hq, hkv, hkv)]

    def one(q, k, v, pools, n):
        B.kv_write(k, v, *pools, dtable, start=n)
        n.add_(1)
        return B.attention_step(q, *pools, dtable, n), B.attention(*prompt, off, window=33)

    eager, pools, n = [], [x.clone() for x in base], slots.clone()
    for t in tokens:
        eager.append([x.clone() for x in one(*t, pools, n)])
    last = [x.clone() for x in pools]
    pools, n = [x.clone() for x in base], slots.clone()
    q, k, v = (x.clone() for x in tokens[0])
    stream = torch.cuda.Stream()
    stream.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(stream):
        one(q, k, v, [x.clone() for x in base], slots.clone())
    torch.cuda.current_stream().wait_stream(stream)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        out = one(q, k, v, pools, n)
    for i, t in enumerate(tokens):
        for dst, src in zip((q, k, v), t):
            dst.copy_(src)
        B.attention(*prompt, off)  # eager work with workspaces of its own
        graph.replay()
        assert torch.equal(out[0], eager[i][0]) and torch.equal(out[1], eager[i][1]), i
    assert all(torch.equal(a, b) for a, b in zip(pools, last))
