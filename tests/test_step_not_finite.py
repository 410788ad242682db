"""Values that are not finite in attention of one token: what they do to the streams that see them."""
import numpy as np
import pytest

from tests.helpers import to_dev, to_np
from tests.test_gpu_attention import _bf16, _dev16, _mask, _table

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def B():
    import byte_level_lm_amd as B
    B.lib()
    return B


@pytest.mark.parametrize("lengths,hq,hkv,d", [([70, 300, 1, 0, 33], 6, 2, 64), ([2048], 12, 4, 128), ([700, 40], 20, 1, 40), ([1500, 9], 4, 2, 256),
                                             ([9000], 3, 1, 128)])
@pytest.mark.parametrize("more", [{}, {"window": 45}, {"window": 300, "prefix": 20}, {"cap": 6.0, "slopes": True}], ids=lambda m: "-".join(m) or "plain")
def test_what_a_stream_sees_of_values_that_are_not_finite(B, lengths, hq, hkv, d, more):
    """Infinities of one sign stay, of both or NaN give NaN, in the columns and heads that have them; everything else is bit for
    bit as without them."""
    rng = np.random.default_rng(sum(lengths) + d)
    lengths, page = np.array(lengths, np.int32), 16
    table, npages = _table(rng, lengths, page)
    k, v = (_bf16(rng, (npages, hkv, page, d), 0.5) for _ in range(2))
    q = _bf16(rng, (len(lengths), hq, d), 0.5)
    host, dev = _mask(more, rng, len(lengths), hq)
    if "slopes" in host:  # no weight becomes zero
        host["slopes"] = np.full(hq, 2.0 ** -10, np.float32)
        dev["slopes"] = to_dev(host["slopes"])
    v2 = v.copy()
    for _ in range(40):
        v2[rng.integers(npages), rng.integers(hkv), rng.integers(page), rng.integers(d)] = rng.choice([np.nan, np.inf, -np.inf])
    s, last = 0, int(lengths[0]) - 1  # and the last row of the first stream, which it sees in any case
    at = table[s, last // page]
    v2[at, 0, last % page, :4] = [np.inf, -np.inf, np.nan, np.inf]
    got, clean = (to_np(B.attention_step(_dev16(q), _dev16(k), _dev16(x), to_dev(table), to_dev(lengths), **dev)).astype(np.float64)
                  for x in (v2, v))
    want = clean.copy()
    for s, n in enumerate(lengths):
        j = np.arange(n)
        seen = j > n - 1 - host["window"] if host.get("window") else np.ones(n, bool)
        if host.get("prefix") is not None:
            seen = seen | (j < host["prefix"][s])
        j = j[seen]
        for h in range(hq):
            x = v2[table[s, j // page], h * hkv // hq, j % page].reshape(len(j), d)
            nan, up, down = np.isnan(x).any(0), (x == np.inf).any(0), (x == -np.inf).any(0)
            part = want[s, h]
            part[up] = np.inf
            part[down] = -np.inf
            part[nan | (up & down)] = np.nan
    assert np.array_equal(got, want, equal_nan=True)


@pytest.mark.parametrize("d", [64, 128, 256])
def test_8_bit_rows_whose_scale_is_not_finite(B, d):
    """Code times scale: infinities where the code is not zero, NaN where it is; one stream of three sees the row."""
    rng = np.random.default_rng(d)
    lengths, page = np.array([100, 40, 64], np.int32), 16
    table, npages = _table(rng, lengths, page)
    k, v = (rng.integers(-127, 128, (npages, 1, page, d)).astype(np.int8) for _ in range(2))
    scale = np.full((npages, 1, page), 1 / 256, np.float32)
    q = _bf16(rng, (3, 2, d), 0.25)
    at = (table[0, 2], 0, 5)
    v[at] = np.where(np.arange(d) % 3 == 0, 0, np.where(np.arange(d) % 3 == 1, 7, -7))
    out = {}
    for x in (1 / 256, np.inf, np.nan):
        vs = scale.copy()
        vs[at] = x
        out[x] = to_np(B.attention_step(_dev16(q), to_dev(k), to_dev(v), to_dev(table), to_dev(lengths), k_scale=to_dev(scale), v_scale=to_dev(vs)))
    want = out[1 / 256].copy()
    want[0] = np.where(np.arange(d) % 3 == 0, np.nan, np.where(np.arange(d) % 3 == 1, np.inf, -np.inf))
    assert np.array_equal(out[np.inf], want, equal_nan=True)
    want[0] = np.nan
    # NaN comes in every column of the stream that sees it and in no other
    assert np.array_equal(out[np.nan], want, equal_nan=True)
